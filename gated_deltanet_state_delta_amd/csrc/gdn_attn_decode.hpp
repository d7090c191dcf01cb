// gdn_attn_decode.hpp -- attention of each row's newest tokens over a paged
// key-value cache (gfx950).
//
//   s_j = scale k_scale <q, K_j>,  out = v_scale sum_j e^{s_j - m} V_j / sum_j e^{s_j - m}
//
// over the positions j that the token sees, in one pass over the cache: a
// running maximum m and sum l per query row, the output rescaled when m
// grows (scores are kept in units of log2, so e^x is one hardware exp2).
//
// What bounds it: every key and value is read once and used for the
// T * hq/hkv query rows of its head only, so the cache's bytes over the HBM
// rate are the floor; the products run on MFMA mostly to keep the VALU free.
//
// Work split: a wave walks keys of one key-value head for 16 or 32 query rows, by
// itself: no barrier, and no LDS where pages are whole subtiles.  The lengths
// are known on the device only, so the keys of all rows, laid end to end in
// steps of one tile, are dealt out evenly: each of a fixed number of waves (as
// many as the card holds at once) finds its share from the lengths and may end
// one row, take some whole ones and begin another.  Whole rows are finished on
// the spot; the parts of a row that several waves share go to the workspace as
// (m, l, unnormalised output) and attn_join_kernel joins them in a fixed order.
//
// No LDS and no shuffles between the cache and MFMA.  Both products are
// taken transposed, so every operand is in the form in which a lane loads
// it (lane l: x = l % 16, g = l / 16):
//  * S^T[key][row] = K Q^T: lane (x, g) loads 16-byte pieces of key x's row;
//    which head dimensions a lane group holds is free as long as q uses the
//    same assignment.  The lane ends with keys 4g .. 4g+3 of query row x.
//  * O^T[dim][row] = V^T P^T: the scores' accumulator is directly the B
//    operand.  Lane (x, g) loads 16-byte pieces of keys 4g .. 4g+3 (16 lanes
//    read a key's row contiguously) and output tile e takes piece element e
//    as its dimension x, so transposing V is a 2 x 2 permute of registers.
//    A lane holds the output of query row x: rescaling by its own factor
//    needs no exchange.
// bf16 weights are split into two bf16 terms (high and rest), so P V keeps
// the weights to 2^-16; the second MFMA is free next to the loads.
#pragma once

#include "gdn_device.hpp"
#include "gdn_paged.hpp"

namespace gdn {

struct AttnParams {
  const void* q;
  int64_t q_sb, q_st, q_sh;  // bytes
  void* out;
  float* lse;
  const void* k;
  const void* v;
  int64_t k_sp, v_sp;            // page strides, bytes
  uint32_t k_st, v_st;           // token strides, bytes
  int64_t k_sh, v_sh;            // head strides, bytes
  const int32_t* table;
  int64_t table_stride;
  const int32_t* lens;
  const float* k_scale;
  const float* v_scale;
  float* part_o;   // [2 * shares][hkv][R][D]; the workspace's arrays are null when each row is one share
  float* part_ml;  // [2 * shares][hkv][R][2]
  int2* plan;      // [batch]: a row's first share and how many it lies in
  float scale_log2;
  uint32_t page_mul, page_shift;  // j / page_size = (j * page_mul) >> page_shift
  int batch, T, hq, hkv, group, R, ntile, n_pages, page_size, cap, shares;
};

__device__ __forceinline__ int attn_len(const AttnParams& p, int b) {
  const int len = p.lens[b];
  return p.n_pages == 0 ? 0 : min(max(len, 0), p.cap);
}

// A row's steps of STEP keys (one tile; every share is whole steps of a row);
// an empty row has one, which writes its zeros.
template <int STEP>
__device__ __forceinline__ int attn_steps(int len) { return max(1, (len + STEP - 1) / STEP); }

__device__ __forceinline__ int wave_scan_add_i(int v) {  // inclusive, in lane order
  v += dpp_i<0x111, 0xF>(0, v);
  v += dpp_i<0x112, 0xF>(0, v);
  v += dpp_i<0x114, 0xF>(0, v);
  v += dpp_i<0x118, 0xF>(0, v);
  v += dpp_i<0x142, 0xA>(0, v);
  v += dpp_i<0x143, 0xC>(0, v);
  return v;
}

// Steps [at, at + n) of row b and, once they end that row, of the rows behind
// it; size: steps of a full share.
struct AttnShare { int b, at, n, size; };

// Share k of `shares` equal ones (the last may be short or empty).  Each lane
// sums the steps of batch / 64 neighbouring rows; every wave finds the share
// for itself, without LDS.  All steps together are below 2^31 (checked on the
// host against the tables' sizes).
template <int STEP>
__device__ __forceinline__ AttnShare attn_share(const AttnParams& p, int k, int lane) {
  AttnShare r;
  if (!p.plan) {
    r.b = k;
    r.at = 0;
    r.n = r.size = k < p.batch ? attn_steps<STEP>(attn_len(p, k)) : 0;
    return r;
  }
  const int per = (p.batch + 63) >> 6, i0 = lane * per, i1 = min(p.batch, i0 + per);
  int mine = 0;
  for (int i = i0; i < i1; ++i) mine += attn_steps<STEP>(attn_len(p, i));
  const int upto = wave_scan_add_i(mine), from = upto - mine;
  const int all = __builtin_amdgcn_readlane(upto, 63);
  r.size = (int)(((int64_t)all + p.shares - 1) / p.shares);
  const int64_t first = (int64_t)k * r.size;
  r.n = (int)max((int64_t)0, min((int64_t)r.size, all - first));
  r.b = r.at = 0;
  if (r.n == 0) return r;
  const bool here = first >= from && first < upto;
  int b = i0, at = (int)first - from;
  if (here)
    for (;; ++b) {
      const int n = attn_steps<STEP>(attn_len(p, b));
      if (at < n) break;
      at -= n;
    }
  const int src = __builtin_ctzll(__ballot(here));
  r.b = __builtin_amdgcn_readlane(b, src);
  r.at = __builtin_amdgcn_readlane(at, src);
  return r;
}

// One output: the weighted sum over the weights' sum l.  l is at least 1 (the
// largest score's weight) unless a row sees nothing or scores of -inf only: then
// it is 0, and the output zero.  The maximum does not tell these rows from one
// whose scores are all NaN (fmaxf drops NaN); there l is NaN and so is the output.
__device__ __forceinline__ float attn_inv(const AttnParams& p, float l, int h) {
  return (p.v_scale ? p.v_scale[h] : 1.0f) / l;
}
__device__ __forceinline__ float attn_out(float o, float l, float inv) { return l == 0.f ? 0.f : o * inv; }
// Natural log of the weights' sum, from the maximum and sum in units of log2.
__device__ __forceinline__ float attn_lse(float m, float l) {
  return l == 0.f ? -__builtin_inff() : (m + __builtin_amdgcn_logf(l)) * 0.6931471805599453f;
}

// N raw bytes of a row piece, as dwords (2 bytes sit in the low half).
template <int N> struct Raw { uint32_t w[(N + 3) / 4]; };

// ONCE: a non-temporal load, for data that no other wave reads.
template <int N, bool ONCE>
__device__ __forceinline__ Raw<N> raw_buf(__amdgpu_buffer_rsrc_t r, uint32_t voff) {
  constexpr int aux = ONCE ? 2 : 0;  // the nt bit
  Raw<N> o;
  if constexpr (N == 16) {
    const u32x4 t = __builtin_amdgcn_raw_buffer_load_b128(r, voff, 0, aux);
    o.w[0] = t[0]; o.w[1] = t[1]; o.w[2] = t[2]; o.w[3] = t[3];
  } else if constexpr (N == 8) {
    const auto t = __builtin_amdgcn_raw_buffer_load_b64(r, voff, 0, aux);
    o.w[0] = t[0]; o.w[1] = t[1];
  } else if constexpr (N == 4) {
    o.w[0] = __builtin_amdgcn_raw_buffer_load_b32(r, voff, 0, aux);
  } else {
    o.w[0] = (uint16_t)__builtin_amdgcn_raw_buffer_load_b16(r, voff, 0, aux);
  }
  return o;
}
template <bool ONCE, typename V>
__device__ __forceinline__ V load_as(const char* p) {
  if constexpr (ONCE) return __builtin_nontemporal_load(reinterpret_cast<const V*>(p));
  else return *reinterpret_cast<const V*>(p);
}
template <int N, bool ONCE>
__device__ __forceinline__ Raw<N> raw_load(const char* p) {
  typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
  Raw<N> o;
  if constexpr (N == 16) {
    const u32x4 t = load_as<ONCE, u32x4>(p);
    o.w[0] = t[0]; o.w[1] = t[1]; o.w[2] = t[2]; o.w[3] = t[3];
  } else if constexpr (N == 8) {
    const u32x2 t = load_as<ONCE, u32x2>(p);
    o.w[0] = t[0]; o.w[1] = t[1];
  } else if constexpr (N == 4) {
    o.w[0] = load_as<ONCE, uint32_t>(p);
  } else {
    o.w[0] = load_as<ONCE, uint16_t>(p);
  }
  return o;
}

typedef __bf16 bf2 __attribute__((ext_vector_type(2)));
typedef float f2 __attribute__((ext_vector_type(2)));
struct e4m3 { uint8_t b; };

// Elements 2i and 2i+1 of a piece as two packed bf16 (exact for e4m3).
template <typename KE, int N>
__device__ __forceinline__ uint32_t bf_pair(const Raw<N>& r, int i) {
  if constexpr (sizeof(KE) == 2) return r.w[i];
  else return __builtin_bit_cast(uint32_t, (i & 1) ? __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(r.w[i >> 1], 1.0f, true)
                                                   : __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(r.w[i >> 1], 1.0f, false));
}
// Elements 2i and 2i+1 of an fp32 piece.
template <int N>
__device__ __forceinline__ f2 f_pair(const Raw<N>& r, int i) {
  return f2{__uint_as_float(r.w[2 * i]), __uint_as_float(r.w[2 * i + 1])};
}

// Reductions over the four lane groups g of the lanes with one x: the halves
// and the 16-lane rows are exchanged in the VALU (permlane swaps).
__device__ __forceinline__ float max_over_g(float v) {
  const uint32_t u = __float_as_uint(v);
  const auto a = __builtin_amdgcn_permlane16_swap(u, u, false, false);
  const float m = fmaxf(__uint_as_float(a[0]), __uint_as_float(a[1]));
  const uint32_t w = __float_as_uint(m);
  const auto b = __builtin_amdgcn_permlane32_swap(w, w, false, false);
  return fmaxf(__uint_as_float(b[0]), __uint_as_float(b[1]));
}
__device__ __forceinline__ float sum_over_g(float v) {
  const uint32_t u = __float_as_uint(v);
  const auto a = __builtin_amdgcn_permlane16_swap(u, u, false, false);
  const float m = __uint_as_float(a[0]) + __uint_as_float(a[1]);
  const uint32_t w = __float_as_uint(m);
  const auto b = __builtin_amdgcn_permlane32_swap(w, w, false, false);
  return __uint_as_float(b[0]) + __uint_as_float(b[1]);
}

__device__ __forceinline__ float exp2_hw(float x) { return __builtin_amdgcn_exp2f(x); }

// How many waves a SIMD holds and the bytes of K in a wave's tile.  Either
// way 64 KiB a CU are in flight; fewer and longer streams read HBM faster as
// long as a wave's own work between its loads is short.  bf16 and fp32 rows of
// 256 bytes and more: one wave, 8 KiB (64 ragged rows up to 8192 tokens, 8
// heads of 128, bf16: 172 us; two waves of 4 KiB 175, two of 8 KiB 184, three
// 193).  Shorter rows, and e4m3 whose conversion is VALU work: two waves, 4
// KiB (256 rows, 2 heads of 256, e4m3: 110 us; one wave 131, three 122).
constexpr int attn_occ(int es, int d) { return es > 1 && d >= 128 ? 1 : 2; }

// IO: type of q and out; KE: cache element.  The products are bf16, or fp32
// for an fp32 cache.  fp32 queries and weights over an e4m3 cache, whose values
// bf16 holds exactly, enter as three bf16 terms (24 bits): 3 products of 16x16x32
// instead of 8 of 16x16x4 at twice the cycles each (64 ragged rows up to 8192 tokens,
// 8 heads of 128: 105 us against 186).
//
// KIND 0: one new token, up to 16 query rows of a key-value head.  1: several
// new tokens, up to 16 rows.  2: up to 32 rows.  3: more.
constexpr int attn_kind(int T, int R) { return R > 32 ? 3 : R > 16 ? 2 : T > 1 ? 1 : 0; }
// Tiles of 16 query rows of a wave, which reads a key once for all of them: two
// where the registers hold them (io: bytes of an element of q), one for fp32
// heads of 256.  64 rows (16 batch rows up to 8192 tokens, 8 heads of 128, bf16):
// 87 us, with four tiles 95, with one 108.
constexpr int attn_rows16(int kind, int d, int io) { return kind < 2 || (io == 4 && d > 128) ? 1 : 2; }
// Waves of a SIMD; with two row tiles a wave needs more than half of its
// registers from heads of 128 on.
constexpr int attn_waves(int es, int d, int kind) { return kind > 1 ? d > 64 ? 1 : 2 : attn_occ(es, d); }

// Keys of a wave's tile, a multiple of the products' depth.
constexpr int attn_tile(int es, int d) {
  const int keys = 8192 / attn_occ(es, d) / (d * es);
  return keys > 64 ? 64 : keys < 16 ? 16 : keys;
}

template <typename IO, typename KE, int D, int KIND>
struct AttnCfg {
  static constexpr int ES = sizeof(KE);
  static constexpr bool BF = ES < 4;
  static constexpr int QT = sizeof(IO) == 2 ? 1 : 3, PT = sizeof(IO) == 2 ? 2 : 3;  // bf16 terms of queries, of weights
  static constexpr int kmin(int a, int b) { return a < b ? a : b; }
  static constexpr int KW = kmin(16 / ES, D / 4), NC = D / (4 * KW);    // elements per K piece, pieces per row and lane
  static constexpr int VW = kmin(16 / ES, D / 16), U = D / (16 * VW);   // the same for V
  static constexpr int OCC = attn_waves(ES, D, KIND), KT = attn_tile(ES, D);
  static constexpr int NT = KT / 16;
  static constexpr int NA = D / 16;  // accumulator tiles
};

// UNI: page_size is a multiple of 16, so every 16-key subtile lies in one
// page: its base is a scalar and rows past the end read zeros through the
// buffer's bound.  Otherwise each key's offset is looked up by one lane and
// passed through LDS.
template <typename IO, typename KE, int D, bool UNI, int KIND>
__global__ void __launch_bounds__(256, (AttnCfg<IO, KE, D, KIND>::OCC)) attn_decode_kernel(AttnParams p) {
  typedef AttnCfg<IO, KE, D, KIND> C;
  constexpr int KT = C::KT, NT = C::NT, NC = C::NC, KW = C::KW, VW = C::VW, U = C::U, NA = C::NA, ES = C::ES;
  constexpr int QT = C::QT, PT = C::PT, RT = attn_rows16(KIND, D, sizeof(IO));
  // Where no second wave reads a key, non-temporal loads leave the caches
  // alone (the bf16 batch above, at two waves of 8 KiB: 184 us against 201 with
  // ordinary ones; 64 rows that share all of their 4096 tokens 94 against 85).
  constexpr bool BF = C::BF, MT = KIND > 0, ONCE = KIND < 2 || (KIND == 2 && RT == 2);
  constexpr uint64_t kNone = ~0ull;
  __shared__ uint64_t offs[UNI ? 1 : 4][2][2][UNI ? 1 : KT];  // [wave][parity][K, V][key]

  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  // Wave -> (share, head, row tile of 16 RT rows).  A workgroup's waves take
  // the row tiles of one (share, head), which read the same keys, or
  // neighbouring heads, whose rows are neighbours in a tokens-first cache;
  // further workgroups of one (share, head) are 8 apart and so on one XCD
  // (workgroups go round the 8).
  const int rtw = p.ntile > 2 ? 4 : p.ntile, nwg = (p.ntile + rtw - 1) / rtw;
  const int unit = (int)((blockIdx.x / (8 * nwg) * 8 + (blockIdx.x & 7)) * (4 / rtw)) + wave / rtw;
  const int rt = (int)(blockIdx.x / 8 % nwg) * rtw + wave % rtw;
  const int h = unit % p.hkv, share_id = unit / p.hkv;
  if (share_id >= p.shares || rt >= p.ntile) return;
  AttnShare share = attn_share<KT>(p, share_id, lane);

  const float s_scale = p.scale_log2 * (p.k_scale ? p.k_scale[h] : 1.0f);

  while (share.n > 0) {
    const int b = share.b, len = attn_len(p, b), row_steps = attn_steps<KT>(len), at = share.at;
    const int take = min(share.n, row_steps - at);
    const int c0 = at * KT, c1 = min(len, (at + take) * KT);
    const bool whole = take == row_steps;
    const int slot = 2 * share_id + (at == 0);  // of a part: one that begins a row, one that does not
    if (p.plan && at == 0 && h == 0 && rt == 0 && lane == 0)
      p.plan[b] = make_int2(share_id, 1 + (row_steps - take + share.size - 1) / share.size);
    share.n -= take;
    share.b = b + 1;
    share.at = 0;

    // The lane's place, opaque to the compiler: what follows from it is computed
    // for each row anew rather than held in registers across the walk.
    int own = lane;
    asm volatile("" : "+v"(own));
    const int x = own & 15, g = own >> 4;
    // This lane's query rows, one of each 16: row r is token r / group, query
    // head h*group + r % group, and sees keys below lim.
    int lim[RT], t_row[RT];
    bf8 qb[RT][BF ? QT : 1][BF ? D / 32 : 1];
    float qf[RT][BF ? 1 : D / 4];
#pragma unroll
    for (int q = 0; q < RT; ++q) {
      const int r = (rt * RT + q) * 16 + x;
      const bool row_ok = r < p.R;
      t_row[q] = row_ok ? r / p.group : 0;
      const int hq_row = h * p.group + (row_ok ? r % p.group : 0);
      lim[q] = row_ok ? max(0, min(len, len - p.T + t_row[q] + 1)) : 0;
      const char* qp = (const char*)p.q + b * p.q_sb + t_row[q] * p.q_st + hq_row * p.q_sh;
#pragma unroll
      for (int i = 0; i < D / 4; i += BF ? 8 : 4) {
        const int c = i / KW, d = 4 * KW * c + KW * g + i % KW;
        if constexpr (BF && sizeof(IO) == 2) {
          bf8 t = {};
          if (row_ok) t = *reinterpret_cast<const bf8*>(qp + d * 2);
          qb[q][0][i / 8] = t;
        } else {
#pragma unroll
          for (int k = 0; k < (BF ? 8 : 4); k += 4) {
            f4 t = {};
            if (row_ok) t = *reinterpret_cast<const f4*>(qp + (d + k) * 4);
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              if constexpr (BF) {
                // cut off, not rounded, so that the largest values stay finite
                float rest = t[e];
#pragma unroll
                for (int n = 0; n < QT; ++n) {
                  const float term = __uint_as_float(__float_as_uint(rest) & 0xffff0000u);
                  qb[q][n][i / 8][k + e] = (__bf16)(fabsf(rest) < __builtin_inff() ? term : rest);
                  rest = fabsf(rest) < __builtin_inff() ? rest - term : 0.f;
                }
              } else {
                qf[q][i + e] = t[e];
              }
            }
          }
        }
      }
    }

    const char* kbase = (const char*)p.k + h * p.k_sh;
    const char* vbase = (const char*)p.v + h * p.v_sh;
    const int32_t* tab = p.table + b * p.table_stride;

    f4 acc[RT][NA];
    float m[RT], l[RT];
#pragma unroll
    for (int q = 0; q < RT; ++q) {
#pragma unroll
      for (int i = 0; i < NA; ++i) acc[q][i] = f4{0.f, 0.f, 0.f, 0.f};
      m[q] = -__builtin_inff();
      l[q] = 0.f;
    }

    Raw<KW * ES> kr[NT][NC];
    Raw<VW * ES> vr[NT][4][U];


    // ---- page lookups
    auto page_of = [&](int key) -> int { return (int)(((uint64_t)(uint32_t)key * p.page_mul) >> p.page_shift); };
    // UNI: the table entries of a tile's subtiles (keys clamped into the row).
    struct Ents { int e[NT]; };
    auto load_ents = [&](int key0) {
      Ents o;
#pragma unroll
      for (int n = 0; n < NT; ++n) o.e[n] = tab[page_of(min(key0 + 16 * n, len - 1))];
      return o;
    };
    // UNI: the resource of one subtile's rows of K or V: `rows` valid rows
    // from its first (none for an entry outside the cache).
    auto sub_rsrc = [&](const char* base, int64_t sp, uint32_t st, int ent, int key) {
      const int off = key - page_of(key) * p.page_size;
      const bool ok = ent >= 0 && ent < p.n_pages;
      const int rows = ok ? min(16, len - key) : 0;
      const uint32_t bytes = rows > 0 ? (uint32_t)(rows - 1) * st + D * ES : 0u;
      return buf_rsrc_n(base + (ok ? (int64_t)ent * sp : 0) + (int64_t)off * st, bytes);
    };
    auto issue_k_uni = [&](const Ents& en, int key0) {
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        const auto rs = sub_rsrc(kbase, p.k_sp, p.k_st, en.e[n], key0 + 16 * n);
#pragma unroll
        for (int c = 0; c < NC; ++c) kr[n][c] = raw_buf<KW * ES, ONCE>(rs, x * p.k_st + (4 * KW * c + KW * g) * ES);
      }
    };
    auto issue_v_uni = [&](const Ents& en, int key0) {
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        const auto rs = sub_rsrc(vbase, p.v_sp, p.v_st, en.e[n], key0 + 16 * n);
#pragma unroll
        for (int j = 0; j < 4; ++j)
#pragma unroll
          for (int u = 0; u < U; ++u)
            vr[n][j][u] = raw_buf<VW * ES, ONCE>(rs, (4 * g + j) * p.v_st + (16 * VW * u + VW * x) * ES);
      }
    };
    // Not UNI: lane l < KT looks up key l of a tile; `publish` leaves the byte
    // offsets of its rows (kNone where there is no row) in this wave's LDS.
    auto load_ent1 = [&](int key0) { return tab[page_of(min(key0 + min(lane, KT - 1), len - 1))]; };
    auto publish = [&](int ent, int key0, int par) {
      const int key = key0 + lane;
      const int off = key - page_of(key) * p.page_size;
      const bool ok = key < len && ent >= 0 && ent < p.n_pages;
      if (lane < KT) {
        offs[wave][par][0][lane] = ok ? (uint64_t)((int64_t)ent * p.k_sp + (int64_t)off * p.k_st) : kNone;
        offs[wave][par][1][lane] = ok ? (uint64_t)((int64_t)ent * p.v_sp + (int64_t)off * p.v_st) : kNone;
      }
      __builtin_amdgcn_wave_barrier();
    };
    auto issue_k_any = [&](int par) {
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        const uint64_t o = offs[wave][par][0][16 * n + x];
        const char* src = kbase + (o == kNone ? 0 : o);  // no row: any row, masked below
#pragma unroll
        for (int c = 0; c < NC; ++c) kr[n][c] = raw_load<KW * ES, ONCE>(src + (4 * KW * c + KW * g) * ES);
      }
    };
    uint32_t held = ~0u;  // bit 4n + j: key 16n + 4g + j has a row
    auto issue_v_any = [&](int par) {
      held = 0;
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const uint64_t o = offs[wave][par][1][16 * n + 4 * g + j];
          held |= (o == kNone ? 0u : 1u) << (4 * n + j);
          const char* src = vbase + (o == kNone ? 0 : o);
#pragma unroll
          for (int u = 0; u < U; ++u) vr[n][j][u] = raw_load<VW * ES, ONCE>(src + (16 * VW * u + VW * x) * ES);
        }
    };

    Ents ent_cur = {}, ent_next = {};
    int ent1_next = 0;
    int par = 0;
    if (c0 < c1) {
      if constexpr (UNI) {
        ent_cur = load_ents(c0);
        issue_k_uni(ent_cur, c0);
        ent_next = load_ents(c0 + KT);
      } else {
        publish(load_ent1(c0), c0, 0);
        issue_k_any(0);
        ent1_next = load_ent1(c0 + KT);
      }
    }
    for (int key0 = c0; key0 < c1; key0 += KT) {
      if constexpr (UNI) issue_v_uni(ent_cur, key0);
      else issue_v_any(par);

      // ---- scores of the tile
      f4 s[RT][NT];
#pragma unroll
      for (int n = 0; n < NT; ++n) {
#pragma unroll
        for (int q = 0; q < RT; ++q) s[q][n] = f4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int c = 0; c < NC; ++c) {
          if constexpr (BF) {
#pragma unroll
            for (int w = 0; w < KW; w += 8) {
              u32x4 t;
#pragma unroll
              for (int i = 0; i < 4; ++i) t[i] = bf_pair<KE>(kr[n][c], w / 2 + i);
#pragma unroll
              for (int k = QT - 1; k >= 0; --k)
#pragma unroll
                for (int q = 0; q < RT; ++q)
                  s[q][n] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf8, t), qb[q][k][(c * KW + w) / 8],
                                                                    s[q][n], 0, 0, 0);
            }
          } else {
#pragma unroll
            for (int i = 0; i < KW / 2; ++i) {
              const f2 t = f_pair(kr[n][c], i);
#pragma unroll
              for (int e = 0; e < 2; ++e)
#pragma unroll
                for (int q = 0; q < RT; ++q)
                  s[q][n] = __builtin_amdgcn_mfma_f32_16x16x4f32(t[e], qf[q][c * KW + 2 * i + e], s[q][n], 0, 0, 0);
            }
          }
        }
      }
      // The next tile's keys into the registers that the scores just read.
      uint32_t sub_ok = ~0u;
      if constexpr (UNI) {
#pragma unroll
        for (int n = 0; n < NT; ++n)
          if (ent_cur.e[n] < 0 || ent_cur.e[n] >= p.n_pages) sub_ok &= ~(1u << n);
        if (key0 + KT < c1) issue_k_uni(ent_next, key0 + KT);
        ent_cur = ent_next;
        ent_next = load_ents(key0 + 2 * KT);
      } else {
        par ^= 1;
        if (key0 + KT < c1) {
          publish(ent1_next, key0 + KT, par);
          issue_k_any(par);
          ent1_next = load_ent1(key0 + 2 * KT);
        }
      }

      // ---- masks, running maximum, weights
#pragma unroll
      for (int q = 0; q < RT; ++q) {
        float mx = m[q];
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const int key = key0 + 16 * n + 4 * g + j;
            const bool sees = key < lim[q] && (UNI ? ((sub_ok >> n) & 1) != 0 : ((held >> (4 * n + j)) & 1) != 0);
            s[q][n][j] = sees ? s[q][n][j] * s_scale : -__builtin_inff();
            mx = fmaxf(mx, s[q][n][j]);
          }
        mx = max_over_g(mx);
        const float mu = mx == -__builtin_inff() ? 0.f : mx;
        const float alpha = exp2_hw(m[q] - mu);
        if (__any(mx != m[q])) {
          l[q] *= alpha;
#pragma unroll
          for (int i = 0; i < NA; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j) acc[q][i][j] *= alpha;
        }
        m[q] = mx;
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            s[q][n][j] = exp2_hw(s[q][n][j] - mu);
            l[q] += s[q][n][j];
          }
      }
      if constexpr (!UNI) {  // a row that is not there must not reach the product
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int j = 0; j < 4; ++j)
            if (!((held >> (4 * n + j)) & 1))
#pragma unroll
              for (int u = 0; u < U; ++u) vr[n][j][u] = {};
      }

      // ---- output += weights x values.  A lane's weights of keys that its row
      // does not see are zero, but zero times an infinity or NaN is not: in a
      // tile where rows see different keys (T > 1, the row's last tokens) and
      // such a value is present, each token takes the product on its own, with
      // the values that it does not see replaced by zeros.
      bool apart = false;
      if (MT && key0 + KT > len - p.T + 1) {
        bool odd = false;
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int j = 0; j < 4; ++j)
#pragma unroll
            for (int u = 0; u < U; ++u)
#pragma unroll
              for (int e = 0; e < VW / 2; ++e) {
                if constexpr (BF) {
                  const uint32_t w = bf_pair<KE>(vr[n][j][u], e);
                  odd |= (w & 0x7f80u) == 0x7f80u || (w & 0x7f800000u) == 0x7f800000u;
                } else {
                  const f2 w = f_pair(vr[n][j][u], e);
                  odd |= (__float_as_uint(w[0]) & 0x7f800000u) == 0x7f800000u ||
                         (__float_as_uint(w[1]) & 0x7f800000u) == 0x7f800000u;
                }
              }
        apart = __any(odd);
      }
      if constexpr (BF) {
        constexpr int NP = NT > 1 ? 2 : 1;  // subtiles of one product: 32 keys deep, or 16
#pragma unroll
        for (int a = 0; a < NT; a += NP) {
          bf4 pw[RT][PT][NP];  // the weights' bf16 terms, largest first
#pragma unroll
          for (int q = 0; q < RT; ++q)
#pragma unroll
            for (int i = 0; i < NP; ++i)
#pragma unroll
              for (int j = 0; j < 4; ++j) {
                float rest = s[q][a + i][j];
#pragma unroll
                for (int k = 0; k < PT; ++k) {
                  pw[q][k][i][j] = (__bf16)rest;
                  rest -= (float)pw[q][k][i][j];
                }
              }
#pragma unroll
          for (int u = 0; u < U; ++u)
#pragma unroll
            for (int e2 = 0; e2 < VW / 2; ++e2) {
              uint32_t c[4 * NP];
#pragma unroll
              for (int j = 0; j < 4 * NP; ++j) c[j] = bf_pair<KE>(vr[a + (j >> 2)][j & 3][u], e2);
              // V^T's operand for the pieces' lower or upper elements
              auto dims = [&](const uint32_t* cc, int half, bf4* t) {
#pragma unroll
                for (int i = 0; i < NP; ++i) {
                  uint2 w;
                  w.x = __builtin_amdgcn_perm(cc[4 * i + 1], cc[4 * i], half ? 0x07060302u : 0x05040100u);
                  w.y = __builtin_amdgcn_perm(cc[4 * i + 3], cc[4 * i + 2], half ? 0x07060302u : 0x05040100u);
                  t[i] = __builtin_bit_cast(bf4, w);
                }
              };
              auto product = [&](const bf4* t, int q, int k, f4 in) {
                if constexpr (NP == 2) return mma_k32(in, t[0], t[1], pw[q][k][0], pw[q][k][1]);
                else return mma_k16(in, t[0], pw[q][k][0]);
              };
              if (!MT || !apart) {
                bf4 t[2][NP];
                dims(c, 0, t[0]);
                dims(c, 1, t[1]);
#pragma unroll
                for (int k = PT - 1; k >= 0; --k)  // the terms outside: neighbouring products are independent
#pragma unroll
                  for (int half = 0; half < 2; ++half)
#pragma unroll
                    for (int q = 0; q < RT; ++q) {
                      f4& o = acc[q][u * VW + 2 * e2 + half];
                      o = product(t[half], q, k, o);
                    }
              } else {
#pragma unroll
                for (int half = 0; half < 2; ++half)
#pragma unroll
                  for (int q = 0; q < RT; ++q) {
                    f4& o = acc[q][u * VW + 2 * e2 + half];
                    const f4 in = o;
                    for (int t = 0; t < p.T; ++t) {
                      uint32_t cz[4 * NP];
#pragma unroll
                      for (int j = 0; j < 4 * NP; ++j)
                        cz[j] = key0 + 16 * (a + (j >> 2)) + 4 * g + (j & 3) < len - p.T + t + 1 ? c[j] : 0u;
                      bf4 tz[NP];
                      dims(cz, half, tz);
                      f4 got = in;
#pragma unroll
                      for (int k = PT - 1; k >= 0; --k) got = product(tz, q, k, got);
                      if (t == t_row[q]) o = got;
                    }
                  }
              }
            }
        }
      } else {
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int u = 0; u < U; ++u)
#pragma unroll
            for (int e2 = 0; e2 < VW / 2; ++e2) {
              f2 c[4];
#pragma unroll
              for (int j = 0; j < 4; ++j) c[j] = f_pair(vr[n][j][u], e2);
#pragma unroll
              for (int half = 0; half < 2; ++half)
#pragma unroll
                for (int q = 0; q < RT; ++q) {
                  f4& o = acc[q][u * VW + 2 * e2 + half];
                  if (!MT || !apart) {
                    o = mma_k16(o, f4{c[0][half], c[1][half], c[2][half], c[3][half]}, s[q][n]);
                  } else {
                    const f4 in = o;
                    for (int t = 0; t < p.T; ++t) {
                      f4 z;
#pragma unroll
                      for (int j = 0; j < 4; ++j)
                        z[j] = key0 + 16 * n + 4 * g + j < len - p.T + t + 1 ? c[j][half] : 0.f;
                      const f4 got = mma_k16(in, z, s[q][n]);
                      if (t == t_row[q]) o = got;
                    }
                  }
                }
            }
      }
    }

    // ---- results: the lane's query rows, VW neighbouring dimensions at a time
    asm volatile("" : "+v"(own));
    const int xo = own & 15, go = own >> 4;
    constexpr int SW = VW < 4 ? VW : 4;
    typedef float fs __attribute__((ext_vector_type(SW)));
    typedef IO ios __attribute__((ext_vector_type(SW)));
#pragma unroll
    for (int q = 0; q < RT; ++q) {
      const float lq = sum_over_g(l[q]);
      const int ro = (rt * RT + q) * 16 + xo;
      if (ro < p.R && !whole) {
        const int64_t to = ((int64_t)slot * p.hkv + h) * p.R + ro;
        float* o = p.part_o + to * D + VW * 4 * go;
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
          for (int j = 0; j < 4; ++j)
#pragma unroll
            for (int e = 0; e < VW; e += SW) {
              fs w;
#pragma unroll
              for (int i = 0; i < SW; ++i) w[i] = acc[q][u * VW + e + i][j];
              *reinterpret_cast<fs*>(o + 16 * VW * u + VW * j + e) = w;
            }
        if (go == 0) *reinterpret_cast<f2*>(p.part_ml + to * 2) = f2{m[q], lq};
      } else if (ro < p.R) {
        const int64_t row = ((int64_t)b * p.T + ro / p.group) * p.hq + h * p.group + ro % p.group;
        IO* o = (IO*)p.out + row * D + VW * 4 * go;
        const float inv = attn_inv(p, lq, h);
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
          for (int j = 0; j < 4; ++j)
#pragma unroll
            for (int e = 0; e < VW; e += SW) {
              ios w;
#pragma unroll
              for (int i = 0; i < SW; ++i) w[i] = from_f32<IO>(attn_out(acc[q][u * VW + e + i][j], lq, inv));
              *reinterpret_cast<ios*>(o + 16 * VW * u + VW * j + e) = w;
            }
        if (p.lse && go == 0) p.lse[row] = attn_lse(m[q], lq);
      }
    }
  }
}

template <typename IO, typename KE>
hipError_t launch_attn_t(const AttnParams& p, int d, dim3 grid, hipStream_t stream) {
  const bool uni = p.page_size % 16 == 0;
  const int kind = attn_kind(p.T, p.R);
#define GDN_ATTN_LAUNCH(DD, UNI, KIND) \
  hipLaunchKernelGGL((attn_decode_kernel<IO, KE, DD, UNI, KIND>), grid, dim3(256), 0, stream, p)
#define GDN_ATTN_KINDS(DD, UNI)                     \
  if (kind == 0) GDN_ATTN_LAUNCH(DD, UNI, 0);       \
  else if (kind == 1) GDN_ATTN_LAUNCH(DD, UNI, 1);  \
  else if (kind == 2) GDN_ATTN_LAUNCH(DD, UNI, 2);  \
  else GDN_ATTN_LAUNCH(DD, UNI, 3);
#define GDN_ATTN_CASE(DD)          \
  case DD:                         \
    if (uni) {                     \
      GDN_ATTN_KINDS(DD, true)     \
    } else {                       \
      GDN_ATTN_KINDS(DD, false)    \
    }                              \
    break;
  switch (d) {
    GDN_ATTN_CASE(32)
    GDN_ATTN_CASE(64)
    GDN_ATTN_CASE(128)
    GDN_ATTN_CASE(256)
    default: return hipErrorInvalidValue;
  }
#undef GDN_ATTN_CASE
#undef GDN_ATTN_KINDS
#undef GDN_ATTN_LAUNCH
  return hipGetLastError();
}

hipError_t launch_attn_bf16(const AttnParams& p, int d, dim3 grid, hipStream_t stream);
hipError_t launch_attn_f32(const AttnParams& p, int d, dim3 grid, hipStream_t stream);
hipError_t launch_attn_bf16_e4m3(const AttnParams& p, int d, dim3 grid, hipStream_t stream);
hipError_t launch_attn_f32_e4m3(const AttnParams& p, int d, dim3 grid, hipStream_t stream);

}  // namespace gdn
