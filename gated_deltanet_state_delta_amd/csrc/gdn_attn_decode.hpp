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
// Work split: a workgroup of 4 waves takes one (row b, key-value head,
// 16 query rows, range of keys); its waves take tiles of KT keys in turn and
// join through LDS at the end.  With more than one range per row, each
// writes (m, l, unnormalised output) to the workspace and
// attn_join_kernel joins them in a fixed order.
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
// the weights to 2^-17; the second MFMA is free next to the loads.
#pragma once

#include "gdn_device.hpp"
#include "gdn_kernels.hpp"

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
  float* part_o;   // [batch * hkv][nsplit][R][D], nsplit > 1 only
  float* part_ml;  // [batch * hkv][nsplit][R][2]
  float scale_log2;
  uint32_t page_mul, page_shift;  // j / page_size = (j * page_mul) >> page_shift
  int batch, T, hq, hkv, group, R, ntile, n_pages, page_size, cap, nsplit, min_chunk;
};

// Keys of one range of a row of len tokens: the row's length over nsplit,
// rounded up to whole tiles of 64, at least min_chunk.
__device__ __forceinline__ int attn_chunk(const AttnParams& p, int len) {
  const int c = (((len + p.nsplit - 1) / p.nsplit) + 63) & ~63;
  return max(c, p.min_chunk);
}
__device__ __forceinline__ int attn_len(const AttnParams& p, int b) {
  const int len = p.lens[b];
  return p.n_pages == 0 ? 0 : min(max(len, 0), p.cap);
}

// Four outputs at element `at`: the weighted sum over the weights' sum.  A
// row that sees nothing (maximum -inf) is zero.
template <typename IO>
__device__ __forceinline__ void attn_store(const AttnParams& p, int64_t at, f4 o, float m, float l, int h) {
  const float inv = (p.v_scale ? p.v_scale[h] : 1.0f) / l;
#pragma unroll
  for (int i = 0; i < 4; ++i) o[i] = m == -__builtin_inff() ? 0.f : o[i] * inv;
  if constexpr (sizeof(IO) == 2)
    *reinterpret_cast<bf4*>((__bf16*)p.out + at) = bf4{(__bf16)o[0], (__bf16)o[1], (__bf16)o[2], (__bf16)o[3]};
  else
    *reinterpret_cast<f4*>((float*)p.out + at) = o;
}
// Natural log of the weights' sum, from the maximum and sum in units of log2.
__device__ __forceinline__ float attn_lse(float m, float l) {
  return m == -__builtin_inff() ? m : (m + __builtin_amdgcn_logf(l)) * 0.6931471805599453f;
}

// N raw bytes of a row piece, as dwords (2 bytes sit in the low half).
template <int N> struct Raw { uint32_t w[(N + 3) / 4]; };

template <int N>
__device__ __forceinline__ Raw<N> raw_buf(__amdgpu_buffer_rsrc_t r, uint32_t voff) {
  Raw<N> o;
  if constexpr (N == 16) {
    const u32x4 t = __builtin_amdgcn_raw_buffer_load_b128(r, voff, 0, 0);
    o.w[0] = t[0]; o.w[1] = t[1]; o.w[2] = t[2]; o.w[3] = t[3];
  } else if constexpr (N == 8) {
    const auto t = __builtin_amdgcn_raw_buffer_load_b64(r, voff, 0, 0);
    o.w[0] = t[0]; o.w[1] = t[1];
  } else if constexpr (N == 4) {
    o.w[0] = __builtin_amdgcn_raw_buffer_load_b32(r, voff, 0, 0);
  } else {
    o.w[0] = (uint16_t)__builtin_amdgcn_raw_buffer_load_b16(r, voff, 0, 0);
  }
  return o;
}
template <int N>
__device__ __forceinline__ Raw<N> raw_load(const char* p) {
  Raw<N> o;
  if constexpr (N == 16) {
    const u32x4 t = *reinterpret_cast<const u32x4*>(p);
    o.w[0] = t[0]; o.w[1] = t[1]; o.w[2] = t[2]; o.w[3] = t[3];
  } else if constexpr (N == 8) {
    const uint2 t = *reinterpret_cast<const uint2*>(p);
    o.w[0] = t.x; o.w[1] = t.y;
  } else if constexpr (N == 4) {
    o.w[0] = *reinterpret_cast<const uint32_t*>(p);
  } else {
    o.w[0] = *reinterpret_cast<const uint16_t*>(p);
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
// Elements 2i and 2i+1 as floats.
template <typename KE, int N>
__device__ __forceinline__ f2 f_pair(const Raw<N>& r, int i) {
  if constexpr (sizeof(KE) == 4) return f2{__uint_as_float(r.w[2 * i]), __uint_as_float(r.w[2 * i + 1])};
  else return (i & 1) ? __builtin_amdgcn_cvt_pk_f32_fp8(r.w[i >> 1], true) : __builtin_amdgcn_cvt_pk_f32_fp8(r.w[i >> 1], false);
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

// IO: type of q and out, and of the products (bf16 or fp32); KE: cache element.
template <typename IO, typename KE, int D>
struct AttnCfg {
  static constexpr int ES = sizeof(KE);
  static constexpr bool BF = sizeof(IO) == 2;
  static constexpr int kmin(int a, int b) { return a < b ? a : b; }
  static constexpr int KW = kmin(16 / ES, D / 4), NC = D / (4 * KW);    // elements per K piece, pieces per row and lane
  static constexpr int VW = kmin(16 / ES, D / 16), U = D / (16 * VW);   // the same for V
  // Keys per wave tile: about 8 KiB of K, a multiple of the products' depth.
  static constexpr int KTW = 8192 / (D * ES);
  static constexpr int KT = KTW > 64 ? 64 : KTW < (BF ? 32 : 16) ? (BF ? 32 : 16) : KTW;
  static constexpr int NT = KT / 16;
  static constexpr int NA = D / 16;  // accumulator tiles
  static constexpr int LDO = D + 4;  // row pitch of the join buffer: rows 4 banks apart
};

// UNI: page_size is a multiple of 16, so every 16-key subtile lies in one
// page: its base is a scalar and rows past the end read zeros through the
// buffer's bound.  Otherwise each key's offset is looked up by one lane and
// passed through LDS.
template <typename IO, typename KE, int D, bool UNI>
__global__ void __launch_bounds__(256) attn_decode_kernel(AttnParams p) {
  typedef AttnCfg<IO, KE, D> C;
  constexpr int KT = C::KT, NT = C::NT, NC = C::NC, KW = C::KW, VW = C::VW, U = C::U, NA = C::NA, ES = C::ES;
  constexpr bool BF = C::BF;
  constexpr uint64_t kNone = ~0ull;
  __shared__ __align__(16) float red[16 * C::LDO];
  __shared__ float red_m[4][16], red_l[4][16];
  __shared__ uint64_t offs[UNI ? 1 : 4][2][2][UNI ? 1 : KT];  // [wave][parity][K, V][key]

  const int lane = threadIdx.x & 63, x = lane & 15, g = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  // Workgroup -> (unit, row tile): the row tiles of a unit, which read the
  // same keys, are 8 apart and so on one XCD (workgroups go round the 8).
  const int nt8 = p.ntile * 8, blk = blockIdx.x;
  const int unit = (blk / nt8) * 8 + (blk & 7), rt = (blk % nt8) >> 3;
  if (unit >= p.batch * p.hkv * p.nsplit) return;
  const int h = unit % p.hkv, split = (unit / p.hkv) % p.nsplit, b = unit / (p.hkv * p.nsplit);
  const int len = attn_len(p, b), chunk = attn_chunk(p, len);
  const int64_t c0l = (int64_t)split * chunk;
  if (split > 0 && c0l >= len) return;  // the join skips the same ranges
  const int c0 = (int)c0l, c1 = min(len, c0 + chunk);

  // This lane's query row: row r is token r / group, query head h*group + r % group.
  const int r = rt * 16 + x;
  const bool row_ok = r < p.R;
  const int t_row = row_ok ? r / p.group : 0, hq_row = h * p.group + (row_ok ? r % p.group : 0);
  const int lim = row_ok ? max(0, min(len, len - p.T + t_row + 1)) : 0;  // it sees keys below lim
  const char* qp = (const char*)p.q + b * p.q_sb + t_row * p.q_st + hq_row * p.q_sh;
  const float s_scale = p.scale_log2 * (p.k_scale ? p.k_scale[h] : 1.0f);

  bf8 qb[BF ? D / 32 : 1];
  float qf[BF ? 1 : D / 4];
#pragma unroll
  for (int c = 0; c < NC; ++c) {
#pragma unroll
    for (int w = 0; w < KW; w += BF ? 8 : 4) {
      const int d = 4 * KW * c + KW * g + w, i = (c * KW + w);
      if constexpr (BF) {
        bf8 t = {};
        if (row_ok) t = *reinterpret_cast<const bf8*>(qp + d * 2);
        qb[i / 8] = t;
      } else {
        f4 t = {};
        if (row_ok) t = *reinterpret_cast<const f4*>(qp + d * 4);
#pragma unroll
        for (int e = 0; e < 4; ++e) qf[i + e] = t[e];
      }
    }
  }

  const char* kbase = (const char*)p.k + h * p.k_sh;
  const char* vbase = (const char*)p.v + h * p.v_sh;
  const int32_t* tab = p.table + b * p.table_stride;

  f4 acc[NA];
#pragma unroll
  for (int i = 0; i < NA; ++i) acc[i] = f4{0.f, 0.f, 0.f, 0.f};
  float m = -__builtin_inff(), l = 0.f;

  Raw<KW * ES> kr[NT][NC];
  Raw<VW * ES> vr[NT][4][U];

  const int first = c0 + wave * KT;
  constexpr int STEP = 4 * KT;

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
      for (int c = 0; c < NC; ++c) kr[n][c] = raw_buf<KW * ES>(rs, x * p.k_st + (4 * KW * c + KW * g) * ES);
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
          vr[n][j][u] = raw_buf<VW * ES>(rs, (4 * g + j) * p.v_st + (16 * VW * u + VW * x) * ES);
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
      for (int c = 0; c < NC; ++c) kr[n][c] = raw_load<KW * ES>(src + (4 * KW * c + KW * g) * ES);
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
        for (int u = 0; u < U; ++u) vr[n][j][u] = raw_load<VW * ES>(src + (16 * VW * u + VW * x) * ES);
      }
  };

  Ents ent_cur = {}, ent_next = {};
  int ent1_next = 0;
  int par = 0;
  if (first < c1) {
    if constexpr (UNI) {
      ent_cur = load_ents(first);
      issue_k_uni(ent_cur, first);
      ent_next = load_ents(first + STEP);
    } else {
      publish(load_ent1(first), first, 0);
      issue_k_any(0);
      ent1_next = load_ent1(first + STEP);
    }
  }
  for (int key0 = first; key0 < c1; key0 += STEP) {
    if constexpr (UNI) issue_v_uni(ent_cur, key0);
    else issue_v_any(par);

    // ---- scores of the tile
    f4 s[NT];
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      s[n] = f4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int c = 0; c < NC; ++c) {
        if constexpr (BF) {
#pragma unroll
          for (int w = 0; w < KW; w += 8) {
            u32x4 t;
#pragma unroll
            for (int i = 0; i < 4; ++i) t[i] = bf_pair<KE>(kr[n][c], w / 2 + i);
            s[n] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf8, t), qb[(c * KW + w) / 8], s[n], 0, 0, 0);
          }
        } else {
#pragma unroll
          for (int i = 0; i < KW / 2; ++i) {
            const f2 t = f_pair<KE>(kr[n][c], i);
            s[n] = __builtin_amdgcn_mfma_f32_16x16x4f32(t[0], qf[c * KW + 2 * i], s[n], 0, 0, 0);
            s[n] = __builtin_amdgcn_mfma_f32_16x16x4f32(t[1], qf[c * KW + 2 * i + 1], s[n], 0, 0, 0);
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
      if (key0 + STEP < c1) issue_k_uni(ent_next, key0 + STEP);
      ent_cur = ent_next;
      ent_next = load_ents(key0 + 2 * STEP);
    } else {
      par ^= 1;
      if (key0 + STEP < c1) {
        publish(ent1_next, key0 + STEP, par);
        issue_k_any(par);
        ent1_next = load_ent1(key0 + 2 * STEP);
      }
    }

    // ---- masks, running maximum, weights
    float mx = m;
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int key = key0 + 16 * n + 4 * g + j;
        const bool sees = key < lim && (UNI ? ((sub_ok >> n) & 1) != 0 : ((held >> (4 * n + j)) & 1) != 0);
        s[n][j] = sees ? s[n][j] * s_scale : -__builtin_inff();
        mx = fmaxf(mx, s[n][j]);
      }
    mx = max_over_g(mx);
    const float mu = mx == -__builtin_inff() ? 0.f : mx;
    const float alpha = exp2_hw(m - mu);
    if (__any(mx != m)) {
      l *= alpha;
#pragma unroll
      for (int i = 0; i < NA; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) acc[i][j] *= alpha;
    }
    m = mx;
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        s[n][j] = exp2_hw(s[n][j] - mu);
        l += s[n][j];
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
    if (p.T > 1 && key0 + KT > len - p.T + 1) {
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
                const f2 w = f_pair<KE>(vr[n][j][u], e);
                odd |= (__float_as_uint(w[0]) & 0x7f800000u) == 0x7f800000u ||
                       (__float_as_uint(w[1]) & 0x7f800000u) == 0x7f800000u;
              }
            }
      apart = __any(odd);
    }
    if constexpr (BF) {
#pragma unroll
      for (int a = 0; a < NT; a += 2) {
        bf8 ph, pl;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const float w = s[a + (j >> 2)][j & 3];
          ph[j] = (__bf16)w;
          pl[j] = (__bf16)(w - (float)ph[j]);
        }
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
          for (int e2 = 0; e2 < VW / 2; ++e2) {
            uint32_t c[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) c[j] = bf_pair<KE>(vr[a + (j >> 2)][j & 3][u], e2);
            auto product = [&](const uint32_t* cc, int half, f4 in) {
              u32x4 t;
#pragma unroll
              for (int i = 0; i < 4; ++i)
                t[i] = __builtin_amdgcn_perm(cc[2 * i + 1], cc[2 * i], half ? 0x07060302u : 0x05040100u);
              in = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf8, t), ph, in, 0, 0, 0);
              return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf8, t), pl, in, 0, 0, 0);
            };
#pragma unroll
            for (int half = 0; half < 2; ++half) {
              f4& o = acc[u * VW + 2 * e2 + half];
              if (__builtin_expect(!apart, 1)) {
                o = product(c, half, o);
              } else {
                const f4 in = o;
                for (int t = 0; t < p.T; ++t) {
                  uint32_t cz[8];
#pragma unroll
                  for (int j = 0; j < 8; ++j)
                    cz[j] = key0 + 16 * (a + (j >> 2)) + 4 * g + (j & 3) < len - p.T + t + 1 ? c[j] : 0u;
                  const f4 got = product(cz, half, in);
                  if (t == t_row) o = got;
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
            for (int j = 0; j < 4; ++j) c[j] = f_pair<KE>(vr[n][j][u], e2);
#pragma unroll
            for (int half = 0; half < 2; ++half) {
              f4& o = acc[u * VW + 2 * e2 + half];
              if (__builtin_expect(!apart, 1)) {
                o = mma_k16(o, f4{c[0][half], c[1][half], c[2][half], c[3][half]}, s[n]);
              } else {
                const f4 in = o;
                for (int t = 0; t < p.T; ++t) {
                  f4 z;
#pragma unroll
                  for (int j = 0; j < 4; ++j)
                    z[j] = key0 + 16 * n + 4 * g + j < len - p.T + t + 1 ? c[j][half] : 0.f;
                  const f4 got = mma_k16(in, z, s[n]);
                  if (t == t_row) o = got;
                }
              }
            }
          }
    }
  }

  // ---- join the waves: a common maximum, then the outputs added in wave order
  l = sum_over_g(l);
  if (g == 0) {
    red_m[wave][x] = m;
    red_l[wave][x] = l;
  }
  __syncthreads();
  float M = red_m[0][x];
#pragma unroll
  for (int w = 1; w < 4; ++w) M = fmaxf(M, red_m[w][x]);
  const float Mu = M == -__builtin_inff() ? 0.f : M;
  float L = 0.f;
#pragma unroll
  for (int w = 0; w < 4; ++w) L += red_l[w][x] * exp2_hw(red_m[w][x] - Mu);
  const float f = exp2_hw(m - Mu);
  // acc tile u*VW + e, register j: dimension 16 VW u + VW (4g + j) + e of row x
  for (int w = 0; w < 4; ++w) {
    if (wave == w) {
#pragma unroll
      for (int u = 0; u < U; ++u)
#pragma unroll
        for (int j = 0; j < 4; ++j)
#pragma unroll
          for (int e = 0; e < VW; ++e) {
            float* o = &red[x * C::LDO + 16 * VW * u + VW * (4 * g + j) + e];
            const float add = acc[u * VW + e][j] * f;
            *o = w == 0 ? add : *o + add;
          }
    }
    __syncthreads();
  }
  // ---- results: row rr of this tile by 16 threads, 4 dimensions at a time
  if (wave == 0 && g == 0) red_l[0][x] = L, red_m[0][x] = M;
  __syncthreads();
  const int rr = threadIdx.x >> 4, ro = rt * 16 + rr;
  if (ro >= p.R) return;
  const float Lr = red_l[0][rr], Mr = red_m[0][rr];
  const int sub = threadIdx.x & 15;
  if (p.nsplit > 1) {
    const int64_t at = ((int64_t)(b * p.hkv + h) * p.nsplit + split) * p.R + ro;
    for (int d = sub * 4; d < D; d += 64)
      *reinterpret_cast<f4*>(p.part_o + at * D + d) = *reinterpret_cast<const f4*>(&red[rr * C::LDO + d]);
    if (sub == 0) {
      p.part_ml[at * 2] = Mr;
      p.part_ml[at * 2 + 1] = Lr;
    }
    return;
  }
  const int t_out = ro / p.group, h_out = h * p.group + ro % p.group;
  const int64_t row = ((int64_t)b * p.T + t_out) * p.hq + h_out;
  for (int d = sub * 4; d < D; d += 64)
    attn_store<IO>(p, row * D + d, *reinterpret_cast<const f4*>(&red[rr * C::LDO + d]), Mr, Lr, h);
  if (p.lse && sub == 0) p.lse[row] = attn_lse(Mr, Lr);
}

template <typename IO, typename KE>
hipError_t launch_attn_t(const AttnParams& p, int d, dim3 grid, hipStream_t stream) {
  const bool uni = p.page_size % 16 == 0;
#define GDN_ATTN_CASE(DD)                                                                                  \
  case DD:                                                                                                 \
    if (uni)                                                                                               \
      hipLaunchKernelGGL((attn_decode_kernel<IO, KE, DD, true>), grid, dim3(256), 0, stream, p);           \
    else                                                                                                   \
      hipLaunchKernelGGL((attn_decode_kernel<IO, KE, DD, false>), grid, dim3(256), 0, stream, p);          \
    break;
  switch (d) {
    GDN_ATTN_CASE(32)
    GDN_ATTN_CASE(64)
    GDN_ATTN_CASE(128)
    GDN_ATTN_CASE(256)
    default: return hipErrorInvalidValue;
  }
#undef GDN_ATTN_CASE
  return hipGetLastError();
}

hipError_t launch_attn_bf16(const AttnParams& p, int d, dim3 grid, hipStream_t stream);
hipError_t launch_attn_f32(const AttnParams& p, int d, dim3 grid, hipStream_t stream);
hipError_t launch_attn_bf16_e4m3(const AttnParams& p, int d, dim3 grid, hipStream_t stream);
hipError_t launch_attn_f32_e4m3(const AttnParams& p, int d, dim3 grid, hipStream_t stream);

}  // namespace gdn
