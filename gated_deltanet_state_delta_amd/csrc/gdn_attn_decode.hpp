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
// itself: no barrier, and no LDS where pages are whole subtiles (but for block
// scales of odd sizes, and for short tables of block-scaled caches, where the
// four waves of a workgroup share a row and join in LDS: attn_team).  The lengths
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

#include <type_traits>

#include "gdn_kv.hpp"

namespace gdn {

// Block scales: a key's factor enters its score, a value's the weight before
// the product (bf16 queries: the two bf16 terms hold weight times factor to
// 2^-16).  A lane holds four neighbouring keys' scores.
//  * kBlocksWide: blocks of 4, 8 or a multiple of 16 tokens, pages of a multiple
//    of 16: one factor for the four, loaded where it is (the subtile's first
//    factor through a scalar, the lane's own at a fixed offset from there);
//  * kBlocksOne: blocks of one token: four factors, likewise;
//  * kBlocksAny: other sizes: read a tile ahead, a key by each lane, and passed
//    through LDS.
// A tile's codes are half the bytes of bf16, so the work between its loads counts
// twice: the places of 64 subtiles are found at a time, one to a lane, and a tile
// whose keys every row sees has no masks.  4 rows of 131 072 tokens, 4 heads of 128,
// e4m3, a block a page, 537 MB: 89 us = 6.0 TB/s, 98 without these; 64 ragged rows
// up to 8192 tokens, 8 heads of 128, int8, blocks of one token, 572 MB: 105 us = 5.4
// TB/s, where the factors of every key are loaded and multiplied in besides.  Rows
// of 64 bytes stay at 4.2 to 4.5 TB/s, of 32 at 2.7: their pieces of V are 4 and 2
// bytes a lane (VW), so a tile takes 8 and 16 loads of values.
// Whether it is one of the first two.
static inline bool attn_lane_blocks(int page_size, int block) {
  return page_size % 16 == 0 && (block == 1 || block == 4 || block == 8 || block % 16 == 0);
}
constexpr int kBlocksNone = 0, kBlocksWide = 1, kBlocksOne = 2, kBlocksAny = 3;

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
  const float* k_blocks;  // block scales, [n_pages][hkv][nblk]
  const float* v_blocks;
  uint32_t blk_mul, blk_shift;  // j / scale_block, as j / page_size below
  int block, nblk;
  int64_t blk_sp;  // scales of a page
  float* part_o;   // [2 * shares][hkv][R][D]; the workspace's arrays are null when each row is one share
  float* part_ml;  // [2 * shares][hkv][R][2]
  int2* plan;      // [batch]: a row's first share and how many it lies in
  float scale_log2;
  uint32_t page_mul, page_shift;  // j / page_size = (j * page_mul) >> page_shift
  int batch, T, hq, hkv, group, R, ntile, n_pages, page_size, cap, shares;
  int team;        // BS: a workgroup's waves share a row, head and row tile, and join in LDS
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

// Elements 2i and 2i+1 of a piece as two packed bf16 (exact for 8-bit types).
template <typename KE, int N>
__device__ __forceinline__ uint32_t bf_pair(const Raw<N>& r, int i) {
  if constexpr (sizeof(KE) == 2) return r.w[i];
  else if constexpr (std::is_same<KE, i8>::value) {
    const uint32_t w = r.w[i >> 1] >> (16 * (i & 1));
    return __builtin_amdgcn_perm(__float_as_uint((float)(int8_t)(w >> 8)), __float_as_uint((float)(int8_t)w), 0x07060302u);
  } else return __builtin_bit_cast(uint32_t, (i & 1) ? __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(r.w[i >> 1], 1.0f, true)
                                                   : __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(r.w[i >> 1], 1.0f, false));
}
// A pointer into device memory that is the same in all lanes, in scalar registers.
template <typename T> __device__ __forceinline__ const T* uniform_ptr(const T* p) {
  const uint32_t lo = __builtin_amdgcn_readfirstlane((uint32_t)(uint64_t)p), hi = __builtin_amdgcn_readfirstlane((uint32_t)((uint64_t)p >> 32));
  return (const T*)(const __attribute__((address_space(1))) T*)((uint64_t)hi << 32 | lo);
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

// How many waves a SIMD holds and the bytes of K in a wave's tile.  Without
// block scales 64 KiB a CU are in flight either way; fewer and longer streams read HBM faster as
// long as a wave's own work between its loads is short.  bf16 and fp32 rows of
// 256 bytes and more: one wave, 8 KiB (64 ragged rows up to 8192 tokens, 8
// heads of 128, bf16: 172 us; two waves of 4 KiB 175, two of 8 KiB 184, three
// 193).  Shorter rows, and e4m3 whose conversion is VALU work: two waves, 4
// KiB (256 rows, 2 heads of 256, e4m3: 110 us; one wave 131, three 122).
// With block scales heads of 64 and fewer take 2 KiB (64 ragged rows up to 8192
// tokens, 16 heads of 64, int8: 140 us, 4 KiB 159; heads of 128 gain 2% or lose 5%),
// and so half as many bytes are in flight, as with one wave (see attn_shares).
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
constexpr int attn_tile(int es, int d, bool bs) {
  const int keys = (bs && d <= 64 ? 2048 : 8192 / attn_occ(es, d)) / (d * es);
  return keys > 64 ? 64 : keys < 16 ? 16 : keys;
}

template <typename IO, typename KE, int D, int KIND, bool BS>
struct AttnCfg {
  static constexpr int ES = sizeof(KE);
  static constexpr bool BF = ES < 4;
  static constexpr int QT = sizeof(IO) == 2 ? 1 : 3, PT = sizeof(IO) == 2 ? 2 : 3;  // bf16 terms of queries, of weights
  static constexpr int kmin(int a, int b) { return a < b ? a : b; }
  static constexpr int KW = kmin(16 / ES, D / 4), NC = D / (4 * KW);    // elements per K piece, pieces per row and lane
  static constexpr int VW = kmin(16 / ES, D / 16), U = D / (16 * VW);   // the same for V
  static constexpr int OCC = attn_waves(ES, D, KIND), KT = attn_tile(ES, D, BS);
  static constexpr int NT = KT / 16;
  static constexpr int NA = D / 16;  // accumulator tiles
};

// UNI: page_size is a multiple of 16, so every 16-key subtile lies in one
// page: its base is a scalar and rows past the end read zeros through the
// buffer's bound.  Otherwise each key's offset is looked up by one lane and
// passed through LDS.
template <typename IO, typename KE, int D, bool UNI, int KIND, int BS>
__global__ void __launch_bounds__(256, (AttnCfg<IO, KE, D, KIND, BS != kBlocksNone>::OCC)) attn_decode_kernel(AttnParams p) {
  typedef AttnCfg<IO, KE, D, KIND, BS != kBlocksNone> C;
  constexpr int KT = C::KT, NT = C::NT, NC = C::NC, KW = C::KW, VW = C::VW, U = C::U, NA = C::NA, ES = C::ES;
  constexpr int QT = C::QT, PT = C::PT, RT = attn_rows16(KIND, D, sizeof(IO));
  // Where no second wave reads a key, non-temporal loads leave the caches
  // alone (the bf16 batch above, at two waves of 8 KiB: 184 us against 201 with
  // ordinary ones; 64 rows that share all of their 4096 tokens 94 against 85).
  // Block-scaled rows of less than 128 bytes lie in one line with the next head's,
  // which stays in the caches for the wave that takes that head (64 ragged rows of
  // up to 8192 tokens, 16 heads of 64, e4m3: 126 us against 136; of 32: 101 against
  // 129).  In caches of heads first there is no such neighbour and this costs 11%
  // (108 us against 97); a branch on the strides here costs every layout its
  // overlapped loads (133 us), an instantiation for each is not built.
  constexpr bool BF = C::BF, MT = KIND > 0;
  constexpr bool ONCE = (KIND < 2 || (KIND == 2 && RT == 2)) && (BS == kBlocksNone || D * ES >= 128);
  constexpr uint64_t kNone = ~0ull;
  __shared__ uint64_t offs[UNI ? 1 : 4][2][2][UNI ? 1 : KT];  // [wave][parity][K, V][key]
  __shared__ __align__(16) float blocks[BS == kBlocksAny ? 4 : 1][2][BS == kBlocksAny ? KT : 4];  // [wave][K, V][key]: a tile's scales

  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  // Wave -> (share, head, row tile of 16 RT rows).  A workgroup's waves take
  // the row tiles of one (share, head), which read the same keys, or
  // neighbouring heads, whose rows are neighbours in a tokens-first cache;
  // further workgroups of one (share, head) are 8 apart and so on one XCD
  // (workgroups go round the 8).
  const int rtw = p.ntile > 2 ? 4 : p.ntile, nwg = (p.ntile + rtw - 1) / rtw;
  const bool team = BS != kBlocksNone && p.team;
  const int unit = team ? (int)(blockIdx.x / (8 * p.ntile) * 8 + (blockIdx.x & 7))
                        : (int)((blockIdx.x / (8 * nwg) * 8 + (blockIdx.x & 7)) * (4 / rtw)) + wave / rtw;
  const int rt = team ? (int)(blockIdx.x / 8 % p.ntile) : (int)(blockIdx.x / 8 % nwg) * rtw + wave % rtw;
  const int h = unit % p.hkv, share_id = unit / p.hkv;
  if (share_id >= p.shares || rt >= p.ntile) return;
  AttnShare share = attn_share<KT>(p, share_id, lane);  // (team: the row)
  // Uniform values that come from loads, into scalar registers: the walk's addresses follow from them.
  auto uniform = [](int v) { return BS != kBlocksNone ? __builtin_amdgcn_readfirstlane(v) : v; };
  share.n = uniform(share.n);

  const float s_scale = BS != kBlocksNone ? p.scale_log2 : p.scale_log2 * (p.k_scale ? p.k_scale[h] : 1.0f);

  while (share.n > 0) {
    const int b = uniform(share.b), len = uniform(attn_len(p, b)), row_steps = attn_steps<KT>(len), part = (row_steps + 3) >> 2;
    const int at = team ? min(wave * part, row_steps) : uniform(share.at);
    const int take = min(team ? part : share.n, row_steps - at);
    const int c0 = at * KT, c1 = min(len, (at + take) * KT);
    const bool whole = take == row_steps || team;
    const int slot = 2 * share_id + (at == 0);  // of a part: one that begins a row, one that does not
    if (p.plan && at == 0 && h == 0 && rt == 0 && lane == 0)
      p.plan[b] = make_int2(share_id, 1 + (row_steps - take + share.size - 1) / share.size);
    share.n = team ? 0 : share.n - take;
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
    if constexpr (BS != kBlocksNone) tab = uniform_ptr(tab);

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
      for (int n = 0; n < NT; ++n) {
        o.e[n] = tab[page_of(min(key0 + 16 * n, len - 1))];
      }
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
    // The factors of the lane's keys in one subtile (kBlocksWide: one).
    constexpr bool LANE = BS == kBlocksWide || BS == kBlocksOne;
    typedef float Four __attribute__((ext_vector_type(BS == kBlocksOne ? 4 : 1), aligned(4)));
    const int fac_at = BS == kBlocksOne ? 4 * g : p.block >= 16 ? 0 : p.block == 8 ? g >> 1 : g;
    const float* kfac = p.k_blocks + (int64_t)h * p.nblk;
    const float* vfac = p.v_blocks + (int64_t)h * p.nblk;
    // LANE: where the next 64 subtiles lie, one to a lane: byte offsets of their
    // rows in K and V, the place of their first factor, and whether they are held.
    // A tile reads its subtiles' from the lanes: a third of the instructions that
    // finding each by itself in scalar registers took.
    struct { int64_t k, v, f; } spot = {};
    uint64_t spot_ok = 0;
    int spot_ent = 0;  // the table entries of the 64 behind
    auto spot_load = [&](int key) { return tab[page_of(min(key + 16 * lane, len - 1))]; };
    auto spot_fill = [&](int first) {
      const int key = first + 16 * lane, off = key - page_of(key) * p.page_size;
      const bool ok = key < c1 && spot_ent >= 0 && spot_ent < p.n_pages;
      const int64_t e = ok ? spot_ent : 0;
      spot.k = e * p.k_sp + (int64_t)off * p.k_st;
      spot.v = e * p.v_sp + (int64_t)off * p.v_st;
      spot.f = e * p.blk_sp + (int)(((uint64_t)(uint32_t)off * p.blk_mul) >> p.blk_shift);
      spot_ok = __ballot(ok);
      spot_ent = spot_load(first + 1024);
    };
    auto from_lane = [&](int64_t v, int l) {
      const uint32_t lo = __builtin_amdgcn_readlane((uint32_t)v, l), hi = __builtin_amdgcn_readlane((uint32_t)((uint64_t)v >> 32), l);
      return (int64_t)((uint64_t)hi << 32 | lo);
    };
    struct Sub { int64_t k, v, f; int rows; bool ok; };
    struct Subs { Sub s[LANE ? NT : 1]; } sub_cur = {}, sub_next = {};
    auto find_subs = [&](int key0) {
      const int at = (key0 - c0) >> 4 & 63;
      if (at == 0) spot_fill(key0);
      Subs o = {};
#pragma unroll
      for (int n = 0; n < (LANE ? NT : 0); ++n) {
        Sub& s = o.s[n];
        s.ok = (spot_ok >> (at + n)) & 1;
        s.k = from_lane(spot.k, at + n);
        s.v = from_lane(spot.v, at + n);
        s.f = from_lane(spot.f, at + n);
        s.rows = s.ok ? min(16, len - key0 - 16 * n) : 0;
      }
      return o;
    };
    auto rows_at = [&](const char* base, int64_t at, uint32_t st, int rows) {
      return buf_rsrc_n(base + at, rows > 0 ? (uint32_t)(rows - 1) * st + D * ES : 0u);
    };
    auto load_factors = [&](const float* base, int64_t at) { return *reinterpret_cast<const Four*>(base + at + fac_at); };
    auto factor_of = [&](const Four& f, int j) { return f[BS == kBlocksOne ? j : 0]; };
    Four kf[LANE ? NT : 1], vf[LANE ? NT : 1];
    auto issue_k_uni = [&](const Ents& en, const Subs& su, int key0) {
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        if constexpr (LANE) kf[n] = load_factors(kfac, su.s[n].f);
        const auto rs = LANE ? rows_at(kbase, su.s[LANE ? n : 0].k, p.k_st, su.s[LANE ? n : 0].rows) : sub_rsrc(kbase, p.k_sp, p.k_st, en.e[n], key0 + 16 * n);
#pragma unroll
        for (int c = 0; c < NC; ++c) kr[n][c] = raw_buf<KW * ES, ONCE>(rs, x * p.k_st + (4 * KW * c + KW * g) * ES);
      }
    };
    auto issue_v_uni = [&](const Ents& en, const Subs& su, int key0) {
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        if constexpr (LANE) vf[n] = load_factors(vfac, su.s[n].f);
        const auto rs = LANE ? rows_at(vbase, su.s[LANE ? n : 0].v, p.v_st, su.s[LANE ? n : 0].rows) : sub_rsrc(vbase, p.v_sp, p.v_st, en.e[n], key0 + 16 * n);
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

    // kBlocksAny: the factors of a tile, lane l's those of key l: 0 where no key is held.
    struct Scales { float k, v; };
    auto load_scales = [&](int ent, int key0) {
      const int key = key0 + lane;
      Scales o = {0.f, 0.f};
      if (lane < KT && key < len && ent >= 0 && ent < p.n_pages) {
        const int blk = (int)(((uint64_t)(uint32_t)key * p.blk_mul) >> p.blk_shift) - page_of(key) * p.nblk;
        o.k = kfac[ent * p.blk_sp + blk];
        o.v = vfac[ent * p.blk_sp + blk];
      }
      return o;
    };

    Ents ent_cur = {}, ent_next = {};
    Scales sc = {};
    int ent1_next = 0;
    int par = 0;
    if (c0 < c1) {
      if constexpr (UNI) {
        if constexpr (LANE) {
          spot_ent = spot_load(c0);
          sub_cur = find_subs(c0);
        } else {
          ent_cur = load_ents(c0);
        }
        issue_k_uni(ent_cur, sub_cur, c0);
        if constexpr (!LANE) ent_next = load_ents(c0 + KT);
      } else {
        const int ent1 = load_ent1(c0);
        publish(ent1, c0, 0);
        issue_k_any(0);
        if constexpr (BS == kBlocksAny) sc = load_scales(ent1, c0);
        ent1_next = load_ent1(c0 + KT);
      }
    }
    for (int key0 = c0; key0 < c1; key0 += KT) {
      if constexpr (UNI) issue_v_uni(ent_cur, sub_cur, key0);
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
      if constexpr (LANE) {
#pragma unroll
        for (int n = 0; n < NT; ++n) {
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const float f = factor_of(kf[n], j) * s_scale;
#pragma unroll
            for (int q = 0; q < RT; ++q) s[q][n][j] *= f;
          }
        }
      }
      f4 ks[BS == kBlocksAny ? NT : 1], vs[BS == kBlocksAny ? NT : 1];  // of the lane's keys
      if constexpr (BS == kBlocksAny) {
        __builtin_amdgcn_wave_barrier();
        if (lane < KT) {
          blocks[wave][0][lane] = sc.k * s_scale;
          blocks[wave][1][lane] = sc.v;
        }
        __builtin_amdgcn_wave_barrier();
#pragma unroll
        for (int n = 0; n < NT; ++n) {
          ks[n] = *reinterpret_cast<const f4*>(&blocks[wave][0][16 * n + 4 * g]);
          vs[n] = *reinterpret_cast<const f4*>(&blocks[wave][1][16 * n + 4 * g]);
        }
      }
      // The next tile's keys into the registers that the scores just read.
      uint32_t sub_ok = ~0u;
      if constexpr (UNI) {
#pragma unroll
        for (int n = 0; n < NT; ++n)
          if (LANE ? !sub_cur.s[LANE ? n : 0].ok : ent_cur.e[n] < 0 || ent_cur.e[n] >= p.n_pages) sub_ok &= ~(1u << n);
        if constexpr (LANE) sub_next = find_subs(key0 + KT);
        // LANE: always, with no rows past the end, so that the values' wait need not count these loads in
        if (LANE || key0 + KT < c1) issue_k_uni(ent_next, sub_next, key0 + KT);
        if constexpr (LANE) {
          sub_cur = sub_next;
        } else {
          ent_cur = ent_next;
          ent_next = load_ents(key0 + 2 * KT);
        }
      } else {
        par ^= 1;
        if (BS != kBlocksNone || key0 + KT < c1) {
          publish(ent1_next, key0 + KT, par);
          issue_k_any(par);
          if constexpr (BS == kBlocksAny) sc = load_scales(ent1_next, key0 + KT);
          ent1_next = load_ent1(key0 + 2 * KT);
        }
      }

      // ---- masks, running maximum, weights
      // all: every row of the wave sees every key of the tile.
      const bool all = BS != kBlocksNone && key0 + KT <= len - p.T + 1 &&
                       (UNI ? sub_ok == ~0u : __all((held & (~0u >> (32 - 4 * NT))) == ~0u >> (32 - 4 * NT)));
#pragma unroll
      for (int q = 0; q < RT; ++q) {
        float mx = m[q];
        if (all) {
#pragma unroll
          for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              if constexpr (!LANE) s[q][n][j] *= ks[BS == kBlocksAny ? n : 0][j];
              mx = fmaxf(mx, s[q][n][j]);
            }
        } else {
#pragma unroll
          for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              const int key = key0 + 16 * n + 4 * g + j;
              const bool sees = key < lim[q] && (UNI ? ((sub_ok >> n) & 1) != 0 : ((held >> (4 * n + j)) & 1) != 0);
              s[q][n][j] = !sees ? -__builtin_inff() : LANE ? s[q][n][j] : s[q][n][j] * (BS == kBlocksAny ? ks[BS == kBlocksAny ? n : 0][j] : s_scale);
              mx = fmaxf(mx, s[q][n][j]);
            }
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
        if constexpr (BS != kBlocksNone) {
          auto vf_of = [&](int n, int j) { return LANE ? factor_of(vf[LANE ? n : 0], j) : vs[LANE ? 0 : n][j]; };
          if (all) {
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
              for (int j = 0; j < 4; ++j) s[q][n][j] *= vf_of(n, j);
          } else {  // a factor of a key that is not seen may be anything
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
              for (int j = 0; j < 4; ++j) {
                const bool sees = key0 + 16 * n + 4 * g + j < lim[q] &&
                                  (UNI ? ((sub_ok >> n) & 1) != 0 : ((held >> (4 * n + j)) & 1) != 0);
                s[q][n][j] = sees ? s[q][n][j] * vf_of(n, j) : 0.f;
              }
          }
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
      if (MT && !std::is_same<KE, i8>::value && key0 + KT > len - p.T + 1) {
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
              if constexpr (!std::is_same<KE, i8>::value) {
#pragma unroll
                for (int j = 0; j < 4 * NP; ++j) c[j] = bf_pair<KE>(vr[a + (j >> 2)][j & 3][u], e2);
              }
              // V^T's operand for the pieces' lower or upper elements
              auto dims = [&](const uint32_t* cc, int half, bf4* t) {
#pragma unroll
                for (int i = 0; i < NP; ++i) {
                  uint2 w;
                  if constexpr (std::is_same<KE, i8>::value) {  // two keys' elements, converted, into one register (107 us -> 105)
                    auto value = [&](int j) { return __float_as_uint((float)(int8_t)(vr[a + i][j][u].w[e2 >> 1] >> (16 * (e2 & 1) + 8 * half))); };
                    w.x = __builtin_amdgcn_perm(value(1), value(0), 0x07060302u);
                    w.y = __builtin_amdgcn_perm(value(3), value(2), 0x07060302u);
                    t[i] = __builtin_bit_cast(bf4, w);
                    continue;
                  }
                  w.x = __builtin_amdgcn_perm(cc[4 * i + 1], cc[4 * i], half ? 0x07060302u : 0x05040100u);
                  w.y = __builtin_amdgcn_perm(cc[4 * i + 3], cc[4 * i + 2], half ? 0x07060302u : 0x05040100u);
                  t[i] = __builtin_bit_cast(bf4, w);
                }
              };
              auto product = [&](const bf4* t, int q, int k, f4 in) {
                if constexpr (NP == 2) return mma_k32(in, t[0], t[1], pw[q][k][0], pw[q][k][1]);
                else return mma_k16(in, t[0], pw[q][k][0]);
              };
              if (!MT || std::is_same<KE, i8>::value || !apart) {
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

    if constexpr (BS != kBlocksNone) {
      if (team) {
        // The upper half of the waves hand what they have to the lower half, and so
        // on down to wave 0, which writes the results: lane by lane, since a lane
        // holds the same rows and dimensions in all of them.
        __shared__ float parts[2][RT * (NA * 4 + 2)][64];
#pragma unroll
        for (int to = 2; to >= 1; to >>= 1) {
          if (wave >= to && wave < 2 * to) {
            int i = 0;
#pragma unroll
            for (int q = 0; q < RT; ++q) {
              parts[wave - to][i++][lane] = m[q];
              parts[wave - to][i++][lane] = l[q];
#pragma unroll
              for (int n = 0; n < NA; ++n)
#pragma unroll
                for (int j = 0; j < 4; ++j) parts[wave - to][i++][lane] = acc[q][n][j];
            }
          }
          __syncthreads();
          if (wave < to) {
            int i = 0;
#pragma unroll
            for (int q = 0; q < RT; ++q) {
              const float mo = parts[wave][i++][lane], lo = parts[wave][i++][lane];
              const float mx = fmaxf(m[q], mo), mu = mx == -__builtin_inff() ? 0.f : mx;
              const float mine = exp2_hw(m[q] - mu), other = exp2_hw(mo - mu);
              m[q] = mx;
              l[q] = l[q] * mine + lo * other;
#pragma unroll
              for (int n = 0; n < NA; ++n)
#pragma unroll
                for (int j = 0; j < 4; ++j) acc[q][n][j] = acc[q][n][j] * mine + parts[wave][i++][lane] * other;
            }
          }
          __syncthreads();
        }
        if (wave != 0) return;
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

template <typename IO, typename KE, bool BLOCKS = false>
hipError_t launch_attn_t(const AttnParams& p, int d, dim3 grid, hipStream_t stream) {
  const bool wide = p.block != 1;
  const bool uni = BLOCKS ? attn_lane_blocks(p.page_size, p.block) : p.page_size % 16 == 0;
  const int kind = attn_kind(p.T, p.R);
#define GDN_ATTN_LAUNCH(DD, UNI, KIND)                                                                              \
  do {                                                                                                              \
    if constexpr (!BLOCKS)                                                                                          \
      hipLaunchKernelGGL((attn_decode_kernel<IO, KE, DD, UNI, KIND, kBlocksNone>), grid, dim3(256), 0, stream, p);   \
    else if constexpr (!UNI)                                                                                        \
      hipLaunchKernelGGL((attn_decode_kernel<IO, KE, DD, UNI, KIND, kBlocksAny>), grid, dim3(256), 0, stream, p);    \
    else if (wide)                                                                                                  \
      hipLaunchKernelGGL((attn_decode_kernel<IO, KE, DD, UNI, KIND, kBlocksWide>), grid, dim3(256), 0, stream, p);   \
    else                                                                                                            \
      hipLaunchKernelGGL((attn_decode_kernel<IO, KE, DD, UNI, KIND, kBlocksOne>), grid, dim3(256), 0, stream, p); \
  } while (0)
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
// with block scales
hipError_t launch_attn_bf16_e4m3_blocks(const AttnParams& p, int d, dim3 grid, hipStream_t stream);
hipError_t launch_attn_f32_e4m3_blocks(const AttnParams& p, int d, dim3 grid, hipStream_t stream);
hipError_t launch_attn_bf16_i8_blocks(const AttnParams& p, int d, dim3 grid, hipStream_t stream);
hipError_t launch_attn_f32_i8_blocks(const AttnParams& p, int d, dim3 grid, hipStream_t stream);

}  // namespace gdn
