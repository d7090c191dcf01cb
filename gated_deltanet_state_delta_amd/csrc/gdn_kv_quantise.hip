// gdn_kv_quantise.hip -- new tokens' keys and values into the pages of an 8-bit
// cache, the scales of their blocks set on the way.
//
// A block is scale_block tokens of a page and head.  With a the largest finite
// |x| of its new tokens and s_old its scale where the row has older tokens in it:
//   e4m3  s = max(s_old, 2^-126, the smallest power of two with a <= 448 s)
//   int8  s = max(s_old, 2^-126, a * (1 / 127))
//   code  = round(x / s); older codes c become round(c s_old / s) where s grew
//
// HBM-bound streaming for prompts, latency-bound for one token a row.  A group
// of lanes takes one unit -- a block, a head, K or V -- whose new tokens it holds
// in registers between the maximum and the codes, so they are read once.
//
// Measured: 32768 tokens of 8 heads of 128, bf16 to int8 in blocks of 32, 201 MB:
// 43 us = 4.7 TB/s, a large copy's rate; 14000 of 2 heads of 256, fp32 to e4m3 in
// blocks of one token, 72 MB: 22 us = 3.3 TB/s (all 1761 workgroups are on the card
// at once and take one pass each of dependent steps, offsets, length, page, loads,
// maximum, stores; the VALU is busy a third of the time); 256 tokens of 8 heads of
// 128: 4.2 us, where no block's scale grows (see quant_older).
#include <type_traits>

#include "gdn_kv.hpp"

namespace gdn {

struct QuantParams {
  const void* k;
  const void* v;
  int64_t k_st, k_sh, v_st, v_sh;  // elements
  void* kc;
  void* vc;
  int64_t kc_sp, kc_st, kc_sh, vc_sp, vc_st, vc_sh;
  const int32_t* table;
  int64_t table_stride;
  const int32_t* lens;
  const int32_t* cu;
  float* ks;
  float* vs;
  int64_t total, ids;
  int batch, T, hkv, d, n_pages, page_size, cap, block, nblk, run, per_row, log_group, splits, dense;
};

// A row's new tokens in one block: n of them (0: nothing to do) behind `old`
// older ones; K's and V's first new token in the inputs and its place in the
// caches (head 0), and the place of head 0's scale.
struct QuantBlock { uint64_t src[2], dst[2]; int64_t scale; int n, old; };

// Blocks are numbered with room for the most that a row can touch: per_row each
// for equal rows; for packed ones row b's begin at cu[b] / block + 2b (n tokens
// touch at most n / block + 2 blocks).  Offsets that decrease mislead the search;
// no number stands for two blocks then, and none for a block of another row.
template <typename IO>
__device__ __forceinline__ QuantBlock quant_block(const QuantParams& p, int64_t id) {
  QuantBlock o = {};
  int b;
  int64_t i, s0, n;
  if (!p.cu) {
    b = (int)((uint32_t)id / (uint32_t)p.per_row);  // ids < 2^29
    i = id - (int64_t)b * p.per_row;
    s0 = (int64_t)b * p.T;
    n = p.T;
  } else {
    auto offset = [&](int r) { return min(max((int64_t)p.cu[r], (int64_t)0), p.total); };
    int lo = 0, hi = p.batch;
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if ((uint32_t)offset(mid) / (uint32_t)p.block + 2 * (int64_t)mid <= id) lo = mid;
      else hi = mid;
    }
    b = lo;
    s0 = offset(b);
    n = offset(b + 1) - s0;
    i = id - (uint32_t)s0 / (uint32_t)p.block - 2 * (int64_t)b;
  }
  const int64_t end = p.lens[b], first = end - n;  // the row's new positions
  const int64_t p0 = max(first, (int64_t)0), p1 = min(end, (int64_t)p.cap);
  if (i < 0 || p0 >= p1) return o;
  const int64_t edge = ((uint32_t)p0 / (uint32_t)p.block + i) * p.block, from = max(edge, p0), to = min(edge + p.block, p1);
  if (from >= to) return o;
  const int page = (int)((uint32_t)from / (uint32_t)p.page_size), ent = p.table[b * p.table_stride + page];
  if (ent < 0 || ent >= p.n_pages) return o;
  const int64_t tok = s0 + (from - first);
  const int slot = (int)(from - (int64_t)page * p.page_size);
  o.src[0] = (uint64_t)((const IO*)p.k + tok * p.k_st);
  o.src[1] = (uint64_t)((const IO*)p.v + tok * p.v_st);
  o.dst[0] = (uint64_t)((uint8_t*)p.kc + ent * p.kc_sp + slot * p.kc_st);
  o.dst[1] = (uint64_t)((uint8_t*)p.vc + ent * p.vc_sp + slot * p.vc_st);
  o.scale = (int64_t)ent * p.hkv * p.nblk + (uint32_t)slot / (uint32_t)p.block;
  o.n = (int)(to - from);
  o.old = (int)(from - edge);
  return o;
}

// Bits of the largest |x| of a piece (NaN and infinity above every number).
__device__ __forceinline__ uint32_t abs_max(const Piece<__bf16>& x) {
  typedef unsigned short u16x2 __attribute__((ext_vector_type(2)));
  u16x2 m = {0, 0};
#pragma unroll
  for (int i = 0; i < 4; ++i) m = __builtin_elementwise_max(m, __builtin_bit_cast(u16x2, x.r[i] & 0x7fff7fffu));
  return (uint32_t)max(m[0], m[1]) << 16;
}
__device__ __forceinline__ uint32_t abs_max(const Piece<float>& x) {
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) m = max(m, __float_as_uint(x.at(i)) & 0x7fffffffu);
  return m;
}
// The same over its finite values.
template <typename IO>
__device__ __forceinline__ uint32_t finite_max(const Piece<IO>& x) {
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const uint32_t u = __float_as_uint(x.at(i)) & 0x7fffffffu;
    m = max(m, u < 0x7f800000u ? u : 0u);
  }
  return m;
}

// The scale that values up to a (bits of a finite number) need.
template <typename KE> __device__ __forceinline__ float scale_for(uint32_t a);
// a = m 2^e with m in [1, 2): 2^(e - 8), one more where m is over 448 / 256.
template <> __device__ __forceinline__ float scale_for<e4m3>(uint32_t a) {
  return __uint_as_float((uint32_t)max((int)((a + 0x1fffffu) >> 23) - 8, 1) << 23);
}
template <> __device__ __forceinline__ float scale_for<i8>(uint32_t a) {
  return fmaxf(__uint_as_float(a) * (1.0f / 127.0f), 1.17549435e-38f);
}

// 8 quotients x / scale as codes, round to nearest even; inv as normal_rcp.
// SURE: every x is finite and at most the limit times scale.
template <bool SURE, typename X>
__device__ __forceinline__ uint2 quotients(e4m3, const X& x, float scale, float inv) {
  const uint32_t s = __float_as_uint(scale);
  float q[8];
  if ((s & 0x807fffffu) == 0 && s >= 0x00800000u && s <= 0x7e000000u) {  // a power of two: its reciprocal is exact
    const float exact = __uint_as_float(0x7f000000u - s);
#pragma unroll
    for (int i = 0; i < 8; ++i) q[i] = SURE ? x.at(i) * exact : e4m3_clamp(x.at(i) * exact);
  } else {
    e4m3_quotients(x, scale, inv, q);
  }
  return make_uint2(e4m3_pack(q), e4m3_pack(q + 4));
}
// Adding 1.5 * 2^23 rounds to a whole number and leaves its low byte in the low
// bits.  A product with inv is less than 2^-14 off the quotient (up to 127), so
// only one that near to the middle of two numbers can round otherwise.
template <bool SURE, typename X>
__device__ __forceinline__ uint2 quotients(i8, const X& x, float scale, float inv) {
  constexpr float magic = 12582912.0f;
  float w[8], far = 0.f;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float q = x.at(i) * inv;
    w[i] = q + magic;
    far = fmaxf(far, fabsf(q - (w[i] - magic)));
  }
  if (!SURE || far > 0.5f - 0x1p-13f || inv == 0.f) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float q = x.at(i) / scale;
      w[i] = (q != q ? 0.f : __builtin_amdgcn_fmed3f(q, -127.0f, 127.0f)) + magic;
    }
  }
  auto word = [&](int i) {
    return __builtin_amdgcn_perm(__float_as_uint(w[i + 1]), __float_as_uint(w[i]), 0x0c0c0400u) |
           __builtin_amdgcn_perm(__float_as_uint(w[i + 3]), __float_as_uint(w[i + 2]), 0x04000c0cu);
  };
  return make_uint2(word(0), word(4));
}

// 8 older codes as the values that they stand for.
struct Older {
  float v[8];
  __device__ __forceinline__ float at(int i) const { return v[i]; }
  __device__ __forceinline__ Older(e4m3, uint2 c, float scale) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const uint32_t w = i ? c.y : c.x;
      v[4 * i] = __builtin_amdgcn_cvt_f32_fp8(w, 0) * scale;
      v[4 * i + 1] = __builtin_amdgcn_cvt_f32_fp8(w, 1) * scale;
      v[4 * i + 2] = __builtin_amdgcn_cvt_f32_fp8(w, 2) * scale;
      v[4 * i + 3] = __builtin_amdgcn_cvt_f32_fp8(w, 3) * scale;
    }
  }
  __device__ __forceinline__ Older(i8, uint2 c, float scale) {
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = (float)(int8_t)((i < 4 ? c.x : c.y) >> (8 * (i & 3))) * scale;
  }
};

// A block's scale: what its new tokens need (m: bits of their largest finite
// value; nan: of int8 tokens), not below that of its older ones.
template <typename KE>
__device__ __forceinline__ float block_scale(uint32_t m, bool nan, bool has_old, float old) {
  float s = scale_for<KE>(m);
  if (std::is_same<KE, i8>::value && nan) s = __builtin_nanf("");
  if (has_old) s = old != old || s != s ? old + s : fmaxf(s, old);
  return s;
}

constexpr int kQuantRun = 64;  // most blocks of one workgroup
// Most pieces of 8 elements that a lane holds between the maximum and the codes.
template <typename IO> constexpr int kQuantHeld = sizeof(IO) == 2 ? 8 : 4;

// The largest value of the 2^log_group lanes of a group (4 to 64), in the VALU.
__device__ __forceinline__ uint32_t group_max(uint32_t m, int log_group) {
  m = max(m, (uint32_t)dpp_i<0xB1, 0xF>(0, (int)m));  // lanes 1 apart, 2 apart
  m = max(m, (uint32_t)dpp_i<0x4E, 0xF>(0, (int)m));
  if (log_group > 2) m = max(m, (uint32_t)dpp_i<0x141, 0xF>(0, (int)m));  // the halves of 8, of 16
  if (log_group > 3) m = max(m, (uint32_t)dpp_i<0x140, 0xF>(0, (int)m));
  if (log_group > 4) {
    const auto a = __builtin_amdgcn_permlane16_swap(m, m, false, false);
    m = max(a[0], a[1]);
  }
  if (log_group > 5) {
    const auto a = __builtin_amdgcn_permlane32_swap(m, m, false, false);
    m = max(a[0], a[1]);
  }
  return m;
}

// Where a unit's new tokens and codes are.
template <typename IO> struct QuantUnit {
  const IO* src;   // of the first new token
  uint8_t* dst;
  float* scale;
  int np, old;     // pieces of new tokens, older tokens
  bool is_v;
};
// Unit r of a block: K's heads, then V's.
template <typename IO>
__device__ __forceinline__ QuantUnit<IO> quant_unit(const QuantParams& p, const QuantBlock& b, int r, int log_head) {
  QuantUnit<IO> o;
  o.is_v = r >= p.hkv;
  const int h = o.is_v ? r - p.hkv : r;
  o.np = b.n << log_head;
  o.old = b.old;
  int64_t in = (int64_t)h << (log_head + 3), out = in;
  if (!p.dense) {
    in = h * (o.is_v ? p.v_sh : p.k_sh);
    out = h * (o.is_v ? p.vc_sh : p.kc_sh);
  }
  o.src = (const IO*)b.src[o.is_v] + in;
  o.dst = (uint8_t*)b.dst[o.is_v] + out;
  o.scale = (o.is_v ? p.vs : p.ks) + b.scale + (int64_t)h * p.nblk;
  return o;
}

// The older codes of a block whose scale grew from `old` to s: pieces first, first + step, ...
// With one new token a row the group's lanes hold one token, so the older ones follow each
// other, a round trip to memory of 0.5 to 0.6 us each: 256 rows of 8 heads of 128, the token at
// its block's last slot, 4.8 us where the scales stay; where all of them grow, int8, 13 us in
// blocks of 16, 44 in blocks of 64, 161 in blocks of 256 (e4m3: 11, 37, 129).
template <typename IO, typename KE>
__device__ __forceinline__ void quant_older(const QuantUnit<IO>& q, int64_t ct, int log_head, int first, int step, float old, float s) {
  const float inv = normal_rcp(s);
  for (int i = first; i < q.old << log_head; i += step) {
    uint2* c = reinterpret_cast<uint2*>(q.dst + ((i >> log_head) - q.old) * ct + (i & ((1 << log_head) - 1)) * 8);
    *c = quotients<false>(KE{}, Older(KE{}, *c, old), s, inv);
  }
}

// Units that a wave or less holds: groups of 2^log_group lanes of a wave, PPL
// pieces a lane, UB units at a time, so that their loads are in flight together.
// The units of p.run blocks are dealt to p.splits workgroups.
template <typename IO, typename KE, int PPL, int UB>
__global__ void __launch_bounds__(256) kv_quantise_kernel(QuantParams p) {
  __shared__ QuantBlock blocks[kQuantRun];
  const uint32_t chunk = blockIdx.x / (uint32_t)p.splits, split = blockIdx.x - chunk * p.splits;
  const int64_t id0 = (int64_t)chunk * p.run;
  const int nid = (int)min((int64_t)p.run, p.ids - id0);
  if ((int)threadIdx.x < nid) blocks[threadIdx.x] = quant_block<IO>(p, id0 + threadIdx.x);
  __syncthreads();

  const int group = 1 << p.log_group, me = threadIdx.x & (group - 1), groups = 256 >> p.log_group;
  const int log_head = 31 - __builtin_clz(p.d / 8);
  const uint32_t per = 2 * p.hkv;
  // a lane's pieces lie at one place of its head's row, step tokens apart
  const int place = (me & ((1 << log_head) - 1)) * 8, tok = me >> log_head, step = group >> log_head;
  const int64_t src_k = tok * p.k_st + place, src_v = tok * p.v_st + place, dst_k = tok * p.kc_st + place, dst_v = tok * p.vc_st + place;
  // the group's units: one of every groups * splits
  const uint32_t stride = groups * p.splits, stride_b = stride / per, stride_r = stride - stride_b * per;
  const uint32_t first = split * groups + (threadIdx.x >> p.log_group);
  uint32_t at = first / per, r = first - at * per;
  while ((int)at < nid) {
    QuantUnit<IO> q[UB];
    Piece<IO> x[UB][PPL];
    float old[UB];
    uint32_t m[UB];
#pragma unroll
    for (int w = 0; w < UB; ++w) {
      q[w] = quant_unit<IO>(p, blocks[min((int)at, nid - 1)], r, log_head);
      if ((int)at >= nid) q[w].np = 0;
      old[w] = 0.f;
      if (q[w].np > 0 && q[w].old > 0) old[w] = *q[w].scale;
      const int64_t st = q[w].is_v ? p.v_st : p.k_st;
      q[w].src += q[w].is_v ? src_v : src_k;
#pragma unroll
      for (int k = 0; k < PPL; ++k)
        if (k * group + me < q[w].np) x[w][k].load(q[w].src + k * (step * st));
      at += stride_b;
      r += stride_r;
      if (r >= per) {
        r -= per;
        ++at;
      }
    }
#pragma unroll
    for (int w = 0; w < UB; ++w) {
      m[w] = 0;
#pragma unroll
      for (int k = 0; k < PPL; ++k)
        if (k * group + me < q[w].np) m[w] = max(m[w], abs_max(x[w][k]));
      m[w] = group_max(m[w], p.log_group);
    }
#pragma unroll
    for (int w = 0; w < UB; ++w) {
      if (q[w].np == 0) continue;
      const bool odd = m[w] >= 0x7f800000u, nan = m[w] > 0x7f800000u;
      if (odd) {  // the largest finite value instead
        m[w] = 0;
#pragma unroll
        for (int k = 0; k < PPL; ++k)
          if (k * group + me < q[w].np) m[w] = max(m[w], finite_max(x[w][k]));
        m[w] = group_max(m[w], p.log_group);
      }
      const float s = block_scale<KE>(m[w], nan, q[w].old > 0, old[w]);
      if (me == 0) *q[w].scale = s;
      const int64_t ct = q[w].is_v ? p.vc_st : p.kc_st;
      if (q[w].old > 0 && s != old[w]) quant_older<IO, KE>(q[w], ct, log_head, me, group, old[w], s);
      const float inv = normal_rcp(s);
      uint8_t* dst = q[w].dst + (q[w].is_v ? dst_v : dst_k);
#pragma unroll
      for (int k = 0; k < PPL; ++k)
        if (k * group + me < q[w].np)
          *reinterpret_cast<uint2*>(dst + k * (step * ct)) =
              odd ? quotients<false>(KE{}, x[w][k], s, inv) : quotients<true>(KE{}, x[w][k], s, inv);
    }
  }
}

// Larger units: a workgroup takes one at a time, in chunks of what its lanes
// hold; the tokens of a unit of several chunks are read twice.
template <typename IO, typename KE>
__global__ void __launch_bounds__(256) kv_quantise_large_kernel(QuantParams p) {
  constexpr int NR = kQuantHeld<IO>;
  __shared__ QuantBlock block;
  __shared__ uint32_t red[4];
  __shared__ float red_scale[2];
  const uint32_t chunk = blockIdx.x / (uint32_t)p.splits, split = blockIdx.x - chunk * p.splits;
  const int64_t id0 = (int64_t)chunk * p.run;
  const int nid = (int)min((int64_t)p.run, p.ids - id0), me = threadIdx.x;
  const int log_head = 31 - __builtin_clz(p.d / 8), place = (me & ((1 << log_head) - 1)) * 8;
  auto over_group = [&](uint32_t m) {
    m = group_max(m, 6);
    __syncthreads();  // the last values are read
    if ((me & 63) == 0) red[me >> 6] = m;
    __syncthreads();
    return max(max(red[0], red[1]), max(red[2], red[3]));
  };
  int par = 0;  // of the units that the workgroup has taken
  for (int u = split; u < nid * 2 * p.hkv; u += p.splits) {
    const int at = (uint32_t)u / (uint32_t)(2 * p.hkv), r = u - at * 2 * p.hkv;
    __syncthreads();  // the last unit's block is read
    if (me == 0 && (r < p.splits || u == (int)split)) block = quant_block<IO>(p, id0 + at);
    __syncthreads();
    const QuantUnit<IO> q = quant_unit<IO>(p, block, r, log_head);
    if (q.np == 0) continue;
    const int64_t st = q.is_v ? p.v_st : p.k_st, ct = q.is_v ? p.vc_st : p.kc_st;
    const int chunks = (q.np + 256 * NR - 1) / (256 * NR);
    Piece<IO> x[NR];
    auto load = [&](int c) {
#pragma unroll
      for (int k = 0; k < NR; ++k) {
        const int i = (c * NR + k) * 256 + me;
        if (i < q.np) x[k].load(q.src + (i >> log_head) * st + place);
      }
    };
    auto held_max = [&](int c, bool finite) {
      uint32_t m = 0;
#pragma unroll
      for (int k = 0; k < NR; ++k)
        if ((c * NR + k) * 256 + me < q.np) m = max(m, finite ? finite_max(x[k]) : abs_max(x[k]));
      return m;
    };
    if (q.old > 0 && me == 0) red_scale[par] = *q.scale;
    uint32_t m = 0;
    for (int c = 0; c < chunks; ++c) {
      load(c);
      m = max(m, held_max(c, false));
    }
    m = over_group(m);
    const bool odd = m >= 0x7f800000u, nan = m > 0x7f800000u;
    if (odd) {  // the largest finite value instead
      m = 0;
      for (int c = 0; c < chunks; ++c) {
        load(c);
        m = max(m, held_max(c, true));
      }
      m = over_group(m);
    }
    const float old = q.old > 0 ? red_scale[par] : 0.f;
    par ^= 1;
    const float s = block_scale<KE>(m, nan, q.old > 0, old), inv = normal_rcp(s);
    if (me == 0) *q.scale = s;
    if (q.old > 0 && s != old) quant_older<IO, KE>(q, ct, log_head, me, 256, old, s);
    for (int c = chunks - 1; c >= 0; --c) {  // the last chunk is in registers
      if (odd || c < chunks - 1) load(c);
#pragma unroll
      for (int k = 0; k < NR; ++k) {
        const int i = (c * NR + k) * 256 + me;
        if (i < q.np)
          *reinterpret_cast<uint2*>(q.dst + (i >> log_head) * ct + place) =
              odd ? quotients<false>(KE{}, x[k], s, inv) : quotients<true>(KE{}, x[k], s, inv);
      }
    }
  }
}

// What a kernel takes at a time: pieces a lane, units.
struct QuantShape { int ppl, ub; };
static QuantShape quant_shape(int64_t pieces, int held) {  // ppl 0: the workgroup takes a unit
  return pieces <= 64 ? QuantShape{1, 4} : pieces <= 128 ? QuantShape{2, 2} : pieces <= 256 ? QuantShape{4, 1} :
         pieces <= 64 * held ? QuantShape{8, 1} : QuantShape{0, 1};
}
template <typename IO, typename KE>
static void launch_quantise(const QuantParams& p, int ppl, dim3 grid, hipStream_t stream) {
  if (ppl == 1) hipLaunchKernelGGL((kv_quantise_kernel<IO, KE, 1, 4>), grid, dim3(256), 0, stream, p);
  else if (ppl == 2) hipLaunchKernelGGL((kv_quantise_kernel<IO, KE, 2, 2>), grid, dim3(256), 0, stream, p);
  else if (ppl == 4) hipLaunchKernelGGL((kv_quantise_kernel<IO, KE, 4, 1>), grid, dim3(256), 0, stream, p);
  else if (ppl == 0) hipLaunchKernelGGL((kv_quantise_large_kernel<IO, KE>), grid, dim3(256), 0, stream, p);
  else if constexpr (kQuantHeld<IO> == 8)
    hipLaunchKernelGGL((kv_quantise_kernel<IO, KE, 8, 1>), grid, dim3(256), 0, stream, p);
}

hipError_t launch_kv_quantise(const gdn_kv_append_args& a, hipStream_t stream) {
  QuantParams p;
  p.k = a.k;
  p.v = a.v;
  p.k_st = a.k_stride_token;
  p.k_sh = a.k_stride_head;
  p.v_st = a.v_stride_token;
  p.v_sh = a.v_stride_head;
  p.kc = a.k_cache;
  p.vc = a.v_cache;
  p.kc_sp = a.kc_stride_page;
  p.kc_st = a.kc_stride_token;
  p.kc_sh = a.kc_stride_head;
  p.vc_sp = a.vc_stride_page;
  p.vc_st = a.vc_stride_token;
  p.vc_sh = a.vc_stride_head;
  p.table = a.page_table;
  p.table_stride = a.page_table_stride;
  p.lens = a.lens;
  p.cu = a.cu_seqlens;
  p.ks = a.k_block_scale;
  p.vs = a.v_block_scale;
  p.total = a.total_tokens;
  p.batch = a.batch;
  p.T = a.cu_seqlens ? 0 : (int)(a.total_tokens / a.batch);
  p.hkv = a.hkv;
  p.d = a.d;
  p.n_pages = a.n_pages;
  p.page_size = a.page_size;
  p.cap = a.max_pages * a.page_size;
  p.block = a.scale_block;
  p.nblk = a.page_size / a.scale_block;
  // T tokens touch (T + block - 2) / block + 1 blocks at most
  p.per_row = a.cu_seqlens ? 0 : (int)(((int64_t)p.T + p.block - 2) / p.block) + 1;
  p.ids = a.cu_seqlens ? a.total_tokens / p.block + 2 * (int64_t)a.batch : (int64_t)a.batch * p.per_row;
  p.dense = a.k_stride_head == a.d && a.v_stride_head == a.d && a.kc_stride_head == a.d && a.vc_stride_head == a.d;
  // Pieces of a unit, and the lanes that take it: as many as it has pieces, up to a wave.  Packed rows may fill
  // their blocks, and are taken to: 256 packed single tokens of 8 heads of 128 in blocks of 64 29 us, the same
  // tokens as equal rows 4.6.
  const int64_t tokens = !a.cu_seqlens && p.T < p.block ? p.T : p.block, pieces = tokens * (a.d / 8);
  p.log_group = 2;
  while (p.log_group < 6 && (1 << p.log_group) < pieces) ++p.log_group;
  const QuantShape shape = quant_shape(pieces, a.io_dtype == GDN_BF16 ? kQuantHeld<__bf16> : kQuantHeld<float>);
  // Units per workgroup: two rounds of what it takes at a time (32768 tokens of
  // 8 heads of 128, bf16 to int8 in blocks of 32: 43.4 us; one round 46, four
  // 47), one where the card holds all workgroups of one at once; but whole blocks
  // only from 1024 workgroups on, and whole rounds of them.
  const int64_t units = 2 * a.hkv, round = shape.ppl == 0 ? 1 : shape.ub * (256 >> p.log_group);
  const int64_t full = a.cu_seqlens ? a.total_tokens / p.block + a.batch : p.ids, most = p.ids / 1024;  // blocks that there are
  const int64_t share = shape.ppl == 0 ? 1 : full * units > 2048 * round ? 2 * round : round;
  int64_t run = share / units < most ? share / units : most;
  if (run * units > round) run = run * units / round * round / units;
  run = run < 1 ? 1 : run > kQuantRun ? kQuantRun : run;
  int64_t splits = (units * run + share - 1) / share;
  if ((p.ids + run - 1) / run > (1 << 23) / splits) {  // a grid's limit; ids < 2^29
    run = kQuantRun;
    splits = 1;
  }
  p.run = (int)run;
  p.splits = (int)splits;
  const dim3 grid((unsigned)((p.ids + run - 1) / run * splits));
  if (a.cache_dtype == GDN_E4M3) {
    if (a.io_dtype == GDN_BF16) launch_quantise<__bf16, e4m3>(p, shape.ppl, grid, stream);
    else launch_quantise<float, e4m3>(p, shape.ppl, grid, stream);
  } else {
    if (a.io_dtype == GDN_BF16) launch_quantise<__bf16, i8>(p, shape.ppl, grid, stream);
    else launch_quantise<float, i8>(p, shape.ppl, grid, stream);
  }
  return hipGetLastError();
}

}  // namespace gdn
