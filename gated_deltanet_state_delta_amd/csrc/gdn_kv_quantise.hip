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
  int batch, T, hkv, d, n_pages, page_size, cap, block, nblk, run, per_row, log_group;
};

// A row's new tokens in one block: n of them from packed token tok on, behind
// `old` older ones; the first goes to `slot` of page `ent`.
struct QuantBlock { int64_t tok; int n, old, ent, slot; };

// Blocks are numbered with room for the most that a row can touch: per_row each
// for equal rows; for packed ones row b's begin at cu[b] / block + 2b (n tokens
// touch at most n / block + 2 blocks).  Offsets that decrease mislead the search;
// no number stands for two blocks then, and none for a block of another row.
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
  o.tok = s0 + (from - first);
  o.n = (int)(to - from);
  o.old = (int)(from - edge);
  o.ent = ent;
  o.slot = (int)(from - (int64_t)page * p.page_size);
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

// 8 quotients x / scale as codes, round to nearest even; inv as in e4m3_quotients.
template <typename X>
__device__ __forceinline__ uint2 quotients(e4m3, const X& x, float scale, float inv) {
  const uint32_t s = __float_as_uint(scale);
  if ((s & 0x807fffffu) == 0 && s >= 0x00800000u && s <= 0x7e000000u) {  // a power of two: its reciprocal is exact
    const float exact = __uint_as_float(0x7f000000u - s);
    float q[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) q[i] = e4m3_clamp(x.at(i) * exact);
    return e4m3_pack(q);
  }
  return e4m3_quotients(x, scale, inv);
}
// Adding 1.5 * 2^23 rounds to a whole number and leaves its low byte in the low
// bits.  A product with inv is less than 2^-14 off the quotient (up to 127), so
// only one that near to the middle of two numbers can round otherwise.
template <typename X>
__device__ __forceinline__ uint2 quotients(i8, const X& x, float scale, float inv) {
  constexpr float magic = 12582912.0f;
  float q[8];
  bool near = inv == 0.f;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    q[i] = x.at(i) * inv;
    const float whole = (q[i] + magic) - magic;
    near |= fabsf(q[i] - whole) > 0.5f - 0x1p-13f;
  }
  if (near) {
#pragma unroll
    for (int i = 0; i < 8; ++i) q[i] = x.at(i) / scale;
  }
  uint32_t w[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float c = __builtin_amdgcn_fmed3f(q[i], -127.0f, 127.0f);
    w[i] = __float_as_uint((q[i] != q[i] ? 0.f : c) + magic);
  }
  uint32_t h[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) h[i] = __builtin_amdgcn_perm(w[2 * i + 1], w[2 * i], 0x0c0c0400u);
  return make_uint2(h[0] | h[1] << 16, h[2] | h[3] << 16);
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

constexpr int kQuantRun = 64;  // most blocks of one workgroup
// Pieces of 8 elements that a lane holds between the maximum and the codes.
template <typename IO> constexpr int kQuantHeld = sizeof(IO) == 2 ? 8 : 4;

// WG: the workgroup is one group (units of more pieces than a wave holds);
// otherwise groups are 2^log_group lanes of a wave.
template <typename IO, typename KE, bool WG>
__global__ void __launch_bounds__(256) kv_quantise_kernel(QuantParams p) {
  constexpr int NR = kQuantHeld<IO>;
  __shared__ QuantBlock blocks[kQuantRun];
  __shared__ uint32_t red[4];
  __shared__ float red_scale[2];
  const int64_t id0 = (int64_t)blockIdx.x * p.run;
  const int nid = (int)min((int64_t)p.run, p.ids - id0);
  if ((int)threadIdx.x < nid) blocks[threadIdx.x] = quant_block(p, id0 + threadIdx.x);
  __syncthreads();

  const int group = WG ? 256 : 1 << p.log_group, me = threadIdx.x & (group - 1);
  const int log_head = 31 - __builtin_clz(p.d / 8), per = 2 * p.hkv, units = nid * per;
  // The largest value of the group's lanes.
  auto over_group = [&](uint32_t m) {
    for (int o = WG ? 32 : group >> 1; o > 0; o >>= 1) m = max(m, (uint32_t)__shfl_xor((int)m, o));
    if constexpr (WG) {
      __syncthreads();  // the last values are read
      if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = m;
      __syncthreads();
      m = max(max(red[0], red[1]), max(red[2], red[3]));
    }
    return m;
  };
  int par = 0;  // of the units that the workgroup has taken
  for (int u = WG ? 0 : threadIdx.x >> p.log_group; u < units; u += WG ? 1 : 256 >> p.log_group) {
    const int at = u / per, r = u - at * per;
    const QuantBlock b = blocks[at];
    if (b.n == 0) continue;
    const bool is_v = r >= p.hkv;
    const int h = is_v ? r - p.hkv : r;
    const int64_t st = is_v ? p.v_st : p.k_st, ct = is_v ? p.vc_st : p.kc_st;
    const IO* src = (const IO*)(is_v ? p.v : p.k) + b.tok * st + h * (is_v ? p.v_sh : p.k_sh);
    uint8_t* dst = (uint8_t*)(is_v ? p.vc : p.kc) + b.ent * (is_v ? p.vc_sp : p.kc_sp) + b.slot * ct + h * (is_v ? p.vc_sh : p.kc_sh);
    float* scale_at = (is_v ? p.vs : p.ks) + ((int64_t)b.ent * p.hkv + h) * p.nblk + b.slot / p.block;
    const int np = b.n << log_head, chunks = (np + group * NR - 1) / (group * NR);
    auto place = [&](int i) { return (i & ((1 << log_head) - 1)) * 8; };

    Piece<IO> x[NR];
    auto load = [&](int c) {
#pragma unroll
      for (int k = 0; k < NR; ++k) {
        const int i = (c * NR + k) * group + me;
        if (i < np) x[k].load(src + (i >> log_head) * st + place(i));
      }
    };
    auto held_max = [&](int c, bool finite) {
      uint32_t m = 0;
#pragma unroll
      for (int k = 0; k < NR; ++k)
        if ((c * NR + k) * group + me < np) m = max(m, finite ? finite_max(x[k]) : abs_max(x[k]));
      return m;
    };
    float old = 0.f;
    if (b.old > 0) {
      if constexpr (WG) {
        if (threadIdx.x == 0) red_scale[par] = *scale_at;
      } else {
        old = *scale_at;
      }
    }
    uint32_t m = 0;
    for (int c = 0; c < chunks; ++c) {
      load(c);
      m = max(m, held_max(c, false));
    }
    m = over_group(m);
    bool nan = false;
    if (m >= 0x7f800000u) {
      nan = m > 0x7f800000u;
      m = 0;
      for (int c = 0; c < chunks; ++c) {
        load(c);
        m = max(m, held_max(c, true));
      }
      m = over_group(m);
    }
    if constexpr (WG) {
      if (b.old > 0) old = red_scale[par];
      par ^= 1;
    }
    float s = scale_for<KE>(m);
    if (std::is_same<KE, i8>::value && nan) s = __builtin_nanf("");
    if (b.old > 0) s = old != old || s != s ? old + s : fmaxf(s, old);
    if (me == 0) *scale_at = s;
    const float inv = normal_rcp(s);
    if (b.old > 0 && s != old) {
      for (int i = me; i < b.old << log_head; i += group) {
        uint2* c = reinterpret_cast<uint2*>(dst + ((i >> log_head) - b.old) * ct + place(i));
        *c = quotients(KE{}, Older(KE{}, *c, old), s, inv);
      }
    }
    for (int c = chunks - 1; c >= 0; --c) {  // the last chunk is in registers
      if (c < chunks - 1) load(c);
#pragma unroll
      for (int k = 0; k < NR; ++k) {
        const int i = (c * NR + k) * group + me;
        if (i < np) *reinterpret_cast<uint2*>(dst + (i >> log_head) * ct + place(i)) = quotients(KE{}, x[k], s, inv);
      }
    }
  }
}

template <typename IO, typename KE>
static void launch_quantise(const QuantParams& p, bool wg, dim3 grid, hipStream_t stream) {
  if (wg) hipLaunchKernelGGL((kv_quantise_kernel<IO, KE, true>), grid, dim3(256), 0, stream, p);
  else hipLaunchKernelGGL((kv_quantise_kernel<IO, KE, false>), grid, dim3(256), 0, stream, p);
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
  // Pieces of a unit, and the lanes that take it: as many as it has pieces, up
  // to a wave, while they hold all of it.
  const int64_t tokens = !a.cu_seqlens && p.T < p.block ? p.T : p.block, pieces = tokens * (a.d / 8);
  const int held = a.io_dtype == GDN_BF16 ? kQuantHeld<__bf16> : kQuantHeld<float>;
  const bool wg = pieces > 64 * held;
  p.log_group = 2;
  while (p.log_group < 6 && (1 << p.log_group) < pieces) ++p.log_group;
  // Blocks per workgroup as the tokens of gdn_kv_append: about 4096 pieces, but
  // at least 1024 workgroups before one takes a second block.
  int64_t run = 4096 / (pieces * 2 * a.hkv), most = p.ids / 1024;
  run = run > most ? most : run;
  run = run < 1 ? 1 : run > kQuantRun ? kQuantRun : run;
  if (p.ids / run >= (1 << 23)) run = kQuantRun;  // a grid's limit; ids < 2^29
  p.run = (int)run;
  const dim3 grid((unsigned)((p.ids + run - 1) / run));
  if (a.cache_dtype == GDN_E4M3) {
    if (a.io_dtype == GDN_BF16) launch_quantise<__bf16, e4m3>(p, wg, grid, stream);
    else launch_quantise<float, e4m3>(p, wg, grid, stream);
  } else {
    if (a.io_dtype == GDN_BF16) launch_quantise<__bf16, i8>(p, wg, grid, stream);
    else launch_quantise<float, i8>(p, wg, grid, stream);
  }
  return hipGetLastError();
}

}  // namespace gdn
