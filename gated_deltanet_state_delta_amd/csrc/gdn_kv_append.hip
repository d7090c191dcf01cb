// gdn_kv_append.hip -- new tokens' keys and values into the pages of a cache.
//
// Row b's n_b tokens go to positions lens[b] - n_b .. lens[b] - 1:
//   cache[table[b][pos / page_size]][pos % page_size] = x   (e4m3: round(x / scale))
//
// HBM-bound streaming for prompts, launch-bound for one token a row.  A
// workgroup takes a run of tokens: one thread a token finds its row, position
// and page and leaves the two row offsets in LDS, then every thread copies
// pieces of 8 elements (16-byte loads and stores for bf16).
#include "gdn_device.hpp"
#include "gdn_kernels.hpp"

namespace gdn {

struct AppendParams {
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
  const float* k_scale;
  const float* v_scale;
  int64_t total;
  int batch, T, hkv, d, n_pages, page_size, cap, run;
};

struct e4m3x8 { uint32_t w[2]; };

// x / scale in e4m3, round to nearest even, beyond +-448 clamped; NaN stays NaN.
__device__ __forceinline__ uint32_t e4m3_pair(float a, float b, float scale, uint32_t old, bool hi) {
  float q[2] = {a / scale, b / scale};
#pragma unroll
  for (int i = 0; i < 2; ++i) q[i] = q[i] != q[i] ? q[i] : fminf(fmaxf(q[i], -448.0f), 448.0f);
  return hi ? __builtin_amdgcn_cvt_pk_fp8_f32(q[0], q[1], old, true) : __builtin_amdgcn_cvt_pk_fp8_f32(q[0], q[1], old, false);
}

template <typename IO>
__device__ __forceinline__ void put8(const IO* src, IO* dst, float) {
#pragma unroll
  for (int i = 0; i < (int)sizeof(IO) / 2; ++i)
    reinterpret_cast<u32x4*>(dst)[i] = reinterpret_cast<const u32x4*>(src)[i];
}
template <typename IO>
__device__ __forceinline__ void put8(const IO* src, uint8_t* dst, float scale) {
  const f4 a = load4(src), b = load4(src + 4);
  uint2 o;
  o.x = e4m3_pair(a[0], a[1], scale, 0, false);
  o.x = e4m3_pair(a[2], a[3], scale, o.x, true);
  o.y = e4m3_pair(b[0], b[1], scale, 0, false);
  o.y = e4m3_pair(b[2], b[3], scale, o.y, true);
  *reinterpret_cast<uint2*>(dst) = o;
}

constexpr int kAppendRun = 64;  // most tokens of one workgroup

template <typename IO, typename KE>
__global__ void __launch_bounds__(256) kv_append_kernel(AppendParams p) {
  __shared__ int64_t off[kAppendRun][2];
  const int64_t t0 = (int64_t)blockIdx.x * p.run;
  const int n = (int)min((int64_t)p.run, p.total - t0);
  if ((int)threadIdx.x < n) {
    const int64_t i = t0 + threadIdx.x;
    int b;
    int64_t back;  // tokens from this one to its row's end
    bool ok = true;
    if (!p.cu) {
      b = (int)(i / p.T);
      back = p.T - i % p.T;
    } else {
      // the last row that starts at or before token i (offsets clamped to
      // [0, total]); a token past that row's end belongs to none
      int lo = 0, hi = p.batch;
      while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (min(max((int64_t)p.cu[mid], (int64_t)0), p.total) <= i) lo = mid;
        else hi = mid;
      }
      b = lo;
      const int64_t s0 = min(max((int64_t)p.cu[b], (int64_t)0), p.total), s1 = min(max((int64_t)p.cu[b + 1], (int64_t)0), p.total);
      ok = s0 <= i && i < s1;
      back = s1 - i;
    }
    const int64_t pos = (int64_t)p.lens[b] - back;
    ok = ok && pos >= 0 && pos < p.cap;
    int64_t ko = -1, vo = -1;
    if (ok) {
      const int page = (int)pos / p.page_size, at = (int)pos - page * p.page_size;
      const int ent = p.table[b * p.table_stride + page];
      if (ent >= 0 && ent < p.n_pages) {
        ko = ent * p.kc_sp + at * p.kc_st;
        vo = ent * p.vc_sp + at * p.vc_st;
      }
    }
    off[threadIdx.x][0] = ko;
    off[threadIdx.x][1] = vo;
  }
  __syncthreads();
  const uint32_t per_head = p.d / 8, per_half = per_head * p.hkv, per_tok = 2 * per_half;
  for (uint32_t i = threadIdx.x; i < n * per_tok; i += 256) {
    const uint32_t tok = i / per_tok, r = i - tok * per_tok;
    const bool is_v = r >= per_half;
    const uint32_t q = is_v ? r - per_half : r, h = q / per_head, e = (q - h * per_head) * 8;
    const int64_t o = off[tok][is_v];
    if (o < 0) continue;
    const IO* src = is_v ? (const IO*)p.v + (t0 + tok) * p.v_st + h * p.v_sh + e
                         : (const IO*)p.k + (t0 + tok) * p.k_st + h * p.k_sh + e;
    KE* dst = is_v ? (KE*)p.vc + o + h * p.vc_sh + e : (KE*)p.kc + o + h * p.kc_sh + e;
    float scale = 1.0f;
    if constexpr (sizeof(KE) == 1) scale = is_v ? p.v_scale[h] : p.k_scale[h];
    put8(src, dst, scale);
  }
}

hipError_t launch_kv_append(const gdn_kv_append_args& a, hipStream_t stream) {
  AppendParams p;
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
  p.k_scale = a.k_scale;
  p.v_scale = a.v_scale;
  p.total = a.total_tokens;
  p.batch = a.batch;
  p.T = a.cu_seqlens ? 0 : (int)(a.total_tokens / a.batch);
  p.hkv = a.hkv;
  p.d = a.d;
  p.n_pages = a.n_pages;
  p.page_size = a.page_size;
  p.cap = a.max_pages * a.page_size;
  // Tokens per workgroup: about 1024 pieces, but at least 1024 workgroups
  // before a workgroup takes a second token.
  const int64_t pieces = 2 * (int64_t)a.hkv * (a.d / 8);
  int64_t run = 1024 / pieces, most = a.total_tokens / 1024;
  run = run > most ? most : run;
  run = run < 1 ? 1 : run > kAppendRun ? kAppendRun : run;
  while (a.total_tokens / run >= (1 << 23)) run *= 2;  // a grid's limit; total_tokens <= 2^28, so run <= kAppendRun
  p.run = (int)run;
  const dim3 grid((unsigned)((a.total_tokens + run - 1) / run));
  if (a.cache_dtype == GDN_E4M3) {
    if (a.io_dtype == GDN_BF16) hipLaunchKernelGGL((kv_append_kernel<__bf16, uint8_t>), grid, dim3(256), 0, stream, p);
    else hipLaunchKernelGGL((kv_append_kernel<float, uint8_t>), grid, dim3(256), 0, stream, p);
  } else if (a.io_dtype == GDN_BF16) {
    hipLaunchKernelGGL((kv_append_kernel<__bf16, __bf16>), grid, dim3(256), 0, stream, p);
  } else {
    hipLaunchKernelGGL((kv_append_kernel<float, float>), grid, dim3(256), 0, stream, p);
  }
  return hipGetLastError();
}

}  // namespace gdn
