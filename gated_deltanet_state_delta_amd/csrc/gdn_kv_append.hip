// gdn_kv_append.hip -- new tokens' keys and values into the pages of a cache.
//
// Row b's n_b tokens go to positions lens[b] - n_b .. lens[b] - 1:
//   cache[table[b][pos / page_size]][pos % page_size] = x   (e4m3: round(x / scale))
//
// HBM-bound streaming for prompts, launch-bound for one token a row.  A
// workgroup takes a run of tokens: one thread a token finds its row, position
// and page and leaves the two row offsets in LDS, then every thread copies
// pieces of 8 elements (16-byte loads and stores for bf16).
#include "gdn_kv.hpp"

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

constexpr int kAppendRun = 64;  // most tokens of one workgroup

template <typename IO, typename KE>
__global__ void __launch_bounds__(256) kv_append_kernel(AppendParams p) {
  __shared__ uint64_t from[kAppendRun][2], to[kAppendRun][2];  // a token's K and V; to: 0 where it is not written
  const int64_t t0 = (int64_t)blockIdx.x * p.run;
  const int n = (int)min((int64_t)p.run, p.total - t0);
  if ((int)threadIdx.x < n) {
    const int64_t i = t0 + threadIdx.x;
    int b;
    int64_t back;  // tokens from this one to its row's end
    bool ok = token_row(p, i, b, back);
    const int64_t pos = (int64_t)p.lens[b] - back;
    ok = ok && pos >= 0 && pos < p.cap;
    uint64_t ko = 0, vo = 0;
    if (ok) {
      const int page = (int)pos / p.page_size, at = (int)pos - page * p.page_size;
      const int ent = p.table[b * p.table_stride + page];
      if (ent >= 0 && ent < p.n_pages) {
        ko = (uint64_t)((KE*)p.kc + ent * p.kc_sp + at * p.kc_st);
        vo = (uint64_t)((KE*)p.vc + ent * p.vc_sp + at * p.vc_st);
      }
    }
    from[threadIdx.x][0] = (uint64_t)((const IO*)p.k + i * p.k_st);
    from[threadIdx.x][1] = (uint64_t)((const IO*)p.v + i * p.v_st);
    to[threadIdx.x][0] = ko;
    to[threadIdx.x][1] = vo;
  }
  __syncthreads();
  // Pieces of the run in order, threads side by side: token, then K before V,
  // head, piece of the head.  A thread steps by 256 pieces, four in flight.
  const uint32_t log_head = 31 - __builtin_clz(p.d / 8), per_half = (uint32_t)p.hkv << log_head, per_tok = 2 * per_half;
  const bool dense = p.k_sh == p.d && p.v_sh == p.d && p.kc_sh == p.d && p.vc_sh == p.d;
  const uint32_t step_tok = 256 / per_tok, step_r = 256 - step_tok * per_tok;
  uint32_t tok = threadIdx.x / per_tok, r = threadIdx.x - tok * per_tok;
  while ((int)tok < n) {
    Piece<IO> x[4];
    KE* dst[4];
    float scale[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      dst[k] = nullptr;
      if ((int)tok < n) {
        const bool is_v = r >= per_half;
        const uint32_t q = is_v ? r - per_half : r, h = q >> log_head;
        const uint64_t o = to[tok][is_v];
        if (o != 0) {
          int64_t in = q * 8, out = q * 8;  // elements from the token's first
          if (!dense) {
            const uint32_t e = (q & ((1u << log_head) - 1)) * 8;
            in = h * (is_v ? p.v_sh : p.k_sh) + e;
            out = h * (is_v ? p.vc_sh : p.kc_sh) + e;
          }
          x[k].load((const IO*)from[tok][is_v] + in);
          dst[k] = (KE*)o + out;
          if constexpr (sizeof(KE) == 1) scale[k] = is_v ? p.v_scale[h] : p.k_scale[h];
        }
      }
      tok += step_tok;
      r += step_r;
      if (r >= per_tok) {
        r -= per_tok;
        ++tok;
      }
    }
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      if (!dst[k]) continue;
      if constexpr (sizeof(KE) == 1) {
        float q[8];
        e4m3_quotients(x[k], scale[k], normal_rcp(scale[k]), q);
        *reinterpret_cast<uint2*>(dst[k]) = make_uint2(e4m3_pack(q), e4m3_pack(q + 4));
      } else {
        x[k].store(dst[k]);
      }
    }
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
  // Tokens per workgroup: about 4096 pieces, but at least 1024 workgroups
  // before a workgroup takes a second token.
  const int64_t pieces = 2 * (int64_t)a.hkv * (a.d / 8);
  int64_t run = 4096 / pieces, most = a.total_tokens / 1024;
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
