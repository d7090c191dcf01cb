// gdn_kv_read.hip -- tokens read back out of the pages of a cache.
//
// Row b's n_b tokens are those of positions lens[b] - n_b .. lens[b] - 1:
//   x = cache[table[b][pos / page_size]][pos % page_size]   (8 bits: code * scale)
//
// HBM-bound streaming, launch-bound for a few tokens.  A workgroup takes a run
// of tokens: one thread a token finds its row, position and page and leaves
// the places in LDS, then every thread copies pieces of 8 elements.
//
// Measured: the histories of 8 rows out of 8 heads of 128, int8 in blocks of 32 to
// bf16, 352 MB, two thirds of it written: 74 us = 4.8 TB/s, a large copy's rate;
// one prompt of 1003 tokens 4.0 us in a graph.
#include <type_traits>

#include "gdn_kv.hpp"

namespace gdn {

struct ReadParams {
  void* k;
  void* v;
  int64_t k_st, k_sh, v_st, v_sh;  // elements
  const void* kc;
  const void* vc;
  int64_t kc_sp, kc_st, kc_sh, vc_sp, vc_st, vc_sh;
  const int32_t* table;
  int64_t table_stride;
  const int32_t* lens;
  const int32_t* cu;
  const float* ks;  // [hkv], or with block > 0 [n_pages][hkv][nblk]
  const float* vs;
  int64_t total;
  int batch, T, hkv, d, n_pages, page_size, cap, run, block, nblk, zero_rest;
};

__device__ __forceinline__ void store8(__bf16* p, const float* x) {
  bf8 o;
#pragma unroll
  for (int i = 0; i < 8; ++i) o[i] = (__bf16)x[i];
  __builtin_nontemporal_store(o, reinterpret_cast<bf8*>(p));
}
__device__ __forceinline__ void store8(float* p, const float* x) {
  st_nt(p, f4{x[0], x[1], x[2], x[3]});
  st_nt(p + 4, f4{x[4], x[5], x[6], x[7]});
}

// 8 elements of a cache, as values without their scale.
template <typename KE> struct Stored {
  Piece<KE> x;
  __device__ __forceinline__ void load(const KE* p) { x.load(p); }
  __device__ __forceinline__ void values(float* o) const {
#pragma unroll
    for (int i = 0; i < 8; ++i) o[i] = x.at(i);
  }
};
struct Stored8 {
  uint32_t w[2];
  __device__ __forceinline__ void load8(const void* p) {
    typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
    const u32x2 t = __builtin_nontemporal_load(reinterpret_cast<const u32x2*>(p));
    w[0] = t[0];
    w[1] = t[1];
  }
};
template <> struct Stored<e4m3> : Stored8 {
  __device__ __forceinline__ void load(const e4m3* p) { load8(p); }
  __device__ __forceinline__ void values(float* o) const {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      o[4 * i] = __builtin_amdgcn_cvt_f32_fp8(w[i], 0);
      o[4 * i + 1] = __builtin_amdgcn_cvt_f32_fp8(w[i], 1);
      o[4 * i + 2] = __builtin_amdgcn_cvt_f32_fp8(w[i], 2);
      o[4 * i + 3] = __builtin_amdgcn_cvt_f32_fp8(w[i], 3);
    }
  }
};
template <> struct Stored<i8> : Stored8 {
  __device__ __forceinline__ void load(const i8* p) { load8(p); }
  __device__ __forceinline__ void values(float* o) const {
#pragma unroll
    for (int i = 0; i < 8; ++i) o[i] = (float)(int8_t)(w[i >> 2] >> (8 * (i & 3)));
  }
};

constexpr int kReadRun = 64;  // most tokens of one workgroup

// A token's place: K and V in the outputs and the cache (cache 0: it holds
// nothing), and its block's scale of head 0; out 0 for a token that is not written.
struct ReadPlace { uint64_t out[2], cache[2]; int64_t scale; };

template <typename IO, typename KE>
__global__ void __launch_bounds__(256) kv_read_kernel(ReadParams p) {
  __shared__ ReadPlace places[kReadRun];
  const int64_t t0 = (int64_t)blockIdx.x * p.run;
  const int n = (int)min((int64_t)p.run, p.total - t0);
  if ((int)threadIdx.x < n) {
    const int64_t i = t0 + threadIdx.x;
    int b;
    int64_t back;  // tokens from this one to its row's end
    ReadPlace o = {};
    const bool ok = token_row(p, i, b, back);
    if (ok || p.zero_rest) {
      o.out[0] = (uint64_t)((IO*)p.k + i * p.k_st);
      o.out[1] = (uint64_t)((IO*)p.v + i * p.v_st);
    }
    if (ok) {
      const int64_t pos = (int64_t)p.lens[b] - back;
      if (pos >= 0 && pos < p.cap && p.n_pages > 0) {
        const int page = (int)pos / p.page_size, at = (int)pos - page * p.page_size;
        const int ent = p.table[b * p.table_stride + page];
        if (ent >= 0 && ent < p.n_pages) {
          o.cache[0] = (uint64_t)((const KE*)p.kc + ent * p.kc_sp + at * p.kc_st);
          o.cache[1] = (uint64_t)((const KE*)p.vc + ent * p.vc_sp + at * p.vc_st);
          if (p.block > 0) o.scale = (int64_t)ent * p.hkv * p.nblk + at / p.block;
        }
      }
    }
    places[threadIdx.x] = o;
  }
  __syncthreads();
  // Pieces of the run in order, threads side by side: token, then K before V,
  // head, piece of the head.  A thread steps by 256 pieces, four in flight.
  const uint32_t log_head = 31 - __builtin_clz(p.d / 8), per_half = (uint32_t)p.hkv << log_head, per_tok = 2 * per_half;
  const uint32_t step_tok = 256 / per_tok, step_r = 256 - step_tok * per_tok;
  uint32_t tok = threadIdx.x / per_tok, r = threadIdx.x - tok * per_tok;
  while ((int)tok < n) {
    Stored<KE> x[4];
    IO* dst[4];
    bool held[4];
    float scale[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      dst[k] = nullptr;
      held[k] = false;
      scale[k] = 1.f;
      if ((int)tok < n) {
        const bool is_v = r >= per_half;
        const uint32_t q = is_v ? r - per_half : r, h = q >> log_head, e = (q & ((1u << log_head) - 1)) * 8;
        const ReadPlace& o = places[tok];
        const uint64_t out = o.out[is_v], from = o.cache[is_v];
        if (out != 0) dst[k] = (IO*)out + h * (is_v ? p.v_sh : p.k_sh) + e;
        held[k] = from != 0;
        if (from != 0) {
          x[k].load((const KE*)from + h * (is_v ? p.vc_sh : p.kc_sh) + e);
          if constexpr (sizeof(KE) == 1)
            scale[k] = (is_v ? p.vs : p.ks)[p.block > 0 ? o.scale + (int64_t)h * p.nblk : h];
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
      float y[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
      if (held[k]) {
        x[k].values(y);
        if constexpr (sizeof(KE) == 1) {
#pragma unroll
          for (int i = 0; i < 8; ++i) y[i] *= scale[k];
        }
      }
      store8(dst[k], y);
    }
  }
}

template <typename IO>
static void launch_read(const gdn_kv_read_args& a, const ReadParams& p, dim3 grid, hipStream_t stream) {
  if (a.cache_dtype == GDN_E4M3) hipLaunchKernelGGL((kv_read_kernel<IO, e4m3>), grid, dim3(256), 0, stream, p);
  else if (a.cache_dtype == GDN_I8) hipLaunchKernelGGL((kv_read_kernel<IO, i8>), grid, dim3(256), 0, stream, p);
  else hipLaunchKernelGGL((kv_read_kernel<IO, IO>), grid, dim3(256), 0, stream, p);
}

hipError_t launch_kv_read(const gdn_kv_read_args& a, hipStream_t stream) {
  ReadParams p;
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
  p.ks = a.scale_block > 0 ? a.k_block_scale : a.k_scale;
  p.vs = a.scale_block > 0 ? a.v_block_scale : a.v_scale;
  p.total = a.total_tokens;
  p.batch = a.batch;
  p.T = a.cu_seqlens ? 0 : (int)(a.total_tokens / a.batch);
  p.hkv = a.hkv;
  p.d = a.d;
  p.n_pages = a.n_pages;
  p.page_size = a.page_size;
  p.cap = a.max_pages * a.page_size;
  p.block = a.scale_block;
  p.nblk = a.scale_block > 0 ? a.page_size / a.scale_block : 0;
  p.zero_rest = a.zero_rest;
  // Tokens per workgroup: about 4096 pieces, but at least 1024 workgroups
  // before a workgroup takes a second token.
  const int64_t pieces = 2 * (int64_t)a.hkv * (a.d / 8);
  int64_t run = 4096 / pieces, most = a.total_tokens / 1024;
  run = run > most ? most : run;
  run = run < 1 ? 1 : run > kReadRun ? kReadRun : run;
  while (a.total_tokens / run >= (1 << 23)) run *= 2;  // a grid's limit; total_tokens <= 2^28, so run <= kReadRun
  p.run = (int)run;
  const dim3 grid((unsigned)((a.total_tokens + run - 1) / run));
  if (a.io_dtype == GDN_BF16) launch_read<__bf16>(a, p, grid, stream);
  else launch_read<float>(a, p, grid, stream);
  return hipGetLastError();
}

}  // namespace gdn
