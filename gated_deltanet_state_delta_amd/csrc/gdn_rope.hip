// gdn_rope.hip -- rotary positions of queries and keys.
//
//   y1 = factor (x1 cos a - x2 sin a),  y2 = factor (x1 sin a + x2 cos a),  a = pos * inv_freq[i]
//
// HBM-bound streaming for prompts, launch-bound for one token a row.  A
// workgroup takes a run of tokens: their rot / 2 sines and cosines, which all
// heads share, are formed once in LDS, then every thread turns pieces.  The
// angle is formed in fp64 and reduced to turns there (fp32 would be 0.06 rad off
// at position 10^6), sine and cosine in fp32.
#include "gdn_kv.hpp"

namespace gdn {

struct RopeParams {
  const void* q;
  const void* k;
  void* qo;
  void* ko;
  int64_t q_st, q_sh, k_st, k_sh, qo_st, qo_sh, ko_st, ko_sh;  // elements
  const double* freq;
  const void* positions;
  const int32_t* lens;
  const int32_t* cu;
  int64_t total;
  float factor;
  int batch, T, hq, hkv, d, rot, run, pos_i64, zero_rest;
  int q_copy, k_copy;  // whether the dimensions behind rot are copied (not in place)
};

constexpr int kRopeRun = 64;      // most tokens of one workgroup
constexpr int kRopeAngles = 1024; // angles that it holds

// V elements at p, as fp32; V = 1, or 16 bytes.
template <int V> __device__ __forceinline__ void load_v(const float* p, float* x) {
  if constexpr (V == 1) {
    x[0] = *p;
  } else {
    const f4 t = ld_nt(p);
#pragma unroll
    for (int i = 0; i < 4; ++i) x[i] = t[i];
  }
}
template <int V> __device__ __forceinline__ void load_v(const __bf16* p, float* x) {
  if constexpr (V == 1) {
    x[0] = (float)*p;
  } else {
    Piece<__bf16> t;
    t.load(p);
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = t.at(i);
  }
}
template <int V, typename IO> __device__ __forceinline__ void store_v(IO* p, const float* x) {
  if constexpr (V == 1) {
    *p = from_f32<IO>(x[0]);
  } else {
    typedef IO vec __attribute__((ext_vector_type(V)));
    vec o;
#pragma unroll
    for (int i = 0; i < V; ++i) o[i] = from_f32<IO>(x[i]);
    *reinterpret_cast<vec*>(p) = o;
  }
}

// V: elements of a piece: 16 bytes where sizes, strides and pointers allow it,
// else 1.  IL: interleaved pairs.
template <typename IO, int V, bool IL>
__global__ void __launch_bounds__(256) rope_kernel(RopeParams p) {
  __shared__ float2 turn[kRopeAngles];  // factor * (cos, sin), [token][pair]
  __shared__ double at[kRopeRun];
  __shared__ int is_row[kRopeRun];
  const int64_t t0 = (int64_t)blockIdx.x * p.run;
  const int n = (int)min((int64_t)p.run, p.total - t0);
  const int half = p.rot / 2;
  if ((int)threadIdx.x < n) {
    const int64_t i = t0 + threadIdx.x;
    bool ok = true;
    double pos = 0.0;
    if (p.positions) {
      pos = p.pos_i64 ? (double)((const int64_t*)p.positions)[i] : (double)((const int32_t*)p.positions)[i];
    } else {
      int b;
      int64_t back;  // tokens from this one to its row's end
      ok = token_row(p, i, b, back);
      if (ok) pos = (double)((int64_t)p.lens[b] - back);
    }
    at[threadIdx.x] = pos;
    is_row[threadIdx.x] = ok;
  }
  __syncthreads();
  for (int i = threadIdx.x; i < n * half; i += 256) {
    const int t = i / half;
    const double turns = at[t] * p.freq[i - t * half] * 0.15915494309189533577;
    float s, c;
    sincospif(2.0f * (float)(turns - __builtin_rint(turns)), &s, &c);
    turn[i] = make_float2(c * p.factor, s * p.factor);
  }
  __syncthreads();
  // Units of the run: token, head (queries before keys), then of a head the
  // pieces of pairs and those that are copied.
  constexpr int PAIRS = IL && V > 1 ? V / 2 : V;  // pairs of a unit
  const int turned = half / PAIRS, per_head = turned + (p.d - p.rot) / V, per_tok = (p.hq + p.hkv) * per_head;
  auto load_or_zero = [](const IO* s, bool row, float* x) {
    if (row) {
      load_v<V>(s, x);
    } else {
#pragma unroll
      for (int k = 0; k < V; ++k) x[k] = 0.f;
    }
  };
  for (int u = threadIdx.x; u < n * per_tok; u += 256) {
    const int t = u / per_tok, r = u - t * per_tok, hh = r / per_head, i = r - hh * per_head;
    const bool row = is_row[t];
    if (!row && !p.zero_rest) continue;
    const bool is_k = hh >= p.hq;
    const int h = is_k ? hh - p.hq : hh;
    const IO* src = is_k ? (const IO*)p.k + (t0 + t) * p.k_st + h * p.k_sh : (const IO*)p.q + (t0 + t) * p.q_st + h * p.q_sh;
    IO* dst = is_k ? (IO*)p.ko + (t0 + t) * p.ko_st + h * p.ko_sh : (IO*)p.qo + (t0 + t) * p.qo_st + h * p.qo_sh;
    float a[V], b[V];
    if (i >= turned) {
      if (is_k ? p.k_copy : p.q_copy) {
        const int e = p.rot + (i - turned) * V;
        load_or_zero(src + e, row, a);
        store_v<V>(dst + e, a);
      }
    } else if constexpr (IL && V > 1) {
      load_or_zero(src + i * V, row, a);
#pragma unroll
      for (int k = 0; k < PAIRS; ++k) {
        const float2 w = turn[t * half + i * PAIRS + k];
        b[2 * k] = a[2 * k] * w.x - a[2 * k + 1] * w.y;
        b[2 * k + 1] = a[2 * k] * w.y + a[2 * k + 1] * w.x;
      }
      store_v<V>(dst + i * V, b);
    } else {
      const int e = IL ? 2 * i : i * V, f = IL ? e + 1 : e + half;
      load_or_zero(src + e, row, a);
      load_or_zero(src + f, row, b);
#pragma unroll
      for (int k = 0; k < V; ++k) {
        const float2 w = turn[t * half + i * V + k];
        const float x = a[k], y = b[k];
        a[k] = x * w.x - y * w.y;
        b[k] = x * w.y + y * w.x;
      }
      store_v<V>(dst + e, a);
      store_v<V>(dst + f, b);
    }
  }
}

template <typename IO, int V>
static void launch_rope_v(const RopeParams& p, bool interleaved, dim3 grid, hipStream_t stream) {
  if (interleaved) hipLaunchKernelGGL((rope_kernel<IO, V, true>), grid, dim3(256), 0, stream, p);
  else hipLaunchKernelGGL((rope_kernel<IO, V, false>), grid, dim3(256), 0, stream, p);
}

hipError_t launch_rope(const gdn_rope_args& a, hipStream_t stream) {
  RopeParams p;
  p.q = a.q;
  p.k = a.k;
  p.qo = a.q_out;
  p.ko = a.k_out;
  p.q_st = a.q_stride_token;
  p.q_sh = a.q_stride_head;
  p.k_st = a.k_stride_token;
  p.k_sh = a.k_stride_head;
  p.qo_st = a.qo_stride_token;
  p.qo_sh = a.qo_stride_head;
  p.ko_st = a.ko_stride_token;
  p.ko_sh = a.ko_stride_head;
  p.freq = a.inv_freq;
  p.positions = a.positions;
  p.pos_i64 = a.positions_i64;
  p.zero_rest = a.zero_rest;
  p.lens = a.lens;
  p.cu = a.positions ? nullptr : a.cu_seqlens;
  p.total = a.total_tokens;
  p.factor = a.factor;
  p.batch = a.batch;
  p.T = a.positions || a.cu_seqlens ? 0 : (int)(a.total_tokens / a.batch);
  p.hq = a.hq;
  p.hkv = a.k ? a.hkv : 0;
  p.d = a.d;
  p.rot = a.rot;
  p.q_copy = a.q != a.q_out;
  p.k_copy = a.k != a.k_out;
  // Pieces of 16 bytes where every one of them is aligned.
  const int es = a.io_dtype == GDN_BF16 ? 2 : 4, v = 16 / es;
  const int64_t strides = a.q_stride_token | a.q_stride_head | a.qo_stride_token | a.qo_stride_head |
                          (a.k ? a.k_stride_token | a.k_stride_head | a.ko_stride_token | a.ko_stride_head : 0);
  const uintptr_t bases = (uintptr_t)a.q | (uintptr_t)a.q_out | (a.k ? (uintptr_t)a.k | (uintptr_t)a.k_out : 0);
  const int step = a.interleaved ? a.rot : a.rot / 2;
  const bool vec = strides % v == 0 && bases % 16 == 0 && a.d % v == 0 && step % v == 0;
  // Tokens per workgroup: as many as their angles' room holds and about 4096
  // pieces, but at least 1024 workgroups before one takes a second token.
  const int64_t pieces = (int64_t)(p.hq + p.hkv) * (vec ? a.d / v : a.d);
  const int64_t room = kRopeAngles / (a.rot / 2);
  int64_t run = 4096 / pieces, most = a.total_tokens / 1024;
  run = run > most ? most : run;
  run = run > kRopeRun ? kRopeRun : run;
  run = run > room ? room : run < 1 ? 1 : run;
  if (a.total_tokens / run > (1 << 23)) run = 2;  // a grid's limit; total_tokens <= 2^24, and there is room for two
  p.run = (int)run;
  const dim3 grid((unsigned)((a.total_tokens + run - 1) / run));
  if (es == 2) {
    if (vec) launch_rope_v<__bf16, 8>(p, a.interleaved != 0, grid, stream);
    else launch_rope_v<__bf16, 1>(p, a.interleaved != 0, grid, stream);
  } else {
    if (vec) launch_rope_v<float, 4>(p, a.interleaved != 0, grid, stream);
    else launch_rope_v<float, 1>(p, a.interleaved != 0, grid, stream);
  }
  return hipGetLastError();
}

}  // namespace gdn
