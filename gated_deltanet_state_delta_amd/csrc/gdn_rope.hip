// gdn_rope.hip -- rotary positions of queries and keys.
//
//   y1 = factor (x1 cos a - x2 sin a),  y2 = factor (x1 sin a + x2 cos a),  a = pos * inv_freq[i]
//
// HBM-bound streaming for prompts, launch-bound for one token a row.  A
// workgroup takes a run of tokens: their rot / 2 sines and cosines, which all
// heads share, are formed once in LDS, then every thread turns pieces.  The
// angle is formed in fp64 and reduced to turns there (fp32 would be 0.06 rad off
// at position 10^6), sine and cosine in fp32: fp32 results are 5.4e-8 off on
// average, 4.0e-8 with sine and cosine in fp64; bf16 rounds 10^4 times as far.
//
// Measured: 32768 tokens of 32 + 8 heads of 128, bf16, 671 MB: 128 us = 5.2 TB/s,
// over a large copy's 4.9; 8192 of 16 + 4 heads of 96, two thirds of each turned,
// neighbouring pairs, fp32, 126 MB: 23 us = 5.4 TB/s; 256 tokens of 40 heads 4.5 us
// in a graph.
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
  int q_copy, k_copy;  // whether the dimensions behind rot are written: not in place, unless tokens of no row get zeros
};

constexpr int kRopeRun = 64;      // most tokens of one workgroup
constexpr int kRopeAngles = 1024; // angles that it holds

// V elements at p, which is aligned to one element (the hardware reads and
// writes whole dwords at any address).
template <typename IO, int V> struct RopeVec {
  typedef IO type __attribute__((ext_vector_type(V), aligned(sizeof(IO))));
};
template <typename IO> struct RopeVec<IO, 1> { typedef IO type; };
template <int V, typename IO> __device__ __forceinline__ void load_v(const IO* p, float* x) {
  const auto t = __builtin_nontemporal_load(reinterpret_cast<const typename RopeVec<IO, V>::type*>(p));
  if constexpr (V == 1) {
    x[0] = to_f32(t);
  } else {
#pragma unroll
    for (int i = 0; i < V; ++i) x[i] = to_f32(t[i]);
  }
}
template <int V, typename IO> __device__ __forceinline__ void store_v(IO* p, const float* x) {
  typename RopeVec<IO, V>::type o;
  if constexpr (V == 1) {
    o = from_f32<IO>(x[0]);
  } else {
#pragma unroll
    for (int i = 0; i < V; ++i) o[i] = from_f32<IO>(x[i]);
  }
  *reinterpret_cast<typename RopeVec<IO, V>::type*>(p) = o;
}

// V: elements of a piece, up to 16 bytes: a power of two that divides the pairs'
// runs and the copied rest.  IL: interleaved pairs.
//
// Units of the run, in order: token, head (queries before keys), then of a head
// the pieces of pairs and those that are copied.  A thread takes one of every 256,
// UB at a time: their loads are in flight together, and the first ones' while
// the angles are formed.
template <typename IO, int V, bool IL>
__global__ void __launch_bounds__(256) rope_kernel(RopeParams p) {
  __shared__ float2 turn[kRopeAngles];  // factor * (cos, sin), [token][pair]
  __shared__ double at[kRopeRun];
  __shared__ int is_row[kRopeRun];
  constexpr bool TWO = !(IL && V > 1);  // a unit of pairs is two pieces, or neighbours in one
  constexpr int PAIRS = TWO ? V : V / 2, UB = TWO ? 2 : 4;
  const int64_t t0 = (int64_t)blockIdx.x * p.run;
  const int n = (int)min((int64_t)p.run, p.total - t0);
  const int half = p.rot / 2;
  const uint32_t turned = half / PAIRS, per_head = turned + (p.d - p.rot) / V, heads = p.hq + p.hkv, per_tok = heads * per_head;
  const uint32_t step_tok = 256 / per_tok, step_in = 256 - step_tok * per_tok, step_head = step_in / per_head,
                 step_i = step_in - step_head * per_head;
  uint32_t tok = threadIdx.x / per_tok, hh = (threadIdx.x - tok * per_tok) / per_head,
           i = threadIdx.x - tok * per_tok - hh * per_head;

  struct Unit { IO* dst; int tok, i; bool skip; float a[V], b[TWO ? V : 1]; } u[UB];
  auto load = [&]() {
#pragma unroll
    for (int k = 0; k < UB; ++k) {
      u[k].tok = tok;
      u[k].i = i;
      const bool is_k = hh >= (uint32_t)p.hq, copied = i >= turned;
      u[k].skip = (int)tok >= n || (copied && !(is_k ? p.k_copy : p.q_copy));
      if (!u[k].skip) {
        const int h = is_k ? hh - p.hq : hh;
        const int64_t t = t0 + tok;
        const int e = copied ? p.rot + (i - turned) * V : IL ? i * (TWO ? 2 : V) : i * V;
        const IO* src = (is_k ? (const IO*)p.k + t * p.k_st + h * p.k_sh : (const IO*)p.q + t * p.q_st + h * p.q_sh) + e;
        u[k].dst = (is_k ? (IO*)p.ko + t * p.ko_st + h * p.ko_sh : (IO*)p.qo + t * p.qo_st + h * p.qo_sh) + e;
        load_v<V>(src, u[k].a);
        if constexpr (TWO)
          if (!copied) load_v<V>(src + (IL ? 1 : half), u[k].b);
      }
      tok += step_tok;
      hh += step_head;
      i += step_i;
      if (i >= per_head) {
        i -= per_head;
        ++hh;
      }
      if (hh >= heads) {
        hh -= heads;
        ++tok;
      }
    }
  };
  load();

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
  while (u[0].tok < n) {
#pragma unroll
    for (int k = 0; k < UB; ++k) {
      if (u[k].skip) continue;
      const bool row = is_row[u[k].tok];
      if (!row) {
        if (!p.zero_rest) continue;
#pragma unroll
        for (int e = 0; e < V; ++e) u[k].a[e] = 0.f;
        if constexpr (TWO)
#pragma unroll
          for (int e = 0; e < V; ++e) u[k].b[e] = 0.f;
      }
      if (u[k].i < (int)turned) {
        const float2* w = turn + u[k].tok * half + u[k].i * PAIRS;
#pragma unroll
        for (int e = 0; e < PAIRS; ++e) {
          float& x = u[k].a[TWO ? e : 2 * e];
          float& y = TWO ? u[k].b[TWO ? e : 0] : u[k].a[TWO ? 0 : 2 * e + 1];
          const float x0 = x, y0 = y, c = row ? w[e].x : 0.f, s = row ? w[e].y : 0.f;
          x = x0 * c - y0 * s;
          y = x0 * s + y0 * c;
        }
        if constexpr (TWO) store_v<V>(u[k].dst + (IL ? 1 : half), u[k].b);
      }
      store_v<V>(u[k].dst, u[k].a);
    }
    load();
  }
}

template <typename IO, int V>
static void launch_rope_v(const RopeParams& p, bool interleaved, dim3 grid, hipStream_t stream) {
  if (interleaved) hipLaunchKernelGGL((rope_kernel<IO, V, true>), grid, dim3(256), 0, stream, p);
  else hipLaunchKernelGGL((rope_kernel<IO, V, false>), grid, dim3(256), 0, stream, p);
}
template <typename IO>
static void launch_rope_t(const RopeParams& p, int v, bool interleaved, dim3 grid, hipStream_t stream) {
  if (v == 8) {
    if constexpr (sizeof(IO) == 2) launch_rope_v<IO, 8>(p, interleaved, grid, stream);
  } else if (v == 4) {
    launch_rope_v<IO, 4>(p, interleaved, grid, stream);
  } else if (v == 2) {
    launch_rope_v<IO, 2>(p, interleaved, grid, stream);
  } else {
    launch_rope_v<IO, 1>(p, interleaved, grid, stream);
  }
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
  p.q_copy = a.q != a.q_out || a.zero_rest;
  p.k_copy = a.k != a.k_out || a.zero_rest;
  const bool interleaved = a.interleaved != 0;
  // One piece size for all of a head: 16384 tokens of 40 heads, bf16, heads of 128 turned whole 59 us, to rot 126 in
  // pieces of 2 bytes 148 (neighbouring pairs, of 4 bytes, 138); heads of 80 whole 48, to rot 20 102 and 59.
  int v = a.io_dtype == GDN_BF16 ? 8 : 4;
  while (((interleaved ? a.rot : a.rot / 2) | (a.d - a.rot)) % v != 0) v /= 2;
  // Tokens per workgroup: about two rounds of what its threads hold (32768 tokens of 40
  // heads of 128, bf16: four tokens 126 us, one 143, eight 132), within the angles'
  // room, but at least 1024 workgroups before one takes a second token.
  const bool two = !interleaved || v == 1;
  const int64_t units = (int64_t)(p.hq + p.hkv) * (two ? a.rot / 2 / v + (a.d - a.rot) / v : a.d / v);
  const int64_t room = kRopeAngles / (a.rot / 2), round = two ? 512 : 1024;
  int64_t run = (2 * round + units / 2) / units, most = a.total_tokens / 1024;
  run = run > most ? most : run;
  run = run > kRopeRun ? kRopeRun : run;
  run = run > room ? room : run < 1 ? 1 : run;
  if (a.total_tokens / run > (1 << 23)) run = 2;  // a grid's limit; total_tokens <= 2^24, and there is room for two
  p.run = (int)run;
  const dim3 grid((unsigned)((a.total_tokens + run - 1) / run));
  if (a.io_dtype == GDN_BF16) launch_rope_t<__bf16>(p, v, interleaved, grid, stream);
  else launch_rope_t<float>(p, v, interleaved, grid, stream);
  return hipGetLastError();
}

}  // namespace gdn
