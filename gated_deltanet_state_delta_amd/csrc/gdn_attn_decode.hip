// gdn_attn_decode.hip -- launch of the attention over a paged cache: the
// split over the rows' lengths and the kernel that joins its parts.
#include "gdn_attn_decode.hpp"

namespace gdn {

// Joins the parts of one (row, head, token): out = sum_s e^{m_s - M} o_s /
// sum_s e^{m_s - M} l_s.  One workgroup each; D/4 threads read one part's
// output, the others further parts, added through LDS in a fixed order.
template <typename IO, int D>
__global__ void __launch_bounds__(256) attn_join_kernel(AttnParams p) {
  constexpr int TPD = D / 4, NG = 256 / TPD;
  __shared__ f4 part[256];
  __shared__ float wave_m[4], wave_l[4];
  const int r = blockIdx.x % p.R, bh = blockIdx.x / p.R, h = bh % p.hkv, b = bh / p.hkv;
  const int len = attn_len(p, b), chunk = attn_chunk(p, len);
  const int n = max(1, (int)(((int64_t)len + chunk - 1) / chunk));  // parts that were written
  const int64_t at0 = (int64_t)bh * p.nsplit * p.R + r;             // part s: at0 + s * R
  const int tid = threadIdx.x;
  float m = -__builtin_inff();
  for (int s = tid; s < n; s += 256) m = fmaxf(m, p.part_ml[(at0 + (int64_t)s * p.R) * 2]);
  for (int o = 32; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor(m, o));
  if ((tid & 63) == 0) wave_m[tid >> 6] = m;
  __syncthreads();
  m = fmaxf(fmaxf(wave_m[0], wave_m[1]), fmaxf(wave_m[2], wave_m[3]));
  const float mu = m == -__builtin_inff() ? 0.f : m;
  float l = 0.f;
  for (int s = tid; s < n; s += 256) {
    const float* ml = p.part_ml + (at0 + (int64_t)s * p.R) * 2;
    l += ml[1] * exp2_hw(ml[0] - mu);
  }
  for (int o = 32; o > 0; o >>= 1) l += __shfl_xor(l, o);
  if ((tid & 63) == 0) wave_l[tid >> 6] = l;

  const int grp = tid / TPD, d = (tid % TPD) * 4;
  f4 acc = {0.f, 0.f, 0.f, 0.f};
  for (int s = grp; s < n; s += NG) {
    const int64_t at = at0 + (int64_t)s * p.R;
    const float w = exp2_hw(p.part_ml[at * 2] - mu);
    const f4 o = *reinterpret_cast<const f4*>(p.part_o + at * D + d);
#pragma unroll
    for (int i = 0; i < 4; ++i) acc[i] += w * o[i];
  }
  part[tid] = acc;
  __syncthreads();
  if (tid >= TPD) return;
  l = (wave_l[0] + wave_l[1]) + (wave_l[2] + wave_l[3]);
#pragma unroll 4
  for (int i = 1; i < NG; ++i) acc += part[i * TPD + tid];
  const int t = r / p.group, hq = h * p.group + r % p.group;
  const int64_t row = ((int64_t)b * p.T + t) * p.hq + hq;
  attn_store<IO>(p, row * D + d, acc, m, l, h);
  if (p.lse && tid == 0) p.lse[row] = attn_lse(m, l);
}

template <typename IO>
static void launch_join(const AttnParams& p, int d, hipStream_t stream) {
  const dim3 grid((unsigned)((int64_t)p.batch * p.hkv * p.R));
  if (d == 32) hipLaunchKernelGGL((attn_join_kernel<IO, 32>), grid, dim3(256), 0, stream, p);
  else if (d == 64) hipLaunchKernelGGL((attn_join_kernel<IO, 64>), grid, dim3(256), 0, stream, p);
  else if (d == 128) hipLaunchKernelGGL((attn_join_kernel<IO, 128>), grid, dim3(256), 0, stream, p);
  else hipLaunchKernelGGL((attn_join_kernel<IO, 256>), grid, dim3(256), 0, stream, p);
}

// Ranges per row: enough workgroups to fill 256 CUs several times over if
// every row is as long as its table allows, none shorter than kMinChunk keys.
constexpr int kMinChunk = 128, kWorkgroups = 2048;
static int attn_splits(const gdn_attn_decode_args& a) {
  const int64_t R = (int64_t)a.T * (a.hq / a.hkv);
  const int64_t units = (int64_t)a.batch * a.hkv * ((R + 15) / 16);
  const int64_t cap = (int64_t)a.max_pages * a.page_size;
  const int64_t most = (cap + kMinChunk - 1) / kMinChunk;
  int64_t n = (kWorkgroups + units - 1) / units;
  if (n > most) n = most;
  return n < 1 ? 1 : (int)n;
}

size_t attn_workspace_bytes(const gdn_attn_decode_args& a) {
  if (a.batch <= 0 || a.T <= 0 || a.hkv <= 0 || a.hq < a.hkv || a.d <= 0 || a.max_pages <= 0 || a.page_size <= 0)
    return 0;
  const int n = attn_splits(a);
  if (n == 1) return 0;
  return (size_t)a.batch * a.hq * a.T * n * (a.d + 2) * sizeof(float);
}

hipError_t launch_attn_decode(const gdn_attn_decode_args& a, hipStream_t stream) {
  const int io = a.io_dtype == GDN_BF16 ? 2 : 4;
  const int ce = a.cache_dtype == GDN_E4M3 ? 1 : io;
  AttnParams p;
  p.q = a.q;
  p.q_sb = a.q_stride_row * io;
  p.q_st = a.q_stride_token * io;
  p.q_sh = a.q_stride_head * io;
  p.out = a.out;
  p.lse = a.lse;
  p.k = a.k_cache;
  p.v = a.v_cache;
  p.k_sp = a.k_stride_page * ce;
  p.v_sp = a.v_stride_page * ce;
  p.k_st = (uint32_t)(a.k_stride_token * ce);
  p.v_st = (uint32_t)(a.v_stride_token * ce);
  p.k_sh = a.k_stride_head * ce;
  p.v_sh = a.v_stride_head * ce;
  p.table = a.page_table;
  p.table_stride = a.page_table_stride;
  p.lens = a.lens;
  p.k_scale = a.k_scale;
  p.v_scale = a.v_scale;
  p.scale_log2 = (float)((double)a.scale * 1.4426950408889634);
  p.batch = a.batch;
  p.T = a.T;
  p.hq = a.hq;
  p.hkv = a.hkv;
  p.group = a.hq / a.hkv;
  p.R = a.T * p.group;
  p.ntile = (p.R + 15) / 16;
  p.n_pages = a.n_pages;
  p.page_size = a.page_size;
  p.cap = a.max_pages * a.page_size;
  p.min_chunk = kMinChunk;
  // j / page_size for j < 2^31: with s = ceil(log2(page_size)) and
  // mul = ceil(2^(31 + s) / page_size), the error of mul is below 2^s.
  int s = 0;
  while ((1 << s) < a.page_size) ++s;
  p.page_mul = (uint32_t)((((uint64_t)1 << (31 + s)) + a.page_size - 1) / a.page_size);
  p.page_shift = 31 + s;
  const size_t need = attn_workspace_bytes(a);
  p.nsplit = 1;
  p.part_o = p.part_ml = nullptr;
  if (need > 0 && a.workspace && a.workspace_bytes >= need) {
    p.nsplit = attn_splits(a);
    p.part_o = (float*)a.workspace;
    p.part_ml = p.part_o + (size_t)a.batch * a.hq * a.T * p.nsplit * a.d;
  }
  const int64_t units = (int64_t)p.batch * p.hkv * p.nsplit;
  const dim3 grid((unsigned)((units + 7) / 8 * 8 * p.ntile));
  hipError_t e;
  if (a.cache_dtype == GDN_E4M3)
    e = a.io_dtype == GDN_BF16 ? launch_attn_bf16_e4m3(p, a.d, grid, stream) : launch_attn_f32_e4m3(p, a.d, grid, stream);
  else
    e = a.io_dtype == GDN_BF16 ? launch_attn_bf16(p, a.d, grid, stream) : launch_attn_f32(p, a.d, grid, stream);
  if (e != hipSuccess || p.nsplit == 1) return e;
  if (a.io_dtype == GDN_BF16) launch_join<__bf16>(p, a.d, stream);
  else launch_join<float>(p, a.d, stream);
  return hipGetLastError();
}

}  // namespace gdn
