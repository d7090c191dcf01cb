// gdn_attn_decode.hip -- launch of the attention over a paged cache: the
// split over the rows' lengths and the kernel that joins its parts.
#include "gdn_attn_decode.hpp"

namespace gdn {

// Joins the parts of one (row, head, token): out = sum_s e^{m_s - M} o_s /
// sum_s e^{m_s - M} l_s.  Latency-bound: WPR waves take its parts in turn,
// eight loads in flight each, the weights in the lanes of one wave.  A row's
// parts: slot 2k + 1 of its first share k, then slots 2k of the shares behind.
// The fewer the rows, the more parts each has: sixteen waves a row (joined
// through LDS) up to 256 rows, four up to 1024, one beyond.  Attention and
// join with sixteen and with four: 12 rows of hundreds of parts (3 rows of
// 19 620 tokens, fp32) 32.8 and 34.8 us, 18 rows (19 870 tokens, heads of 256)
// 42.0 and 45.8, 156 rows of few parts the same.  Four also for up to 32 parts a
// row, taken over the batch, of a block-scaled cache, which they load at once (1 row
// of 1003 tokens, 8 heads of 128: 9.6 us against 10.1; 4 rows 10.6 and 11.2; 2 rows
// of 1500 the same).  Other caches keep the choice that was measured for them.
template <typename IO, int D, int WPR>
__global__ void __launch_bounds__(WPR > 1 ? 64 * WPR : 256) attn_join_kernel(AttnParams p) {
  constexpr int V = D < 64 ? 1 : D / 64;  // dimensions of a lane (the first 32 lanes' for D = 32)
  __shared__ float red[WPR > 1 ? WPR : 1][64 * V];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int64_t id = WPR > 1 ? blockIdx.x : (int64_t)blockIdx.x * 4 + wave;
  if (id >= (int64_t)p.batch * p.hkv * p.R) return;
  const int r = (int)(id % p.R), bh = (int)(id / p.R), h = bh % p.hkv, b = bh / p.hkv;
  const int2 row = p.plan[b];
  const int k0 = __builtin_amdgcn_readfirstlane(row.x), n = __builtin_amdgcn_readfirstlane(row.y);
  if (n == 1) return;  // a whole row, finished where it was walked
  const int d = min(lane * V, D - V);
  auto part = [&](int s) { return ((int64_t)(s == 0 ? 2 * k0 + 1 : 2 * (k0 + s)) * p.hkv + h) * p.R + r; };

  float m = -__builtin_inff();
  for (int s = lane; s < n; s += 64) m = fmaxf(m, p.part_ml[part(s) * 2]);
  for (int o = 32; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor(m, o));
  const float mu = m == -__builtin_inff() ? 0.f : m;
  float l = 0.f, acc[V];
#pragma unroll
  for (int v = 0; v < V; ++v) acc[v] = 0.f;
  for (int s0 = 0; s0 < n; s0 += 64) {
    float w = 0.f;
    if (s0 + lane < n) {
      const float* ml = p.part_ml + part(s0 + lane) * 2;
      w = exp2_hw(ml[0] - mu);
      l += ml[1] * w;
    }
    const int top = min(64, n - s0);
    for (int j = WPR > 1 ? wave : 0; j < top; j += 8 * WPR) {
      float o[8][V];
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float* src = p.part_o + part(s0 + min(j + i * WPR, top - 1)) * D + d;
#pragma unroll
        for (int v = 0; v < V; ++v) o[i][v] = src[v];
      }
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int at = j + i * WPR;
        const float e = __int_as_float(__builtin_amdgcn_readlane(__float_as_int(w), min(at, 63)));
        if (at < top)
#pragma unroll
          for (int v = 0; v < V; ++v) acc[v] += e * o[i][v];
      }
    }
  }
  for (int o = 32; o > 0; o >>= 1) l += __shfl_xor(l, o);
  if constexpr (WPR > 1) {
#pragma unroll
    for (int v = 0; v < V; ++v) red[wave][lane * V + v] = acc[v];
    __syncthreads();
    if (wave != 0) return;
#pragma unroll
    for (int w = 1; w < WPR; ++w)
#pragma unroll
      for (int v = 0; v < V; ++v) acc[v] += red[w][lane * V + v];
  }
  const int t = r / p.group, hq = h * p.group + r % p.group;
  const int64_t at = ((int64_t)b * p.T + t) * p.hq + hq;
  if (lane * V < D) {
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const float out = attn_out(acc[v], l, attn_inv(p, l, h));
      if constexpr (sizeof(IO) == 2) ((__bf16*)p.out)[at * D + d + v] = (__bf16)out;
      else ((float*)p.out)[at * D + d + v] = out;
    }
  }
  if (p.lse && lane == 0) p.lse[at] = attn_lse(m, l);
}

template <typename IO, int D>
static void launch_join_d(const AttnParams& p, hipStream_t stream) {
  const int64_t rows = (int64_t)p.batch * p.hkv * p.R;
  const bool few_parts = p.block > 0 && p.shares <= 32 * (int64_t)p.batch;
  if (rows <= 256 && !few_parts) hipLaunchKernelGGL((attn_join_kernel<IO, D, 16>), dim3((unsigned)rows), dim3(1024), 0, stream, p);
  else if (rows <= 1024) hipLaunchKernelGGL((attn_join_kernel<IO, D, 4>), dim3((unsigned)rows), dim3(256), 0, stream, p);
  else hipLaunchKernelGGL((attn_join_kernel<IO, D, 1>), dim3((unsigned)((rows + 3) / 4)), dim3(256), 0, stream, p);
}
template <typename IO>
static void launch_join(const AttnParams& p, int d, hipStream_t stream) {
  if (d == 32) launch_join_d<IO, 32>(p, stream);
  else if (d == 64) launch_join_d<IO, 64>(p, stream);
  else if (d == 128) launch_join_d<IO, 128>(p, stream);
  else launch_join_d<IO, 256>(p, stream);
}

// Shares of all rows' steps: waves to fill 256 CUs of 4 SIMDs once (each share
// as large as the next, so that they end together), but no more shares than
// steps if every row is as long as its table.  0: one wave per row, head and
// row tile -- tables of at most four tiles of 32 keys (128 tokens, 8 heads of
// 128, bf16: 8.9 us on the GPU against 10.5 with the second launch; 256 tokens
// 13.2 against 10.6, and four tiles of 16 keys gain nothing), heads and row
// tiles that fill the card by themselves, and batches of so many rows that
// finding the shares would cost more than their evenness gives.
constexpr int kMostRows = 4096;
static int cache_bytes(int dtype) { return dtype == GDN_F32 ? 4 : dtype == GDN_BF16 ? 2 : 1; }
// Row tiles (see attn_rows16) of a key-value head.
static int attn_tiles(const gdn_attn_decode_args& a) {
  const int R = a.T * (a.hq / a.hkv), rows = 16 * attn_rows16(attn_kind(a.T, R), a.d, a.io_dtype == GDN_BF16 ? 2 : 4);
  return (R + rows - 1) / rows;
}
static int attn_shares(const gdn_attn_decode_args& a) {
  const int es = cache_bytes(a.cache_dtype), tile = attn_tile(es, a.d, a.scale_block > 0);
  const int64_t cap = (int64_t)a.max_pages * a.page_size, steps = a.batch * ((cap + tile - 1) / tile);
  const int alone = tile < 32 ? 64 : 128;
  if (cap <= alone || a.batch > kMostRows || (int64_t)a.batch * a.hq * a.T > (1 << 24)) return 0;
  const int64_t each = (int64_t)a.hkv * attn_tiles(a);  // waves of a share
  // Block-scaled caches, bf16 queries, heads of 128 and more, factors at a lane's own place: one wave a SIMD, though
  // there is room for two (4 rows of 131 072 tokens, 4 heads of 128, e4m3: 90 us, two 99; 256 ragged rows up to 4096, 2
  // heads of 256, e4m3 104 and 114, int8 106 and 114; heads of 128 in tokens-first pages 1% either way; fp32 queries
  // 121 and 111, heads of 64 144 and 137).
  const bool one = a.scale_block > 0 && a.io_dtype == GDN_BF16 && a.d >= 128 && attn_lane_blocks(a.page_size, a.scale_block);
  const int64_t fill = 1024 * (one ? 1 : attn_waves(es, a.d, attn_kind(a.T, a.T * (a.hq / a.hkv)))) / each;
  const int64_t n = fill < steps ? fill : steps;
  return n < 2 ? 0 : (int)n;
}

// Instead of shares and the second launch, for short tables of block-scaled
// caches: the four waves of a workgroup take a quarter each of a row, head and
// row tile, and join in LDS.  From 64 tokens, where one wave does as well, to 512,
// while two such workgroups a CU hold everything at a time or two (8 heads of 128,
// bf16 over e4m3: 1 row of 256 tokens 7.3 us against 10.3, of 512 9.6 against
// 11.0, of 1024 16 against 11; 64 rows of 256 12.6 against 17, of 512 19 against
// 23; 256 rows of 256 35 against 30).  Teams of eight waves were slower.  Other
// caches keep one wave, up to the 128 tokens that attn_shares measured for them.
static bool attn_team(const gdn_attn_decode_args& a) {
  const int64_t cap = (int64_t)a.max_pages * a.page_size;
  return a.scale_block > 0 && cap > 64 && cap <= 512 && (int64_t)a.batch * a.hkv * attn_tiles(a) <= 1024;
}

size_t attn_workspace_bytes(const gdn_attn_decode_args& a) {
  if (a.batch == 0 || a.max_pages == 0 || attn_team(a)) return 0;
  const int shares = attn_shares(a);
  if (shares == 0) return 0;
  return (2 * (size_t)shares * a.hq * a.T * (a.d + 2) + 2 * (size_t)a.batch) * sizeof(float);
}

// j / n = (j * mul) >> shift for j < 2^31 and n up to 2^30: with s = ceil(log2(n)) and
// mul = ceil(2^(31 + s) / n), the error of mul is below 2^s.
static void divider(int n, uint32_t& mul, uint32_t& shift) {
  int s = 0;
  while ((1 << s) < n) ++s;
  mul = (uint32_t)((((uint64_t)1 << (31 + s)) + n - 1) / n);
  shift = 31 + s;
}

hipError_t launch_attn_decode(const gdn_attn_decode_args& a, hipStream_t stream) {
  const int io = a.io_dtype == GDN_BF16 ? 2 : 4;
  const int ce = cache_bytes(a.cache_dtype);
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
  p.k_blocks = a.k_block_scale;
  p.v_blocks = a.v_block_scale;
  p.block = a.scale_block;
  p.blk_sp = a.scale_block > 0 ? (int64_t)a.hkv * (a.page_size / a.scale_block) : 0;
  p.nblk = a.scale_block > 0 ? a.page_size / a.scale_block : 0;
  p.scale_log2 = (float)((double)a.scale * 1.4426950408889634);
  p.batch = a.batch;
  p.T = a.T;
  p.hq = a.hq;
  p.hkv = a.hkv;
  p.group = a.hq / a.hkv;
  p.R = a.T * p.group;
  p.ntile = attn_tiles(a);
  p.n_pages = a.n_pages;
  p.page_size = a.page_size;
  p.cap = a.max_pages * a.page_size;
  divider(a.page_size, p.page_mul, p.page_shift);
  divider(a.scale_block > 0 ? a.scale_block : 1, p.blk_mul, p.blk_shift);
  const size_t need = attn_workspace_bytes(a);
  p.team = attn_team(a);
  p.shares = a.batch;
  p.plan = nullptr;
  p.part_o = p.part_ml = nullptr;
  if (need > 0 && a.workspace && a.workspace_bytes >= need) {
    p.shares = attn_shares(a);
    const size_t parts = 2 * (size_t)p.shares * a.hq * a.T;
    p.part_o = (float*)a.workspace;
    p.part_ml = p.part_o + parts * a.d;
    p.plan = (int2*)(p.part_ml + parts * 2);
  }
  // Workgroups of 4 waves: see the kernel's mapping.
  const int rtw = p.ntile > 2 ? 4 : p.ntile, nwg = (p.ntile + rtw - 1) / rtw, per = 8 * (4 / rtw);
  const int64_t units = (int64_t)p.shares * p.hkv;
  const dim3 grid((unsigned)(p.team ? (units + 7) / 8 * 8 * p.ntile : (units + per - 1) / per * 8 * nwg));
  hipError_t e;
  if (a.cache_dtype == GDN_I8)  // block scales always
    e = a.io_dtype == GDN_BF16 ? launch_attn_bf16_i8_blocks(p, a.d, grid, stream) : launch_attn_f32_i8_blocks(p, a.d, grid, stream);
  else if (a.scale_block > 0)
    e = a.io_dtype == GDN_BF16 ? launch_attn_bf16_e4m3_blocks(p, a.d, grid, stream) : launch_attn_f32_e4m3_blocks(p, a.d, grid, stream);
  else if (a.cache_dtype == GDN_E4M3)
    e = a.io_dtype == GDN_BF16 ? launch_attn_bf16_e4m3(p, a.d, grid, stream) : launch_attn_f32_e4m3(p, a.d, grid, stream);
  else
    e = a.io_dtype == GDN_BF16 ? launch_attn_bf16(p, a.d, grid, stream) : launch_attn_f32(p, a.d, grid, stream);
  if (e != hipSuccess || !p.plan) return e;
  if (a.io_dtype == GDN_BF16) launch_join<__bf16>(p, a.d, stream);
  else launch_join<float>(p, a.d, stream);
  return hipGetLastError();
}

}  // namespace gdn
