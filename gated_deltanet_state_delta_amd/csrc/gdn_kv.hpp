// gdn_kv.hpp -- what the calls that move tokens into and out of a paged cache
// share: pieces of 8 elements, 8-bit codes, the place of a packed token.
#pragma once

#include "gdn_device.hpp"
#include "gdn_paged.hpp"

namespace gdn {

// Cache elements of 8 bits.
struct e4m3 { uint8_t b; };
struct i8 { int8_t b; };

// 8 elements of a new token, read once.
template <typename IO> struct Piece;
template <> struct Piece<__bf16> {
  u32x4 r;
  __device__ __forceinline__ void load(const __bf16* p) { r = __builtin_nontemporal_load(reinterpret_cast<const u32x4*>(p)); }
  __device__ __forceinline__ float at(int i) const {
    return __uint_as_float((i & 1) ? r[i >> 1] & 0xffff0000u : r[i >> 1] << 16);
  }
  __device__ __forceinline__ void store(__bf16* p) const { *reinterpret_cast<u32x4*>(p) = r; }
};
template <> struct Piece<float> {
  f4 r[2];
  __device__ __forceinline__ void load(const float* p) {
    r[0] = ld_nt(p);
    r[1] = ld_nt(p + 4);
  }
  __device__ __forceinline__ float at(int i) const { return r[i >> 2][i & 3]; }
  __device__ __forceinline__ void store(float* p) const {
    reinterpret_cast<f4*>(p)[0] = r[0];
    reinterpret_cast<f4*>(p)[1] = r[1];
  }
};

// Beyond +-448 clamped; NaN stays NaN.
__device__ __forceinline__ float e4m3_clamp(float q) {
  const float c = __builtin_amdgcn_fmed3f(q, -448.0f, 448.0f);
  return q != q ? q : c;
}

// 4 numbers within +-448 (or NaN) in e4m3, round to nearest even.
__device__ __forceinline__ uint32_t e4m3_pack(const float* q) {
  const uint32_t lo = __builtin_amdgcn_cvt_pk_fp8_f32(q[0], q[1], 0, false);
  return __builtin_amdgcn_cvt_pk_fp8_f32(q[2], q[3], lo, true);
}

// 8 quotients x / scale, clamped, that e4m3_pack rounds as it rounds the fp32
// quotients.  They come from a product with 1 / scale, at most 3 units in the
// last place off; e4m3's values and the midpoints between them have 19 zero bits
// at the end of an fp32 mantissa, so only a product within 16 units of such a
// number can round otherwise than the quotient, and then the lane divides (IEEE
// division, about 12 instructions each: 57 us instead of 40 for 32768 tokens of 8
// heads of 128 with it alone).  inv is 0 where 1 / scale is not a normal number:
// always divide.
template <typename X>
__device__ __forceinline__ void e4m3_quotients(const X& x, float scale, float inv, float* q) {
  uint32_t near = 0x7ffffu;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    q[i] = x.at(i) * inv;
    near = min(near, (__float_as_uint(q[i]) + 16u) & 0x7ffffu);
  }
  if (near < 32u || inv == 0.f) {
#pragma unroll
    for (int i = 0; i < 8; ++i) q[i] = x.at(i) / scale;
  }
#pragma unroll
  for (int i = 0; i < 8; ++i) q[i] = e4m3_clamp(q[i]);
}

// 1 / scale to 1 unit in the last place, 0 where it is not a normal number.
__device__ __forceinline__ float normal_rcp(float scale) {
  const float one = __builtin_amdgcn_rcpf(scale);
  return fabsf(one) >= 1.2e-38f && fabsf(one) <= 3.0e38f ? one : 0.f;
}

// Token i of a packed batch: its row b and how many tokens there are from it to
// its row's end, or false for a token of no row.  P has cu, batch, T, total.
// (A copy of the offsets in LDS, searched there, gained nothing: 2048 tokens of
// 256 rows read back in 7.5 us with it, 7.2 without.)
template <typename P>
__device__ __forceinline__ bool token_row(const P& p, int64_t i, int& b, int64_t& back) {
  if (!p.cu) {
    b = (int)(i / p.T);
    back = p.T - i % p.T;
    return true;
  }
  // the last row that starts at or before token i (offsets clamped to
  // [0, total]); a token past that row's end belongs to none.  Offsets that
  // decrease mislead the search, and the check of the range then leaves the
  // token out.
  int lo = 0, hi = p.batch;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (min(max((int64_t)p.cu[mid], (int64_t)0), p.total) <= i) lo = mid;
    else hi = mid;
  }
  b = lo;
  const int64_t s0 = min(max((int64_t)p.cu[b], (int64_t)0), p.total), s1 = min(max((int64_t)p.cu[b + 1], (int64_t)0), p.total);
  back = s1 - i;
  return s0 <= i && i < s1;
}

}  // namespace gdn
