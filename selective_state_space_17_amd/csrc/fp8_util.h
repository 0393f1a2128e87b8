// Matrices in 8 bits as the kernels read and write them.
//
// A matrix [rows, cols]: e4m3 codes [rows][128 blocks], blocks = ceil(cols / 128), zeros past cols, and a power of two
// for each block as e8m0 (a byte b: 2^(b - 127)): of 128 columns of a row, [blocks][lines], lines = rows rounded up to 4,
// or of 128 x 128, [blocks][ceil(rows / 128)].  Blocks stand outermost, so that the scales of a tile's rows are one
// stretch of memory, four of them a word.
//
// The scale is the least power of two that brings the block's largest finite magnitude to 448 or less, e4m3's largest
// value (2^-126 at the least; 1 for a block without a value but zero).  A power of two, so that dividing by it is exact
// and the codes alone carry the rounding: half a step of e4m3 (2^-4 of the value; 2^-10 of the scale below 2^-6 of it).
#pragma once

#include "device_util.h"

namespace mssm {

constexpr int kBlock = 128;      // values that share a scale, along a row
constexpr int kOne = 127;        // the byte of 2^0

inline __host__ __device__ int64_t fp8_blocks(int64_t cols) { return (cols + kBlock - 1) / kBlock; }
inline __host__ __device__ int64_t fp8_lines(int64_t rows) { return (rows + 3) / 4 * 4; }

// |v| where it is finite, else 0
__device__ __forceinline__ float finite_abs(float v) {
  const float a = __builtin_fabsf(v);
  return a < __builtin_inff() ? a : 0.f;   // (NaN: 0)
}
// a block's scale from its largest finite magnitude: 448 = 1.75 x 2^8, and what is above 1.75 x 2^k needs one power more
__device__ __forceinline__ uint32_t fp8_scale(float top) {
  const int e = static_cast<int>((__float_as_uint(top) + 0x1fffffu) >> 23) - 8;
  return top == 0.f ? kOne : e < 1 ? 1 : e;
}
// what a value is multiplied by before its rounding
__device__ __forceinline__ float fp8_inverse(uint32_t scale) { return __uint_as_float((254u - scale) << 23); }
// and a code's value by after it (byte 0: 2^-127, 255: NaN)
__device__ __forceinline__ float fp8_power(uint32_t scale) {
  return scale == 0 ? 0x1p-127f : scale == 255 ? __builtin_nanf("") : __uint_as_float(scale << 23);
}
// four values of magnitude 448 or less to codes, to nearest even; infinities and NaN to NaN
__device__ __forceinline__ uint32_t fp8_codes(float a, float b, float c, float d) {
  int v = __builtin_amdgcn_cvt_pk_fp8_f32(a, b, 0, false);
  v = __builtin_amdgcn_cvt_pk_fp8_f32(c, d, v, true);
  return static_cast<uint32_t>(v);
}
__device__ __forceinline__ void fp8_values(uint32_t codes, float (&v)[4]) {
  const f32x2_t lo = __builtin_amdgcn_cvt_pk_f32_fp8(static_cast<int>(codes), false);
  const f32x2_t hi = __builtin_amdgcn_cvt_pk_f32_fp8(static_cast<int>(codes), true);
  v[0] = lo[0]; v[1] = lo[1]; v[2] = hi[0]; v[3] = hi[1];
}
// largest of a row of 16 lanes, in each of them
__device__ __forceinline__ float row16_max(float v) {
  v = __builtin_fmaxf(v, __uint_as_float(dpp_or_zero<0x128, 0xf>(__float_as_uint(v))));   // row_ror:8
  v = __builtin_fmaxf(v, __uint_as_float(dpp_or_zero<0x124, 0xf>(__float_as_uint(v))));
  v = __builtin_fmaxf(v, __uint_as_float(dpp_or_zero<0x122, 0xf>(__float_as_uint(v))));
  return __builtin_fmaxf(v, __uint_as_float(dpp_or_zero<0x121, 0xf>(__float_as_uint(v))));
}
// 16 lanes with 8 neighbouring values each hold a block of a row: their codes, and the block's scale (in each lane)
__device__ __forceinline__ u32x2_t fp8_block_codes(const float (&v)[8], uint32_t& scale) {
  float top = 0.f;
#pragma unroll
  for (int i = 0; i < 8; ++i) top = __builtin_fmaxf(top, finite_abs(v[i]));
  scale = fp8_scale(row16_max(top));
  const float s = fp8_inverse(scale);
  return u32x2_t{fp8_codes(v[0] * s, v[1] * s, v[2] * s, v[3] * s), fp8_codes(v[4] * s, v[5] * s, v[6] * s, v[7] * s)};
}

}  // namespace mssm
