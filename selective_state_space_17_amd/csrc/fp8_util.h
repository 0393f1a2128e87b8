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
struct E4m3 {};                  // the type of a kernel's inputs that are in 8 bits

inline __host__ __device__ int64_t fp8_blocks(int64_t cols) { return (cols + kBlock - 1) / kBlock; }
inline __host__ __device__ int64_t fp8_lines(int64_t rows) { return (rows + 3) / 4 * 4; }

// Magnitudes are compared as the bits of |v|, where infinities and NaN are above every finite value.
constexpr uint32_t kInfinite = 0x7f800000u;
__device__ __forceinline__ uint32_t magnitude(float v) { return __float_as_uint(v) & 0x7fffffffu; }
// of a finite value; 0 otherwise
__device__ __forceinline__ uint32_t finite_magnitude(float v) {
  const uint32_t m = magnitude(v);
  return m < kInfinite ? m : 0;
}
__device__ __forceinline__ uint32_t larger(uint32_t a, uint32_t b) { return a > b ? a : b; }
// a block's scale from its largest finite magnitude: 448 = 1.75 x 2^8, and what is above 1.75 x 2^k needs one power more
__device__ __forceinline__ uint32_t fp8_scale(uint32_t top) {
  const int e = static_cast<int>((top + 0x1fffffu) >> 23) - 8;
  return top == 0 ? kOne : e < 1 ? 1 : e;
}
// and a code's factor from its scale (byte 0: 2^-127, 255: NaN, whose bits beside the exponent are the same)
__device__ __forceinline__ float fp8_power(uint32_t scale) {
  return __uint_as_float(scale << 23 | (((scale + 1) & 255u) < 2 ? 0x400000u : 0u));
}
// four values, divided by a scale from fp8_scale() that brings them to 448 or less, to codes, to nearest even;
// infinities and NaN to NaN
typedef short i16x2_t __attribute__((ext_vector_type(2)));
__device__ __forceinline__ uint32_t fp8_codes(float a, float b, float c, float d, uint32_t scale) {
  const float s = __uint_as_float(scale << 23);
  i16x2_t v = __builtin_amdgcn_cvt_scalef32_pk_fp8_f32(i16x2_t{0, 0}, a, b, s, false);
  v = __builtin_amdgcn_cvt_scalef32_pk_fp8_f32(v, c, d, s, true);
  return __builtin_bit_cast(uint32_t, v);
}
__device__ __forceinline__ void fp8_values(uint32_t codes, float (&v)[4]) {
  const f32x2_t lo = __builtin_amdgcn_cvt_pk_f32_fp8(static_cast<int>(codes), false);
  const f32x2_t hi = __builtin_amdgcn_cvt_pk_f32_fp8(static_cast<int>(codes), true);
  v[0] = lo[0]; v[1] = lo[1]; v[2] = hi[0]; v[3] = hi[1];
}
// largest of a row of 16 lanes, in each of them
__device__ __forceinline__ uint32_t row16_max(uint32_t v) {
  v = larger(v, dpp_or_zero<0x128, 0xf>(v));   // row_ror:8
  v = larger(v, dpp_or_zero<0x124, 0xf>(v));
  v = larger(v, dpp_or_zero<0x122, 0xf>(v));
  return larger(v, dpp_or_zero<0x121, 0xf>(v));
}
// largest of the lanes 16, 32 and 48 apart, in each of them
__device__ __forceinline__ uint32_t column4_max(uint32_t v) {
  const auto a = __builtin_amdgcn_permlane16_swap(v, v, false, false);
  const uint32_t w = larger(a[0], a[1]);
  const auto b = __builtin_amdgcn_permlane32_swap(w, w, false, false);
  return larger(b[0], b[1]);
}
// 16 lanes with 8 neighbouring values each hold a block of a row: their codes, and the block's scale (in each lane)
__device__ __forceinline__ u32x2_t fp8_block_codes(const float (&v)[8], uint32_t& scale) {
  uint32_t top = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) top = larger(top, magnitude(v[i]));
  top = row16_max(top);
  if (top >= kInfinite) {   // (the 16 lanes together)
    top = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) top = larger(top, finite_magnitude(v[i]));
    top = row16_max(top);
  }
  scale = fp8_scale(top);
  return u32x2_t{fp8_codes(v[0], v[1], v[2], v[3], scale), fp8_codes(v[4], v[5], v[6], v[7], scale)};
}

}  // namespace mssm
