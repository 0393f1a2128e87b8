// Device helpers shared by the embedding, norm and cross-entropy kernels.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace mssm {

constexpr int kLanes = 64;   // a gfx950 wave

typedef __bf16 bf16x2_t __attribute__((ext_vector_type(2)));
typedef float f32x2_t __attribute__((ext_vector_type(2)));
typedef float f32x4_t __attribute__((ext_vector_type(4)));
typedef unsigned int u32x2_t __attribute__((ext_vector_type(2)));
typedef unsigned int u32x4_t __attribute__((ext_vector_type(4)));

// two floats -> packed bf16 pair, round to nearest even
__device__ __forceinline__ uint32_t pack_bf16(float a, float b) {
  return __builtin_bit_cast(uint32_t, __builtin_convertvector(f32x2_t{a, b}, bf16x2_t));
}

__device__ __forceinline__ float widen(float v) { return v; }
__device__ __forceinline__ float widen(uint16_t v) { return __uint_as_float(static_cast<uint32_t>(v) << 16); }
template <typename T> __device__ __forceinline__ T narrow(float v);
template <> __device__ __forceinline__ float narrow<float>(float v) { return v; }
template <> __device__ __forceinline__ uint16_t narrow<uint16_t>(float v) {
  return __builtin_bit_cast(uint16_t, static_cast<__bf16>(v));
}
// v as it reads back after being stored as T
template <typename T> __device__ __forceinline__ float rounded(float v) { return widen(narrow<T>(v)); }

// The same vectors at any element's address: gfx950 takes wide global accesses at any alignment, so rows of an
// odd length are read as widely as others.
typedef f32x4_t f32x4_u __attribute__((aligned(4)));
typedef u32x4_t u32x4_u __attribute__((aligned(2)));
typedef u32x2_t u32x2_u __attribute__((aligned(2)));

// V = 4 or 8 consecutive elements at p, any alignment
template <int V> __device__ __forceinline__ void load_row(const float* p, float (&v)[V]) {
#pragma unroll
  for (int i = 0; i < V / 4; ++i) {
    const f32x4_t t = *reinterpret_cast<const f32x4_u*>(p + 4 * i);
    v[4 * i] = t[0]; v[4 * i + 1] = t[1]; v[4 * i + 2] = t[2]; v[4 * i + 3] = t[3];
  }
}
__device__ __forceinline__ void split_bf16(uint32_t w, float& a, float& b) {
  a = __uint_as_float(w << 16);
  b = __uint_as_float(w & 0xffff0000u);
}
template <int V> __device__ __forceinline__ void load_row(const uint16_t* p, float (&v)[V]) {
  if constexpr (V == 8) {
    const u32x4_t t = *reinterpret_cast<const u32x4_u*>(p);
#pragma unroll
    for (int i = 0; i < 4; ++i) split_bf16(t[i], v[2 * i], v[2 * i + 1]);
  } else {
    const u32x2_t t = *reinterpret_cast<const u32x2_u*>(p);
    split_bf16(t[0], v[0], v[1]);
    split_bf16(t[1], v[2], v[3]);
  }
}
template <int V> __device__ __forceinline__ void store_row(float* p, const float (&v)[V]) {
#pragma unroll
  for (int i = 0; i < V / 4; ++i)
    *reinterpret_cast<f32x4_u*>(p + 4 * i) = f32x4_t{v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]};
}
template <int V> __device__ __forceinline__ void store_row(uint16_t* p, const float (&v)[V]) {
  if constexpr (V == 8) {
    *reinterpret_cast<u32x4_u*>(p) = u32x4_t{pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3]), pack_bf16(v[4], v[5]),
                                             pack_bf16(v[6], v[7])};
  } else {
    *reinterpret_cast<u32x2_u*>(p) = u32x2_t{pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3])};
  }
}
// the first n of V elements (n <= 0: none, and n >= V: all); what is not there reads as zero
template <int V, typename T> __device__ __forceinline__ void load_row(const T* p, float (&v)[V], int64_t n) {
  if (n >= V) {
    load_row<V>(p, v);
  } else {
#pragma unroll
    for (int i = 0; i < V; ++i) v[i] = i < n ? widen(p[i]) : 0.f;
  }
}
template <int V, typename T> __device__ __forceinline__ void store_row(T* p, const float (&v)[V], int64_t n) {
  if (n >= V) {
    store_row<V>(p, v);
  } else {
#pragma unroll
    for (int i = 0; i < V; ++i)
      if (i < n) p[i] = narrow<T>(v[i]);
  }
}

// v of another lane by a DPP move; lanes outside the row mask, or without a source, get 0
template <int CTRL, int ROWS> __device__ __forceinline__ uint32_t dpp_or_zero(uint32_t v) {
  return static_cast<uint32_t>(__builtin_amdgcn_update_dpp(0, static_cast<int>(v), CTRL, ROWS, 0xf, true));
}
// sum over the lanes up to and including this one: within rows of 16, then across rows (row_bcast)
__device__ __forceinline__ uint32_t wave_prefix(uint32_t v) {
  v += dpp_or_zero<0x111, 0xf>(v);   // row_shr:1
  v += dpp_or_zero<0x112, 0xf>(v);
  v += dpp_or_zero<0x114, 0xf>(v);
  v += dpp_or_zero<0x118, 0xf>(v);
  v += dpp_or_zero<0x142, 0xa>(v);   // row_bcast:15 into rows 1 and 3
  v += dpp_or_zero<0x143, 0xc>(v);   // row_bcast:31 into rows 2 and 3
  return v;
}
// sum over the wave's 64 lanes, in every lane (the same order of additions every time)
__device__ __forceinline__ float wave_sum(float v) {
  auto add = [&](uint32_t o) { v += __uint_as_float(o); };
  add(dpp_or_zero<0x111, 0xf>(__float_as_uint(v)));
  add(dpp_or_zero<0x112, 0xf>(__float_as_uint(v)));
  add(dpp_or_zero<0x114, 0xf>(__float_as_uint(v)));
  add(dpp_or_zero<0x118, 0xf>(__float_as_uint(v)));
  add(dpp_or_zero<0x142, 0xa>(__float_as_uint(v)));
  add(dpp_or_zero<0x143, 0xc>(__float_as_uint(v)));
  return __uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(v), 63));
}

// ids and targets are int32 or int64
__device__ __forceinline__ int64_t id_at(const void* ids, int id_bytes, int64_t i) {
  return id_bytes == 8 ? static_cast<const int64_t*>(ids)[i] : static_cast<const int32_t*>(ids)[i];
}
// those at first, first + step, ...: all loads at once (id_at's branch would have each wait for the one before);
// from end on the last one again
template <int E>
__device__ __forceinline__ void ids_at(const void* ids, int id_bytes, int64_t first, int64_t step, int64_t end,
                                       int64_t (&v)[E]) {
  auto all = [&](auto* from) {
#pragma unroll
    for (int e = 0; e < E; ++e) {
      const int64_t i = first + e * step;
      v[e] = from[i < end ? i : end - 1];
    }
  };
  if (id_bytes == 8) all(static_cast<const int64_t*>(ids));
  else all(static_cast<const int32_t*>(ids));
}

}  // namespace mssm
