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

// V consecutive elements (V = 1, 2, 4 or 8; p aligned to min(16, V * sizeof(T)) bytes)
template <int V> __device__ __forceinline__ void load_row(const float* p, float (&v)[V]) {
  if constexpr (V >= 4) {
#pragma unroll
    for (int i = 0; i < V / 4; ++i) {
      const f32x4_t t = *reinterpret_cast<const f32x4_t*>(p + 4 * i);
      v[4 * i] = t[0]; v[4 * i + 1] = t[1]; v[4 * i + 2] = t[2]; v[4 * i + 3] = t[3];
    }
  } else if constexpr (V == 2) {
    const f32x2_t t = *reinterpret_cast<const f32x2_t*>(p);
    v[0] = t[0]; v[1] = t[1];
  } else {
    v[0] = *p;
  }
}
__device__ __forceinline__ void split_bf16(uint32_t w, float& a, float& b) {
  a = __uint_as_float(w << 16);
  b = __uint_as_float(w & 0xffff0000u);
}
template <int V> __device__ __forceinline__ void load_row(const uint16_t* p, float (&v)[V]) {
  if constexpr (V == 8) {
    const u32x4_t t = *reinterpret_cast<const u32x4_t*>(p);
#pragma unroll
    for (int i = 0; i < 4; ++i) split_bf16(t[i], v[2 * i], v[2 * i + 1]);
  } else if constexpr (V == 4) {
    const u32x2_t t = *reinterpret_cast<const u32x2_t*>(p);
    split_bf16(t[0], v[0], v[1]);
    split_bf16(t[1], v[2], v[3]);
  } else if constexpr (V == 2) {
    split_bf16(*reinterpret_cast<const uint32_t*>(p), v[0], v[1]);
  } else {
    v[0] = widen(*p);
  }
}
template <int V> __device__ __forceinline__ void store_row(float* p, const float (&v)[V]) {
  if constexpr (V >= 4) {
#pragma unroll
    for (int i = 0; i < V / 4; ++i)
      *reinterpret_cast<f32x4_t*>(p + 4 * i) = f32x4_t{v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]};
  } else if constexpr (V == 2) {
    *reinterpret_cast<f32x2_t*>(p) = f32x2_t{v[0], v[1]};
  } else {
    *p = v[0];
  }
}
template <int V> __device__ __forceinline__ void store_row(uint16_t* p, const float (&v)[V]) {
  if constexpr (V == 8) {
    *reinterpret_cast<u32x4_t*>(p) = u32x4_t{pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3]), pack_bf16(v[4], v[5]),
                                             pack_bf16(v[6], v[7])};
  } else if constexpr (V == 4) {
    *reinterpret_cast<u32x2_t*>(p) = u32x2_t{pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3])};
  } else if constexpr (V == 2) {
    *reinterpret_cast<uint32_t*>(p) = pack_bf16(v[0], v[1]);
  } else {
    *p = narrow<uint16_t>(v[0]);
  }
}

template <int CTRL> __device__ __forceinline__ float dpp_mov(float v) {
  return __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, v), CTRL, 0xf, 0xf, false));
}
// sum over the wave's 64 lanes, in every lane (the same order of additions every time)
__device__ __forceinline__ float wave_sum(float v) {
  v += dpp_mov<0xB1>(v);    // quad_perm [1,0,3,2]
  v += dpp_mov<0x4E>(v);    // quad_perm [2,3,0,1]
  v += dpp_mov<0x141>(v);   // row_half_mirror
  v += dpp_mov<0x140>(v);   // row_mirror
  v += __shfl_xor(v, 16, 64);
  v += __shfl_xor(v, 32, 64);
  return v;
}

// ids and targets are int32 or int64
__device__ __forceinline__ int64_t id_at(const void* ids, int id_bytes, int64_t i) {
  return id_bytes == 8 ? static_cast<const int64_t*>(ids)[i] : static_cast<const int32_t*>(ids)[i];
}

// largest element count of 8, 4, 2, 1 that divides dim and that every pointer's alignment allows, for
// elements of at most `es` bytes (16-byte accesses at most need 16-byte alignment)
inline int vector_width(int64_t dim, const void* const* ptrs, const int* elem_bytes, int n, int most) {
  for (int v = most; v > 1; v /= 2) {
    bool ok = dim % v == 0;
    for (int i = 0; ok && i < n; ++i) {
      const uintptr_t need = static_cast<uintptr_t>(v * elem_bytes[i] < 16 ? v * elem_bytes[i] : 16);
      ok = ptrs[i] == nullptr || reinterpret_cast<uintptr_t>(ptrs[i]) % need == 0;
    }
    if (ok) return v;
  }
  return 1;
}

}  // namespace mssm
