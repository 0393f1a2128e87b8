// Matrices kept in 8 bits with a power of two for each block of 128 (fp8_util.h): rounded from fp32 or bf16, in either
// order or both from one read; laid out the other way from 8 bits; read back.
//
// A workgroup takes tiles of 128 x 128, so that a tile is one block along either axis: a thread holds 8 rows x 8
// columns in registers, finds the largest magnitudes of its rows (over 16 lanes) and of its columns (over the
// workgroup), and rounds with either; the transposed codes change places in LDS.  Bound by memory: each input is read
// once and each output written once.
// A matrix in 8 bits laid out the other way loses little: with powers of two its values are e4m3 numbers whatever the
// scale, so under another block's scale they stay what they are, except below 2^-6 of it, where e4m3's steps stop
// shrinking.
#include <type_traits>

#include "fp8_util.h"
#include "internal.h"

namespace mssm {
namespace {

struct TileParams {
  int64_t rows, cols, tiles;
  int tiles_c;
  const void* x;                 // fp32, bf16, or e4m3 codes
  const unsigned char* x_scales; // of the codes (of rows)
  unsigned char* codes;          // nullable
  unsigned char* scales;
  unsigned char* codes_t;        // nullable
  unsigned char* scales_t;
};

constexpr int kThreads = 256;
struct E4m3 {};   // the type of inputs that are in 8 bits

template <typename T, bool SQUARE> __global__ __launch_bounds__(kThreads) void tile_kernel(TileParams p) {
  __shared__ float tops[4][kBlock];
  __shared__ __attribute__((aligned(16))) uint64_t turned[kBlock][16];   // [column][8 rows], its place xor-ed with the chunk
  const int chunk = threadIdx.x % 16, rg = threadIdx.x / 16;
  const int wave = threadIdx.x / kLanes, lane = threadIdx.x % kLanes;
  const int64_t pitch = static_cast<int64_t>(p.tiles_c) * kBlock;            // of the codes
  const int64_t tiles_r = fp8_blocks(p.rows), pitch_t = tiles_r * kBlock;    // of the transposed ones
  const int64_t lines = fp8_lines(p.rows), lines_t = fp8_lines(p.cols);
  for (int64_t tile = blockIdx.x; tile < p.tiles; tile += gridDim.x) {
    const int64_t tr = tile / p.tiles_c, r0 = tr * kBlock + rg * 8;
    const int tc = static_cast<int>(tile - tr * p.tiles_c), c0 = tc * kBlock + chunk * 8;
    float v[8][8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int64_t r = r0 + i;
      if constexpr (std::is_same_v<T, E4m3>) {
        u32x2_t q = {0, 0};
        float s = 1.f;
        if (r < p.rows) {
          q = *reinterpret_cast<const u32x2_t*>(static_cast<const unsigned char*>(p.x) + r * pitch + c0);
          s = fp8_power(p.x_scales[tc * lines + r]);
        }
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          float f[4];
          fp8_values(q[h], f);
#pragma unroll
          for (int e = 0; e < 4; ++e) v[i][4 * h + e] = f[e] * s;
        }
      } else {
        load_row<8>(static_cast<const T*>(p.x) + r * p.cols + c0, v[i], r < p.rows ? p.cols - c0 : 0);
      }
    }
    float col_top[8];
    if (SQUARE || p.codes_t != nullptr) {
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        float t = 0.f;
#pragma unroll
        for (int i = 0; i < 8; ++i) t = __builtin_fmaxf(t, finite_abs(v[i][j]));
        t = __builtin_fmaxf(t, __shfl_xor(t, 16, kLanes));
        col_top[j] = __builtin_fmaxf(t, __shfl_xor(t, 32, kLanes));
      }
      __syncthreads();   // (the tile before may still be read)
      if (lane < 16) {
#pragma unroll
        for (int j = 0; j < 8; ++j) tops[wave][chunk * 8 + j] = col_top[j];
      }
      __syncthreads();
#pragma unroll
      for (int j = 0; j < 8; ++j)
#pragma unroll
        for (int w = 0; w < 4; ++w) col_top[j] = __builtin_fmaxf(col_top[j], tops[w][chunk * 8 + j]);
    }
    uint32_t all = 0;
    if constexpr (SQUARE) {
      float t = 0.f;
#pragma unroll
      for (int j = 0; j < 8; ++j) t = __builtin_fmaxf(t, col_top[j]);
      all = fp8_scale(row16_max(t));
      if (threadIdx.x == 0) {
        if (p.codes != nullptr) p.scales[tc * tiles_r + tr] = static_cast<unsigned char>(all);
        if (p.codes_t != nullptr) p.scales_t[tr * p.tiles_c + tc] = static_cast<unsigned char>(all);
      }
    }
    if (p.codes != nullptr) {
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int64_t r = r0 + i;
        u32x2_t q;
        if constexpr (SQUARE) {
          const float s = fp8_inverse(all);
          q = u32x2_t{fp8_codes(v[i][0] * s, v[i][1] * s, v[i][2] * s, v[i][3] * s),
                      fp8_codes(v[i][4] * s, v[i][5] * s, v[i][6] * s, v[i][7] * s)};
        } else {
          uint32_t scale;
          q = fp8_block_codes(v[i], scale);   // (1 for the rows that pad the scales' lines)
          if (chunk == 0 && r < lines) p.scales[tc * lines + r] = static_cast<unsigned char>(scale);
        }
        if (r < p.rows) *reinterpret_cast<u32x2_t*>(p.codes + r * pitch + c0) = q;
      }
    }
    if (p.codes_t != nullptr) {
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const uint32_t scale = SQUARE ? all : fp8_scale(col_top[j]);
        const float s = fp8_inverse(scale);
        const int64_t c = c0 + j;
        if (!SQUARE && rg == 0 && c < lines_t) p.scales_t[tr * lines_t + c] = static_cast<unsigned char>(scale);
        const uint64_t lo = fp8_codes(v[0][j] * s, v[1][j] * s, v[2][j] * s, v[3][j] * s);
        const uint64_t hi = fp8_codes(v[4][j] * s, v[5][j] * s, v[6][j] * s, v[7][j] * s);
        turned[chunk * 8 + j][rg ^ chunk] = lo | hi << 32;
      }
      __syncthreads();
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const int c = k * 32 + threadIdx.x / 8, pair = threadIdx.x % 8 * 2;
        const uint64_t a = turned[c][pair ^ (c / 8)], b = turned[c][(pair + 1) ^ (c / 8)];
        if (tc * kBlock + c < p.cols)
          *reinterpret_cast<u32x4_t*>(p.codes_t + (tc * static_cast<int64_t>(kBlock) + c) * pitch_t + tr * kBlock + pair * 8) =
              u32x4_t{static_cast<uint32_t>(a), static_cast<uint32_t>(a >> 32), static_cast<uint32_t>(b),
                      static_cast<uint32_t>(b >> 32)};
      }
    }
  }
}

// values back from 8 bits, 8 a thread
struct BackParams {
  int64_t rows, cols, chunks;    // chunks of 8 columns, rows x (cols / 8 rounded up)
  int square;
  const unsigned char* codes;
  const unsigned char* scales;
  void* out;
};
template <typename T> __global__ __launch_bounds__(kThreads) void back_kernel(BackParams p) {
  const int64_t per = (p.cols + 7) / 8, pitch = fp8_blocks(p.cols) * kBlock;
  const int64_t lines = p.square ? fp8_blocks(p.rows) : fp8_lines(p.rows);
  for (int64_t i = static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x; i < p.chunks;
       i += static_cast<int64_t>(gridDim.x) * kThreads) {
    const int64_t r = i / per, c = (i - r * per) * 8;
    const u32x2_t q = *reinterpret_cast<const u32x2_t*>(p.codes + r * pitch + c);
    const float s = fp8_power(p.scales[c / kBlock * lines + (p.square ? r / kBlock : r)]);
    float v[8];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      float f[4];
      fp8_values(q[h], f);
#pragma unroll
      for (int e = 0; e < 4; ++e) v[4 * h + e] = f[e] * s;
    }
    store_row<8>(static_cast<T*>(p.out) + r * p.cols + c, v, p.cols - c);
  }
}

// workgroups of a kernel that walks over its work
unsigned grid(int64_t work) { return static_cast<unsigned>(work < (1 << 20) ? work : 1 << 20); }

TileParams tile_params(const Fp8Args& a) {
  TileParams p{};
  p.rows = a.rows; p.cols = a.cols; p.tiles_c = static_cast<int>(fp8_blocks(a.cols));
  p.tiles = fp8_blocks(a.rows) * p.tiles_c;
  p.codes_t = static_cast<unsigned char*>(a.t.codes); p.scales_t = static_cast<unsigned char*>(a.t.scales);
  return p;
}

}  // namespace

hipError_t fp8_quantize_launch(const Fp8Args& a, hipStream_t stream) {
  if (a.rows == 0) return hipSuccess;
  TileParams p = tile_params(a);
  p.x = a.x;
  p.codes = static_cast<unsigned char*>(a.m.codes); p.scales = static_cast<unsigned char*>(a.m.scales);
  auto go = [&](auto kernel) { kernel<<<dim3(grid(p.tiles)), kThreads, 0, stream>>>(p); };
  if (a.io) go(a.square ? tile_kernel<uint16_t, true> : tile_kernel<uint16_t, false>);
  else go(a.square ? tile_kernel<float, true> : tile_kernel<float, false>);
  return hipGetLastError();
}

hipError_t fp8_transpose_launch(const Fp8Args& a, hipStream_t stream) {
  if (a.rows == 0) return hipSuccess;
  TileParams p = tile_params(a);
  p.x = a.m.codes; p.x_scales = static_cast<const unsigned char*>(a.m.scales);
  tile_kernel<E4m3, false><<<dim3(grid(p.tiles)), kThreads, 0, stream>>>(p);
  return hipGetLastError();
}

hipError_t fp8_dequantize_launch(const Fp8Args& a, hipStream_t stream) {
  if (a.rows == 0) return hipSuccess;
  BackParams p{};
  p.rows = a.rows; p.cols = a.cols; p.chunks = a.rows * ((a.cols + 7) / 8); p.square = a.square;
  p.codes = static_cast<const unsigned char*>(a.m.codes); p.scales = static_cast<const unsigned char*>(a.m.scales);
  p.out = a.out;
  const unsigned blocks = grid((p.chunks + kThreads - 1) / kThreads);
  if (a.io) back_kernel<uint16_t><<<dim3(blocks), kThreads, 0, stream>>>(p);
  else back_kernel<float><<<dim3(blocks), kThreads, 0, stream>>>(p);
  return hipGetLastError();
}

}  // namespace mssm
