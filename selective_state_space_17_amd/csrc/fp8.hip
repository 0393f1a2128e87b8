// Matrices kept in 8 bits with a power of two for each block of 128 (fp8_util.h): rounded from fp32 or bf16, in either
// order or both from one read; laid out the other way from 8 bits; read back.
//
// A workgroup takes tiles of 128 x 128, so that a tile is one block along either axis: a thread holds 4 rows x 8
// columns in registers, finds the largest magnitudes of its rows (over 16 lanes) and of its columns (over the
// workgroup), and rounds with either; the transposed codes change places in LDS.  Bound by memory: each input is read
// once and each output written once (both orders of 16384 x 10240 in bf16: 143 us, 671 MB, 4.7 TB/s, in blocks of 128 x 128
// 150; of 16384 x 1536: 24 us, 4.2 TB/s; 16384 x 1536 back to bf16: 14 us, 5.4 TB/s).  With 8 x 8 values a thread registers
// spilled (the first: 218 us).  Laid out the other way from 8 bits less of the rate is reached (16384 x 2560: 27 us, 84 MB,
// 3.2 TB/s; 16384 x 10240: 91, 3.7): half the bytes for the same work on each value, transposed codes leave as 128 bytes a
// column, and the words that change places in LDS meet on banks for a seventh of a CU's cycles.
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
constexpr int kTileThreads = 512;
constexpr int kHigh = 4;   // rows of a thread

struct TileShared {
  uint32_t tops[kTileThreads / kLanes][kBlock];
  uint32_t turned[kBlock][kBlock / kHigh];   // [column][4 rows], the place xor-ed
};

// workgroup `group` of `groups`
template <typename T, bool SQUARE>
__device__ __forceinline__ void tiles(const TileParams& p, int64_t group, int64_t groups, TileShared& shared) {
  constexpr int kWaves = kTileThreads / kLanes;
  auto& tops = shared.tops;
  auto& turned = shared.turned;
  const int chunk = threadIdx.x % 16, rg = threadIdx.x / 16;
  const int wave = threadIdx.x / kLanes, lane = threadIdx.x % kLanes;
  const int64_t pitch = static_cast<int64_t>(p.tiles_c) * kBlock;            // of the codes
  const int64_t tiles_r = fp8_blocks(p.rows), pitch_t = tiles_r * kBlock;    // of the transposed ones
  const int64_t lines = fp8_lines(p.rows), lines_t = fp8_lines(p.cols);
  for (int64_t tile = group; tile < p.tiles; tile += groups) {
    const int64_t tr = tile / p.tiles_c, r0 = tr * kBlock + rg * kHigh;
    const int tc = static_cast<int>(tile - tr * p.tiles_c), c0 = tc * kBlock + chunk * 8;
    float v[kHigh][8];
    if constexpr (std::is_same_v<T, E4m3>) {
      u32x2_t q[kHigh];
#pragma unroll
      for (int i = 0; i < kHigh; ++i)
        q[i] = r0 + i < p.rows
                   ? *reinterpret_cast<const u32x2_t*>(static_cast<const unsigned char*>(p.x) + (r0 + i) * pitch + c0)
                   : u32x2_t{0, 0};
      const uint32_t s = r0 < lines ? *reinterpret_cast<const uint32_t*>(p.x_scales + tc * lines + r0) : 0;
#pragma unroll
      for (int i = 0; i < kHigh; ++i) {
        const float power = r0 + i < p.rows ? fp8_power((s >> (8 * i)) & 255u) : 0.f;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          float f[4];
          fp8_values(q[i][h], f);
#pragma unroll
          for (int e = 0; e < 4; ++e) v[i][4 * h + e] = f[e] * power;
        }
      }
    } else {
#pragma unroll
      for (int i = 0; i < kHigh; ++i)
        load_row<8>(static_cast<const T*>(p.x) + (r0 + i) * p.cols + c0, v[i], r0 + i < p.rows ? p.cols - c0 : 0);
    }
    // largest magnitudes of this thread's part of its rows and columns
    uint32_t row_top[kHigh] = {}, col_top[8] = {}, most = 0;
#pragma unroll
    for (int i = 0; i < kHigh; ++i) {
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const uint32_t m = magnitude(v[i][j]);
        row_top[i] = larger(row_top[i], m);
        col_top[j] = larger(col_top[j], m);
      }
      most = larger(most, row_top[i]);
    }
    if (most >= kInfinite) {
#pragma unroll
      for (int i = 0; i < kHigh; ++i) row_top[i] = 0;
#pragma unroll
      for (int j = 0; j < 8; ++j) col_top[j] = 0;
#pragma unroll
      for (int i = 0; i < kHigh; ++i)
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          row_top[i] = larger(row_top[i], finite_magnitude(v[i][j]));
          col_top[j] = larger(col_top[j], finite_magnitude(v[i][j]));
        }
    }
    if (SQUARE || p.codes_t != nullptr) {
#pragma unroll
      for (int j = 0; j < 8; ++j) col_top[j] = column4_max(col_top[j]);
      __syncthreads();   // (the tile before may still be read)
      if (lane < 16) {
#pragma unroll
        for (int h = 0; h < 2; ++h)
          *reinterpret_cast<u32x4_t*>(&tops[wave][chunk * 8 + 4 * h]) =
              u32x4_t{col_top[4 * h], col_top[4 * h + 1], col_top[4 * h + 2], col_top[4 * h + 3]};
      }
      __syncthreads();
#pragma unroll
      for (int w = 0; w < kWaves; ++w)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const u32x4_t t = *reinterpret_cast<const u32x4_t*>(&tops[w][chunk * 8 + 4 * h]);
#pragma unroll
          for (int e = 0; e < 4; ++e) col_top[4 * h + e] = larger(col_top[4 * h + e], t[e]);
        }
    }
    uint32_t all = 0;
    if constexpr (SQUARE) {
      uint32_t t = 0;
#pragma unroll
      for (int j = 0; j < 8; ++j) t = larger(t, col_top[j]);
      all = fp8_scale(row16_max(t));
      if (threadIdx.x == 0) {
        if (p.codes != nullptr) p.scales[tc * tiles_r + tr] = static_cast<unsigned char>(all);
        if (p.codes_t != nullptr) p.scales_t[tr * p.tiles_c + tc] = static_cast<unsigned char>(all);
      }
    }
    if (p.codes != nullptr) {
      uint32_t word = 0;   // the scales of the four rows (1 for the rows that pad the lines)
#pragma unroll
      for (int i = 0; i < kHigh; ++i) {
        const uint32_t scale = SQUARE ? all : fp8_scale(row16_max(row_top[i]));
        word |= scale << (8 * i);
        if (r0 + i < p.rows)
          *reinterpret_cast<u32x2_t*>(p.codes + (r0 + i) * pitch + c0) =
              u32x2_t{fp8_codes(v[i][0], v[i][1], v[i][2], v[i][3], scale),
                      fp8_codes(v[i][4], v[i][5], v[i][6], v[i][7], scale)};
      }
      if (!SQUARE && chunk == 0 && r0 < lines) *reinterpret_cast<uint32_t*>(p.scales + tc * lines + r0) = word;
    }
    if (p.codes_t != nullptr) {
      uint32_t word[2] = {0, 0};
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const uint32_t scale = SQUARE ? all : fp8_scale(col_top[j]);
        word[j / 4] |= scale << (8 * (j % 4));
        // (a place is 4 rows, and the ways of 16 lanes differ in their chunk's low three bits)
        turned[chunk * 8 + j][rg ^ (chunk % 8 * 4)] = fp8_codes(v[0][j], v[1][j], v[2][j], v[3][j], scale);
      }
      if (!SQUARE && rg == 0) {
#pragma unroll
        for (int h = 0; h < 2; ++h)
          if (c0 + 4 * h < lines_t) *reinterpret_cast<uint32_t*>(p.scales_t + tr * lines_t + c0 + 4 * h) = word[h];
      }
      __syncthreads();
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        const int c = k * 64 + threadIdx.x / 8, at = threadIdx.x % 8 * 4;
        const u32x4_t q = *reinterpret_cast<const u32x4_t*>(&turned[c][at ^ (c / 8 % 8 * 4)]);
        if (tc * kBlock + c < p.cols)
          *reinterpret_cast<u32x4_t*>(p.codes_t + (tc * static_cast<int64_t>(kBlock) + c) * pitch_t + tr * kBlock + at * 4) = q;
      }
    }
  }
}

template <typename T, bool SQUARE> __global__ __launch_bounds__(kTileThreads, 4) void tile_kernel(TileParams p) {
  __shared__ __attribute__((aligned(16))) TileShared shared;
  tiles<T, SQUARE>(p, blockIdx.x, gridDim.x, shared);
}

// a plain matrix and one in 8 bits side by side: the first `split` workgroups have the plain one
template <typename T>
__global__ __launch_bounds__(kTileThreads, 4) void two_kernel(TileParams plain, TileParams packed, unsigned split) {
  __shared__ __attribute__((aligned(16))) TileShared shared;
  if (blockIdx.x < split) tiles<T, false>(plain, blockIdx.x, split, shared);
  else tiles<E4m3, false>(packed, blockIdx.x - split, gridDim.x - split, shared);
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

namespace {
TileParams quantize_params(const Fp8Args& a) {
  TileParams p = tile_params(a);
  p.x = a.x;
  p.codes = static_cast<unsigned char*>(a.m.codes); p.scales = static_cast<unsigned char*>(a.m.scales);
  return p;
}
TileParams transpose_params(const Fp8Args& a) {
  TileParams p = tile_params(a);
  p.x = a.m.codes; p.x_scales = static_cast<const unsigned char*>(a.m.scales);
  return p;
}
}  // namespace

hipError_t fp8_quantize_launch(const Fp8Args& a, hipStream_t stream) {
  if (a.rows == 0) return hipSuccess;
  const TileParams p = quantize_params(a);
  auto go = [&](auto kernel) { kernel<<<dim3(grid(p.tiles)), kTileThreads, 0, stream>>>(p); };
  if (a.io) go(a.square ? tile_kernel<uint16_t, true> : tile_kernel<uint16_t, false>);
  else go(a.square ? tile_kernel<float, true> : tile_kernel<float, false>);
  return hipGetLastError();
}

hipError_t fp8_transpose_launch(const Fp8Args& a, hipStream_t stream) {
  if (a.rows == 0) return hipSuccess;
  const TileParams p = transpose_params(a);
  tile_kernel<E4m3, false><<<dim3(grid(p.tiles)), kTileThreads, 0, stream>>>(p);
  return hipGetLastError();
}

hipError_t fp8_both_launch(const Fp8Args& plain, const Fp8Args& packed, hipStream_t stream) {
  if (plain.rows == 0) return hipSuccess;
  const TileParams a = quantize_params(plain), b = transpose_params(packed);
  const unsigned split = grid(a.tiles), all = split + grid(b.tiles);
  if (plain.io) two_kernel<uint16_t><<<dim3(all), kTileThreads, 0, stream>>>(a, b, split);
  else two_kernel<float><<<dim3(all), kTileThreads, 0, stream>>>(a, b, split);
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
