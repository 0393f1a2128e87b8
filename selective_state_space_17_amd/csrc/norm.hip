// Layer norm and RMS norm with the residual add in front, and their gradients, for gfx950 (MI355X).
//
//   h    = x + residual            (kept rounded to the residual stream's type; what is normalised is what is kept)
//   xh   = (h - mu) rstd,  mu = mean h (layer norm) or 0 (RMS norm),  rstd = (mean (h - mu)^2 + eps)^(-1/2)
//   out  = xh w + b
// and with g = dout w and the gradient dr of the stream that goes on:
//   dh   = rstd (g - xh mean(g xh) - [layer] mean g) + dr
//   dw   = sum_rows dout xh,   db = sum_rows dout
//
// Bound by memory: a row is read once and kept in registers between its statistics and its output, so every
// tensor crosses HBM once.  A row belongs to one wave (up to 1024 columns) or one workgroup (up to 16384); each
// thread owns the same columns of every row it visits.  In the backward pass the workgroups walk over rows and keep
// their columns' dw and db in registers, write them once as partial sums, and a second kernel adds the partial sums
// in a fixed order: no atomics, the same result on every run.
// Statistics, sums and gradients are fp32 whatever the types.
// Measured, where a large copy reaches 5.1 to 5.2 TB/s: RMS norm of 32768 x 2560, bf16 with an fp32 stream, forward
// 183 us (1.01 GB, 5.5 TB/s), gradients 250 us (1.34 GB, 5.4 TB/s) and 5 us of sums.  Layer norm of 16384 x 768 in
// bf16: 15, 19 and 4 us (50 and 75 MB: launches and the first loads' latency are a third of it); 5001 x 1023 in
// fp32, whose rows start at any element: 16, 21 and 5 us.  Loading the gradients' next row ahead took 287 us at 2560
// columns: a kernel with a workgroup a row is compiled for 1024 threads, the most that a row takes, and its 128
// registers spilled.
#include <type_traits>

#include "device_util.h"
#include "internal.h"

namespace mssm {
namespace {

struct NormParams {
  int64_t rows;
  int dim;
  float eps;
  int layer;                // 1: layer norm, 0: RMS norm
  const void* x;            // forward: [rows, dim]
  const void* residual;     // nullable
  const float* weight;
  const float* bias;        // nullable
  void* out;
  void* residual_out;       // nullable
  float* mean;              // nullable
  float* rstd;              // forward: nullable
  // backward
  const void* h;
  const void* dout;
  const void* dresidual;    // nullable
  void* dx;                 // nullable
  void* dresidual_in;       // nullable
  float* part;              // [groups][2][dim] (RMS norm without a bias gradient: the second half unused)
};

constexpr int kMaxWaves = 16;

// Sum of v over the row's threads.  WAVE: the row is one wave.  Else the whole workgroup; slot: one of two
// LDS lines taken in turn, so that one barrier per sum is enough.
template <bool WAVE>
__device__ __forceinline__ float row_sum(float v, float (*red)[kMaxWaves], int slot) {
  v = wave_sum(v);
  if constexpr (WAVE) {
    return v;
  } else {
    const int waves = blockDim.x / kLanes;
    if (threadIdx.x % kLanes == 0) red[slot][threadIdx.x / kLanes] = v;
    __syncthreads();
    float s = 0.f;
    for (int w = 0; w < waves; ++w) s += red[slot][w];
    return s;
  }
}

// one value of what is normalised
template <typename T, typename R> __device__ __forceinline__ float norm_at(const NormParams& p, int64_t i) {
  float v = widen(static_cast<const T*>(p.x)[i]);
  if (p.residual != nullptr) v += widen(static_cast<const R*>(p.residual)[i]);
  return p.residual_out != nullptr ? rounded<R>(v) : v;
}

template <typename T, typename R, int V, int C, bool WAVE>
__global__ __launch_bounds__(WAVE ? 256 : 1024) void norm_fwd_kernel(NormParams p) {
  __shared__ float red[2][kMaxWaves];
  const int per = WAVE ? blockDim.x / kLanes : 1;            // rows at a time
  const int tr = WAVE ? kLanes : blockDim.x;                 // threads of a row
  const int tid = WAVE ? threadIdx.x % kLanes : threadIdx.x;
  const int64_t row = static_cast<int64_t>(blockIdx.x) * per + (WAVE ? threadIdx.x / kLanes : 0);
  if (row >= p.rows) return;
  const int64_t base = row * p.dim;
  const float inv = 1.f / static_cast<float>(p.dim);
  float h[C][V];
#pragma unroll
  for (int c = 0; c < C; ++c) {
    const int col = (c * tr + tid) * V;
    const int left = p.dim - col;
    load_row<V>(static_cast<const T*>(p.x) + base + col, h[c], left);
    if (left > 0) {
      if (p.residual != nullptr) {
        float r[V];
        load_row<V>(static_cast<const R*>(p.residual) + base + col, r, left);
#pragma unroll
        for (int i = 0; i < V; ++i) h[c][i] += r[i];
      }
      if (p.residual_out != nullptr) {
        store_row<V>(static_cast<R*>(p.residual_out) + base + col, h[c], left);
#pragma unroll
        for (int i = 0; i < V; ++i) h[c][i] = rounded<R>(h[c][i]);
      }
    }
  }
  float mu = 0.f;
  if (p.layer) {
    // the mean as the row's first value plus the mean distance from it: rows whose values lie far from zero
    // lose nothing to the size of their sum, and the mean of equal values is that value
    const float first = norm_at<T, R>(p, base);
    float s = 0.f;
#pragma unroll
    for (int c = 0; c < C; ++c) {
      const int left = p.dim - (c * tr + tid) * V;
#pragma unroll
      for (int i = 0; i < V; ++i) s += i < left ? h[c][i] - first : 0.f;
    }
    mu = first + row_sum<WAVE>(s, red, 0) * inv;
  }
  float q = 0.f;
#pragma unroll
  for (int c = 0; c < C; ++c) {
    const int left = p.dim - (c * tr + tid) * V;
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const float d = i < left ? h[c][i] - mu : 0.f;
      q = __builtin_fmaf(d, d, q);
    }
  }
  const float rs = 1.f / __builtin_sqrtf(row_sum<WAVE>(q, red, 1) * inv + p.eps);
  if (tid == 0) {
    if (p.mean != nullptr) p.mean[row] = mu;
    if (p.rstd != nullptr) p.rstd[row] = rs;
  }
#pragma unroll
  for (int c = 0; c < C; ++c) {
    const int col = (c * tr + tid) * V;
    const int left = p.dim - col;
    if (left > 0) {
      float w[V], y[V];
      load_row<V>(p.weight + col, w, left);
#pragma unroll
      for (int i = 0; i < V; ++i) y[i] = (h[c][i] - mu) * rs * w[i];
      if (p.bias != nullptr) {
        float b[V];
        load_row<V>(p.bias + col, b, left);
#pragma unroll
        for (int i = 0; i < V; ++i) y[i] += b[i];
      }
      store_row<V>(static_cast<T*>(p.out) + base + col, y, left);
    }
  }
}

template <typename T, typename R, int V, int C, bool WAVE>
__global__ __launch_bounds__(WAVE ? 256 : 1024) void norm_bwd_kernel(NormParams p) {
  __shared__ float red[4][kMaxWaves];
  const int per = WAVE ? blockDim.x / kLanes : 1;
  const int tr = WAVE ? kLanes : blockDim.x;
  const int tid = WAVE ? threadIdx.x % kLanes : threadIdx.x;
  const int64_t group = static_cast<int64_t>(blockIdx.x) * per + (WAVE ? threadIdx.x / kLanes : 0);
  const int64_t groups = static_cast<int64_t>(gridDim.x) * per;
  const float inv = 1.f / static_cast<float>(p.dim);
  float dw[C][V], db[C][V], w[C][V];
#pragma unroll
  for (int c = 0; c < C; ++c) {
    const int col = (c * tr + tid) * V;
#pragma unroll
    for (int i = 0; i < V; ++i) dw[c][i] = db[c][i] = 0.f;
    load_row<V>(p.weight + col, w[c], p.dim - col);
  }
  int turn = 0;
  for (int64_t row = group; row < p.rows; row += groups, turn ^= 2) {
    const int64_t base = row * p.dim;
    const float mu = p.layer ? p.mean[row] : 0.f, rs = p.rstd[row];
    float xh[C][V], g[C][V];
    float s1 = 0.f, s2 = 0.f;
#pragma unroll
    for (int c = 0; c < C; ++c) {
      const int col = (c * tr + tid) * V;
      const int left = p.dim - col;
      load_row<V>(static_cast<const R*>(p.h) + base + col, xh[c], left);
      load_row<V>(static_cast<const T*>(p.dout) + base + col, g[c], left);   // zeros past the row's end
      if (left > 0) {
#pragma unroll
        for (int i = 0; i < V; ++i) {
          xh[c][i] = (xh[c][i] - mu) * rs;
          dw[c][i] = __builtin_fmaf(g[c][i], xh[c][i], dw[c][i]);
          db[c][i] += g[c][i];
          g[c][i] *= w[c][i];
          s1 = __builtin_fmaf(g[c][i], xh[c][i], s1);
          s2 += g[c][i];
        }
      }
    }
    s1 = row_sum<WAVE>(s1, red, turn) * inv;
    s2 = p.layer ? row_sum<WAVE>(s2, red, turn + 1) * inv : 0.f;
#pragma unroll
    for (int c = 0; c < C; ++c) {
      const int col = (c * tr + tid) * V;
      const int left = p.dim - col;
      if (left > 0) {
        float d[V];
#pragma unroll
        for (int i = 0; i < V; ++i) d[i] = rs * (g[c][i] - xh[c][i] * s1 - s2);
        if (p.dresidual != nullptr) {
          float r[V];
          load_row<V>(static_cast<const R*>(p.dresidual) + base + col, r, left);
#pragma unroll
          for (int i = 0; i < V; ++i) d[i] += r[i];
        }
        if (p.dx != nullptr) store_row<V>(static_cast<T*>(p.dx) + base + col, d, left);
        if (p.dresidual_in != nullptr) store_row<V>(static_cast<R*>(p.dresidual_in) + base + col, d, left);
      }
    }
  }
  if constexpr (WAVE) {
    // the workgroup's waves add up first, in order
    __shared__ float sums[3][C * kLanes * V];
    const int wave = threadIdx.x / kLanes;
#pragma unroll
    for (int half = 0; half < 2; ++half) {
      if (half == 1 && !p.layer) break;
      float(&mine)[C][V] = half == 0 ? dw : db;
      __syncthreads();
      if (wave > 0) {
#pragma unroll
        for (int c = 0; c < C; ++c)
#pragma unroll
          for (int i = 0; i < V; ++i) sums[wave - 1][(c * V + i) * kLanes + tid] = mine[c][i];
      }
      __syncthreads();
      if (wave == 0) {
#pragma unroll
        for (int c = 0; c < C; ++c)
#pragma unroll
          for (int i = 0; i < V; ++i) {
            const int at = (c * V + i) * kLanes + tid;
            mine[c][i] = ((mine[c][i] + sums[0][at]) + sums[1][at]) + sums[2][at];
          }
      }
    }
    if (wave > 0) return;
  }
  float* const out = p.part + static_cast<int64_t>(blockIdx.x) * 2 * p.dim;
#pragma unroll
  for (int c = 0; c < C; ++c) {
    const int col = (c * tr + tid) * V;
    store_row<V>(out + col, dw[c], p.dim - col);
    if (p.layer) store_row<V>(out + p.dim + col, db[c], p.dim - col);
  }
}

// Rows too wide for one workgroup's registers: the row is read again for each of its passes (from the L2,
// where it still is), an element a lane: layer norm of 4096 x 20000 in bf16 224 us, gradients 307 us, 1.5 TB/s.
constexpr int kWideThreads = 1024;
template <typename T, typename R>
__global__ __launch_bounds__(kWideThreads) void norm_fwd_wide_kernel(NormParams p) {
  __shared__ float red[2][kMaxWaves];
  const int64_t base = static_cast<int64_t>(blockIdx.x) * p.dim;
  const float inv = 1.f / static_cast<float>(p.dim);
  auto at = [&](int col) { return norm_at<T, R>(p, base + col); };
  float mu = 0.f;
  if (p.layer) {
    const float first = at(0);
    float s = 0.f;
    for (int c = threadIdx.x; c < p.dim; c += kWideThreads) s += at(c) - first;
    mu = first + row_sum<false>(s, red, 0) * inv;
  }
  float q = 0.f;
  for (int c = threadIdx.x; c < p.dim; c += kWideThreads) {
    const float d = at(c) - mu;
    q = __builtin_fmaf(d, d, q);
  }
  const float rs = 1.f / __builtin_sqrtf(row_sum<false>(q, red, 1) * inv + p.eps);
  if (threadIdx.x == 0) {
    if (p.mean != nullptr) p.mean[blockIdx.x] = mu;
    if (p.rstd != nullptr) p.rstd[blockIdx.x] = rs;
  }
  for (int c = threadIdx.x; c < p.dim; c += kWideThreads) {
    const float v = at(c);
    if (p.residual_out != nullptr) static_cast<R*>(p.residual_out)[base + c] = narrow<R>(v);
    static_cast<T*>(p.out)[base + c] = narrow<T>((v - mu) * rs * p.weight[c] + (p.bias != nullptr ? p.bias[c] : 0.f));
  }
}

template <typename T, typename R>
__global__ __launch_bounds__(kWideThreads) void norm_bwd_wide_kernel(NormParams p) {
  __shared__ float red[2][kMaxWaves];
  const int64_t base = static_cast<int64_t>(blockIdx.x) * p.dim;
  const float inv = 1.f / static_cast<float>(p.dim);
  const float mu = p.layer ? p.mean[blockIdx.x] : 0.f, rs = p.rstd[blockIdx.x];
  float s1 = 0.f, s2 = 0.f;
  for (int c = threadIdx.x; c < p.dim; c += kWideThreads) {
    const float xh = (widen(static_cast<const R*>(p.h)[base + c]) - mu) * rs;
    const float g = widen(static_cast<const T*>(p.dout)[base + c]) * p.weight[c];
    s1 = __builtin_fmaf(g, xh, s1);
    s2 += g;
  }
  s1 = row_sum<false>(s1, red, 0) * inv;
  s2 = p.layer ? row_sum<false>(s2, red, 1) * inv : 0.f;
  for (int c = threadIdx.x; c < p.dim; c += kWideThreads) {
    const float xh = (widen(static_cast<const R*>(p.h)[base + c]) - mu) * rs;
    const float g = widen(static_cast<const T*>(p.dout)[base + c]) * p.weight[c];
    float d = rs * (g - xh * s1 - s2);
    if (p.dresidual != nullptr) d += widen(static_cast<const R*>(p.dresidual)[base + c]);
    if (p.dx != nullptr) static_cast<T*>(p.dx)[base + c] = narrow<T>(d);
    if (p.dresidual_in != nullptr) static_cast<R*>(p.dresidual_in)[base + c] = narrow<R>(d);
  }
}

// their dw and db: a thread owns a column and walks over a block of rows
constexpr int kColThreads = 256;
template <typename T, typename R>
__global__ __launch_bounds__(kColThreads) void norm_cols_wide_kernel(NormParams p) {
  const int c = blockIdx.x * kColThreads + threadIdx.x;
  if (c >= p.dim) return;
  const int64_t per = (p.rows + gridDim.y - 1) / gridDim.y;
  const int64_t lo = blockIdx.y * per, hi = lo + per < p.rows ? lo + per : p.rows;
  float dw = 0.f, db = 0.f;
  for (int64_t r = lo; r < hi; ++r) {
    const float mu = p.layer ? p.mean[r] : 0.f;
    const float g = widen(static_cast<const T*>(p.dout)[r * p.dim + c]);
    dw = __builtin_fmaf(g, (widen(static_cast<const R*>(p.h)[r * p.dim + c]) - mu) * p.rstd[r], dw);
    db += g;
  }
  p.part[blockIdx.y * 2 * static_cast<int64_t>(p.dim) + c] = dw;
  if (p.layer) p.part[(blockIdx.y * 2 + 1) * static_cast<int64_t>(p.dim) + c] = db;
}

// dw, db = sum over the groups, in a fixed order: a workgroup of 1024 owns 64 columns, wave w every 16th group
// from w on, eight loads in flight.
constexpr int kSumWaves = 16;
__global__ __launch_bounds__(kSumWaves * kLanes) void norm_sum_kernel(const float* part, int64_t groups, int dim,
                                                                      float* dw, float* db) {
  __shared__ float red[kSumWaves][kLanes];
  const int wave = threadIdx.x / kLanes, lane = threadIdx.x % kLanes;
  const int c = blockIdx.x * kLanes + lane;
  float s = 0.f;
  if (c < dim) {
#pragma unroll 8
    for (int64_t g = wave; g < groups; g += kSumWaves) s += part[(g * 2 + blockIdx.y) * dim + c];
  }
  red[wave][lane] = s;
  __syncthreads();
  if (wave == 0 && c < dim) {
#pragma unroll
    for (int w = 1; w < kSumWaves; ++w) s += red[w][lane];
    (blockIdx.y == 0 ? dw : db)[c] = s;
  }
}

// ---------------------------------------------------------------------------------------------- plan
// C accesses of kVec elements per thread and row, whether a row is one wave, threads per workgroup
constexpr int kVec = 8, kMostC = 2;
struct NormPlan {
  int C = 0, threads = 0;
  bool wave = false, wide = false;
};

NormPlan norm_plan(int64_t dim) {
  NormPlan n;
  const int64_t chunks = (dim + kVec - 1) / kVec;
  if (chunks <= kLanes * kMostC) {
    n.wave = true;
    n.threads = 256;
    n.C = static_cast<int>((chunks + kLanes - 1) / kLanes);
  } else {
    n.C = chunks > 256 ? 2 : 1;
    const int64_t t = ((chunks + n.C - 1) / n.C + kLanes - 1) / kLanes * kLanes;
    n.wide = t > kMaxWaves * kLanes;
    n.threads = static_cast<int>(t);
  }
  return n;
}

// workgroups of the backward pass, each of which leaves a partial sum of dw (and db): four to a CU, fewer for
// few rows
int64_t norm_groups(int64_t rows) { return rows < 1024 ? rows : 1024; }

template <typename K> hipError_t norm_dispatch(const NormPlan& n, K&& k) {
  using One = std::integral_constant<int, 1>;
  using Two = std::integral_constant<int, 2>;
  if (n.wave) {
    if (n.C == 1) k(One{}, std::true_type{});
    else k(Two{}, std::true_type{});
  } else {
    if (n.C == 1) k(One{}, std::false_type{});
    else k(Two{}, std::false_type{});
  }
  return hipGetLastError();
}

NormParams params(const NormArgs& a) {
  NormParams p{};
  p.rows = a.rows; p.dim = static_cast<int>(a.dim); p.eps = a.eps; p.layer = a.layer;
  p.x = a.x; p.residual = a.residual; p.weight = a.weight; p.bias = a.bias; p.out = a.out;
  p.residual_out = a.residual_out; p.mean = a.mean; p.rstd = a.rstd;
  p.h = a.h; p.dout = a.dout; p.dresidual = a.dresidual; p.dx = a.dx; p.dresidual_in = a.dresidual_in;
  p.part = static_cast<float*>(a.workspace);
  return p;
}

template <typename T, typename R> hipError_t norm_fwd_t(const NormArgs& a, hipStream_t stream) {
  const NormParams p = params(a);
  const NormPlan n = norm_plan(a.dim);
  if (n.wide) {
    norm_fwd_wide_kernel<T, R><<<dim3(static_cast<unsigned>(a.rows)), kWideThreads, 0, stream>>>(p);
    return hipGetLastError();
  }
  const int64_t blocks = n.wave ? (a.rows + 3) / 4 : a.rows;
  return norm_dispatch(n, [&](auto C, auto W) {
    norm_fwd_kernel<T, R, kVec, decltype(C)::value, decltype(W)::value>
        <<<dim3(static_cast<unsigned>(blocks)), n.threads, 0, stream>>>(p);
  });
}

template <typename T, typename R> hipError_t norm_bwd_t(const NormArgs& a, hipStream_t stream) {
  const NormParams p = params(a);
  const NormPlan n = norm_plan(a.dim);
  int64_t groups = norm_groups(n.wave ? (a.rows + 3) / 4 : a.rows);
  hipError_t e = hipSuccess;
  if (a.rows == 0) {
    groups = 0;   // the sums over no rows are written as zeros
  } else if (n.wide) {
    norm_bwd_wide_kernel<T, R><<<dim3(static_cast<unsigned>(a.rows)), kWideThreads, 0, stream>>>(p);
    groups = groups < 64 ? groups : 64;
    norm_cols_wide_kernel<T, R><<<dim3(static_cast<unsigned>((a.dim + kColThreads - 1) / kColThreads),
                                       static_cast<unsigned>(groups)), kColThreads, 0, stream>>>(p);
    e = hipGetLastError();
  } else {
    e = norm_dispatch(n, [&](auto C, auto W) {
      norm_bwd_kernel<T, R, kVec, decltype(C)::value, decltype(W)::value>
          <<<dim3(static_cast<unsigned>(groups)), n.threads, 0, stream>>>(p);
    });
  }
  if (e != hipSuccess) return e;
  norm_sum_kernel<<<dim3(static_cast<unsigned>((a.dim + kLanes - 1) / kLanes), a.dbias != nullptr ? 2 : 1),
                    kSumWaves * kLanes, 0, stream>>>(p.part, groups, p.dim, a.dweight, a.dbias);
  return hipGetLastError();
}

}  // namespace

size_t norm_bwd_workspace_bytes(int64_t rows, int64_t dim) {
  return static_cast<size_t>(norm_groups(rows)) * 2 * static_cast<size_t>(dim) * 4;
}

hipError_t norm_fwd_launch(const NormArgs& a, hipStream_t stream) {
  if (a.rows == 0) return hipSuccess;
  if (!a.io) return norm_fwd_t<float, float>(a, stream);
  return a.res_io ? norm_fwd_t<uint16_t, uint16_t>(a, stream) : norm_fwd_t<uint16_t, float>(a, stream);
}

hipError_t norm_bwd_launch(const NormArgs& a, hipStream_t stream) {
  if (!a.io) return norm_bwd_t<float, float>(a, stream);
  return a.res_io ? norm_bwd_t<uint16_t, uint16_t>(a, stream) : norm_bwd_t<uint16_t, float>(a, stream);
}

}  // namespace mssm
