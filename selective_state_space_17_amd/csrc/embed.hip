// Embedding lookup and the gradient of its table, for gfx950 (MI355X).
//
//   out[t]      = scale * W[id_t]              (an id outside [0, vocab): a zero row)
//   dW[v] (+)=    scale * sum_{t: id_t = v} dout[t]
//
// Both move bytes only.  The lookup reads one row and writes one row per token.  The gradient reads every
// row of dout once and writes every row of dW once; what makes it more than a copy is that text repeats a
// few ids very often, so a row of dW may be the sum of one token or of a tenth of the batch.  The tokens
// are therefore sorted by id (a stable radix sort: equal ids keep their token order, so the sums are taken
// in a fixed order and the result is the same on every run), and the sorted list is cut into slices of
// equal length: a wave sums the runs of equal ids inside its slice, writes the rows of runs that lie wholly
// inside, and leaves the sums of runs that cross a border in the workspace, where a second kernel adds
// them slice by slice.  No atomics on data, no slice longer than another.
#include "device_util.h"
#include "internal.h"

namespace mssm {
namespace {

constexpr int kThreads = 256;
constexpr int kWaves = kThreads / kLanes;

// ------------------------------------------------------------------------------------------------ lookup
struct EmbedParams {
  const void* ids;
  int id_bytes;
  float scale;
  int64_t tokens, vocab, dim;
  const void* weight;
  void* out;
};

// WPR waves share a row: one when the tokens alone fill the chip, four for a few tokens, where the row's
// own load-store latency is all there is.
template <typename T, int V, int WPR>
__global__ __launch_bounds__(kThreads) void embed_kernel(EmbedParams p) {
  constexpr int kRows = kWaves / WPR;
  const int wave = threadIdx.x / kLanes, lane = threadIdx.x % kLanes;
  const int64_t t = static_cast<int64_t>(blockIdx.x) * kRows + wave / WPR;
  if (t >= p.tokens) return;
  const int64_t id = id_at(p.ids, p.id_bytes, t);
  const bool in = id >= 0 && id < p.vocab;
  const T* src = static_cast<const T*>(p.weight) + (in ? id : 0) * p.dim;
  T* dst = static_cast<T*>(p.out) + t * p.dim;
  const float s = in ? p.scale : 0.f;
  const int chunks = static_cast<int>(p.dim / V);
  for (int c = (wave % WPR) * kLanes + lane; c < chunks; c += WPR * kLanes) {
    float v[V];
    if (in) {
      load_row<V>(src + static_cast<int64_t>(c) * V, v);
    } else {
#pragma unroll
      for (int i = 0; i < V; ++i) v[i] = 0.f;
    }
#pragma unroll
    for (int i = 0; i < V; ++i) v[i] *= s;
    store_row<V>(dst + static_cast<int64_t>(c) * V, v);
  }
}

// ---------------------------------------------------------------------------------------- sort by id
// Least-significant-digit radix sort of (id, token) pairs, ids outside [0, vocab) sorted last as `vocab`.
constexpr int kTile = 2048;                    // pairs per workgroup
constexpr int kPerWave = kTile / kWaves;       // a wave's pairs are consecutive, so its order is the input's
constexpr int kMaxDigits = 512;

struct SortParams {
  const void* ids;         // first pass: keys come from here, tokens are positions
  int id_bytes;
  int64_t vocab;
  const uint32_t* keys;    // later passes
  const uint32_t* toks;
  uint32_t* out_keys;
  uint32_t* out_toks;
  uint32_t* hist;          // [digit][tile]
  int n, tiles, shift, bits;
};

__device__ __forceinline__ uint32_t key_at(const SortParams& p, int i) {
  if (p.ids == nullptr) return p.keys[i];
  const int64_t id = id_at(p.ids, p.id_bytes, i);
  return static_cast<uint32_t>(id < 0 || id > p.vocab ? p.vocab : id);
}

__global__ __launch_bounds__(kThreads) void sort_hist_kernel(SortParams p) {
  __shared__ uint32_t cnt[kMaxDigits];
  const int digits = 1 << p.bits;
  for (int d = threadIdx.x; d < digits; d += kThreads) cnt[d] = 0;
  __syncthreads();
  const int64_t base = static_cast<int64_t>(blockIdx.x) * kTile;
  for (int e = threadIdx.x; e < kTile; e += kThreads)
    if (base + e < p.n) atomicAdd(&cnt[(key_at(p, static_cast<int>(base) + e) >> p.shift) & (digits - 1)], 1u);
  __syncthreads();
  for (int d = threadIdx.x; d < digits; d += kThreads)
    p.hist[static_cast<int64_t>(d) * p.tiles + blockIdx.x] = cnt[d];
}

// exclusive prefix sum of n counts in place, one workgroup
constexpr int kScanThreads = 1024;
__global__ __launch_bounds__(kScanThreads) void sort_scan_kernel(uint32_t* v, int64_t n) {
  __shared__ uint32_t part[kScanThreads];
  const int64_t per = (n + kScanThreads - 1) / kScanThreads;
  const int64_t lo = threadIdx.x * per, hi = lo + per < n ? lo + per : n;
  uint32_t s = 0;
  for (int64_t i = lo; i < hi; ++i) s += v[i];
  part[threadIdx.x] = s;
  __syncthreads();
  for (int step = 1; step < kScanThreads; step *= 2) {
    const uint32_t add = static_cast<int>(threadIdx.x) >= step ? part[threadIdx.x - step] : 0u;
    __syncthreads();
    part[threadIdx.x] += add;
    __syncthreads();
  }
  uint32_t run = part[threadIdx.x] - s;
  for (int64_t i = lo; i < hi; ++i) {
    const uint32_t c = v[i];
    v[i] = run;
    run += c;
  }
}

// Lanes of this wave whose digit equals mine (among the lanes where `on` holds).
__device__ __forceinline__ uint64_t same_digit(uint32_t digit, int bits, bool on) {
  uint64_t m = __ballot(on);
  for (int b = 0; b < bits; ++b) {
    const uint64_t set = __ballot((digit >> b) & 1u);
    m &= ((digit >> b) & 1u) ? set : ~set;
  }
  return m;
}

__global__ __launch_bounds__(kThreads) void sort_scatter_kernel(SortParams p) {
  __shared__ uint32_t at[kWaves][kMaxDigits];   // where the wave's next pair of each digit goes
  const int wave = threadIdx.x / kLanes, lane = threadIdx.x % kLanes;
  const int digits = 1 << p.bits;
  for (int d = threadIdx.x; d < digits; d += kThreads)
#pragma unroll
    for (int w = 0; w < kWaves; ++w) at[w][d] = 0;
  __syncthreads();
  const int64_t first = static_cast<int64_t>(blockIdx.x) * kTile + wave * kPerWave;
  for (int e = lane; e < kPerWave; e += kLanes)
    if (first + e < p.n)
      atomicAdd(&at[wave][(key_at(p, static_cast<int>(first) + e) >> p.shift) & (digits - 1)], 1u);
  __syncthreads();
  for (int d = threadIdx.x; d < digits; d += kThreads) {
    uint32_t run = p.hist[static_cast<int64_t>(d) * p.tiles + blockIdx.x];
#pragma unroll
    for (int w = 0; w < kWaves; ++w) {
      const uint32_t c = at[w][d];
      at[w][d] = run;
      run += c;
    }
  }
  __syncthreads();
  volatile uint32_t* const mine = at[wave];
  for (int e = lane; e < kPerWave; e += kLanes) {
    const bool on = first + e < p.n;
    const int i = static_cast<int>(first) + e;
    const uint32_t key = on ? key_at(p, i) : 0u;
    const uint32_t digit = (key >> p.shift) & (digits - 1);
    const uint64_t m = same_digit(digit, p.bits, on);
    const int rank = __popcll(m & ((1ull << lane) - 1));
    if (on) {
      const uint32_t to = mine[digit] + rank;
      p.out_keys[to] = key;
      p.out_toks[to] = p.ids != nullptr ? static_cast<uint32_t>(i) : p.toks[i];
    }
    __builtin_amdgcn_wave_barrier();
    if (on && rank == 0) mine[digit] += __popcll(m);
    __builtin_amdgcn_wave_barrier();
  }
}

// ------------------------------------------------------------------------------------------- gradient
struct EmbedGradParams {
  const uint32_t* keys;    // sorted
  const uint32_t* toks;
  const void* dout;
  void* dweight;
  float* part;             // [slices][2][dim]: the slice's first run if it began earlier; its last if it goes on
  float scale;
  int64_t dim;
  int n, slice, slices;
  uint32_t vocab;
  int accumulate;
};

template <typename G, int V>
__device__ __forceinline__ void write_grad(G* row, const float (&acc)[V], float scale, bool accumulate) {
  float v[V];
#pragma unroll
  for (int i = 0; i < V; ++i) v[i] = acc[i] * scale;
  if (accumulate) {
    float old[V];
    load_row<V>(row, old);
#pragma unroll
    for (int i = 0; i < V; ++i) v[i] += old[i];
  }
  store_row<V>(row, v);
}

// One wave: one slice of the sorted list x one chunk of 64 V columns.
template <typename T, typename G, int V>
__global__ __launch_bounds__(kThreads) void embed_grad_kernel(EmbedGradParams p) {
  const int wave = threadIdx.x / kLanes, lane = threadIdx.x % kLanes;
  const int64_t s = static_cast<int64_t>(blockIdx.x) * kWaves + wave;
  if (s >= p.slices) return;
  const int64_t col = (static_cast<int64_t>(blockIdx.y) * kLanes + lane) * V;
  const bool on = col < p.dim;
  const int lo = static_cast<int>(s) * p.slice;
  const int hi = lo + p.slice < p.n ? lo + p.slice : p.n;
  const T* dout = static_cast<const T*>(p.dout);
  float acc[V];
#pragma unroll
  for (int i = 0; i < V; ++i) acc[i] = 0.f;
  bool head = lo > 0 && p.keys[lo - 1] == p.keys[lo];
  for (int i = lo; i < hi; ++i) {
    const uint32_t key = p.keys[i];
    if (key >= p.vocab) break;   // ids outside the table come last
    if (on) {
      float v[V];
      load_row<V>(dout + static_cast<int64_t>(p.toks[i]) * p.dim + col, v);
#pragma unroll
      for (int j = 0; j < V; ++j) acc[j] += v[j];
    }
    const bool last = i + 1 == p.n || p.keys[i + 1] != key;
    if (last || i + 1 == hi) {
      if (on) {
        if (head || !last) {
          store_row<V>(p.part + (s * 2 + (head ? 0 : 1)) * p.dim + col, acc);
        } else {
          write_grad<G, V>(static_cast<G*>(p.dweight) + key * p.dim + col, acc, p.scale, p.accumulate != 0);
        }
      }
      head = false;
#pragma unroll
      for (int j = 0; j < V; ++j) acc[j] = 0.f;
    }
  }
}

// Runs that cross slices: the wave of the slice where such a run begins adds its parts in order.
template <typename G, int V>
__global__ __launch_bounds__(kThreads) void embed_join_kernel(EmbedGradParams p) {
  const int wave = threadIdx.x / kLanes, lane = threadIdx.x % kLanes;
  const int64_t s = static_cast<int64_t>(blockIdx.x) * kWaves + wave;
  if (s + 1 >= p.slices) return;
  const int lo = static_cast<int>(s) * p.slice, next = lo + p.slice;
  const uint32_t key = p.keys[next - 1];
  if (key >= p.vocab || p.keys[next] != key) return;        // nothing goes on past this slice
  if (lo > 0 && p.keys[lo - 1] == key) return;              // the run began in an earlier slice
  const int64_t col = (static_cast<int64_t>(blockIdx.y) * kLanes + lane) * V;
  if (col >= p.dim) return;
  float acc[V];
  load_row<V>(p.part + (s * 2 + 1) * p.dim + col, acc);
  for (int64_t j = s + 1; j < p.slices && p.keys[j * p.slice] == key; ++j) {
    float v[V];
    load_row<V>(p.part + j * 2 * p.dim + col, v);
#pragma unroll
    for (int i = 0; i < V; ++i) acc[i] += v[i];
  }
  write_grad<G, V>(static_cast<G*>(p.dweight) + key * p.dim + col, acc, p.scale, p.accumulate != 0);
}

// rows without a token
template <typename G>
__global__ __launch_bounds__(kThreads) void embed_zero_kernel(G* p, int64_t n) {
  constexpr int V = 16 / sizeof(G);
  const float z[V] = {};
  int64_t i = (static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x) * V;
  const int64_t step = static_cast<int64_t>(gridDim.x) * kThreads * V;
  if (reinterpret_cast<uintptr_t>(p) % 16 == 0) {
    for (; i + V <= n; i += step) store_row<V>(p + i, z);
    for (int64_t j = i; j < n && j < i + V; ++j) p[j] = 0;
  } else {
    for (; i < n; i += step)
      for (int64_t j = i; j < n && j < i + V; ++j) p[j] = 0;
  }
}

int sort_passes(int64_t vocab, int* bits) {
  int need = 1;
  while ((int64_t{1} << need) <= vocab) ++need;   // the keys are 0 .. vocab
  const int passes = (need + 8) / 9;
  *bits = (need + passes - 1) / passes;
  return passes;
}

// a slice long enough that the crossing runs' parts stay few, short enough that the slices fill the chip
int slice_len(int64_t tokens) { return tokens >= (1 << 17) ? 64 : tokens >= (1 << 15) ? 32 : 16; }

constexpr size_t up256(size_t b) { return (b + 255) / 256 * 256; }

template <typename F> hipError_t launch_width(int v, F&& f) {
  switch (v) {
    case 8: f(std::integral_constant<int, 8>{}); break;
    case 4: f(std::integral_constant<int, 4>{}); break;
    case 2: f(std::integral_constant<int, 2>{}); break;
    default: f(std::integral_constant<int, 1>{}); break;
  }
  return hipGetLastError();
}

template <typename T> hipError_t embed_fwd_t(const EmbedArgs& a, hipStream_t stream) {
  EmbedParams p{a.ids, a.id_bytes, a.scale, a.tokens, a.vocab, a.dim, a.weight, a.out};
  const void* ptrs[] = {a.weight, a.out};
  const int es[] = {sizeof(T), sizeof(T)};
  const int v = vector_width(a.dim, ptrs, es, 2, 16 / sizeof(T));
  return launch_width(v, [&](auto V) {
    constexpr int kV = decltype(V)::value > static_cast<int>(16 / sizeof(T)) ? 1 : decltype(V)::value;
    if (a.tokens < 4096)
      embed_kernel<T, kV, kWaves><<<dim3(static_cast<unsigned>(a.tokens)), kThreads, 0, stream>>>(p);
    else
      embed_kernel<T, kV, 1><<<dim3(static_cast<unsigned>((a.tokens + kWaves - 1) / kWaves)), kThreads, 0, stream>>>(p);
  });
}

template <typename T, typename G> hipError_t embed_bwd_t(const EmbedArgs& a, hipStream_t stream) {
  const int n = static_cast<int>(a.tokens);
  int bits = 0;
  const int passes = sort_passes(a.vocab, &bits);
  const int tiles = (n + kTile - 1) / kTile;
  unsigned char* ws = static_cast<unsigned char*>(a.workspace);
  uint32_t* buf[4];
  for (int i = 0; i < 4; ++i) buf[i] = reinterpret_cast<uint32_t*>(ws + i * up256(size_t(n) * 4));
  uint32_t* hist = reinterpret_cast<uint32_t*>(ws + 4 * up256(size_t(n) * 4));
  float* part = reinterpret_cast<float*>(ws + 4 * up256(size_t(n) * 4) + up256((size_t(1) << bits) * tiles * 4));

  if (!a.accumulate) {
    const int64_t total = a.vocab * a.dim;
    const int64_t want = (total + kThreads * 8 - 1) / (kThreads * 8);
    embed_zero_kernel<G><<<dim3(static_cast<unsigned>(want < 8192 ? want : 8192)), kThreads, 0, stream>>>(
        static_cast<G*>(a.dweight), total);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  if (n == 0) return hipSuccess;
  SortParams sp{};
  sp.n = n; sp.tiles = tiles; sp.bits = bits; sp.vocab = a.vocab; sp.hist = hist; sp.id_bytes = a.id_bytes;
  for (int k = 0; k < passes; ++k) {
    sp.ids = k == 0 ? a.ids : nullptr;
    sp.keys = buf[(k & 1) ? 0 : 2];
    sp.toks = buf[(k & 1) ? 1 : 3];
    sp.out_keys = buf[(k & 1) ? 2 : 0];
    sp.out_toks = buf[(k & 1) ? 3 : 1];
    sp.shift = k * bits;
    sort_hist_kernel<<<dim3(tiles), kThreads, 0, stream>>>(sp);
    sort_scan_kernel<<<dim3(1), kScanThreads, 0, stream>>>(hist, (int64_t{1} << bits) * tiles);
    sort_scatter_kernel<<<dim3(tiles), kThreads, 0, stream>>>(sp);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  EmbedGradParams p{};
  p.keys = sp.out_keys; p.toks = sp.out_toks; p.dout = a.dout; p.dweight = a.dweight; p.part = part;
  p.scale = a.scale; p.dim = a.dim; p.n = n; p.slice = slice_len(n); p.slices = (n + p.slice - 1) / p.slice;
  p.vocab = static_cast<uint32_t>(a.vocab); p.accumulate = a.accumulate;
  const void* ptrs[] = {a.dout, a.dweight, part};
  const int es[] = {sizeof(T), sizeof(G), 4};
  const int v = vector_width(a.dim, ptrs, es, 3, 16 / sizeof(T));
  return launch_width(v, [&](auto V) {
    constexpr int kV = decltype(V)::value > static_cast<int>(16 / sizeof(T)) ? 1 : decltype(V)::value;
    const dim3 grid(static_cast<unsigned>((p.slices + kWaves - 1) / kWaves),
                    static_cast<unsigned>((a.dim + kLanes * kV - 1) / (kLanes * kV)));
    embed_grad_kernel<T, G, kV><<<grid, kThreads, 0, stream>>>(p);
    embed_join_kernel<G, kV><<<grid, kThreads, 0, stream>>>(p);
  });
}

}  // namespace

size_t embed_bwd_workspace_bytes(int64_t tokens, int64_t vocab, int64_t dim) {
  if (tokens <= 0) return 0;
  int bits = 0;
  sort_passes(vocab, &bits);
  const size_t n = static_cast<size_t>(tokens), tiles = (n + kTile - 1) / kTile;
  const size_t slice = static_cast<size_t>(slice_len(tokens)), slices = (n + slice - 1) / slice;
  return 4 * up256(n * 4) + up256((size_t{1} << bits) * tiles * 4) + up256(slices * 2 * dim * 4);
}

hipError_t embed_fwd_launch(const EmbedArgs& a, hipStream_t stream) {
  if (a.tokens == 0) return hipSuccess;
  return a.io ? embed_fwd_t<uint16_t>(a, stream) : embed_fwd_t<float>(a, stream);
}

hipError_t embed_bwd_launch(const EmbedArgs& a, hipStream_t stream) {
  if (!a.io) return embed_bwd_t<float, float>(a, stream);
  return a.grad_io ? embed_bwd_t<uint16_t, uint16_t>(a, stream) : embed_bwd_t<uint16_t, float>(a, stream);
}

}  // namespace mssm
