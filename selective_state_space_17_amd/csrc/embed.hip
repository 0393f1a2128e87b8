// Embedding lookup and the gradient of its table, for gfx950 (MI355X).
//
//   out[t]      = scale * W[id_t]              (an id outside [0, vocab): a zero row)
//   dW[v] (+)=    scale * sum_{t: id_t = v} dout[t]
//
// Both move bytes only.  The lookup reads one row and writes one row per token.  The gradient reads every
// row of dout once and writes every row of dW once; what makes it more than a copy is that text repeats a
// few ids very often, so a row of dW may be the sum of one token or of a tenth of the batch.  The tokens
// are therefore sorted by id (equal ids keep their token order, so the sums are taken in a fixed order and the
// result is the same on every run), and the sorted list is cut into slices of
// sixteen: a wave loads its slice's rows at once, sums the runs of equal ids, writes the rows of runs that lie
// wholly inside, and leaves the sums of runs that cross a border in the workspace, where a second kernel adds
// them in order.  No atomics on data, no slice longer than another.  The rows of ids that do not occur are
// zeroed beforehand, by workgroups that run beside the sort.
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
// own load-store latency is all there is.  16384 x 768 in bf16: 8.1 us, 6.2 TB/s of rows read and written (a table
// of 77 MB stays in the 256 MB cache); 8 x 2560: 2.9 us.
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
  const int chunks = static_cast<int>((p.dim + V - 1) / V);
  for (int c = (wave % WPR) * kLanes + lane; c < chunks; c += WPR * kLanes) {
    const int64_t col = static_cast<int64_t>(c) * V;
    float v[V];
    load_row<V>(src + col, v, in ? p.dim - col : 0);
#pragma unroll
    for (int i = 0; i < V; ++i) v[i] *= s;
    store_row<V>(dst + col, v, p.dim - col);
  }
}

// ---------------------------------------------------------------------------------------- rows without a token
// What a launch zeroes with the workgroups behind its own: n units of two bytes.  A workgroup writes one stretch, the
// workgroups stretches in order.
struct Zeros {
  uint16_t* p;
  int64_t n;
};
constexpr int kZeroBlocks = 1 << 20;   // (a launch has less than 2^32 threads)
// Stores of a thread at a time: one where zeroing is all that a launch does (716 MB at 6.6 TB/s; four: 5.9), four
// beside a sort, whose workgroups then wait for fewer others (16384 x 768 of 50280: 34.2 us; one: 37.1).
constexpr int kStoresAlone = 1, kStoresBeside = 4;
template <int STORES = kStoresBeside>
__device__ __forceinline__ void zero_rows(const Zeros& z, int64_t block, int64_t blocks, int threads) {
  const float none[8] = {};
  const int64_t piece = static_cast<int64_t>(threads) * 8 * STORES;
  for (int64_t at = block * piece; at < z.n; at += blocks * piece) {
#pragma unroll
    for (int k = 0; k < STORES; ++k) {
      const int64_t i = at + (k * threads + threadIdx.x) * 8;
      store_row<8>(z.p + i, none, z.n - i);
    }
  }
}
unsigned zero_blocks(const Zeros& z, int threads, int stores = kStoresBeside) {
  const int64_t piece = static_cast<int64_t>(threads) * 8 * stores, want = (z.n + piece - 1) / piece;
  return static_cast<unsigned>(want < kZeroBlocks ? want : kZeroBlocks);
}

__global__ __launch_bounds__(kThreads) void embed_zero_kernel(Zeros z) {
  zero_rows<kStoresAlone>(z, blockIdx.x, gridDim.x, kThreads);
}

__device__ __forceinline__ uint32_t sort_key(int64_t id, int64_t vocab) {
  return static_cast<uint32_t>(id < 0 || id > vocab ? vocab : id);
}

// ------------------------------------------------------------------------------- sort of up to 16384 by id
// No passes: a token's place is the number of words key << 14 | token below its own.  A workgroup finds the places
// of 64 tokens, spread evenly over the batch; it sorts them, looks every word of the batch up between them (six
// reads of 64 words that stand in 64 banks: no conflicts) and counts the words in each gap; the places are those
// counts' prefix sums.  Workgroups of the same launch behind them zero dW meanwhile.  16384 ids, table of 50280 x
// 768 in bf16: 16 us, 11 us without the zeroing, which alone takes 14 us; a radix sort by one workgroup, four bits
// a pass in LDS, took 26 us beside the same zeroing.  The work grows with the square of the tokens; at the limit, to
// which a word has bits for them, the whole gradient takes 35 us, one token above, sorted as below, 52 us.
constexpr int kRankThreads = 1024, kTokenBits = 14, kRankMost = 1 << kTokenBits, kPivots = kLanes;

struct RankParams {
  const void* ids;
  int id_bytes;
  int64_t vocab;
  int n, groups;     // groups: workgroups with tokens
  uint32_t* keys;
  uint32_t* toks;
  Zeros zeros;
};

template <int E> __global__ __launch_bounds__(kRankThreads, 8) void rank_kernel(RankParams p) {
  __shared__ uint32_t pivots[kPivots], counts[kPivots + 1];
  if (static_cast<int>(blockIdx.x) >= p.groups) {
    zero_rows(p.zeros, blockIdx.x - p.groups, gridDim.x - p.groups, kRankThreads);
    return;
  }
  const int tid = threadIdx.x, lane = tid % kLanes;
  auto word = [&](int64_t id, int i) {   // (what lies past the end sorts last)
    return i < p.n ? sort_key(id, p.vocab) << kTokenBits | static_cast<uint32_t>(i) : ~0u;
  };
  int64_t ids[E], one[1];
  const int mine = static_cast<int>(blockIdx.x) + lane * p.groups;
  ids_at<1>(p.ids, p.id_bytes, mine, 0, p.n, one);
  ids_at<E>(p.ids, p.id_bytes, tid, kRankThreads, p.n, ids);
  uint32_t v[E];
#pragma unroll
  for (int e = 0; e < E; ++e) v[e] = word(ids[e], e * kRankThreads + tid);
  if (tid < kLanes) {
    const uint32_t own = word(one[0], mine);
    int at = 0;
#pragma unroll 8
    for (int l = 0; l < kLanes; ++l) {
      const uint32_t o = __builtin_amdgcn_readlane(own, l);
      at += o < own || (o == own && l < lane);
    }
    pivots[at] = own;
    counts[lane] = 0;
    if (lane == 0) counts[kPivots] = 0;
  }
  __syncthreads();
  const uint32_t top = pivots[kPivots - 1];
  constexpr int kAtOnce = E < 8 ? E : 8;
#pragma unroll
  for (int e0 = 0; e0 < E; e0 += kAtOnce) {
    uint32_t below[kAtOnce];   // pivots below the word
#pragma unroll
    for (int e = 0; e < kAtOnce; ++e) below[e] = 0;
#pragma unroll
    for (int step = kPivots / 2; step > 0; step /= 2) {
      uint32_t x[kAtOnce];
#pragma unroll
      for (int e = 0; e < kAtOnce; ++e) x[e] = pivots[below[e] + step - 1];
#pragma unroll
      for (int e = 0; e < kAtOnce; ++e) below[e] += x[e] < v[e0 + e] ? step : 0;
    }
#pragma unroll
    for (int e = 0; e < kAtOnce; ++e) {
      below[e] += top < v[e0 + e];
      if (v[e0 + e] != ~0u)
        __hip_atomic_fetch_add(&counts[below[e]], 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_WORKGROUP);
    }
    __builtin_amdgcn_sched_barrier(0);
  }
  __syncthreads();
  if (tid >= kLanes) return;
  const uint32_t own = pivots[lane];
  const uint32_t at = wave_prefix(counts[lane]) - 1;   // the words up to this one, but for itself
  if (own != ~0u) {
    p.keys[at] = own >> kTokenBits;
    p.toks[at] = own & (kRankMost - 1);
  }
}

// ---------------------------------------------------------------------------------- sort of any number by id
// Least-significant-digit radix sort of (id, token) pairs, ids outside [0, vocab) sorted last as `vocab`.  Each of
// its launches, few workgroups that wait for memory, zeroes a share of dW beside.  Up to nine bits a pass: 65536 ids of
// a table of 50280 take two passes of three launches, 6 + 6 + 7 us each, of 84 us for the gradient (768 columns).
constexpr int kTile = 1024;                    // pairs per workgroup
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
  Zeros zeros;
};

// keys first, first + step, ..., all loads at once; past the end the last one again
template <int E> __device__ __forceinline__ void keys_at(const SortParams& p, int64_t first, int64_t step, uint32_t (&key)[E]) {
  if (p.ids == nullptr) {
#pragma unroll
    for (int e = 0; e < E; ++e) {
      const int64_t i = first + e * step;
      key[e] = p.keys[i < p.n ? i : p.n - 1];
    }
  } else {
    int64_t id[E];
    ids_at<E>(p.ids, p.id_bytes, first, step, p.n, id);
#pragma unroll
    for (int e = 0; e < E; ++e) key[e] = sort_key(id[e], p.vocab);
  }
}

__global__ __launch_bounds__(kThreads) void sort_hist_kernel(SortParams p) {
  __shared__ uint32_t cnt[kMaxDigits];
  if (static_cast<int>(blockIdx.x) >= p.tiles) {
    zero_rows(p.zeros, blockIdx.x - p.tiles, gridDim.x - p.tiles, kThreads);
    return;
  }
  const int digits = 1 << p.bits;
  for (int d = threadIdx.x; d < digits; d += kThreads) cnt[d] = 0;
  __syncthreads();
  const int64_t mine = static_cast<int64_t>(blockIdx.x) * kTile + threadIdx.x;
  uint32_t key[kTile / kThreads];
  keys_at(p, mine, kThreads, key);
#pragma unroll
  for (int e = 0; e < kTile / kThreads; ++e)
    if (mine + e * kThreads < p.n) atomicAdd(&cnt[(key[e] >> p.shift) & (digits - 1)], 1u);
  __syncthreads();
  for (int d = threadIdx.x; d < digits; d += kThreads)
    p.hist[static_cast<int64_t>(d) * p.tiles + blockIdx.x] = cnt[d];
}

// Exclusive prefix sum of n counts in place, one workgroup: 16 counts a thread at a time, all loads at once.
// 16384 counts (65536 tokens) in 5.5 us; count after count through a thread's share took 26 us.
constexpr int kScanThreads = 1024, kScanPer = 16, kScanWaves = kScanThreads / kLanes;
__global__ __launch_bounds__(kScanThreads) void sort_scan_kernel(uint32_t* v, int64_t n, Zeros zeros) {
  __shared__ uint32_t totals[2][kScanWaves];
  if (blockIdx.x > 0) {
    zero_rows(zeros, blockIdx.x - 1, gridDim.x - 1, kScanThreads);
    return;
  }
  const int wave = threadIdx.x / kLanes, lane = threadIdx.x % kLanes;
  uint32_t before = 0;   // counts of the rounds before
  int turn = 0;
  for (int64_t base = 0; base < n; base += kScanThreads * kScanPer, turn ^= 1) {
    const int64_t at = base + threadIdx.x * kScanPer;
    const bool whole = at + kScanPer <= n;
    uint32_t c[kScanPer], s = 0;
    if (whole) {
#pragma unroll
      for (int k = 0; k < kScanPer / 4; ++k) {
        const u32x4_t t = *reinterpret_cast<const u32x4_t*>(v + at + 4 * k);
        c[4 * k] = t[0]; c[4 * k + 1] = t[1]; c[4 * k + 2] = t[2]; c[4 * k + 3] = t[3];
      }
    } else {
#pragma unroll
      for (int k = 0; k < kScanPer; ++k) c[k] = at + k < n ? v[at + k] : 0u;
    }
#pragma unroll
    for (int k = 0; k < kScanPer; ++k) s += c[k];
    const uint32_t upto = wave_prefix(s);
    if (lane == kLanes - 1) totals[turn][wave] = upto;
    __syncthreads();
    uint32_t run = before + upto - s;
#pragma unroll
    for (int w = 0; w < kScanWaves; ++w) {
      const uint32_t t = totals[turn][w];
      run += w < wave ? t : 0u;
      before += t;
    }
#pragma unroll
    for (int k = 0; k < kScanPer; ++k) {
      const uint32_t t = c[k];
      c[k] = run;
      run += t;
    }
    if (whole) {
#pragma unroll
      for (int k = 0; k < kScanPer / 4; ++k)
        *reinterpret_cast<u32x4_t*>(v + at + 4 * k) = u32x4_t{c[4 * k], c[4 * k + 1], c[4 * k + 2], c[4 * k + 3]};
    } else {
#pragma unroll
      for (int k = 0; k < kScanPer; ++k)
        if (at + k < n) v[at + k] = c[k];
    }
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
  if (static_cast<int>(blockIdx.x) >= p.tiles) {
    zero_rows(p.zeros, blockIdx.x - p.tiles, gridDim.x - p.tiles, kThreads);
    return;
  }
  const int wave = threadIdx.x / kLanes, lane = threadIdx.x % kLanes;
  const int digits = 1 << p.bits;
  for (int d = threadIdx.x; d < digits; d += kThreads)
#pragma unroll
    for (int w = 0; w < kWaves; ++w) at[w][d] = 0;
  __syncthreads();
  const int64_t first = static_cast<int64_t>(blockIdx.x) * kTile + wave * kPerWave + lane;
  constexpr int kEach = kPerWave / kLanes;
  uint32_t key[kEach], tok[kEach];
  keys_at(p, first, kLanes, key);
#pragma unroll
  for (int e = 0; e < kEach; ++e) {
    const int64_t i = first + e * kLanes;
    tok[e] = p.ids != nullptr ? static_cast<uint32_t>(i) : p.toks[i < p.n ? i : p.n - 1];
  }
#pragma unroll
  for (int e = 0; e < kEach; ++e)
    if (first + e * kLanes < p.n) atomicAdd(&at[wave][(key[e] >> p.shift) & (digits - 1)], 1u);
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
#pragma unroll
  for (int e = 0; e < kEach; ++e) {
    const bool on = first + e * kLanes < p.n;
    const uint32_t digit = (key[e] >> p.shift) & (digits - 1);
    const uint64_t m = same_digit(digit, p.bits, on);
    const int rank = __popcll(m & ((1ull << lane) - 1));
    if (on) {
      const uint32_t to = mine[digit] + rank;
      p.out_keys[to] = key[e];
      p.out_toks[to] = tok[e];
    }
    __builtin_amdgcn_wave_barrier();
    if (on && rank == 0) mine[digit] += __popcll(m);
    __builtin_amdgcn_wave_barrier();
  }
}

// ------------------------------------------------------------------------------------------- gradient
constexpr int kSlice = 16;

struct EmbedGradParams {
  const uint32_t* keys;    // sorted
  const uint32_t* toks;
  const void* dout;
  void* dweight;
  float* part;             // [slices][2][dim]: the slice's first run if it began earlier; its last if it goes on
  float scale;
  int64_t dim;
  int n, slices;
  uint32_t vocab;
  int accumulate;
};

template <typename G, int V>
__device__ __forceinline__ void write_grad(G* row, const float (&acc)[V], float scale, bool accumulate, int64_t n) {
  float v[V];
#pragma unroll
  for (int i = 0; i < V; ++i) v[i] = acc[i] * scale;
  if (accumulate) {
    float old[V];
    load_row<V>(row, old, n);
#pragma unroll
    for (int i = 0; i < V; ++i) v[i] += old[i];
  }
  store_row<V>(row, v, n);
}

// Up to 64 tokens need no sort: a wave for every token and chunk of 64 V columns compares the token's id with all
// others', and where none before it has that id adds the rows of those that do, in order.  Two launches instead of
// three, which is what so small a call's time is: 64 x 768 of 50280 in bf16 15 us (25 by the sort below), 38 x 1856
// of 96414 in fp32, where 716 MB of zeros are the work, 108 us (142).
constexpr int kFew = kLanes;
template <typename T, typename G, int V>
__global__ __launch_bounds__(kThreads) void embed_few_kernel(EmbedGradParams p, const void* ids, int id_bytes) {
  const int lane = threadIdx.x % kLanes;
  const int t = __builtin_amdgcn_readfirstlane(static_cast<int>(blockIdx.x) * kWaves + threadIdx.x / kLanes);
  if (t >= p.n) return;
  const uint32_t key = sort_key(id_at(ids, id_bytes, lane < p.n ? lane : p.n - 1), p.vocab);
  const uint32_t mine = __builtin_amdgcn_readlane(key, t);
  uint64_t same = __ballot(lane < p.n && key == mine);
  if (mine >= p.vocab || (same & ((1ull << t) - 1)) != 0) return;
  const int64_t col = (static_cast<int64_t>(blockIdx.y) * kLanes + lane) * V;
  const int64_t left = p.dim - col;
  float acc[V];
#pragma unroll
  for (int j = 0; j < V; ++j) acc[j] = 0.f;
  constexpr int kAtOnce = 4;
  while (same != 0) {
    float v[kAtOnce][V];
#pragma unroll
    for (int k = 0; k < kAtOnce; ++k) {
      const bool has = same != 0;
      const int64_t i = has ? __builtin_ctzll(same) : 0;
      same &= same - (has ? 1 : 0);
      load_row<V>(static_cast<const T*>(p.dout) + i * p.dim + col, v[k], has ? left : 0);
    }
#pragma unroll
    for (int k = 0; k < kAtOnce; ++k)
#pragma unroll
      for (int j = 0; j < V; ++j) acc[j] += v[k][j];
  }
  if (left > 0) write_grad<G, V>(static_cast<G*>(p.dweight) + mine * p.dim + col, acc, p.scale, p.accumulate != 0, left);
}

// One wave: one slice of the sorted list x one chunk of 64 V columns.  Lane i holds the slice's i-th key and token.
// 16384 x 768 in bf16: 14 us for 25 MB of rows and some 11 MB written; what it waits for is one chain of three
// dependent loads (key, token, row), once, with all rows of a slice in flight.
template <typename T, typename G, int V>
__global__ __launch_bounds__(kThreads) void embed_grad_kernel(EmbedGradParams p) {
  const int wave = threadIdx.x / kLanes, lane = threadIdx.x % kLanes;
  const int64_t s = static_cast<int64_t>(blockIdx.x) * kWaves + wave;
  if (s >= p.slices) return;
  const int64_t col = (static_cast<int64_t>(blockIdx.y) * kLanes + lane) * V;
  const int64_t left = p.dim - col;
  const bool on = left > 0;
  const int lo = static_cast<int>(s) * kSlice;
  // lanes 0 .. 15: the slice; 16: what follows it; 17: what stands before it (~0: nothing)
  const int at = lane <= kSlice ? lo + lane : lo - 1;
  const uint32_t key = lane <= kSlice + 1 && at >= 0 && at < p.n ? p.keys[at] : ~0u;
  const uint32_t tok = lane < kSlice && at < p.n ? p.toks[at] : 0u;
  const T* dout = static_cast<const T*>(p.dout) + (on ? col : 0);
  float v[kSlice][V];
#pragma unroll
  for (int i = 0; i < kSlice; ++i) {
    // (a token that is not to be counted is not read: its row may hold anything)
    if (static_cast<uint32_t>(__builtin_amdgcn_readlane(key, i)) < p.vocab)
      load_row<V>(dout + static_cast<int64_t>(static_cast<uint32_t>(__builtin_amdgcn_readlane(tok, i))) * p.dim, v[i], left);
  }
  float acc[V];
#pragma unroll
  for (int j = 0; j < V; ++j) acc[j] = 0.f;
  bool head = __builtin_amdgcn_readlane(key, kSlice + 1) == __builtin_amdgcn_readlane(key, 0);
#pragma unroll
  for (int i = 0; i < kSlice; ++i) {
    const uint32_t k = __builtin_amdgcn_readlane(key, i);
    if (k >= p.vocab) break;   // ids outside the table come last
#pragma unroll
    for (int j = 0; j < V; ++j) acc[j] += v[i][j];
    const bool last = static_cast<uint32_t>(__builtin_amdgcn_readlane(key, i + 1)) != k;
    if (last || i + 1 == kSlice) {
      if (on) {
        if (head || !last) {
          store_row<V>(p.part + (s * 2 + (head ? 0 : 1)) * p.dim + col, acc, left);
        } else {
          write_grad<G, V>(static_cast<G*>(p.dweight) + k * p.dim + col, acc, p.scale, p.accumulate != 0, left);
        }
      }
      head = false;
#pragma unroll
      for (int j = 0; j < V; ++j) acc[j] = 0.f;
    }
  }
}

// Runs that cross slices: the workgroup of the slice where such a run begins adds its parts, each wave a
// quarter of them in order, the quarters in order.  6 us for the same sizes (a launch, two rounds of probes for the
// run's end, up to a hundred parts) and more with the longest run: 40 us where every id is the same.  Halving the interval instead of 64 places at once took 7.5 us.
template <typename G, int V>
__global__ __launch_bounds__(kThreads) void embed_join_kernel(EmbedGradParams p) {
  __shared__ float red[kWaves][kLanes * V];
  const int wave = threadIdx.x / kLanes, lane = threadIdx.x % kLanes;
  const int64_t s = blockIdx.x;
  if (s + 1 >= p.slices) return;
  const int lo = static_cast<int>(s) * kSlice, next = lo + kSlice;
  const uint32_t key = p.keys[next - 1];
  if (key >= p.vocab || p.keys[next] != key) return;        // nothing goes on past this slice
  if (lo > 0 && p.keys[lo - 1] == key) return;              // the run began in an earlier slice
  // the last slice the run reaches into: its first key is still the run's
  int64_t have = s + 1, not_in = p.slices;
  while (not_in - have > 1) {   // 63 or 64 places between, a lane each
    const int64_t step = (not_in - have + kLanes - 1) / kLanes, at = have + (lane + 1) * step;
    const int in = __popcll(__ballot(at < not_in && p.keys[at < not_in ? at * kSlice : 0] == key));
    have += in * step;
    not_in = have + step < not_in ? have + step : not_in;
  }
  const int parts = static_cast<int>(have - s) + 1;          // the first from the second half of its line
  const int64_t col = (static_cast<int64_t>(blockIdx.y) * kLanes + lane) * V;
  const int64_t left = p.dim - col;
  const bool on = left > 0;
  const int quarter = (parts + kWaves - 1) / kWaves;
  const int end = (wave + 1) * quarter < parts ? (wave + 1) * quarter : parts;
  float acc[V];
#pragma unroll
  for (int j = 0; j < V; ++j) acc[j] = 0.f;
  if (on) {
#pragma unroll 8
    for (int k = wave * quarter; k < end; ++k) {
      float v[V];
      load_row<V>(p.part + ((s + k) * 2 + (k == 0 ? 1 : 0)) * p.dim + col, v, left);
#pragma unroll
      for (int j = 0; j < V; ++j) acc[j] += v[j];
    }
  }
#pragma unroll
  for (int j = 0; j < V; ++j) red[wave][j * kLanes + lane] = acc[j];
  __syncthreads();
  if (wave != 0 || !on) return;
#pragma unroll
  for (int w = 1; w < kWaves; ++w)
#pragma unroll
    for (int j = 0; j < V; ++j) acc[j] += red[w][j * kLanes + lane];
  write_grad<G, V>(static_cast<G*>(p.dweight) + key * p.dim + col, acc, p.scale, p.accumulate != 0, left);
}

int sort_passes(int64_t vocab, int* bits) {
  int need = 1;
  while ((int64_t{1} << need) <= vocab) ++need;   // the keys are 0 .. vocab
  const int passes = (need + 8) / 9;
  *bits = (need + passes - 1) / passes;
  return passes;
}

constexpr size_t up256(size_t b) { return (b + 255) / 256 * 256; }

template <typename T> hipError_t embed_fwd_t(const EmbedArgs& a, hipStream_t stream) {
  EmbedParams p{a.ids, a.id_bytes, a.scale, a.tokens, a.vocab, a.dim, a.weight, a.out};
  constexpr int kV = 16 / sizeof(T);
  if (a.tokens < 4096)
    embed_kernel<T, kV, kWaves><<<dim3(static_cast<unsigned>(a.tokens)), kThreads, 0, stream>>>(p);
  else
    embed_kernel<T, kV, 1><<<dim3(static_cast<unsigned>((a.tokens + kWaves - 1) / kWaves)), kThreads, 0, stream>>>(p);
  return hipGetLastError();
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

  const Zeros all{static_cast<uint16_t*>(a.dweight), a.accumulate ? 0 : a.vocab * a.dim * static_cast<int64_t>(sizeof(G) / 2)};
  EmbedGradParams g{};
  g.dout = a.dout; g.dweight = a.dweight; g.part = part;
  g.scale = a.scale; g.dim = a.dim; g.n = n; g.slices = (n + kSlice - 1) / kSlice;
  g.vocab = static_cast<uint32_t>(a.vocab); g.accumulate = a.accumulate;
  constexpr int kV = 16 / sizeof(T);
  const unsigned chunks = static_cast<unsigned>((a.dim + kLanes * kV - 1) / (kLanes * kV));
  if (n <= kFew) {
    if (all.n > 0) embed_zero_kernel<<<dim3(zero_blocks(all, kThreads, kStoresAlone)), kThreads, 0, stream>>>(all);
    if (n > 0)
      embed_few_kernel<T, G, kV><<<dim3((n + kWaves - 1) / kWaves, chunks), kThreads, 0, stream>>>(g, a.ids, a.id_bytes);
    return hipGetLastError();
  }
  if (n <= kRankMost && a.vocab < (int64_t{1} << (32 - kTokenBits)) - 1) {
    const RankParams rp{a.ids, a.id_bytes, a.vocab, n, (n + kPivots - 1) / kPivots, buf[0], buf[1], all};
    const dim3 grid(rp.groups + zero_blocks(all, kRankThreads));
    if (n <= kRankThreads) rank_kernel<1><<<grid, kRankThreads, 0, stream>>>(rp);
    else if (n <= 4 * kRankThreads) rank_kernel<4><<<grid, kRankThreads, 0, stream>>>(rp);
    else if (n <= 8 * kRankThreads) rank_kernel<8><<<grid, kRankThreads, 0, stream>>>(rp);
    else rank_kernel<16><<<grid, kRankThreads, 0, stream>>>(rp);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    g.keys = buf[0];
    g.toks = buf[1];
  } else {
    const int launches = 3 * passes;
    const int64_t share = ((all.n + launches - 1) / launches + 7) / 8 * 8;   // of a launch, in whole stores
    int64_t done = 0;
    auto next = [&]() {
      const int64_t left = all.n - done;
      const Zeros z{all.p + done, left < share ? left : share};
      done += z.n;
      return z;
    };
    SortParams sp{};
    sp.n = n; sp.tiles = tiles; sp.bits = bits; sp.vocab = a.vocab; sp.hist = hist; sp.id_bytes = a.id_bytes;
    for (int k = 0; k < passes; ++k) {
      sp.ids = k == 0 ? a.ids : nullptr;
      sp.keys = buf[(k & 1) ? 0 : 2];
      sp.toks = buf[(k & 1) ? 1 : 3];
      sp.out_keys = buf[(k & 1) ? 2 : 0];
      sp.out_toks = buf[(k & 1) ? 3 : 1];
      sp.shift = k * bits;
      sp.zeros = next();
      sort_hist_kernel<<<dim3(tiles + zero_blocks(sp.zeros, kThreads)), kThreads, 0, stream>>>(sp);
      const Zeros z = next();
      sort_scan_kernel<<<dim3(1 + zero_blocks(z, kScanThreads)), kScanThreads, 0, stream>>>(
          hist, (int64_t{1} << bits) * tiles, z);
      sp.zeros = next();
      sort_scatter_kernel<<<dim3(tiles + zero_blocks(sp.zeros, kThreads)), kThreads, 0, stream>>>(sp);
      const hipError_t e = hipGetLastError();
      if (e != hipSuccess) return e;
    }
    g.keys = sp.out_keys;
    g.toks = sp.out_toks;
  }
  embed_grad_kernel<T, G, kV><<<dim3(static_cast<unsigned>((g.slices + kWaves - 1) / kWaves), chunks), kThreads, 0,
                                stream>>>(g);
  embed_join_kernel<G, kV><<<dim3(static_cast<unsigned>(g.slices - 1), chunks), kThreads, 0, stream>>>(g);
  return hipGetLastError();
}

}  // namespace

size_t embed_bwd_workspace_bytes(int64_t tokens, int64_t vocab, int64_t dim) {
  if (tokens <= 0) return 0;
  int bits = 0;
  sort_passes(vocab, &bits);
  const size_t n = static_cast<size_t>(tokens), tiles = (n + kTile - 1) / kTile;
  const size_t slices = (n + kSlice - 1) / kSlice;
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
