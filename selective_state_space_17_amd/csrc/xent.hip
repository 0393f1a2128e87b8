// Softmax cross entropy of a linear head over a large vocabulary, and its gradients, for gfx950 (MI355X).
//
//   l[t,v]  = x_t . W_v            lse_t = log sum_v exp l[t,v]        loss_t = lse_t - l[t, y_t]
//   G[t,v]  = exp(l[t,v] - lse_t) (dloss_t + dlse_t) - [v = y_t] dloss_t
//   dx      = G W                  dW (+)= G^T x
// over the tokens whose target counts; the others' x is not read into any sum, their loss, lse and dx are 0.
//
// The logits [tokens, vocab] are never kept.  The forward pass forms them tile by tile on the matrix cores
// and keeps, per token and tile, the maximum and the sum of exponentials (and the target's logit); a second
// kernel joins those.  The gradients take the vocabulary in pieces: a piece's logits are formed again, G of
// the piece goes to the workspace in 16-bit terms, and two more products take it to dx (summed over the pieces in
// fp32) and to the piece's rows of dW.
//
// One tiled product serves all four: out[m, n] = sum_k A[m, k] B[n, k] with m on the weight's side (so that
// a lane's four accumulators are neighbours along the vocabulary or the width, and a token is one column).
// An operand is read K-contiguous (rows of k) or K-strided (k is the row: G^T, x^T, W^T), the latter through
// transposing LDS reads.  Tiles go from global memory straight into LDS.
//
// bf16 inputs enter the matrix cores as they are; products are summed in fp32.  G is rounded to bf16 (the
// gradients' own type) once; for up to 256 tokens, where few roundings average out and the weight's bytes are what
// the time goes into, or where the caller asks for it, it is kept in two bf16 terms.  (8192 x 768 x 50280, relative
// errors of dx in the 2-norm: 2.34e-3 with one rounding of G, 1.66e-3 with two terms, which is dx's own rounding; loss
// and gradients 2.12 and 3.33 ms.)
// fp32 matrices carry a power of two each, s, that brings their largest finite magnitude to [2^14, 2^15).  x and the
// weight enter the logits as two fp16 terms, v s = hi + lo: exact for three values in four, one unit in the last of 24
// bits off (2^-23) for the rest.  A product is the three term products hi lo + lo hi + hi hi, summed in fp32; lo lo is
// left out, below 2^-22 of the product (2^-25 in the mean square).  Over a row of products both vanish beside the
// roundings of the sum.  fp16's smallest step lies 2^39 below the largest value, so values down to 2^-16 of it keep the
// bits said, smaller ones are right to 2^-39 of the largest.  That serves the logits, whose absolute error is what
// counts, and not the gradients: a word's row of dW is made of p dloss with p down to 1e-30, and its error relative to
// its own size is what an optimiser sees.  There x, the weight and G enter as three bf16 terms, all 24 bits of what is
// within 2^-117 of the largest, and a product is the six term products whose places add up to two at most (what is left
// out is below 2^-23 of the product, 2^-26 in the mean square).  One product at the matrix cores' fp32 rate, a sixteenth
// of fp16's, would take 2.7 times the time of six.
#include <type_traits>

#include "device_util.h"
#include "internal.h"

namespace mssm {
namespace {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));
typedef short i16x4 __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) i16x4 lds_i16x4;

constexpr float kLog2e = 1.44269504088896340736f;
constexpr int kBK = 64;                 // k per step: two matrix instructions'
constexpr int kRow = kBK * 2;           // bytes of a row of a step
constexpr int kPlane = 64 * kRow;       // LDS tiles are planes of 64 rows x 128 bytes
constexpr int kTokTile = 256;           // compacted tokens are padded to this
constexpr int kSkew = 34;               // rows between panels: 4352 bytes, see Operand
constexpr int kTerms = 2;               // fp16 terms of an fp32 value in the logits
constexpr int kFineTerms = 3;           // bf16 terms of an fp32 value in the gradients' products
constexpr int kMostPairs = 6;           // term products kept
constexpr int kFewTokens = 256;         // up to these G is kept in two terms with bf16 too

// v (already scaled) = t[0] + t[1]: each the nearest fp16 of what is left.  Infinities and NaN stay what they are.
__device__ __forceinline__ void split_half(float v, uint16_t (&t)[kTerms]) {
  const _Float16 hi = static_cast<_Float16>(v);
  const float r = v - static_cast<float>(hi);
  t[0] = __builtin_bit_cast(uint16_t, hi);
  t[1] = __builtin_bit_cast(uint16_t, static_cast<_Float16>(r == r ? r : 0.f));   // (inf - inf)
}
// the same in bf16 terms
__device__ __forceinline__ void split_bf(float v, uint16_t (&t)[kFineTerms]) {
#pragma unroll
  for (int k = 0; k < kFineTerms; ++k) {
    t[k] = narrow<uint16_t>(v);
    v -= widen(t[k]);
    v = v == v ? v : 0.f;
  }
}

__device__ __forceinline__ uint32_t lds_addr(const void* p) {
  return static_cast<uint32_t>(reinterpret_cast<uintptr_t>(p));   // low half of a flat LDS address
}
// lane l's 16 bytes at base + off go to LDS offset lds + 16 l (base and lds are wave-uniform).  Written as asm
// so that the compiler does not wait for these loads before the LDS reads of the other buffer; they are
// waited for by count.  No output register: nothing can be overwritten while a load is in flight.
__device__ __forceinline__ void dma16(const void* base, uint32_t off, uint32_t lds) {
  asm volatile("s_mov_b32 m0, %2\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %0, %1"
               :: "v"(off), "s"(base), "s"(__builtin_amdgcn_readfirstlane(lds)) : "memory", "m0");
}

// ------------------------------------------------------------------------------------------------ product
// An operand as the products read it, in bytes.  K-contiguous: `row` from one output row to the next, `step`
// per 64 k.  K-strided: `row` from one k to the next, `plane` per 64 output columns, `step` per 64 k.  What
// this library lays out itself (x, G, and the weight where it must) is kept in panels of 64 columns, [panel]
// [row][64]: 64 k of a tile's rows, or 64 rows of a panel, are then one contiguous stretch either way it is read.
// Panels stand kSkew rows further apart than they are long, off the powers of two at which every workgroup
// would be at the same memory channels at the same time.
struct Operand {
  const unsigned char* p;
  int64_t row, step, plane;
  int64_t term;            // between the terms of a split operand
  int rows, planes;        // what may be read: rows, and (K-strided) panels of 64 columns
};

// What the kernels find in the workspace about the call.
enum Plan { kCount = 0, kSlicesX = 1, kSlicesW = 2, kSlicesLastW = 3, kScaleW = 4, kScaleX = 5, kScaleG = 6, kPlanInts = 8 };

struct ProductParams {
  Operand A, B;
  int M, N;                // rows of the output on either side (what lies past them is not stored)
  int K;                   // multiple of 64; with k_is_tokens: the compacted count, rounded up, instead
  int k_is_tokens, n_is_tokens;
  int pairs;               // term products, and the terms of either operand in each
  int ta[kMostPairs], tb[kMostPairs];
  const int* plan;         // see Plan
  int scale_a, scale_b;    // fp32: which of its scales the operands carry
  int slices_at;           // dx, dW: where in plan the slices of the tiles of the last round stand
  // epilogues
  int v0;                  // first vocabulary row of this piece
  const int* tgt;          // compacted targets
  float2* part;            // [tile_m][wave row][tok_cap]: maximum, sum of exponentials
  int64_t tok_cap;
  float* tlogit;           // target's logit
  const float* lse;        // compacted
  const float* gl;         // dloss + dlse
  const float* g;          // dloss
  int g_terms;
  uint16_t* dl;            // panels [vocabulary / 64][token][64], one to three terms
  int64_t pdl;             // elements between them
  float* sums;             // [job][BN][BM]: a slice's sums
  float* over;             // [n][ld_over]: sums over pieces, or null
  int64_t ld_over;
  int first, last;         // of the pieces
  const int* rows;         // compacted -> token
  void* out;               // dx or dW
  int64_t dim;
  int out_f32, accumulate;
};

enum { kLogits = 0, kGradLogits = 1, kGradX = 2, kGradW = 3 };

// Rows 4 q .. 4 q + 3 of two neighbouring row tiles (as bf16; q: the lane's sixteen) to rows 8 q .. 8 q + 7 of the
// 32 rows that they form: tile and q's high bit change places, then that and q's low bit.
__device__ __forceinline__ u32x4_t two_tiles(u32x2_t a, u32x2_t b) {
  u32x4_t v;
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const auto s = __builtin_amdgcn_permlane32_swap(a[i], b[i], false, false);
    const auto t = __builtin_amdgcn_permlane16_swap(s[0], s[1], false, false);
    v[i] = t[0];
    v[2 + i] = t[1];
  }
  return v;
}

// Four neighbouring elements (m .. m + 3, of row n of the other side) of a product's output, to where they belong.
template <int EPI>
__device__ __forceinline__ void put_four(const ProductParams& p, int64_t row, int n, int m, float (&v)[4]) {
  if (EPI == kGradX && p.over != nullptr) {
    float* const to = p.over + n * p.ld_over + m;
    if (!p.first) {
      float o[4];
      load_row<4>(to, o);
#pragma unroll
      for (int e = 0; e < 4; ++e) v[e] += o[e];
    }
    if (!p.last) {
      store_row<4>(to, v);
      return;
    }
  }
  auto put = [&](auto* to) {
    if (EPI == kGradW && p.accumulate) {
      float o[4];
      load_row<4>(to, o, p.M - m);
#pragma unroll
      for (int e = 0; e < 4; ++e) v[e] += o[e];
    }
    store_row<4>(to, v, p.M - m);
  };
  if (p.out_f32) put(static_cast<float*>(p.out) + row * p.dim + m);
  else put(static_cast<uint16_t*>(p.out) + row * p.dim + m);
}

template <typename T> __device__ __forceinline__ T lds_at(uint32_t addr) {
  return *(__attribute__((address_space(3))) const T*)static_cast<uintptr_t>(addr);
}
// the scheduler keeps what stands before this before it
__device__ __forceinline__ void fence_schedule() { __builtin_amdgcn_sched_barrier(0); }

// One workgroup stays on a CU (two of the small tile) and takes tile after tile.  The loads run two steps of
// 64 k ahead of the matrix cores and cross tile borders: a tile's first steps are on their way while the
// tile before it is finished and stored.
// Bound by the matrix cores at the clock that the power limit leaves them (1.8 to 1.9 GHz): 16384 x 2048 x 131072 in
// bf16 runs at 1.32 PFLOP/s (logits, 6.6 ms; a library product of the same sizes, which writes them, at 1.40), 1.21
// (G), 1.28 (dx) and 1.23 (dW), with the matrix cores busy 69, 60, 66 and 64 % of the cycles and no LDS bank
// conflicts; 7373 x 768 x 50280 at 1.03 PFLOP/s (553 us; the library: 0.82).  With few tokens bound by the weight's
// bytes: 16 x 2560 x 50280 in 49 us, 5.2 TB/s with part of the weight left in the 256 MB cache by the call before (a
// kernel that streamed the weight straight into registers was no faster).  Tried and slower: a ring of five
// buffers of 32 k (8.3 against 7.5 ms for the logits at the time), two groups of waves taking turns (8.8 ms), 32 x
// 32 x 16 instructions (8.6 ms, spills), all loads in a step's first two rows (7.9 ms), G stored past the cache
// (1.78 against 1.55 ms a piece).
template <int BM, int BN, int WM, int WN, bool ATR, bool BTR, bool FP32, int EPI>
__global__ __launch_bounds__(WM * WN * 64, 2) void product_kernel(ProductParams p) {
  constexpr int kW = WM * WN;
  constexpr int TM = BM / WM / 16, TN = BN / WN / 16;      // 16 x 16 tiles of a wave
  constexpr int LA = BM / 8 / kW, LB = BN / 8 / kW;        // 1 KB loads of a wave per step
  constexpr int LR = (LA + LB + TM - 1) / TM;              // loads between two rows of multiplications
  constexpr int RR = (TM + TN + TM - 2) / (TM - 1);        // fragments read there
  static_assert(LA * 8 * kW == BM && LB * 8 * kW == BN, "loads split evenly over the waves");
  static_assert(TM % 4 == 0 && TN % 4 == 0, "a wave's share of a tile is whole panels");
  constexpr int kA = BM * kRow, kB = BN * kRow;            // bytes of a buffer
  __shared__ __attribute__((aligned(128))) unsigned char as[2][kA];
  __shared__ __attribute__((aligned(128))) unsigned char bs[2][kB];

  const int lane = threadIdx.x % kLanes;
  const int w = __builtin_amdgcn_readfirstlane(threadIdx.x / kLanes);
  const int wm = w / WN, wn = w % WN;
  const int count = p.plan[kCount];

  // Jobs.  Whole tiles as long as every workgroup gets one; the tiles of the last, partial round are cut along
  // k where that fills the chip, each slice with sums of its own that are added afterwards.  Workgroups b,
  // b + 8, ... share an XCD and its L2: each XCD takes a contiguous range of an order that walks bands of 4
  // n-tiles, m outer, so that what runs on it at one time is a block of 8 m-tiles by 4 n-tiles (bands of 16: 2 %
  // slower, of 8: 1 %).
  const int tiles_m = (p.M + BM - 1) / BM;
  const int tiles_n = ((p.n_is_tokens ? count : p.N) + BN - 1) / BN;
  const int tiles = tiles_m * tiles_n;
  constexpr bool kSliced = EPI == kGradX || EPI == kGradW;
  const int whole = kSliced ? tiles / static_cast<int>(gridDim.x) * static_cast<int>(gridDim.x) : 0;
  const int slices = kSliced ? p.plan[p.slices_at] : 1;
  const int rest = tiles - whole, cut = rest * slices;
  const int xcd = blockIdx.x % 8, stride = gridDim.x / 8;
  const int whole8 = whole / 8, cut8 = (cut + 7) / 8;      // of an XCD
  const int mine = cut - xcd * cut8 < cut8 ? cut - xcd * cut8 : cut8;
  const int job_first = blockIdx.x / 8, job_end = whole8 + (mine > 0 ? mine : 0);
  const int steps1 = ((p.k_is_tokens ? count : p.K) + kBK - 1) / kBK;   // of one pair of terms
  const int all = steps1 * p.pairs;
  struct Job {
    int m0, n0, sum, begin, steps;   // sum: which sums, or -1
  };
  auto job_at = [&](int i) {
    Job j;
    int tile;
    if (!kSliced || i < whole8) {
      tile = kSliced ? xcd * whole8 + i : xcd * cut8 + i;
      j.sum = -1;
      j.begin = 0;
      j.steps = all;
    } else {
      const int c = xcd * cut8 + i - whole8;
      const int slice = c / rest;
      tile = whole + c - slice * rest;
      j.sum = slices > 1 ? c : -1;
      j.begin = static_cast<int>(static_cast<int64_t>(all) * slice / slices);
      j.steps = static_cast<int>(static_cast<int64_t>(all) * (slice + 1) / slices) - j.begin;
    }
    const int band = tile / (tiles_m * 4);
    const int left = tiles_n - band * 4, wide = left < 4 ? left : 4;
    const int in_band = tile - band * tiles_m * 4;
    j.m0 = in_band / wide * BM;
    j.n0 = (band * 4 + in_band % wide) * BN;
    return j;
  };

  // ---- loads.  A load is 8 rows x 128 bytes (K-strided: of a plane of 64 columns), a lane's part row
  // lane / 8 and the 16-byte chunk lane % 8 as stored.  The chunk it holds is xor-ed with a key of the row that
  // keeps the reads below free of bank conflicts: K-contiguous, where 16 lanes read one chunk of 16 rows, the
  // row's low three bits; K-strided, where 32 lanes read a pair of chunks of rows r .. r + 3 and r + 8 .. r + 11,
  // its bits 1 and 3 (above the bit within the pair).  Rows past the matrix are its last row again, panels its
  // last panel.
  const int lrow = lane / 8;
  int ljob = job_first;   // job, step and pair of terms of the next loads
  int lleft = 0, lk = 0, lseg = 0;
  const unsigned char *la = nullptr, *lb = nullptr;
  uint32_t oa[LA], ob[LB];
  auto offsets = [&](const Operand& o, bool tr, int o0, auto& off) {
#pragma unroll
    for (int i = 0; i < static_cast<int>(sizeof(off) / sizeof(off[0])); ++i) {
      const int r = (i * kW + w) * 8 + lrow;
      if (!tr) {
        off[i] = static_cast<uint32_t>((o0 + r < o.rows ? r : o.rows - 1 - o0) * o.row) + ((lane % 8) ^ lrow) * 16;
      } else {
        off[i] = static_cast<uint32_t>(r % 64 * o.row) + ((lane % 8) ^ ((r & 2) | (r & 8) / 2)) * 16;
      }
    }
  };
  Job lj{};
  auto start_pair = [&]() {
    la = p.A.p + p.ta[lseg] * p.A.term + (ATR ? 0 : lj.m0 * p.A.row);
    lb = p.B.p + p.tb[lseg] * p.B.term + (BTR ? 0 : lj.n0 * p.B.row);
  };
  auto start_load = [&]() {   // the next job with steps, if there is one; else the last loads are repeated
    while (ljob < job_end) {
      const Job j = job_at(ljob);
      if (j.steps > 0) {
        lj = j;
        lleft = j.steps;
        lseg = j.begin / steps1;
        lk = j.begin - lseg * steps1;
        offsets(p.A, ATR, j.m0, oa);
        offsets(p.B, BTR, j.n0, ob);
        start_pair();
        return;
      }
      ljob += stride;
    }
  };
  const uint32_t as_a = lds_addr(&as[0][0]), bs_a = lds_addr(&bs[0][0]);
  // load i of a step into buffer `buf`
  auto load_a = [&](int i, int buf) {
    const unsigned char* a = la + lk * p.A.step;
    uint32_t o = oa[i];
    if constexpr (ATR) {
      const int plane = lj.m0 / 64 + i * kW / 8;
      a += (plane < p.A.planes ? plane : p.A.planes - 1) * p.A.plane;
      if ((lk + 1) * kBK > p.A.rows) {   // k rows past the matrix: its last row again
        const int over = lk * kBK + (i * kW + w) % 8 * 8 + lrow - (p.A.rows - 1);
        if (over > 0) o -= static_cast<uint32_t>(over * p.A.row);
      }
    }
    dma16(a, o, as_a + buf * kA + (i * kW + w) * 1024);
  };
  auto load_b = [&](int i, int buf) {
    const unsigned char* b = lb + lk * p.B.step;
    if constexpr (BTR) {
      const int plane = lj.n0 / 64 + i * kW / 8;
      b += (plane < p.B.planes ? plane : p.B.planes - 1) * p.B.plane;
    }
    dma16(b, ob[i], bs_a + buf * kB + (i * kW + w) * 1024);
  };
  auto load_one = [&](int i, int buf) {
    if (i < LA) load_a(i < LA ? i : 0, buf);
    else load_b(i - LA < LB ? i - LA : 0, buf);
  };
  auto loaded = [&]() {   // after a step's last load
    if (lleft > 1) {
      --lleft;
      if (++lk == steps1) {
        lk = 0;
        ++lseg;
        start_pair();
      }
    } else if (ljob < job_end) {
      ljob += stride;
      start_load();
    }
  };

  // ---- fragments.  K-strided: in each 16-lane group, lane j receives element j of the four 16-element rows
  // that its lanes point at.
  uint32_t fa_at[2], fb_at[2];   // by k half
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const int r = lane % 16;
    const uint32_t kc = r * kRow + (((h * 4 + lane / 16) ^ (r & 7)) << 4);
    const int j = lane % 16, tr = lane / 16 * 8 + j / 4;
    const uint32_t ks = (h * 32 + tr) * kRow + (((j % 4 / 2) ^ ((tr & 2) | (tr & 8) / 2)) << 4) + j % 2 * 8;
    fa_at[h] = as_a + (ATR ? ks + wm * (TM / 4) * kPlane : kc + wm * TM * 16 * kRow);
    fb_at[h] = bs_a + (BTR ? ks + wn * (TN / 4) * kPlane : kc + wn * TN * 16 * kRow);
  }
  auto frag = [&](uint32_t at, bool tr, int t) -> bf16x8 {
    if (!tr) return lds_at<bf16x8>(at + t * 16 * kRow);
    u32x4_t f;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const uint32_t addr = (at ^ (t % 4 * 32)) + t / 4 * kPlane + h * 4 * kRow;
      const u32x2_t v = __builtin_bit_cast(
          u32x2_t, __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_i16x4*)static_cast<uintptr_t>(addr)));
      f[2 * h] = v[0];
      f[2 * h + 1] = v[1];
    }
    return __builtin_bit_cast(bf16x8, f);
  };
  f32x4_t acc[TM][TN];
  bf16x8 fa[2][TM], fb[2][TN];
  auto read_one = [&](int q, uint32_t at_a, uint32_t at_b, int set) {
    if (q < TN) fb[set][q < TN ? q : 0] = frag(at_b, BTR, q < TN ? q : 0);
    else fa[set][q - TN < TM ? q - TN : 0] = frag(at_a, ATR, q - TN < TM ? q - TN : 0);
  };
  auto multiply_row = [&](int i, int set) {
#pragma unroll
    for (int j = 0; j < TN; ++j)
      if constexpr (FP32 && !kSliced)
        acc[i][j] = __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8, fa[set][i]),
                                                           __builtin_bit_cast(f16x8, fb[set][j]), acc[i][j], 0, 0, 0);
      else
        acc[i][j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(fa[set][i], fb[set][j], acc[i][j], 0, 0, 0);
  };

  // ---- Two LDS buffers, two sets of fragments.  A step's second half is read while its first half is
  // multiplied; between the halves every wave has read all of the step's buffer, so one barrier there frees it
  // for the loads two steps ahead and publishes the next step's, whose first half is then read while the
  // second half is multiplied.  Reads and loads are spread between the multiplications: all waves at once
  // would queue for the LDS with the matrix cores idle.
  start_load();
  if (lleft > 0) {   // (no steps at all where no token counts: the tiles are then stored as zeros)
#pragma unroll
    for (int b = 0; b < 2; ++b) {
#pragma unroll
      for (int q = 0; q < LA + LB; ++q) load_one(q, b);
      loaded();
    }
    asm volatile("s_waitcnt vmcnt(%0)" ::"n"(LA + LB) : "memory");
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
  }
  int buf = 0;
#pragma unroll
  for (int q = 0; q < TM + TN; ++q) read_one(q, fa_at[0], fb_at[0], 0);
  for (int job = job_first; job < job_end; job += stride) {
    const Job cur = job_at(job);
    const int m0 = cur.m0, n0 = cur.n0;
#pragma unroll
    for (int i = 0; i < TM; ++i)
#pragma unroll
      for (int j = 0; j < TN; ++j) acc[i][j] = f32x4_t{0.f, 0.f, 0.f, 0.f};
    for (int s = 0; s < cur.steps; ++s, buf ^= 1) {
      fence_schedule();
      {
        const uint32_t at_a = fa_at[1] + buf * kA, at_b = fb_at[1] + buf * kB;
#pragma unroll
        for (int i = 0; i < TM; ++i) {
          multiply_row(i, 0);
          fence_schedule();
#pragma unroll
          for (int q = i * RR; q < (i + 1) * RR && q < TM + TN; ++q) read_one(q, at_a, at_b, 1);
          fence_schedule();
        }
      }
      asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)" ::: "memory");
      __builtin_amdgcn_s_barrier();
      asm volatile("" ::: "memory");
      fence_schedule();
      {
        const uint32_t at_a = fa_at[0] + (buf ^ 1) * kA, at_b = fb_at[0] + (buf ^ 1) * kB;
#pragma unroll
        for (int i = 0; i < TM; ++i) {
          multiply_row(i, 1);
          fence_schedule();
#pragma unroll
          for (int q = i * LR; q < (i + 1) * LR && q < LA + LB; ++q) load_one(q, buf);
#pragma unroll
          for (int q = i * RR; q < (i + 1) * RR && q < TM + TN; ++q) read_one(q, at_a, at_b, 0);
          fence_schedule();
        }
      }
      loaded();
    }

    // accumulator e of tile (i, j): row m = m0 + (wm TM + i) 16 + 4 (lane / 16) + e, column n = n0 + (wn TN + j) 16 + lane % 16
    const int wave_m = m0 + wm * TM * 16;
    const int mrow = wave_m + lane / 16 * 4;
    const int ncol = n0 + wn * TN * 16 + lane % 16;
    // What undoes the operands' scales: their product may lie outside fp32, so two powers of two, one after the
    // other, each half of it: what is in between lies between the accumulator and the result, and overflows only if
    // one of them does.  For the logits the product is kept at 2^-126 or more: they are then as good as 0, but 0
    // times the mask's -inf would not be -inf.
    const float* const scales = reinterpret_cast<const float*>(p.plan);
    const int back = FP32 ? 254 - (__float_as_uint(scales[p.scale_a]) >> 23) - (__float_as_uint(scales[p.scale_b]) >> 23) : 0;
    const float ua = __uint_as_float((127 + back / 2) << 23), ub = __uint_as_float((127 + back - back / 2) << 23);
    const float unit = __builtin_fmaxf(ua * ub, 0x1p-126f);
    const float to_log2 = kLog2e * unit;
    auto each = [&](int j, auto&& f) {   // accumulator = f(accumulator, row)
#pragma unroll
      for (int i = 0; i < TM; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e) acc[i][j][e] = f(acc[i][j][e], mrow + i * 16 + e);
    };
    if constexpr (EPI == kLogits) {
#pragma unroll
      for (int j = 0; j < TN; ++j) {
        const int n = ncol + j * 16;
        if (m0 + BM > p.M) each(j, [&](float a, int m) { return m < p.M ? a : -__builtin_inff(); });
        const int y = p.tgt[n] - p.v0;   // padded tokens have target -1
        if (__ballot(y >= wave_m && y < wave_m + TM * 16) != 0) {
          float hit = 0.f;   // (one store: as many as there are rows cost each wave 0.8 us a tile)
          each(j, [&](float a, int m) {
            hit = m == y ? a : hit;
            return a;
          });
          const int at = y - mrow;
          if (at >= 0 && at < TM * 16 && at % 16 < 4) p.tlogit[n] = hit * unit;
        }
        float mx = -__builtin_inff();
        each(j, [&](float a, int) {
          mx = __builtin_fmaxf(mx, a);
          return a;
        });
        mx = __builtin_fmaxf(mx, __shfl_xor(mx, 16, 64));
        mx = __builtin_fmaxf(mx, __shfl_xor(mx, 32, 64)) * unit;
        // exp(a - mx) = 2^(a log2e - c) 2^(c - mx log2e): one multiply-add an element, and the rounding of
        // c = mx log2e taken out of the sum once
        const float ref = mx == -__builtin_inff() ? 0.f : mx, c = ref * kLog2e;
        float s = 0.f;
        each(j, [&](float a, int) {
          s += __builtin_amdgcn_exp2f(__builtin_fmaf(a, to_log2, -c));
          return a;
        });
        s += __shfl_xor(s, 16, 64);
        s += __shfl_xor(s, 32, 64);
        s *= __builtin_amdgcn_exp2f(__builtin_fmaf(-ref, kLog2e, c));
        if (lane < 16) p.part[(static_cast<int64_t>(m0 / BM) * WM + wm) * p.tok_cap + n] = float2{mx, s};
      }
    } else if constexpr (EPI == kGradLogits) {
#pragma unroll
      for (int j = 0; j < TN; ++j) {
        const int n = ncol + j * 16;
        const float sg = FP32 ? scales[kScaleG] : 1.f;
        const float lse = p.lse[n], g = p.g[n] * sg, c = lse * kLog2e;
        const float gl = p.gl[n] * sg * __builtin_amdgcn_exp2f(__builtin_fmaf(-lse, kLog2e, c));   // as in the forward pass
        each(j, [&](float a, int) { return __builtin_amdgcn_exp2f(__builtin_fmaf(a, to_log2, -c)) * gl; });
        const int y = p.tgt[n] - p.v0;
        if (__ballot(y >= wave_m && y < wave_m + TM * 16) != 0) each(j, [&](float a, int m) { return a - (m == y ? g : 0.f); });
        if (m0 + BM > p.M || n0 + BN > count) each(j, [&](float a, int m) { return n < count && m < p.M ? a : 0.f; });
        // two row tiles together: a lane gets 8 neighbouring elements, the four lanes of a token 64 bytes
        uint16_t* const to = p.dl + (wave_m / 64 * (p.tok_cap + kSkew) + n) * 64 + lane / 16 * 8;
#pragma unroll
        for (int i = 0; i < TM; i += 2) {
          uint16_t* const at = to + (i / 4 * (p.tok_cap + kSkew)) * 64 + i % 4 * 16;
          if (FP32 || p.g_terms == 2) {
            // term after term of what is left
            f32x4_t r[2] = {acc[i][j], acc[i + 1][j]};
#pragma unroll
            for (int k = 0; k < (FP32 ? kFineTerms : 2); ++k) {
              u32x2_t d[2];
#pragma unroll
              for (int h = 0; h < 2; ++h)
#pragma unroll
                for (int e = 0; e < 4; e += 2) {
                  float a, b;
                  d[h][e / 2] = pack_bf16(r[h][e], r[h][e + 1]);
                  split_bf16(d[h][e / 2], a, b);
                  a = r[h][e] - a;
                  b = r[h][e + 1] - b;
                  r[h][e] = a == a ? a : 0.f;   // (inf - inf)
                  r[h][e + 1] = b == b ? b : 0.f;
                }
              *reinterpret_cast<u32x4_t*>(at + k * p.pdl) = two_tiles(d[0], d[1]);
            }
          } else {
            const f32x4_t x = acc[i][j], y = acc[i + 1][j];
            *reinterpret_cast<u32x4_t*>(at) =
                two_tiles(u32x2_t{pack_bf16(x[0], x[1]), pack_bf16(x[2], x[3])},
                          u32x2_t{pack_bf16(y[0], y[1]), pack_bf16(y[2], y[3])});
          }
        }
      }
    } else {
#pragma unroll
      for (int j = 0; j < TN; ++j) {
        const int n = ncol + j * 16;
        if (EPI == kGradX ? n >= count : n >= p.N) continue;
        if (cur.sum >= 0) {
          float* const to = p.sums + (static_cast<int64_t>(cur.sum) * BN + n - n0) * BM + mrow - m0;
#pragma unroll
          for (int i = 0; i < TM; ++i) *reinterpret_cast<f32x4_t*>(to + i * 16) = acc[i][j] * ua * ub;
          continue;
        }
        const int64_t row = EPI == kGradX ? static_cast<int64_t>(p.rows[n]) : n;
#pragma unroll
        for (int i = 0; i < TM; ++i) {
          const f32x4_t d = acc[i][j] * ua * ub;
          float v[4] = {d[0], d[1], d[2], d[3]};
          if (mrow + i * 16 < p.M) put_four<EPI>(p, row, n, mrow + i * 16, v);
        }
      }
    }
  }
  // the last loads may still be on their way into this workgroup's LDS
  asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
}

// Adds the slices of the tiles of the last round, in order: workgroup (tile, share of its n).
constexpr int kShares = 8;
template <int BM, int BN, int EPI>
__global__ __launch_bounds__(256) void sum_kernel(ProductParams p, int slots) {
  const int count = p.plan[kCount], slices = p.plan[p.slices_at];
  if (slices == 1) return;
  const int tiles_m = (p.M + BM - 1) / BM;
  const int tiles_n = ((p.n_is_tokens ? count : p.N) + BN - 1) / BN;
  const int tiles = tiles_m * tiles_n, rest = tiles % slots;
  const int t = blockIdx.x / kShares;
  if (t >= rest) return;
  const int tile = tiles - rest + t;
  const int band = tile / (tiles_m * 4);
  const int left = tiles_n - band * 4, wide = left < 4 ? left : 4;
  const int in_band = tile - band * tiles_m * 4;
  const int m = in_band / wide * BM + threadIdx.x % (BM / 4) * 4, n0 = (band * 4 + in_band % wide) * BN;
  if (m >= p.M) return;
  constexpr int kRows = BN / kShares, kAtOnce = 256 / (BM / 4);
  const int first = blockIdx.x % kShares * kRows + threadIdx.x / (BM / 4);
  for (int i = 0; i < kRows; i += kAtOnce) {
    const int n = n0 + first + i;
    if (n >= (EPI == kGradX ? count : p.N)) return;
    float v[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll 4
    for (int s = 0; s < slices; ++s) {
      float o[4];
      load_row<4>(p.sums + ((static_cast<int64_t>(s) * rest + t) * BN + first + i) * BM + threadIdx.x % (BM / 4) * 4, o);
#pragma unroll
      for (int e = 0; e < 4; ++e) v[e] += o[e];
    }
    put_four<EPI>(p, EPI == kGradX ? static_cast<int64_t>(p.rows[n]) : n, n, m, v);
  }
}

// How many slices the tiles of the last round are cut into: the least time, in steps of a workgroup.  A slice
// costs some four steps more (its start, its sums' way out) and the addition some eight (of a few slices; of hundreds,
// which only a tile or two of very many steps come to, far more: 83 us of 165 at 64 x 128 x 131072).  At most two
// rounds of slices, which bounds the sums' memory.  Of a workgroup of 256, every thread with some of the up to 1024 counts:
// one thread after another's three divisions took 150 us for 64 x 128 x 131072.
__device__ int pick_slices(int tiles, int steps, int slots, uint64_t (&red)[4]) {
  const int rest = tiles % slots;
  uint64_t best = ~0ull;   // time and, for equal times, the fewer slices
  for (int s = 1 + threadIdx.x; s == 1 || (rest > 0 && rest * s <= 2 * slots && steps / s >= 4); s += 256) {
    const int time = s == 1 ? steps : (rest * s + slots - 1) / slots * ((steps + s - 1) / s + 4) + 8;
    const uint64_t mine = static_cast<uint64_t>(time) << 32 | static_cast<uint32_t>(s);
    best = mine < best ? mine : best;
  }
#pragma unroll
  for (int step = 1; step < kLanes; step *= 2) {
    const uint64_t o = __shfl_xor(best, step, kLanes);
    best = o < best ? o : best;
  }
  __syncthreads();
  if (threadIdx.x % kLanes == 0) red[threadIdx.x / kLanes] = best;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < 4; ++w) best = red[w] < best ? red[w] : best;
  return static_cast<int>(best & 0xffffffffu);
}

// -------------------------------------------------------------------------------------- around the products
struct PrepParams {
  const void* targets;
  int id_bytes;
  int64_t ignore, vocab, tokens, dim, dpad, tok_cap;
  const void* x;
  uint16_t* xc;            // panels [term][dpad / 64][tok_cap][64]
  uint16_t* xf;            // fp32 gradients: the same in bf16 terms, or null
  int* tally;              // counted tokens of each group of kGroup, or null: counted again where needed
  int* plan;               // written: the count, the slices, the scales
  const uint32_t* range;   // fp32: the largest magnitudes, see range_kernel
  int pairs, steps_x, tile_x, tile_w, tiles_mx, tiles_w, tiles_w_last;
  int* rows;
  int* tgt;
  int per;                 // tokens of a workgroup (64 at most)
  int work_blocks;         // workgroups with tokens; the ones after them pad
  // forward
  float* loss;
  float* lse_out;
  // gradients
  const float* lse;
  const float* dloss;
  const float* dlse;       // nullable
  float* c_lse;
  float* c_gl;
  float* c_g;
  void* dx;                // nullable: rows of tokens left out are zeroed
};

constexpr int kCUs = 256;
constexpr int kBig = 256, kSmall = 128;   // tiles: one workgroup to a CU, or two
__host__ __device__ constexpr int slots_of(int tile) { return tile == kBig ? kCUs : 2 * kCUs; }

constexpr int kPadBlocks = 16;
constexpr int kGroup = 4096;

__device__ __forceinline__ bool target_counts(const PrepParams& p, int64_t y) {
  return y >= 0 && y < p.vocab && y != p.ignore;
}
__device__ __forceinline__ bool token_counts(const PrepParams& p, int64_t t) {
  return target_counts(p, id_at(p.targets, p.id_bytes, t));
}
// how many of a thread's tokens lo + tid, lo + tid + 256, ... below hi count, E at a time
template <int E>
__device__ __forceinline__ int counted(const PrepParams& p, int64_t lo, int64_t hi) {
  int n = 0;
  for (int64_t t = lo + threadIdx.x; t < hi; t += E * 256) {
    int64_t y[E];
    ids_at<E>(p.targets, p.id_bytes, t, 256, hi, y);
#pragma unroll
    for (int e = 0; e < E; ++e) n += t + e * 256 < hi && target_counts(p, y[e]);
  }
  return n;
}

// the sum of every thread's n over the workgroup of 256
__device__ __forceinline__ int block_count(int n, int* red) {
#pragma unroll
  for (int step = 1; step < kLanes; step *= 2) n += __shfl_xor(n, step, kLanes);
  if (threadIdx.x % kLanes == 0) red[threadIdx.x / kLanes] = n;
  __syncthreads();
  return red[0] + red[1] + red[2] + red[3];
}

__global__ __launch_bounds__(256) void tally_kernel(PrepParams p) {
  __shared__ int red[4];
  const int64_t lo = static_cast<int64_t>(blockIdx.x) * kGroup;
  const int n = block_count(counted<kGroup / 256>(p, lo, lo + kGroup < p.tokens ? lo + kGroup : p.tokens), red);
  if (threadIdx.x == 0) p.tally[blockIdx.x] = n;
}

// 8 elements of a row, laid out: bf16 as it is, fp32 scaled and in two fp16 terms, and with `fine` in three bf16 terms
// there; past the row's end zeros
template <typename T>
__device__ __forceinline__ void lay_out(const T* row, int64_t col, int64_t dim, uint16_t* to, uint16_t* fine,
                                        int64_t term, float scale) {
  if constexpr (sizeof(T) == 2) {
    u32x4_t v = {0, 0, 0, 0};
    if (col + 8 <= dim) {
      v = *reinterpret_cast<const u32x4_u*>(row + col);
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e)
        if (col + e < dim) v[e / 2] |= static_cast<uint32_t>(row[col + e]) << (e % 2 * 16);
    }
    *reinterpret_cast<u32x4_t*>(to) = v;
  } else {
    float f[8];
    load_row<8>(row + col, f, dim - col);
    auto put = [&](auto n, uint16_t* at, auto&& split) {
      constexpr int kN = decltype(n)::value;
      uint16_t t[8][kN];
#pragma unroll
      for (int e = 0; e < 8; ++e) split(f[e], t[e]);
#pragma unroll
      for (int k = 0; k < kN; ++k) {
        u32x4_t v;
#pragma unroll
        for (int e = 0; e < 4; ++e) v[e] = t[2 * e][k] | static_cast<uint32_t>(t[2 * e + 1][k]) << 16;
        *reinterpret_cast<u32x4_t*>(at + k * term) = v;
      }
    };
    put(std::integral_constant<int, kTerms>{}, to, [&](float v, auto& t) { split_half(v * scale, t); });
    if (fine != nullptr)
      put(std::integral_constant<int, kFineTerms>{}, fine, [&](float v, auto& t) { split_bf(v * scale, t); });
  }
}

// The largest finite magnitudes, of the weight, of the counted tokens' x and of their dloss and dloss + dlse
// (fp32 only), each workgroup's.
struct RangeParams {
  PrepParams prep;
  const float* weight;
  int64_t elems;
  uint32_t* part;          // [3][kRangeBlocks]
};
constexpr int kRangeBlocks = 1024;

__device__ __forceinline__ uint32_t magnitude(float v) {
  const uint32_t m = __float_as_uint(v) & 0x7fffffffu;
  return m < 0x7f800000u ? m : 0u;
}
__device__ __forceinline__ uint32_t wave_max(uint32_t v) {
#pragma unroll
  for (int step = 1; step < kLanes; step *= 2) {
    const uint32_t o = __shfl_xor(v, step, kLanes);
    v = o > v ? o : v;
  }
  return v;
}

__global__ __launch_bounds__(256) void range_kernel(RangeParams r) {
  __shared__ uint32_t red[4][3];
  const PrepParams& p = r.prep;
  const int wave = threadIdx.x / kLanes, lane = threadIdx.x % kLanes;
  uint32_t m[3] = {0, 0, 0};
  auto scan = [&](const float* v, int64_t n, int64_t first, int64_t step, uint32_t& most) {
#pragma unroll 4
    for (int64_t i = first * 4; i < n; i += step * 4) {
      float f[4];
      load_row<4>(v + i, f, n - i);
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const uint32_t a = magnitude(f[e]);
        most = a > most ? a : most;
      }
    }
  };
  scan(r.weight, r.elems, static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x, int64_t{kRangeBlocks} * 256, m[0]);
  for (int64_t t = static_cast<int64_t>(blockIdx.x) * 4 + wave; t < p.tokens; t += kRangeBlocks * 4) {
    if (!token_counts(p, t)) continue;
    scan(static_cast<const float*>(p.x) + t * p.dim, p.dim, lane, kLanes, m[1]);
    if (p.dloss != nullptr) {
      const float g = p.dloss[t];
      const uint32_t a = magnitude(g), b = magnitude(p.dlse != nullptr ? g + p.dlse[t] : g);
      m[2] = a > m[2] ? a : m[2];
      m[2] = b > m[2] ? b : m[2];
    }
  }
#pragma unroll
  for (int k = 0; k < 3; ++k) {
    m[k] = wave_max(m[k]);
    if (lane == 0) red[wave][k] = m[k];
  }
  __syncthreads();
  if (threadIdx.x < 3) {
    uint32_t v = 0;
    for (int w = 0; w < 4; ++w) v = red[w][threadIdx.x] > v ? red[w][threadIdx.x] : v;
    r.part[threadIdx.x * kRangeBlocks + blockIdx.x] = v;
  }
}

// 2^e as fp32 that brings the k-th maximum to [2^14, 2^15), but at most 2^126; for a workgroup of 256
__device__ __forceinline__ uint32_t scale_of(const uint32_t* range, int k, uint32_t (&red)[4]) {
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < kRangeBlocks / 256; ++i) {
    const uint32_t v = range[k * kRangeBlocks + i * 256 + threadIdx.x];
    m = v > m ? v : m;
  }
  m = wave_max(m);
  __syncthreads();
  if (threadIdx.x % kLanes == 0) red[threadIdx.x / kLanes] = m;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < 4; ++w) m = red[w] > m ? red[w] : m;
  const int e = 14 - (static_cast<int>(m >> 23) - 127);
  return static_cast<uint32_t>((m == 0 ? 0 : e > 126 ? 126 : e) + 127) << 23;
}

// Which tokens count, in order, and their x as the products read it: in panels of 64 columns, padded with
// zeros, fp32 as two fp16 terms (and for the gradients three bf16 terms beside); after the last one, zero rows up to
// the end of its tile of 256.
template <typename T>
__global__ __launch_bounds__(256) void prep_kernel(PrepParams p) {
  __shared__ int red[4];
  const int wave = threadIdx.x / kLanes, lane = threadIdx.x % kLanes;
  const bool pad = static_cast<int>(blockIdx.x) >= p.work_blocks;
  const int64_t lo = pad ? p.tokens : static_cast<int64_t>(blockIdx.x) * p.per;
  int before = 0;
  int64_t from = 0;
  if (p.tally != nullptr) {
    const int groups = static_cast<int>(lo / kGroup);
    for (int g = threadIdx.x; g < groups; g += 256) before += p.tally[g];
    from = static_cast<int64_t>(groups) * kGroup;
  }
  before += counted<8>(p, from, lo);
  before = block_count(before, red);

  const int64_t term = (p.tok_cap + kSkew) * p.dpad;
  float scale = 1.f;
  if constexpr (sizeof(T) == 4) {   // (every workgroup finds the scale of x for itself: a launch between took 5 us)
    __shared__ uint32_t most[4];
    scale = __uint_as_float(scale_of(p.range, 1, most));
    if (blockIdx.x == static_cast<unsigned>(p.work_blocks)) {
      const uint32_t w = scale_of(p.range, 0, most), g = scale_of(p.range, 2, most);
      if (threadIdx.x < 3)
        p.plan[kScaleW + threadIdx.x] = static_cast<int>(threadIdx.x == 0 ? w : threadIdx.x == 1 ? __float_as_uint(scale) : g);
    }
  }
  auto put = [&](int64_t i, int64_t t, bool real) {
    const T* row = static_cast<const T*>(p.x) + t * p.dim;
    for (int64_t c = lane * 8; c < p.dpad; c += kLanes * 8) {
      const int64_t at = (c / 64 * (p.tok_cap + kSkew) + i) * 64 + c % 64;
      lay_out<T>(row, c, real ? p.dim : 0, p.xc + at, p.xf != nullptr ? p.xf + at : nullptr, term, scale);
    }
  };
  if (pad) {
    if (blockIdx.x == static_cast<unsigned>(p.work_blocks)) {
      __shared__ uint64_t least[4];
      int slices[3] = {1, 1, 1};
      if (p.c_lse != nullptr) {
        const int steps_w = (before + kBK - 1) / kBK * p.pairs;
        const int tiles_x = p.tiles_mx * ((before + p.tile_x - 1) / p.tile_x);
        slices[0] = pick_slices(tiles_x, p.steps_x, slots_of(p.tile_x), least);
        slices[1] = pick_slices(p.tiles_w, steps_w, slots_of(p.tile_w), least);
        slices[2] = p.tiles_w_last == p.tiles_w ? slices[1] : pick_slices(p.tiles_w_last, steps_w, slots_of(p.tile_w), least);
      }
      if (threadIdx.x == 0) {
        p.plan[kCount] = before;
        p.plan[kSlicesX] = slices[0];
        p.plan[kSlicesW] = slices[1];
        p.plan[kSlicesLastW] = slices[2];
      }
    }
    const int64_t end = (before + kTokTile - 1) / kTokTile * int64_t{kTokTile};
    for (int64_t i = before + (blockIdx.x - p.work_blocks) * 4 + wave; i < end; i += kPadBlocks * 4) {
      put(i, 0, false);
      if (lane == 0) {
        p.rows[i] = 0;
        p.tgt[i] = -1;
        if (p.c_lse != nullptr) p.c_lse[i] = p.c_gl[i] = p.c_g[i] = 0.f;
      }
    }
    return;
  }
  const int64_t hi = lo + p.per < p.tokens ? lo + p.per : p.tokens;
  // lane l of every wave looks at token lo + l
  const bool mine = lo + lane < hi && token_counts(p, lo + lane);
  const uint64_t mask = __ballot(mine);
  for (int64_t t = lo + wave; t < hi; t += 4) {
    const int l = static_cast<int>(t - lo);
    if ((mask >> l) & 1) {
      const int64_t i = before + __popcll(mask & ((1ull << l) - 1));
      put(i, t, true);
      if (lane == 0) {
        p.rows[i] = static_cast<int>(t);
        p.tgt[i] = static_cast<int>(id_at(p.targets, p.id_bytes, t));
        if (p.c_lse != nullptr) {
          const float g = p.dloss[t];
          p.c_lse[i] = p.lse[t];
          p.c_g[i] = g;
          p.c_gl[i] = p.dlse != nullptr ? g + p.dlse[t] : g;
        }
      }
    } else {
      if (p.loss != nullptr && lane == 0) p.loss[t] = p.lse_out[t] = 0.f;
      if (p.dx != nullptr)
        for (int64_t c = lane; c < p.dim; c += kLanes) static_cast<T*>(p.dx)[t * p.dim + c] = 0;
    }
  }
}

// rows of the weight as the products read them (width not a multiple of 64, or fp32), in panels
// [term][dpad / 64][rows][64]: 32 rows a workgroup; `fine`: see lay_out
template <typename T>
__global__ __launch_bounds__(256) void weight_kernel(const T* w, uint16_t* to, uint16_t* fine, int64_t rows, int64_t dim,
                                                     int64_t dpad, const int* plan) {
  const int64_t r = static_cast<int64_t>(blockIdx.x) * 32 + threadIdx.x / 8;
  if (r >= rows) return;
  const float scale = sizeof(T) == 2 ? 1.f : reinterpret_cast<const float*>(plan)[kScaleW];
  for (int64_t c = threadIdx.x % 8 * 8; c < dpad; c += 64) {
    const int64_t at = (c / 64 * (rows + kSkew) + r) * 64 + c % 64;
    lay_out<T>(w + r * dim, c, dim, to + at, fine != nullptr ? fine + at : nullptr, (rows + kSkew) * dpad, scale);
  }
}

// Joins the tiles' (maximum, sum) of a piece with those of the pieces before it; after the last piece, the loss.
struct JoinParams {
  const float2* part;
  int tiles, first, last;
  int64_t tok_cap;
  const int* plan;
  const int* rows;
  float2* run;
  const float* tlogit;
  float* loss;
  float* lse;
};

__device__ __forceinline__ float2 join(float2 a, float2 b) {
  const float m = __builtin_fmaxf(a.x, b.x);
  const float ref = m == -__builtin_inff() ? 0.f : m;
  // (a part of maximum -inf holds a sum of zeros or, where a logit was NaN, NaN)
  return {m, a.y * __builtin_amdgcn_exp2f((a.x - ref) * kLog2e) + b.y * __builtin_amdgcn_exp2f((b.x - ref) * kLog2e)};
}

// TL tokens x 256 / TL shares of the tiles a workgroup: many tokens side by side, or many shares of a few.
template <int TL>
__global__ __launch_bounds__(256) void join_kernel(JoinParams p) {
  constexpr int kShareN = 256 / TL;
  __shared__ float2 red[kShareN][TL + 1];
  const int tl = threadIdx.x % TL, share = threadIdx.x / TL;
  const int64_t n = static_cast<int64_t>(blockIdx.x) * TL + tl;
  const int count = p.plan[kCount];
  if (static_cast<int64_t>(blockIdx.x) * TL >= count) return;
  float2 r = {-__builtin_inff(), 0.f};
  if (n < count) {
#pragma unroll 4
    for (int k = share; k < p.tiles; k += kShareN) r = join(r, p.part[k * p.tok_cap + n]);
  }
  red[share][tl] = r;
  __syncthreads();
  for (int step = kShareN / 2; step > 0; step /= 2) {
    if (share < step) red[share][tl] = join(red[share][tl], red[share + step][tl]);
    __syncthreads();
  }
  if (share != 0 || n >= count) return;
  r = red[0][tl];
  if (!p.first) r = join(p.run[n], r);
  if (!p.last) {
    p.run[n] = r;
    return;
  }
  const float lse = r.x + __builtin_logf(r.y);
  p.lse[p.rows[n]] = lse;
  p.loss[p.rows[n]] = lse - p.tlogit[n];
}

// ---------------------------------------------------------------------------------------------- host side
constexpr size_t up256(size_t b) { return (b + 255) / 256 * 256; }
// of a piece's G (or partial sums) and laid-out weight, and of the bf16 terms of x, which leave the rest half at least
constexpr int64_t kPieceBytes = int64_t{896} << 20;

int64_t tiles_of(int64_t m, int64_t n, int tile) { return (m + tile - 1) / tile * ((n + tile - 1) / tile); }

// The tile of a product whose last round is sliced: the large one unless it is more than a quarter empty (the
// small one takes 1.25 times as long for the same work: twice the loads and LDS reads a multiplication).
int tile_sliced(int64_t m, int64_t n) { return 4 * tiles_of(m, n, kBig) <= 1.25 * tiles_of(m, n, kSmall) ? kBig : kSmall; }

// The tile of a product that is not: the one that takes fewer rounds, in units of a large tile's.
int tile_whole(int64_t m, int64_t n) {
  const int64_t big = (tiles_of(m, n, kBig) + kCUs - 1) / kCUs, small = (tiles_of(m, n, kSmall) + 2 * kCUs - 1) / (2 * kCUs);
  return static_cast<double>(big) <= 0.5 * 1.25 * static_cast<double>(small) ? kBig : kSmall;
}

// Most that the slices' sums of a product may take (see pick_slices): two rounds of slices of four steps or more.
int64_t sums_bytes(int64_t tiles, int64_t steps, int tile) {
  const int64_t most = 2 * int64_t{slots_of(tile)};
  if (steps < 8) return 0;
  const int64_t jobs = tiles < slots_of(tile) && tiles * (steps / 4) < most ? tiles * (steps / 4) : most;
  return jobs * tile * tile * 4;
}

struct XentPlan {
  bool copy_w;             // the weight needs a laid-out copy
  int terms, pairs;        // in the logits
  int fine, g_terms, g_pairs;           // fp32 gradients: bf16 terms of x and the weight (else 0: read as in the logits); of G
  int64_t dpad, tok_cap, piece;    // piece: vocabulary rows, a multiple of 256
  int pieces;
  int logits, gx, gw;      // tiles
  size_t off_plan, off_range, off_rows, off_tgt, off_a, off_b, off_c, off_xc, off_xf, off_tally, off_part, off_w, off_wf, off_dl, off_over, off_sums, bytes;
};

XentPlan xent_plan(const XentArgs& a, bool grad) {
  XentPlan n{};
  n.terms = a.io ? 1 : kTerms;
  n.pairs = a.io ? 1 : 3;
  n.fine = a.io || !grad ? 0 : kFineTerms;
  n.g_terms = !a.io ? kFineTerms : a.tokens <= kFewTokens || a.fine_g ? 2 : 1;
  n.g_pairs = a.io ? n.g_terms : kMostPairs;
  n.dpad = (a.dim + 63) / 64 * 64;
  n.tok_cap = (a.tokens + kTokTile - 1) / kTokTile * kTokTile;
  n.copy_w = !a.io || a.dim % 64 != 0;
  const int64_t vpad = (a.vocab + 255) / 256 * 256;
  int64_t row = 1;   // bytes a vocabulary row of a piece costs
  if (grad) row += n.tok_cap * 2 * n.g_terms;
  else row += n.tok_cap / 8;   // a partial of 8 bytes per 64 rows
  if (n.copy_w) row += n.dpad * 2 * (n.terms + n.fine);
  const int64_t fine_x = (n.tok_cap + kSkew) * n.dpad * 2 * n.fine;
  n.piece = (fine_x < kPieceBytes / 2 ? kPieceBytes - fine_x : kPieceBytes / 2) / row / 256 * 256;
  if (n.piece < 256) n.piece = 256;
  if (n.piece > vpad) n.piece = vpad;
  n.pieces = static_cast<int>((a.vocab + n.piece - 1) / n.piece);
  n.piece = ((a.vocab + n.pieces - 1) / n.pieces + 255) / 256 * 256;   // pieces of equal size
  n.pieces = static_cast<int>((a.vocab + n.piece - 1) / n.piece);
  const int64_t tok = a.tokens > 0 ? a.tokens : 1, rows = n.piece < a.vocab ? n.piece : a.vocab;
  n.logits = tile_whole(rows, tok);
  n.gx = tile_sliced(a.dim, tok);
  n.gw = tile_sliced(a.dim, rows);
  size_t at = 0;
  auto take = [&](size_t b) { const size_t o = at; at += up256(b); return o; };
  const size_t tc = static_cast<size_t>(n.tok_cap);
  n.off_plan = take(kPlanInts * 4);
  n.off_range = take(a.io ? 0 : size_t{kRangeBlocks} * 3 * 4);
  n.off_rows = take(tc * 4);
  n.off_tgt = take(tc * 4);
  n.off_a = take(tc * 4);
  n.off_b = take(tc * (grad ? 4 : 8));
  n.off_c = take(tc * 4);
  n.off_xc = take((tc + kSkew) * n.dpad * 2 * n.terms);
  n.off_xf = take(static_cast<size_t>(fine_x));
  n.off_tally = take((tc + kGroup - 1) / kGroup * 4);
  n.off_w = take(n.copy_w ? size_t(n.piece + kSkew) * n.dpad * 2 * n.terms : 0);
  n.off_wf = take(size_t(n.piece + kSkew) * n.dpad * 2 * n.fine);
  n.off_part = take(grad ? 0 : size_t(n.piece) / 64 * tc * 8);
  n.off_dl = take(grad ? (tc + kSkew) * n.piece * 2 * n.g_terms : 0);
  n.off_over = take(grad && n.pieces > 1 ? tc * n.dpad * 4 : 0);
  const int64_t pairs = n.g_pairs;
  const int64_t sx = sums_bytes(tiles_of(a.dim, tok, n.gx), (rows + kBK - 1) / kBK * pairs, n.gx);
  const int64_t sw = sums_bytes(tiles_of(a.dim, rows, n.gw), (tok + kBK - 1) / kBK * pairs, n.gw);
  n.off_sums = take(grad ? static_cast<size_t>(sx > sw ? sx : sw) : 0);   // dx and dW in turn
  n.bytes = at;
  return n;
}

template <int BM, int WM, int WN, bool ATR, bool BTR, bool FP32, int EPI>
hipError_t product(const ProductParams& p, hipStream_t stream) {
  constexpr int kSlots = slots_of(BM);
  const int64_t tiles = tiles_of(p.M, p.N, BM);
  if (tiles == 0) return hipSuccess;
  const int64_t want = EPI == kGradX || EPI == kGradW ? kSlots : (tiles + 7) / 8 * 8;
  product_kernel<BM, BM, WM, WN, ATR, BTR, FP32, EPI>
      <<<dim3(static_cast<unsigned>(want < kSlots ? want : kSlots)), WM * WN * 64, 0, stream>>>(p);
  if constexpr (EPI == kGradX || EPI == kGradW) {
    const int64_t sliced = tiles < kSlots ? tiles : kSlots;
    sum_kernel<BM, BM, EPI><<<dim3(static_cast<unsigned>(sliced * kShares)), 256, 0, stream>>>(p, kSlots);
  }
  return hipGetLastError();
}

template <bool ATR, bool BTR, bool FP32, int EPI>
hipError_t product_any(int tile, const ProductParams& p, hipStream_t stream) {
  return tile == kBig ? product<kBig, 2, 4, ATR, BTR, FP32, EPI>(p, stream)
                      : product<kSmall, 2, 2, ATR, BTR, FP32, EPI>(p, stream);
}

template <typename T> hipError_t prep(const XentArgs& a, const XentPlan& n, unsigned char* ws, bool grad, hipStream_t stream) {
  PrepParams p{};
  p.targets = a.targets; p.id_bytes = a.id_bytes; p.ignore = a.ignore; p.vocab = a.vocab; p.tokens = a.tokens;
  p.dim = a.dim; p.dpad = n.dpad; p.tok_cap = n.tok_cap; p.x = a.x;
  p.xc = reinterpret_cast<uint16_t*>(ws + n.off_xc);
  p.plan = reinterpret_cast<int*>(ws + n.off_plan);
  p.rows = reinterpret_cast<int*>(ws + n.off_rows);
  p.tgt = reinterpret_cast<int*>(ws + n.off_tgt);
  // about a thousand workgroups, of at most 64 tokens
  const int64_t per = (a.tokens + 1023) / 1024;
  p.per = static_cast<int>(per < 1 ? 1 : per > 64 ? 64 : per);
  p.work_blocks = static_cast<int>((a.tokens + p.per - 1) / p.per);
  if (grad) {
    const int64_t rows = n.piece < a.vocab ? n.piece : a.vocab, last = a.vocab - (n.pieces - 1) * n.piece;
    p.pairs = n.g_pairs;
    p.steps_x = static_cast<int>((rows + kBK - 1) / kBK) * p.pairs;
    p.tile_x = n.gx; p.tile_w = n.gw;
    p.tiles_mx = static_cast<int>((a.dim + n.gx - 1) / n.gx);
    p.tiles_w = static_cast<int>(tiles_of(a.dim, rows, n.gw));
    p.tiles_w_last = static_cast<int>(tiles_of(a.dim, last, n.gw));
    if (n.fine != 0) p.xf = reinterpret_cast<uint16_t*>(ws + n.off_xf);
    p.lse = a.lse_in; p.dloss = a.dloss; p.dlse = a.dlse; p.dx = a.dx;
    p.c_lse = reinterpret_cast<float*>(ws + n.off_a);
    p.c_gl = reinterpret_cast<float*>(ws + n.off_b);
    p.c_g = reinterpret_cast<float*>(ws + n.off_c);
  } else {
    p.loss = a.loss; p.lse_out = a.lse;
  }
  // a few thousand tokens are counted again by every workgroup; more are counted group by group first
  if (a.tokens > 2 * kGroup) {
    p.tally = reinterpret_cast<int*>(ws + n.off_tally);
    tally_kernel<<<dim3(static_cast<unsigned>((a.tokens + kGroup - 1) / kGroup)), 256, 0, stream>>>(p);
  }
  if constexpr (sizeof(T) == 4) {
    RangeParams r{p, static_cast<const float*>(a.weight), a.vocab * a.dim, reinterpret_cast<uint32_t*>(ws + n.off_range)};
    range_kernel<<<dim3(kRangeBlocks), 256, 0, stream>>>(r);
    p.range = r.part;
  }
  prep_kernel<T><<<dim3(static_cast<unsigned>(p.work_blocks + kPadBlocks)), 256, 0, stream>>>(p);
  return hipGetLastError();
}

// a matrix in panels of 64 columns, [panel][rows][64], one or two of them
Operand panels(const void* p, int64_t rows, int64_t cols, bool k_strided) {
  Operand o{};
  o.p = static_cast<const unsigned char*>(p);
  o.row = kRow;
  o.plane = (rows + kSkew) * kRow;
  o.step = k_strided ? kBK * int64_t{kRow} : o.plane;
  o.term = o.plane * (cols / 64);
  o.rows = static_cast<int>(rows);
  o.planes = static_cast<int>(cols / 64);
  return o;
}

// the piece's rows of the weight, laid out first where they cannot be read in place (fp32 with dx: for both products)
template <typename T>
hipError_t lay_out_weight(const XentArgs& a, const XentPlan& n, unsigned char* ws, int64_t v0, int64_t rows,
                          hipStream_t stream) {
  if (!n.copy_w) return hipSuccess;
  weight_kernel<T><<<dim3(static_cast<unsigned>((rows + 31) / 32)), 256, 0, stream>>>(
      static_cast<const T*>(a.weight) + v0 * a.dim, reinterpret_cast<uint16_t*>(ws + n.off_w),
      n.fine != 0 && a.dx != nullptr ? reinterpret_cast<uint16_t*>(ws + n.off_wf) : nullptr, rows, a.dim, n.dpad,
      reinterpret_cast<const int*>(ws + n.off_plan));
  return hipGetLastError();
}

// the term products (of A, of B), smallest first: one term of either; two of B alone; two of either; three of either
void set_pairs(ProductParams* p, int pairs) {
  constexpr int kOf[4][kMostPairs][2] = {{{0, 0}}, {{0, 1}, {0, 0}}, {{1, 0}, {0, 1}, {0, 0}},
                                         {{2, 0}, {1, 1}, {0, 2}, {1, 0}, {0, 1}, {0, 0}}};
  p->pairs = pairs;
  for (int i = 0; i < pairs; ++i) {
    p->ta[i] = kOf[pairs < 4 ? pairs - 1 : 3][i][0];
    p->tb[i] = kOf[pairs < 4 ? pairs - 1 : 3][i][1];
  }
}

Operand weight_operand(const XentArgs& a, const XentPlan& n, unsigned char* ws, int64_t v0, int64_t rows, bool k_strided) {
  if (n.copy_w) return panels(ws + (n.fine != 0 && k_strided ? n.off_wf : n.off_w), rows, n.dpad, k_strided);
  Operand o{};
  o.p = static_cast<const unsigned char*>(a.weight) + v0 * a.dim * 2;
  o.row = a.dim * 2;
  o.step = k_strided ? kBK * a.dim * 2 : kRow;
  o.plane = kRow;
  o.rows = static_cast<int>(rows);
  o.planes = static_cast<int>(a.dim / 64);
  return o;
}

template <typename T> hipError_t xent_fwd_t(const XentArgs& a, hipStream_t stream) {
  constexpr bool kFp32 = sizeof(T) == 4;
  const XentPlan n = xent_plan(a, false);
  unsigned char* ws = static_cast<unsigned char*>(a.workspace);
  hipError_t e = prep<T>(a, n, ws, false, stream);
  for (int k = 0; k < n.pieces && e == hipSuccess; ++k) {
    const int64_t v0 = k * n.piece, rows = v0 + n.piece < a.vocab ? n.piece : a.vocab - v0;
    ProductParams p{};
    e = lay_out_weight<T>(a, n, ws, v0, rows, stream);
    if (e != hipSuccess) return e;
    p.A = weight_operand(a, n, ws, v0, rows, false);
    p.B = panels(ws + n.off_xc, n.tok_cap, n.dpad, false);
    p.M = static_cast<int>(rows); p.N = static_cast<int>(n.tok_cap); p.K = static_cast<int>(n.dpad);
    p.n_is_tokens = 1;
    set_pairs(&p, n.pairs);
    p.scale_a = kScaleW; p.scale_b = kScaleX;
    p.plan = reinterpret_cast<int*>(ws + n.off_plan);
    p.tgt = reinterpret_cast<int*>(ws + n.off_tgt);
    p.v0 = static_cast<int>(v0);
    p.part = reinterpret_cast<float2*>(ws + n.off_part);
    p.tok_cap = n.tok_cap;
    p.tlogit = reinterpret_cast<float*>(ws + n.off_a);
    e = product_any<false, false, kFp32, kLogits>(n.logits, p, stream);
    if (e != hipSuccess) return e;
    JoinParams j{};
    j.part = p.part; j.tiles = static_cast<int>((rows + n.logits - 1) / n.logits * 2); j.first = k == 0; j.last = k + 1 == n.pieces;
    j.tok_cap = n.tok_cap; j.plan = p.plan; j.rows = reinterpret_cast<int*>(ws + n.off_rows);
    j.run = reinterpret_cast<float2*>(ws + n.off_b); j.tlogit = p.tlogit; j.loss = a.loss; j.lse = a.lse;
    if (a.tokens <= 512) join_kernel<2><<<dim3(static_cast<unsigned>((a.tokens + 1) / 2)), 256, 0, stream>>>(j);
    else join_kernel<16><<<dim3(static_cast<unsigned>((a.tokens + 15) / 16)), 256, 0, stream>>>(j);
    e = hipGetLastError();
  }
  return e;
}

template <typename T> hipError_t xent_bwd_t(const XentArgs& a, hipStream_t stream) {
  constexpr bool kFp32 = sizeof(T) == 4;
  const XentPlan n = xent_plan(a, true);
  unsigned char* ws = static_cast<unsigned char*>(a.workspace);
  hipError_t e = prep<T>(a, n, ws, true, stream);
  for (int k = 0; k < n.pieces && e == hipSuccess; ++k) {
    const int64_t v0 = k * n.piece, rows = v0 + n.piece < a.vocab ? n.piece : a.vocab - v0;
    const int64_t rpad = (rows + 255) / 256 * 256;
    ProductParams p{};
    e = lay_out_weight<T>(a, n, ws, v0, rows, stream);
    if (e != hipSuccess) return e;
    uint16_t* const dl = reinterpret_cast<uint16_t*>(ws + n.off_dl);
    p.plan = reinterpret_cast<int*>(ws + n.off_plan);
    // G of the piece
    p.A = weight_operand(a, n, ws, v0, rows, false);
    p.B = panels(ws + n.off_xc, n.tok_cap, n.dpad, false);
    p.M = static_cast<int>(rows); p.N = static_cast<int>(n.tok_cap); p.K = static_cast<int>(n.dpad);
    p.n_is_tokens = 1;
    set_pairs(&p, n.pairs);
    p.scale_a = kScaleW; p.scale_b = kScaleX;
    p.g_terms = n.g_terms;
    p.tgt = reinterpret_cast<int*>(ws + n.off_tgt);
    p.v0 = static_cast<int>(v0);
    p.lse = reinterpret_cast<float*>(ws + n.off_a);
    p.gl = reinterpret_cast<float*>(ws + n.off_b);
    p.g = reinterpret_cast<float*>(ws + n.off_c);
    p.dl = dl; p.pdl = (n.tok_cap + kSkew) * rpad;
    p.tok_cap = n.tok_cap;
    e = product_any<false, false, kFp32, kGradLogits>(n.logits, p, stream);
    if (e != hipSuccess) return e;
    if (a.dx != nullptr) {     // dx += G W: m = width, n = token, k = vocabulary
      ProductParams q{};
      q.plan = p.plan;
      q.A = weight_operand(a, n, ws, v0, rows, true);
      q.B = panels(dl, n.tok_cap, rpad, false);
      q.M = static_cast<int>(a.dim); q.N = static_cast<int>(n.tok_cap); q.K = static_cast<int>((rows + 63) / 64 * 64);
      q.n_is_tokens = 1;
      set_pairs(&q, n.g_pairs);
      q.scale_a = kScaleW; q.scale_b = kScaleG;
      q.slices_at = kSlicesX;
      q.first = k == 0; q.last = k + 1 == n.pieces;
      q.rows = reinterpret_cast<int*>(ws + n.off_rows);
      q.out = a.dx; q.dim = a.dim; q.out_f32 = kFp32;
      q.sums = reinterpret_cast<float*>(ws + n.off_sums);
      if (n.pieces > 1) {
        q.over = reinterpret_cast<float*>(ws + n.off_over);
        q.ld_over = n.dpad;
      }
      e = product_any<true, false, kFp32, kGradX>(n.gx, q, stream);
      if (e != hipSuccess) return e;
    }
    if (a.dweight != nullptr) {   // dW of the piece = G^T x: m = width, n = vocabulary row, k = token
      ProductParams q{};
      const size_t gs = a.grad_io ? sizeof(T) : 4;
      q.plan = p.plan;
      q.A = panels(ws + (n.fine != 0 ? n.off_xf : n.off_xc), n.tok_cap, n.dpad, true);
      q.B = panels(dl, n.tok_cap, rpad, true);
      q.M = static_cast<int>(a.dim); q.N = static_cast<int>(rows);
      q.k_is_tokens = 1;
      q.out = static_cast<unsigned char*>(a.dweight) + v0 * a.dim * gs;
      q.dim = a.dim; q.out_f32 = gs == 4; q.accumulate = a.accumulate;
      set_pairs(&q, n.g_pairs);
      q.scale_a = kScaleX; q.scale_b = kScaleG;
      q.slices_at = k + 1 == n.pieces ? kSlicesLastW : kSlicesW;
      q.sums = reinterpret_cast<float*>(ws + n.off_sums);
      e = product_any<true, true, kFp32, kGradW>(n.gw, q, stream);
    }
  }
  return e;
}

}  // namespace

size_t xent_workspace_bytes(const XentArgs& a, bool grad) { return xent_plan(a, grad).bytes; }

hipError_t xent_fwd_launch(const XentArgs& a, hipStream_t stream) {
  if (a.tokens == 0) return hipSuccess;
  return a.io ? xent_fwd_t<uint16_t>(a, stream) : xent_fwd_t<float>(a, stream);
}

hipError_t xent_bwd_launch(const XentArgs& a, hipStream_t stream) {
  return a.io ? xent_bwd_t<uint16_t>(a, stream) : xent_bwd_t<float>(a, stream);
}

}  // namespace mssm
