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
// the piece goes to the workspace in bf16, and two more products take it to dx (summed over the pieces in
// fp32) and to the piece's rows of dW.
//
// One tiled product serves all four: out[m, n] = sum_k A[m, k] B[n, k] with m on the weight's side (so that
// a lane's four accumulators are neighbours along the vocabulary or the width, and a token is one column).
// An operand is read K-contiguous (rows of k) or K-strided (k is the row: G^T, x^T, W^T), the latter through
// transposing LDS reads.  Tiles go from global memory straight into LDS.
//
// bf16 inputs enter the matrix cores as they are; products are summed in fp32.  G is rounded to bf16 (the
// gradients' own type) once.  fp32 inputs are split into three bf16 terms, v = hi + mid + lo with 24
// significant bits in all, and a product is the six term products that matter,
//   hi hi + hi mid + mid hi + hi lo + lo hi + mid mid
// (what is left out is below 2^-24 of the product), summed in fp32 smallest first: six bf16 products at the
// matrix cores' bf16 rate beat one product at their fp32 rate, a sixteenth of it.
#include <type_traits>

#include "device_util.h"
#include "internal.h"

namespace mssm {
namespace {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef short i16x4 __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) i16x4 lds_i16x4;

constexpr float kLog2e = 1.44269504088896340736f;
constexpr int kBK = 64;                 // k per step
constexpr int kRow = kBK * 2;           // bytes of an LDS row
constexpr int kPlane = 64 * kRow;       // LDS tiles are planes of 64 rows x 128 bytes
constexpr int kTokTile = 256;           // compacted tokens are padded to this
constexpr int kTerms = 3;               // bf16 terms of an fp32 value
constexpr int kPairs = 6;               // term products kept
__device__ __constant__ const int kPairA[kPairs] = {2, 0, 1, 1, 0, 0};
__device__ __constant__ const int kPairB[kPairs] = {0, 2, 1, 0, 1, 0};

// v = t[0] + t[1] + t[2] exactly: each term is the nearest bf16 of what is left (8 + 8 + 8 significant bits),
// |t[1]| <= 2^-8 |v|, |t[2]| <= 2^-16 |v|.  A finite v that would round to infinity is cut off instead;
// infinities and NaN stay what they are.
__device__ __forceinline__ void split3(float v, uint16_t (&t)[kTerms]) {
  constexpr uint32_t kExp = 0x7f800000u;
  const uint32_t u = __float_as_uint(v);
  t[0] = narrow<uint16_t>(v);
  t[1] = t[2] = 0;
  if ((u & kExp) == kExp) return;
  if ((t[0] & 0x7fffu) == 0x7f80u) t[0] = static_cast<uint16_t>(u >> 16);
  const float r = v - widen(t[0]);
  t[1] = narrow<uint16_t>(r);
  t[2] = narrow<uint16_t>(r - widen(t[1]));
}

__device__ __forceinline__ uint32_t lds_addr(const void* p) {
  return static_cast<uint32_t>(reinterpret_cast<uintptr_t>(p));   // low half of a flat LDS address
}
// lane l's 16 bytes go from global memory to LDS offset lds + 16 l (lds is wave-uniform)
__device__ __forceinline__ void dma16(const void* g, uint32_t lds) {
  asm volatile("s_mov_b32 m0, %1\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %0, off"
               :: "v"(g), "s"(__builtin_amdgcn_readfirstlane(lds)) : "memory", "m0");
}

// ------------------------------------------------------------------------------------------------ product
struct ProductParams {
  const uint16_t* A;
  const uint16_t* B;
  int64_t lda, ldb;        // elements between rows
  int64_t pa, pb;          // elements between an operand's bf16 terms (split operands)
  int M, N;                // rows of the output on either side (columns past them are not stored)
  int rows_a, cols_a;      // what may be read of A: rows, and (K-strided) columns
  int rows_b, cols_b;
  int K;                   // multiple of 64; with k_is_tokens: the compacted count, rounded up, instead
  int tiles_m, tiles_n;
  int k_is_tokens, n_is_tokens;
  const int* count;        // compacted tokens
  // epilogues
  int v0, vocab;           // first vocabulary row of this piece
  const int* tgt;          // compacted targets
  float2* part;            // [2 * tiles_m][tok_cap]: maximum, sum of exponentials
  int64_t tok_cap;
  float* tlogit;           // target's logit
  const float* lse;        // compacted
  const float* gl;         // dloss + dlse
  const float* g;          // dloss
  uint16_t* dl;            // [tok][piece], one or three terms
  int64_t ldl, pdl;
  float* dxacc;            // [tok_cap][ldx], sums over pieces
  int64_t ldx;
  int first, last;         // piece
  const int* rows;         // compacted -> token
  void* out;               // dx or dW
  int64_t dim;
  int out_f32, accumulate, vec;
};

enum { kLogits = 0, kGradLogits = 1, kGradX = 2, kGradW = 3 };

template <int BM, int BN, int WM, int WN, bool ATR, bool BTR, bool SPLIT, int EPI>
__global__ __launch_bounds__(WM * WN * 64) void product_kernel(ProductParams p) {
  constexpr int kWavesN = WM * WN;
  constexpr int TM = BM / WM / 16, TN = BN / WN / 16;      // 16 x 16 tiles of a wave
  constexpr int LA = BM / 8 / kWavesN, LB = BN / 8 / kWavesN;   // 1 KB loads of a wave per step
  static_assert(LA * 8 * kWavesN == BM && LB * 8 * kWavesN == BN, "loads split evenly over the waves");
  __shared__ __attribute__((aligned(16))) unsigned char as[2][BM * kRow];
  __shared__ __attribute__((aligned(16))) unsigned char bs[2][BN * kRow];

  const int lane = threadIdx.x % kLanes;
  const int w = __builtin_amdgcn_readfirstlane(threadIdx.x / kLanes);
  const int wm = w / WN, wn = w % WN;
  const int count = *p.count;

  // workgroup -> tile.  Workgroups b, b + 8, ... share an XCD and its L2: each XCD takes a contiguous range
  // of an order that walks bands of 8 n-tiles, m outer, so that what runs on it at one time is a block of
  // few m-tiles by 8 n-tiles.
  const int total = p.tiles_m * p.tiles_n;
  const int per = (total + 7) / 8;
  const int tile = (blockIdx.x % 8) * per + blockIdx.x / 8;
  if (tile >= total || blockIdx.x / 8 >= per) return;
  const int band = tile / (p.tiles_m * 8);
  const int left = p.tiles_n - band * 8, wide = left < 8 ? left : 8;
  const int in_band = tile - band * p.tiles_m * 8;
  const int m0 = in_band / wide * BM, n0 = (band * 8 + in_band % wide) * BN;
  if (p.n_is_tokens && n0 >= count) return;
  const int steps1 = (p.k_is_tokens ? (count + kBK - 1) / kBK * kBK : p.K) / kBK;
  const int steps = SPLIT ? steps1 * kPairs : steps1;

  // this lane's part of the loads: row lane / 8 of an 8-row group, 16-byte chunk lane % 8 as stored; the
  // chunk it holds is xor-ed with the row, so that both kinds of reads below are free of bank conflicts
  const int lrow = lane / 8;
  auto src = [&](const uint16_t* base, int64_t ld, bool tr, int group, int o0, int rows, int cols) {
    if (!tr) {     // rows of the tile are output rows, 64 k each
      const int r = group * 8 + lrow;
      const int c = (lane % 8) ^ (r & 7);
      const int row = o0 + r < rows ? o0 + r : rows - 1;
      return base + static_cast<int64_t>(row) * ld + c * 8;
    }
    const int r = group % 8 * 8 + lrow;               // k within the step
    const int c = (lane % 8) ^ (r & 7);
    const int col = o0 + group / 8 * 64 + c * 8;
    return base + static_cast<int64_t>(r) * ld + (col < cols ? col : 0);
  };
  const uint16_t* ga[LA];
  const uint16_t* gb[LB];
#pragma unroll
  for (int i = 0; i < LA; ++i) ga[i] = src(p.A, p.lda, ATR, i * kWavesN + w, m0, p.rows_a, p.cols_a);
#pragma unroll
  for (int i = 0; i < LB; ++i) gb[i] = src(p.B, p.ldb, BTR, i * kWavesN + w, n0, p.rows_b, p.cols_b);
  const uint32_t as_a = lds_addr(&as[0][0]), bs_a = lds_addr(&bs[0][0]);

  auto issue = [&](int step, int buf) {
    int seg = 0, k = step;
    if constexpr (SPLIT) {
      seg = step / steps1;
      k = step - seg * steps1;
    }
    const int64_t oa = (SPLIT ? kPairA[seg] * p.pa : 0) + static_cast<int64_t>(k) * kBK * (ATR ? p.lda : 1);
    const int64_t ob = (SPLIT ? kPairB[seg] * p.pb : 0) + static_cast<int64_t>(k) * kBK * (BTR ? p.ldb : 1);
#pragma unroll
    for (int i = 0; i < LA; ++i) {
      const uint16_t* a = ga[i] + oa;
      if constexpr (ATR) {   // k rows past the matrix (the last step of a piece): its last row again
        const int r = k * kBK + (i * kWavesN + w) % 8 * 8 + lrow;
        if (r >= p.rows_a) a -= static_cast<int64_t>(r - (p.rows_a - 1)) * p.lda;
      }
      dma16(a, as_a + buf * BM * kRow + (i * kWavesN + w) * 1024);
    }
#pragma unroll
    for (int i = 0; i < LB; ++i) dma16(gb[i] + ob, bs_a + buf * BN * kRow + (i * kWavesN + w) * 1024);
  };

  auto frag = [&](const unsigned char* base, bool tr, int t16, int ks) -> bf16x8 {
    if (!tr) {
      const int r = t16 * 16 + lane % 16;
      const int c = ks * 4 + lane / 16;
      return *reinterpret_cast<const bf16x8*>(base + r * kRow + ((c ^ (r & 7)) << 4));
    }
    // in each 16-lane group, lane j receives element j of the four 16-element rows its lanes point at
    const int j = lane % 16;
    const int col = t16 * 16 + j % 4 * 4;
    const unsigned char* plane = base + col / 64 * kPlane;
    u32x4_t f;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int r = ks * 32 + lane / 16 * 8 + h * 4 + j / 4;
      const unsigned char* at = plane + r * kRow + (((col % 64 / 8) ^ (r & 7)) << 4) + col % 8 * 2;
      const u32x2_t v = __builtin_bit_cast(
          u32x2_t, __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_i16x4*)(const_cast<unsigned char*>(at))));
      f[2 * h] = v[0];
      f[2 * h + 1] = v[1];
    }
    return __builtin_bit_cast(bf16x8, f);
  };

  f32x4_t acc[TM][TN];
#pragma unroll
  for (int i = 0; i < TM; ++i)
#pragma unroll
    for (int j = 0; j < TN; ++j) acc[i][j] = f32x4_t{0.f, 0.f, 0.f, 0.f};

  if (steps > 0) issue(0, 0);
  for (int s = 0; s < steps; ++s) {
    asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)" ::: "memory");
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
    if (s + 1 < steps) issue(s + 1, (s + 1) & 1);
    const unsigned char* a = as[s & 1];
    const unsigned char* b = bs[s & 1];
#pragma unroll
    for (int ks = 0; ks < 2; ++ks) {
      bf16x8 fa[TM], fb[TN];
#pragma unroll
      for (int i = 0; i < TM; ++i) fa[i] = frag(a, ATR, wm * TM + i, ks);
#pragma unroll
      for (int j = 0; j < TN; ++j) fb[j] = frag(b, BTR, wn * TN + j, ks);
#pragma unroll
      for (int i = 0; i < TM; ++i)
#pragma unroll
        for (int j = 0; j < TN; ++j) acc[i][j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(fa[i], fb[j], acc[i][j], 0, 0, 0);
    }
  }

  // accumulator e of tile (i, j): row m = m0 + (wm TM + i) 16 + 4 (lane / 16) + e, column n = n0 + (wn TN + j) 16 + lane % 16
  const int mrow = m0 + wm * TM * 16 + lane / 16 * 4;
  const int ncol = n0 + wn * TN * 16 + lane % 16;
  if constexpr (EPI == kLogits) {
#pragma unroll
    for (int j = 0; j < TN; ++j) {
      const int n = ncol + j * 16;
      const int y = p.tgt[n] - p.v0;   // padded tokens have target -1
      float mx = -__builtin_inff();
#pragma unroll
      for (int i = 0; i < TM; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int m = mrow + i * 16 + e;
          if (m < p.M) mx = __builtin_fmaxf(mx, acc[i][j][e]);
          if (m == y && n < count) p.tlogit[n] = acc[i][j][e];
        }
      mx = __builtin_fmaxf(mx, __shfl_xor(mx, 16, 64));
      mx = __builtin_fmaxf(mx, __shfl_xor(mx, 32, 64));
      const float ref = mx == -__builtin_inff() ? 0.f : mx;
      float s = 0.f;
#pragma unroll
      for (int i = 0; i < TM; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int m = mrow + i * 16 + e;
          if (m < p.M) s += __builtin_amdgcn_exp2f((acc[i][j][e] - ref) * kLog2e);
        }
      s += __shfl_xor(s, 16, 64);
      s += __shfl_xor(s, 32, 64);
      if (lane < 16) p.part[(static_cast<int64_t>(m0 / BM) * WM + wm) * p.tok_cap + n] = float2{mx, s};
    }
  } else if constexpr (EPI == kGradLogits) {
#pragma unroll
    for (int j = 0; j < TN; ++j) {
      const int n = ncol + j * 16;
      const bool on = n < count;
      const int y = p.tgt[n] - p.v0;
      const float lse = p.lse[n], gl = p.gl[n], g = p.g[n];
#pragma unroll
      for (int i = 0; i < TM; ++i) {
        float d[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int m = mrow + i * 16 + e;
          const float v = __builtin_amdgcn_exp2f((acc[i][j][e] - lse) * kLog2e) * gl - (m == y ? g : 0.f);
          d[e] = on && m < p.M ? v : 0.f;
        }
        uint16_t* const to = p.dl + n * p.ldl + mrow + i * 16;
        if constexpr (SPLIT) {
          uint16_t t[4][kTerms];
#pragma unroll
          for (int e = 0; e < 4; ++e) split3(d[e], t[e]);
#pragma unroll
          for (int k = 0; k < kTerms; ++k)
            *reinterpret_cast<u32x2_t*>(to + k * p.pdl) =
                u32x2_t{t[0][k] | static_cast<uint32_t>(t[1][k]) << 16, t[2][k] | static_cast<uint32_t>(t[3][k]) << 16};
        } else {
          *reinterpret_cast<u32x2_t*>(to) = u32x2_t{pack_bf16(d[0], d[1]), pack_bf16(d[2], d[3])};
        }
      }
    }
  } else {
#pragma unroll
    for (int j = 0; j < TN; ++j) {
      const int n = ncol + j * 16;
      if (EPI == kGradX ? n >= count : n >= p.N) continue;
      const int64_t row = EPI == kGradX ? static_cast<int64_t>(p.rows[n]) : n;
#pragma unroll
      for (int i = 0; i < TM; ++i) {
        const int m = mrow + i * 16;
        if (m >= p.M) continue;
        float v[4] = {acc[i][j][0], acc[i][j][1], acc[i][j][2], acc[i][j][3]};
        if constexpr (EPI == kGradX) {
          if (!p.first) {
            float o[4];
            load_row<4>(p.dxacc + n * p.ldx + m, o);
#pragma unroll
            for (int e = 0; e < 4; ++e) v[e] += o[e];
          }
          if (!p.last) {
            store_row<4>(p.dxacc + n * p.ldx + m, v);
            continue;
          }
        }
        const int64_t at = row * p.dim + m;
        auto put = [&](auto* to) {
          using T = std::remove_reference_t<decltype(*to)>;
          if (p.vec) {   // dim and the pointer allow four elements at once; m is a multiple of 4
            if (EPI == kGradW && p.accumulate) {
              float o[4];
              load_row<4>(to, o);
#pragma unroll
              for (int e = 0; e < 4; ++e) v[e] += o[e];
            }
            store_row<4>(to, v);
          } else {
#pragma unroll
            for (int e = 0; e < 4; ++e)
              if (m + e < p.M) to[e] = narrow<T>(EPI == kGradW && p.accumulate ? v[e] + widen(to[e]) : v[e]);
          }
        };
        if (SPLIT || p.out_f32) put(static_cast<float*>(p.out) + at);
        else put(static_cast<uint16_t*>(p.out) + at);
      }
    }
  }
}

// -------------------------------------------------------------------------------------- around the products
struct PrepParams {
  const void* targets;
  int id_bytes;
  int64_t ignore, vocab, tokens, dim, dpad, tok_cap;
  const void* x;
  uint16_t* xc;            // [terms][tok_cap][dpad]
  int* count;
  int* rows;
  int* tgt;
  int per;                 // tokens of a workgroup
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

constexpr int kPadBlocks = 16;

// Which tokens count, in order, and their x as the products read it: rows padded to a multiple of 64 with
// zeros, fp32 as three bf16 terms; after the last one, zero rows up to the end of its tile of 256.
template <typename T>
__global__ __launch_bounds__(256) void prep_kernel(PrepParams p) {
  __shared__ int red[4];
  const int wave = threadIdx.x / kLanes, lane = threadIdx.x % kLanes;
  const bool pad = static_cast<int>(blockIdx.x) >= p.work_blocks;
  const int64_t lo = pad ? p.tokens : static_cast<int64_t>(blockIdx.x) * p.per;
  auto counts = [&](int64_t t) {
    const int64_t y = id_at(p.targets, p.id_bytes, t);
    return y >= 0 && y < p.vocab && y != p.ignore;
  };
  int before = 0;
  for (int64_t t = threadIdx.x; t < lo; t += 256) before += counts(t);
#pragma unroll
  for (int step = 1; step < kLanes; step *= 2) before += __shfl_xor(before, step, kLanes);
  if (lane == 0) red[wave] = before;
  __syncthreads();
  before = red[0] + red[1] + red[2] + red[3];

  constexpr int kT = sizeof(T) == 4 ? kTerms : 1;
  const int64_t plane = p.tok_cap * p.dpad;
  auto put = [&](int64_t i, int64_t t, bool real) {
    uint16_t* to = p.xc + i * p.dpad;
    const T* from = static_cast<const T*>(p.x) + t * p.dim;
    for (int c = lane; c < p.dpad; c += kLanes) {
      if constexpr (kT == 1) {
        to[c] = real && c < p.dim ? from[c] : 0;
      } else {
        uint16_t s[kTerms] = {0, 0, 0};
        if (real && c < p.dim) split3(from[c], s);
#pragma unroll
        for (int k = 0; k < kTerms; ++k) to[k * plane + c] = s[k];
      }
    }
  };
  if (pad) {
    if (blockIdx.x == static_cast<unsigned>(p.work_blocks) && threadIdx.x == 0) *p.count = before;
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
  // per <= 64: lane l of every wave looks at token lo + l
  const bool mine = lo + lane < hi && counts(lo + lane);
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

// rows of the weight as the products read them (width not a multiple of 64, or fp32)
template <typename T>
__global__ __launch_bounds__(256) void weight_kernel(const T* w, uint16_t* to, int64_t rows, int64_t dim, int64_t dpad) {
  constexpr int kT = sizeof(T) == 4 ? kTerms : 1;
  const int wave = threadIdx.x / kLanes, lane = threadIdx.x % kLanes;
  const int64_t r = static_cast<int64_t>(blockIdx.x) * 4 + wave;
  if (r >= rows) return;
  for (int64_t c = lane; c < dpad; c += kLanes) {
    if constexpr (kT == 1) {
      to[r * dpad + c] = c < dim ? w[r * dim + c] : 0;
    } else {
      uint16_t s[kTerms] = {0, 0, 0};
      if (c < dim) split3(w[r * dim + c], s);
#pragma unroll
      for (int k = 0; k < kTerms; ++k) to[(k * rows + r) * dpad + c] = s[k];
    }
  }
}

// Joins the tiles' (maximum, sum) of a piece with those of the pieces before it; after the last piece, the
// loss.  16 tokens x 16 shares of the tiles a workgroup.
struct JoinParams {
  const float2* part;
  int tiles, first, last;
  int64_t tok_cap;
  const int* count;
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

__global__ __launch_bounds__(256) void join_kernel(JoinParams p) {
  __shared__ float2 red[16][17];
  const int tl = threadIdx.x % 16, share = threadIdx.x / 16;
  const int64_t n = static_cast<int64_t>(blockIdx.x) * 16 + tl;
  const int count = *p.count;
  if (static_cast<int64_t>(blockIdx.x) * 16 >= count) return;
  float2 r = {-__builtin_inff(), 0.f};
  if (n < count)
    for (int k = share; k < p.tiles; k += 16) r = join(r, p.part[k * p.tok_cap + n]);
  red[share][tl] = r;
  __syncthreads();
  if (share != 0 || n >= count) return;
  for (int k = 1; k < 16; ++k) r = join(r, red[k][tl]);
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
constexpr int64_t kPieceBytes = int64_t{512} << 20;   // of G, or of the weight as the products read it

struct XentPlan {
  bool copy_w;             // the weight needs a laid-out copy
  int terms;
  int64_t dpad, tok_cap, piece;    // piece: vocabulary rows, a multiple of 256
  int pieces;
  size_t off_count, off_rows, off_tgt, off_a, off_b, off_c, off_xc, off_part, off_w, off_dl, off_dx, bytes;
};

XentPlan xent_plan(const XentArgs& a, bool grad) {
  XentPlan n{};
  n.terms = a.io ? 1 : kTerms;
  n.dpad = (a.dim + 63) / 64 * 64;
  n.tok_cap = (a.tokens + kTokTile - 1) / kTokTile * kTokTile;
  n.copy_w = !a.io || a.dim % 64 != 0;
  const int64_t vpad = (a.vocab + 255) / 256 * 256;
  int64_t row = 1;   // bytes a vocabulary row of a piece costs
  if (grad) row += n.tok_cap * 2 * n.terms;
  else row += n.tok_cap / 8;   // a partial of 8 bytes per 64 rows
  if (n.copy_w && n.dpad * 2 * n.terms > row) row = n.dpad * 2 * n.terms;
  n.piece = kPieceBytes / row / 256 * 256;
  if (n.piece < 256) n.piece = 256;
  if (n.piece > vpad) n.piece = vpad;
  n.pieces = static_cast<int>((a.vocab + n.piece - 1) / n.piece);
  size_t at = 0;
  auto take = [&](size_t b) { const size_t o = at; at += up256(b); return o; };
  const size_t tc = static_cast<size_t>(n.tok_cap);
  n.off_count = take(4);
  n.off_rows = take(tc * 4);
  n.off_tgt = take(tc * 4);
  n.off_a = take(tc * 4);
  n.off_b = take(tc * (grad ? 4 : 8));
  n.off_c = take(tc * 4);
  n.off_xc = take(tc * n.dpad * 2 * n.terms);
  n.off_w = take(n.copy_w ? size_t(n.piece) * n.dpad * 2 * n.terms : 0);
  n.off_part = take(grad ? 0 : size_t(n.piece) / 64 * tc * 8);
  n.off_dl = take(grad ? tc * n.piece * 2 * n.terms : 0);
  n.off_dx = take(grad && n.pieces > 1 ? tc * n.dpad * 4 : 0);
  n.bytes = at;
  return n;
}

template <int BM, int BN, int WM, int WN, bool ATR, bool BTR, bool SPLIT, int EPI>
hipError_t product(ProductParams p, hipStream_t stream) {
  p.tiles_m = (p.M + BM - 1) / BM;
  p.tiles_n = (p.N + BN - 1) / BN;
  const int total = p.tiles_m * p.tiles_n;
  if (total == 0) return hipSuccess;
  product_kernel<BM, BN, WM, WN, ATR, BTR, SPLIT, EPI>
      <<<dim3(static_cast<unsigned>((total + 7) / 8 * 8)), WM * WN * 64, 0, stream>>>(p);
  return hipGetLastError();
}

template <bool ATR, bool BTR, bool SPLIT, int EPI>
hipError_t product_any(const ProductParams& p, hipStream_t stream) {
  return product<128, 128, 2, 2, ATR, BTR, SPLIT, EPI>(p, stream);
}

template <typename T> hipError_t prep(const XentArgs& a, const XentPlan& n, unsigned char* ws, bool grad, hipStream_t stream) {
  PrepParams p{};
  p.targets = a.targets; p.id_bytes = a.id_bytes; p.ignore = a.ignore; p.vocab = a.vocab; p.tokens = a.tokens;
  p.dim = a.dim; p.dpad = n.dpad; p.tok_cap = n.tok_cap; p.x = a.x;
  p.xc = reinterpret_cast<uint16_t*>(ws + n.off_xc);
  p.count = reinterpret_cast<int*>(ws + n.off_count);
  p.rows = reinterpret_cast<int*>(ws + n.off_rows);
  p.tgt = reinterpret_cast<int*>(ws + n.off_tgt);
  // about a thousand workgroups, of at most 64 tokens
  const int64_t per = (a.tokens + 1023) / 1024;
  p.per = static_cast<int>(per < 1 ? 1 : per > 64 ? 64 : per);
  p.work_blocks = static_cast<int>((a.tokens + p.per - 1) / p.per);
  if (grad) {
    p.lse = a.lse_in; p.dloss = a.dloss; p.dlse = a.dlse; p.dx = a.dx;
    p.c_lse = reinterpret_cast<float*>(ws + n.off_a);
    p.c_gl = reinterpret_cast<float*>(ws + n.off_b);
    p.c_g = reinterpret_cast<float*>(ws + n.off_c);
  } else {
    p.loss = a.loss; p.lse_out = a.lse;
  }
  prep_kernel<T><<<dim3(static_cast<unsigned>(p.work_blocks + kPadBlocks)), 256, 0, stream>>>(p);
  return hipGetLastError();
}

// the piece's rows of the weight as an operand
template <typename T>
hipError_t weight_operand(const XentArgs& a, const XentPlan& n, unsigned char* ws, int64_t v0, int64_t rows,
                          ProductParams* p, hipStream_t stream) {
  p->A = static_cast<const uint16_t*>(a.weight) + v0 * a.dim;
  p->lda = n.dpad;
  p->pa = rows * n.dpad;
  p->rows_a = static_cast<int>(rows);
  p->cols_a = static_cast<int>(n.dpad);
  if (!n.copy_w) return hipSuccess;
  uint16_t* to = reinterpret_cast<uint16_t*>(ws + n.off_w);
  weight_kernel<T><<<dim3(static_cast<unsigned>((rows + 3) / 4)), 256, 0, stream>>>(
      static_cast<const T*>(a.weight) + v0 * a.dim, to, rows, a.dim, n.dpad);
  p->A = to;
  return hipGetLastError();
}

template <typename T> hipError_t xent_fwd_t(const XentArgs& a, hipStream_t stream) {
  constexpr bool kSplit = sizeof(T) == 4;
  const XentPlan n = xent_plan(a, false);
  unsigned char* ws = static_cast<unsigned char*>(a.workspace);
  hipError_t e = prep<T>(a, n, ws, false, stream);
  for (int k = 0; k < n.pieces && e == hipSuccess; ++k) {
    const int64_t v0 = k * n.piece, rows = v0 + n.piece < a.vocab ? n.piece : a.vocab - v0;
    ProductParams p{};
    e = weight_operand<T>(a, n, ws, v0, rows, &p, stream);
    if (e != hipSuccess) return e;
    p.B = reinterpret_cast<uint16_t*>(ws + n.off_xc);
    p.ldb = n.dpad; p.pb = n.tok_cap * n.dpad;
    p.rows_b = static_cast<int>(n.tok_cap); p.cols_b = static_cast<int>(n.dpad);
    p.M = static_cast<int>(rows); p.N = static_cast<int>(n.tok_cap); p.K = static_cast<int>(n.dpad);
    p.n_is_tokens = 1;
    p.count = reinterpret_cast<int*>(ws + n.off_count);
    p.tgt = reinterpret_cast<int*>(ws + n.off_tgt);
    p.v0 = static_cast<int>(v0);
    p.part = reinterpret_cast<float2*>(ws + n.off_part);
    p.tok_cap = n.tok_cap;
    p.tlogit = reinterpret_cast<float*>(ws + n.off_a);
    e = product_any<false, false, kSplit, kLogits>(p, stream);
    if (e != hipSuccess) return e;
    JoinParams j{};
    j.part = p.part; j.tiles = static_cast<int>((rows + 127) / 128 * 2); j.first = k == 0; j.last = k + 1 == n.pieces;
    j.tok_cap = n.tok_cap; j.count = p.count; j.rows = reinterpret_cast<int*>(ws + n.off_rows);
    j.run = reinterpret_cast<float2*>(ws + n.off_b); j.tlogit = p.tlogit; j.loss = a.loss; j.lse = a.lse;
    join_kernel<<<dim3(static_cast<unsigned>((a.tokens + 15) / 16)), 256, 0, stream>>>(j);
    e = hipGetLastError();
  }
  return e;
}

template <typename T> hipError_t xent_bwd_t(const XentArgs& a, hipStream_t stream) {
  constexpr bool kSplit = sizeof(T) == 4;
  const XentPlan n = xent_plan(a, true);
  unsigned char* ws = static_cast<unsigned char*>(a.workspace);
  hipError_t e = prep<T>(a, n, ws, true, stream);
  for (int k = 0; k < n.pieces && e == hipSuccess; ++k) {
    const int64_t v0 = k * n.piece, rows = v0 + n.piece < a.vocab ? n.piece : a.vocab - v0;
    const int64_t rpad = (rows + 255) / 256 * 256;
    ProductParams p{};
    e = weight_operand<T>(a, n, ws, v0, rows, &p, stream);
    if (e != hipSuccess) return e;
    const ProductParams w = p;
    uint16_t* const xc = reinterpret_cast<uint16_t*>(ws + n.off_xc);
    uint16_t* const dl = reinterpret_cast<uint16_t*>(ws + n.off_dl);
    p.count = reinterpret_cast<int*>(ws + n.off_count);
    // G of the piece, [token][rpad]
    p.B = xc; p.ldb = n.dpad; p.pb = n.tok_cap * n.dpad;
    p.rows_b = static_cast<int>(n.tok_cap); p.cols_b = static_cast<int>(n.dpad);
    p.M = static_cast<int>(rows); p.N = static_cast<int>(n.tok_cap); p.K = static_cast<int>(n.dpad);
    p.n_is_tokens = 1;
    p.tgt = reinterpret_cast<int*>(ws + n.off_tgt);
    p.v0 = static_cast<int>(v0);
    p.lse = reinterpret_cast<float*>(ws + n.off_a);
    p.gl = reinterpret_cast<float*>(ws + n.off_b);
    p.g = reinterpret_cast<float*>(ws + n.off_c);
    p.dl = dl; p.ldl = rpad; p.pdl = n.tok_cap * rpad;
    p.tok_cap = n.tok_cap;
    e = product_any<false, false, kSplit, kGradLogits>(p, stream);
    if (e != hipSuccess) return e;
    if (a.dx != nullptr) {     // dx += G W: m = width, n = token, k = vocabulary
      ProductParams q = w;
      q.count = p.count;
      q.B = dl; q.ldb = rpad; q.pb = p.pdl;
      q.rows_b = static_cast<int>(n.tok_cap); q.cols_b = static_cast<int>(rpad);
      q.M = static_cast<int>(a.dim); q.N = static_cast<int>(n.tok_cap); q.K = static_cast<int>((rows + 63) / 64 * 64);
      q.n_is_tokens = 1;
      q.dxacc = reinterpret_cast<float*>(ws + n.off_dx); q.ldx = n.dpad;
      q.first = k == 0; q.last = k + 1 == n.pieces;
      q.rows = reinterpret_cast<int*>(ws + n.off_rows);
      q.out = a.dx; q.dim = a.dim; q.out_f32 = kSplit;
      q.vec = a.dim % 4 == 0 && reinterpret_cast<uintptr_t>(a.dx) % (4 * sizeof(T)) == 0;
      e = product_any<true, false, kSplit, kGradX>(q, stream);
      if (e != hipSuccess) return e;
    }
    if (a.dweight != nullptr) {   // dW of the piece = G^T x: m = width, n = vocabulary row, k = token
      ProductParams q{};
      const size_t gs = a.grad_io ? sizeof(T) : 4;
      q.count = p.count;
      q.A = xc; q.lda = n.dpad; q.pa = n.tok_cap * n.dpad;
      q.rows_a = static_cast<int>(n.tok_cap); q.cols_a = static_cast<int>(n.dpad);
      q.B = dl; q.ldb = rpad; q.pb = p.pdl;
      q.rows_b = static_cast<int>(n.tok_cap); q.cols_b = static_cast<int>(rpad);
      q.M = static_cast<int>(a.dim); q.N = static_cast<int>(rows);
      q.k_is_tokens = 1;
      q.out = static_cast<unsigned char*>(a.dweight) + v0 * a.dim * gs;
      q.dim = a.dim; q.out_f32 = gs == 4; q.accumulate = a.accumulate;
      q.vec = a.dim % 4 == 0 && reinterpret_cast<uintptr_t>(a.dweight) % (4 * gs) == 0;
      e = product_any<true, true, kSplit, kGradW>(q, stream);
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
