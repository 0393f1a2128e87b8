// Product of two matrices in 8 bits (fp8_util.h), for gfx950 (MI355X):
//   out[r, c] (+)= sum_k R[r, k] C[c, k],   R with scales of rows, C with scales of rows or of 128 x 128
// which is a linear layer's output (R: tokens, C: the weight), the gradient of its input (R: the output's gradient,
// C: the weight transposed) and of its weight (both transposed, k over the tokens).
//
// bf16 results: the 8-bit matrix instructions with a scale, 128 k at a time, which is one block: they multiply by the
// two e8m0 scales themselves and sum in fp32.  Within 8 neighbouring k they drop what lies some 14 bits below the
// largest product (measured: 1.2e-5 of the result's 2-norm for normally distributed values, 1 / 300 of bf16's own
// rounding).  fp32 results are to be better than that: the codes are widened to bf16, which holds them and their
// scales exactly, and the bf16 instructions' sums keep fp32's bits, at half the rate.
#include <type_traits>
#include <utility>

#include "fp8_util.h"
#include "internal.h"

namespace mssm {
namespace {

typedef float f32x16_t __attribute__((ext_vector_type(16)));
typedef int i32x8_t __attribute__((ext_vector_type(8)));
typedef __bf16 bf16x8_t __attribute__((ext_vector_type(8)));

struct Fp8Params {
  const unsigned char *r, *rs, *c, *cs;
  int64_t rows, cols;
  int64_t r_lines, c_lines;      // of the scales
  int64_t pitch;                 // bytes of a row of either
  int steps;                     // of 128 k
  int square;
  void* out;
  int accumulate;
  // tiles: see tile_product_kernel
  int tiles_c, tiles_r, whole, slices;
  float* sums;                   // [slice][BR][BC]
};

// 8 codes (words 2 q and 2 q + 1) times s, as bf16: exact
__device__ __forceinline__ bf16x8_t wide_codes(const i32x8_t& v, int q, float s) {
  bf16x8_t o;
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const bf16x2_t a = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(v[2 * q + h], s, false);
    const bf16x2_t b = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(v[2 * q + h], s, true);
    o[4 * h] = a[0]; o[4 * h + 1] = a[1]; o[4 * h + 2] = b[0]; o[4 * h + 3] = b[1];
  }
  return o;
}

// -------------------------------------------------------------------------------------------------- tiles
constexpr int kRow = kBlock / 2;         // bytes of a row of half a step
constexpr int kRing = 4;                 // halves in LDS
constexpr int kBand = 4;                 // tiles of R side by side in the order of tiles

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
// the same with up to four bytes a lane, each of which becomes a word at lds + 4 l
template <int BYTES> __device__ __forceinline__ void dma_word(const void* base, uint32_t off, uint32_t lds) {
  const uint32_t to = __builtin_amdgcn_readfirstlane(lds);
  if constexpr (BYTES == 4)
    asm volatile("s_mov_b32 m0, %2\n\ts_nop 0\n\tglobal_load_lds_dword %0, %1" :: "v"(off), "s"(base), "s"(to) : "memory", "m0");
  else if constexpr (BYTES == 2)
    asm volatile("s_mov_b32 m0, %2\n\ts_nop 0\n\tglobal_load_lds_ushort %0, %1" :: "v"(off), "s"(base), "s"(to) : "memory", "m0");
  else
    asm volatile("s_mov_b32 m0, %2\n\ts_nop 0\n\tglobal_load_lds_ubyte %0, %1" :: "v"(off), "s"(base), "s"(to) : "memory", "m0");
}
template <typename V> __device__ __forceinline__ V lds_at(uint32_t addr) {
  return *(__attribute__((address_space(3))) const V*)static_cast<uintptr_t>(addr);
}
// the scheduler keeps what stands before this before it
__device__ __forceinline__ void fence_schedule() { __builtin_amdgcn_sched_barrier(0); }

template <int... I, typename F> __device__ __forceinline__ void unrolled(std::integer_sequence<int, I...>, F&& f) {
  (f(std::integral_constant<int, I>{}), ...);
}
template <int N, typename F> __device__ __forceinline__ void unrolled(F&& f) {
  unrolled(std::make_integer_sequence<int, N>{}, f);
}

// where tile `tile` of the order below lies
struct Place {
  int c0, r0;
};
template <int BC, int BR> __device__ __forceinline__ Place place_of(const Fp8Params& p, int tile) {
  const int band = tile / (p.tiles_c * kBand);
  const int left = p.tiles_r - band * kBand, wide = left < kBand ? left : kBand;
  const int in_band = tile - band * p.tiles_c * kBand;
  // (the same for all lanes, which the divisions hide from the compiler)
  return {__builtin_amdgcn_readfirstlane(in_band / wide * BC),
          __builtin_amdgcn_readfirstlane((band * kBand + in_band % wide) * BR)};
}

// 8 neighbouring elements of a row of the output, the first `left` of which exist, to where they belong
template <typename T> __device__ __forceinline__ void put(T* to, float (&v)[8], int64_t left, int accumulate) {
  if (accumulate) {
    float o[8];
    load_row<8>(to, o, left);
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] += o[e];
  }
  store_row<8>(to, v, left);
}

// C's rows are the matrix instructions' rows: a lane's accumulators are neighbours in the output.
//
// One workgroup stays on a CU (two of the small tile) and takes tile after tile, each 128 k (a block) a step, in halves
// of 64 k.  Four halves are in LDS or on their way there.  While a half is multiplied from registers the next one's
// fragments are read, and the place that it was read from before takes the loads of the half four ahead; one barrier
// after each half, before which a wave waits for its loads of the half after the next, by count.  So a load has three
// halves of multiplications to arrive in, and crosses the borders of tiles (with two whole steps in LDS and a barrier a
// step it had two: 497 us at 8192^3).
//
// A wave holds TC x TR tiles of 32 x 32.  Row i of tile t is row TC i + t of its share: a lane's scales for its tiles
// are then TC neighbouring bytes of memory, one word, from which the instruction picks a byte; and what a lane holds of
// an output row are runs of 4 TC neighbouring elements.
template <int BC, int BR, int WC, int WR, typename T>
__global__ __launch_bounds__(WC * WR * 64, 2) void tile_product_kernel(Fp8Params p) {
  constexpr bool kFine = std::is_same_v<T, float>;
  constexpr int kW = WC * WR;
  constexpr int TC = BC / WC / 32, TR = BR / WR / 32;      // 32 x 32 tiles of a wave
  constexpr int LC = BC / 16 / kW, LR = BR / 16 / kW;      // 1 KB loads of a wave per half
  constexpr int kLoads = (LC + LR + TC - 1) / TC;          // loads between two rows of multiplications
  constexpr int kReads = (TC + TR + TC - 1) / TC;          // fragments read there
  constexpr int kAhead = 2 * (LC + LR) + 2;                // loads of two neighbouring halves, scales among them
  constexpr int kStores = TC * TR * static_cast<int>(sizeof(T));   // a whole tile's stores of a wave, 16 bytes a lane
  static_assert(LC * 16 * kW == BC && LR * 16 * kW == BR, "loads split evenly over the waves");
  static_assert(TC == 2 || TC == 4, "a lane's scales of C are a word or half of one");
  static_assert(TR == 2, "and those of R half of one");
  static_assert(kAhead + kStores < 64, "what the wait instruction can count");
  constexpr int kC = BC * kRow, kR = BR * kRow;            // bytes of a half
  __shared__ __attribute__((aligned(256))) unsigned char cbuf[kRing][kC];
  __shared__ __attribute__((aligned(256))) unsigned char rbuf[kRing][kR];
  __shared__ uint32_t sbuf[kRing / 2][kW][2][kLanes];      // scales of a step, each wave's own: C's, R's

  const int lane = threadIdx.x % kLanes;
  const int w = __builtin_amdgcn_readfirstlane(threadIdx.x / kLanes);
  const int wc = w / WR, wr = w % WR;

  // Jobs.  Whole tiles as long as every workgroup gets one; the tiles of the last, partial round are cut along k where
  // that fills the chip, each slice with sums of its own that are added afterwards.  Workgroups b, b + 8, ... share an
  // XCD and its L2: each XCD takes a contiguous range of an order that walks bands of 4 tiles of R, C outer.
  const int tiles = p.tiles_c * p.tiles_r;
  const int rest = tiles - p.whole, cut = rest * p.slices;
  const int xcd = blockIdx.x % 8, stride = gridDim.x / 8;
  const int whole8 = p.whole / 8, cut8 = (cut + 7) / 8;    // of an XCD
  const int mine = cut - xcd * cut8 < cut8 ? cut - xcd * cut8 : cut8;
  const int job_first = blockIdx.x / 8, job_end = whole8 + (mine > 0 ? mine : 0);
  struct Job {
    int c0, r0, sum, begin, steps;   // sum: which sums, or -1
  };
  auto job_at = [&](int i) {
    Job j;
    int tile;
    if (i < whole8) {
      tile = xcd * whole8 + i;
      j.sum = -1;
      j.begin = 0;
      j.steps = p.steps;
    } else {
      const int c = xcd * cut8 + i - whole8;
      const int slice = c / rest;
      tile = p.whole + c - slice * rest;
      j.sum = p.slices > 1 ? c : -1;
      // (steps < 2^16, slices <= 2 workgroups)
      j.begin = __builtin_amdgcn_readfirstlane(p.steps * slice / p.slices);
      j.steps = __builtin_amdgcn_readfirstlane(p.steps * (slice + 1) / p.slices) - j.begin;
    }
    const Place at = place_of<BC, BR>(p, tile);
    j.c0 = at.c0;
    j.r0 = at.r0;
    return j;
  };

  // ---- loads.  A load is 16 rows x 64 bytes, a lane's part row lane / 4 and the 16-byte chunk lane % 4 as stored.  The
  // chunk it holds is xor-ed with bits 2 and 3 of the row: the reads below, where 32 lanes read one chunk of 32 rows, are
  // served 16 lanes, 256 bytes, at a time, four rows of 64 bytes side by side.  LDS row 32 t + i of a wave's share holds
  // row TC i + t of it.  Rows past the matrix are its last row again.
  const int lrow = lane / 4;
  const uint32_t chunk = static_cast<uint32_t>(((lane % 4) ^ (lane / 16)) * 16);
  int ljob = job_first, lleft = 0, lk = 0;   // job and step of the next loads
  const unsigned char *lc = nullptr, *lr = nullptr, *lcs = nullptr, *lrs = nullptr;
  uint32_t oc[LC], orr[LR], ocs = 0, ors = 0;
  const uint32_t pitch = static_cast<uint32_t>(p.pitch);
  auto offsets = [&](int64_t rows, int of, auto& off) {   // rows: of the matrix, from the tile's first on
    const int last = rows < 256 ? static_cast<int>(rows) - 1 : 255;
#pragma unroll
    for (int i = 0; i < static_cast<int>(sizeof(off) / sizeof(off[0])); ++i) {
      const int at = (i * kW + w) * 16 + lrow;
      const int r = at / (32 * of) * (32 * of) + at % 32 * of + at / 32 % of;
      off[i] = static_cast<uint32_t>(r < last ? r : last) * pitch + chunk;   // (pitch <= 2^22)
    }
  };
  auto start_load = [&]() {   // the next job with steps, if there is one; else the last loads are repeated
    while (ljob < job_end) {
      const Job j = job_at(ljob);
      if (j.steps > 0) {
        lleft = j.steps;
        lk = j.begin;
        offsets(p.cols - j.c0, TC, oc);
        offsets(p.rows - j.r0, TR, orr);
        lc = p.c + static_cast<int64_t>(j.c0) * p.pitch;
        lr = p.r + static_cast<int64_t>(j.r0) * p.pitch;
        const int c = wc * (32 * TC) + lane % 32 * TC, r = wr * (32 * TR) + lane % 32 * TR;
        const int64_t left_c = p.c_lines - j.c0 - TC, left_r = p.r_lines - j.r0 - TR;
        lcs = p.cs + (p.square ? j.c0 / kBlock : j.c0);
        lrs = p.rs + j.r0;
        if (p.square) ocs = j.c0 / kBlock + wc * (32 * TC) / kBlock < p.c_lines ? wc * (32 * TC) / kBlock : 0;
        else ocs = c < left_c ? c : static_cast<int>(left_c);
        ors = r < left_r ? r : static_cast<int>(left_r);
        return;
      }
      ljob += stride;
    }
  };
  const uint32_t c_lds = lds_addr(&cbuf[0][0]), r_lds = lds_addr(&rbuf[0][0]);
  const uint32_t s_lds = lds_addr(&sbuf[0][w][0][0]);
  constexpr int kScales = sizeof(sbuf[0]);
  // load i of half h of a step into the place of half h of steps of parity `turn`
  auto load_one = [&](int i, int h, int turn) {
    const int64_t k = static_cast<int64_t>(lk) * kBlock + h * kRow;
    const int slot = 2 * turn + h;
    if (i < LC) dma16(lc + k, oc[i < LC ? i : 0], c_lds + slot * kC + (i * kW + w) * 1024);
    else dma16(lr + k, orr[i - LC < LR && i >= LC ? i - LC : 0], r_lds + slot * kR + ((i - LC) * kW + w) * 1024);
  };
  auto load_scales = [&](int turn) {
    const uint32_t to = s_lds + turn * kScales;
    const unsigned char* const c = lcs + lk * p.c_lines;
    if (p.square) dma_word<1>(c, ocs, to);
    else dma_word<TC>(c, ocs, to);
    dma_word<TR>(lrs + lk * p.r_lines, ors, to + 4 * kLanes);
  };
  auto loaded = [&]() {   // after a step's last load
    if (lleft > 1) {
      --lleft;
      ++lk;
    } else if (ljob < job_end) {
      ljob += stride;
      start_load();
    }
  };

  // ---- fragments: a lane's 32 codes are chunks 2 (lane / 32) and the next of its row
  uint32_t fc_at[2], fr_at[2];   // by chunk
#pragma unroll
  for (int q = 0; q < 2; ++q) {
    const int i = lane % 32;
    const uint32_t at = i * kRow + (((lane / 32 * 2 + q) ^ (i / 4 % 4)) << 4);
    fc_at[q] = c_lds + at + wc * TC * 32 * kRow;
    fr_at[q] = r_lds + at + wr * TR * 32 * kRow;
  }
  f32x16_t acc[TC][TR];
  i32x8_t fc[2][TC], fr[2][TR];
  auto frag = [&](const uint32_t (&at)[2], uint32_t more) {
    const u32x4_t a = lds_at<u32x4_t>(at[0] + more), b = lds_at<u32x4_t>(at[1] + more);
    return i32x8_t{static_cast<int>(a[0]), static_cast<int>(a[1]), static_cast<int>(a[2]), static_cast<int>(a[3]),
                   static_cast<int>(b[0]), static_cast<int>(b[1]), static_cast<int>(b[2]), static_cast<int>(b[3])};
  };
  auto read_one = [&](int q, int h, int slot) {
    if (q < TR) fr[h][q < TR ? q : 0] = frag(fr_at, slot * kR + (q < TR ? q : 0) * 32 * kRow);
    else fc[h][q - TR < TC && q >= TR ? q - TR : 0] = frag(fc_at, slot * kC + (q - TR) * 32 * kRow);
  };
  struct Scales {
    uint32_t c, r;
  };
  auto read_scales = [&](int turn) {
    const uint32_t at = s_lds + turn * kScales + lane * 4;
    return Scales{lds_at<uint32_t>(at) * (p.square ? 0x01010101u : 1u), lds_at<uint32_t>(at + 4 * kLanes)};
  };
  auto multiply_row = [&](auto i, int h, const Scales& s) {
    constexpr int I = decltype(i)::value;
    if constexpr (kFine) {
      // 16 k at a time, every fragment widened once
      float sc[TC], sr[TR];
#pragma unroll
      for (int c = 0; c < TC; ++c) sc[c] = fp8_power((s.c >> (8 * c)) & 255u);
#pragma unroll
      for (int r = 0; r < TR; ++r) sr[r] = fp8_power((s.r >> (8 * r)) & 255u);
#pragma unroll
      for (int q = I * 4 / TC; q < (I + 1) * 4 / TC; ++q) {
        bf16x8_t b[TR];
#pragma unroll
        for (int r = 0; r < TR; ++r) b[r] = wide_codes(fr[h][r], q, sr[r]);
#pragma unroll
        for (int c = 0; c < TC; ++c) {
          const bf16x8_t a = wide_codes(fc[h][c], q, sc[c]);
#pragma unroll
          for (int r = 0; r < TR; ++r) acc[c][r] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(a, b[r], acc[c][r], 0, 0, 0);
        }
      }
    } else {
      unrolled<TR>([&](auto j) {
        constexpr int J = decltype(j)::value;
        acc[I][J] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(fc[h][I], fr[h][J], acc[I][J], 0, 0, I,
                                                                    static_cast<int>(s.c), J, static_cast<int>(s.r));
        // stays here: the compiler knows of no reason not to move a multiplication to where its result is used
        asm volatile("" : "+v"(acc[I][J]));
      });
    }
  };

  int stored = 0;   // halves whose wait may leave the last tile's stores outstanding too
  // the end of a half: this wave's reads of the next one are done, and its loads of the one after that have arrived
  auto turn_over = [&]() {
    if (stored > 0) {
      --stored;
      asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)" ::"n"(kAhead + kStores) : "memory");
    } else {
      asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)" ::"n"(kAhead) : "memory");
    }
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
    fence_schedule();
  };
  start_load();
  Scales now{}, next{};
  if (lleft > 0) {   // (no steps at all where k is empty: the tiles are then stored as zeros)
#pragma unroll
    for (int turn = 0; turn < 2; ++turn) {
      load_scales(turn);
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int q = 0; q < LC + LR; ++q) load_one(q, h, turn);
      loaded();
    }
    turn_over();
#pragma unroll
    for (int q = 0; q < TC + TR; ++q) read_one(q, 0, 0);
    now = read_scales(0);
    turn_over();
  }
  int turn = 0;   // parity of the step, counted over all tiles
  for (int job = job_first; job < job_end; job += stride) {
    const Job cur = job_at(job);
#pragma unroll
    for (int i = 0; i < TC; ++i)
#pragma unroll
      for (int j = 0; j < TR; ++j) acc[i][j] = f32x16_t{};
    for (int s = 0; s < cur.steps; ++s, turn ^= 1) {
      fence_schedule();
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        if (h == 0) load_scales(turn);
        else next = read_scales(turn ^ 1);
        unrolled<TC>([&](auto i) {
          multiply_row(i, h, now);
          fence_schedule();
#pragma unroll
          for (int q = i * kLoads; q < (i + 1) * kLoads && q < LC + LR; ++q) load_one(q, h, turn);
#pragma unroll
          for (int q = i * kReads; q < (i + 1) * kReads && q < TC + TR; ++q)
            read_one(q, h ^ 1, h == 0 ? 2 * turn + 1 : 2 * (turn ^ 1));
          fence_schedule();
        });
        turn_over();
      }
      now = next;
      loaded();
    }

    // accumulator e = 4 q + f of tile (i, j): C's row TC (8 q + 4 (lane / 32) + f) + i and R's row TR (lane % 32) + j of
    // the wave's shares
    const int wave_c = wc * TC * 32 + lane / 32 * 4 * TC, wave_r = wr * TR * 32 + lane % 32 * TR;
    auto each = [&](auto&& to) {   // every run of 8 neighbouring elements: (row of the tile, column of it, values)
#pragma unroll
      for (int j = 0; j < TR; ++j)
#pragma unroll
        for (int q = 0; q < 4; ++q)
#pragma unroll
          for (int h = 0; h < TC / 2; ++h) {
            float v[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) v[e] = acc[e % TC][j][4 * q + (8 * h + e) / TC];
            to(wave_r + j, wave_c + 8 * TC * q + 8 * h, v);
          }
    };
    if (cur.sum >= 0) {
      float* const to = p.sums + static_cast<int64_t>(cur.sum) * BR * BC;
      each([&](int r, int c, float (&v)[8]) { store_row<8>(to + r * BC + c, v); });
    } else {
      T* const to = static_cast<T*>(p.out) + cur.r0 * p.cols + cur.c0;
      const int64_t rows = p.rows - cur.r0, cols = p.cols - cur.c0;
      if (rows >= BR && cols >= BC && !p.accumulate) {
        if constexpr (kFine) {
          each([&](int r, int c, float (&v)[8]) { store_row<8>(to + r * p.cols + c, v); });
        } else {
          // A run of a row is 16 (TC 2) or 32 bytes of lane l and as many after it of lane l + 32.  Pieces of 16 bytes change
          // places between lanes 16 apart, so that a store writes 64 bytes of each of 16 rows, past the cache: kept there,
          // the output pushed the operands out of it (32768 x 2560 x 10240, which writes 671 MB: 817 us, as here 767; past
          // the cache but in pieces of 32 bytes 955).
          constexpr bool kTwo = TC == 4;             // a run is two pieces: they change places, else runs q and q + 1
          const int row16 = lane / 16 % 2;
#pragma unroll
          for (int j = 0; j < TR; ++j)
#pragma unroll
            for (int q = 0; q < 4; q += kTwo ? 1 : 2) {
              u32x4_t piece[2];
#pragma unroll
              for (int h = 0; h < 2; ++h)
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                  const int at = (kTwo ? 8 * h : 0) + 2 * e, run = 4 * (kTwo ? q : q + h);
                  piece[h][e] = pack_bf16(acc[at % TC][j][run + at / TC], acc[(at + 1) % TC][j][run + (at + 1) / TC]);
                }
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                const auto t = __builtin_amdgcn_permlane16_swap(piece[0][e], piece[1][e], false, false);
                piece[0][e] = t[0];
                piece[1][e] = t[1];
              }
              const int c = wave_c + 8 * TC * q + row16 * (kTwo ? 8 : 8 * TC);
#pragma unroll
              for (int h = 0; h < 2; ++h) {
                const int r = wr * TR * 32 + (lane % 16 + 16 * h) * TR + j;
                __builtin_nontemporal_store(piece[h], reinterpret_cast<u32x4_u*>(to + r * p.cols + c));
              }
            }
        }
        stored = 2;
      } else {
        each([&](int r, int c, float (&v)[8]) {
          if (r < rows) put(to + r * p.cols + c, v, cols - c, p.accumulate);
        });
      }
    }
  }
  // the last loads may still be on their way into this workgroup's LDS
  asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
}

// Adds the slices of the tiles of the last round, in order: workgroup (tile, share of its rows).
constexpr int kShares = 8;
template <int BC, int BR, typename T> __global__ __launch_bounds__(256) void slices_kernel(Fp8Params p) {
  const int t = blockIdx.x / kShares, rest = p.tiles_c * p.tiles_r - p.whole;
  const Place at = place_of<BC, BR>(p, p.whole + t);
  const int c = threadIdx.x % (BC / 8) * 8;
  const int64_t left = p.cols - at.c0 - c;
  if (left <= 0) return;
  constexpr int kRowsOf = BR / kShares, kAtOnce = 256 / (BC / 8);
  const int first = blockIdx.x % kShares * kRowsOf + threadIdx.x / (BC / 8);
  for (int i = 0; i < kRowsOf; i += kAtOnce) {
    const int64_t row = static_cast<int64_t>(at.r0) + first + i;
    if (row >= p.rows) return;
    float v[8] = {};
#pragma unroll 4
    for (int s = 0; s < p.slices; ++s) {
      float o[8];
      load_row<8>(p.sums + ((static_cast<int64_t>(s) * rest + t) * BR + first + i) * BC + c, o);
#pragma unroll
      for (int e = 0; e < 8; ++e) v[e] += o[e];
    }
    put(static_cast<T*>(p.out) + row * p.cols + at.c0 + c, v, left, p.accumulate);
  }
}

// ---------------------------------------------------------------------------------------------- plan
struct Tiling {
  int bc, br;              // tile
  int grid;                // workgroups
  int64_t tiles;
  int whole, slices;
  int64_t cost;
};

// Slices of the last, partial round: the least time, in steps of a workgroup.  A slice costs some four steps more (its
// start, its sums' way out) and the addition some eight.  At most two rounds of slices, which bounds the sums' memory.
Tiling tiling(const Fp8ProductArgs& a, int bc, int br, int grid, int64_t weight) {
  Tiling t{bc, br, grid, 0, 0, 1, 0};
  t.tiles = ((a.cols + bc - 1) / bc) * ((a.rows + br - 1) / br);
  const int64_t steps = fp8_blocks(a.k), rest = t.tiles % grid;
  int64_t best = rest > 0 ? steps : 0;
  for (int64_t s = 2; rest > 0 && rest * s <= 2 * grid && steps / s >= 4; ++s) {
    const int64_t time = (rest * s + grid - 1) / grid * ((steps + s - 1) / s + 4) + 8;
    if (time < best) {
      best = time;
      t.slices = static_cast<int>(s);
    }
  }
  t.whole = static_cast<int>(t.tiles - rest);
  t.cost = weight * (t.tiles / grid * steps + best);
  return t;
}

constexpr int kCus = 256;
// Tiles of 256 x 256, one workgroup to a CU, or of 128 x 128, two to a CU.
Tiling pick(const Fp8ProductArgs& a) {
  const Tiling small = tiling(a, 128, 128, 2 * kCus, 5);
  const Tiling large = tiling(a, 256, 256, kCus, 8);
  return large.cost <= small.cost ? large : small;
}

}  // namespace

size_t fp8_product_workspace_bytes(const Fp8ProductArgs& a) {
  if (a.rows == 0 || a.cols == 0) return 0;
  const Tiling t = pick(a);
  return t.slices > 1 ? static_cast<size_t>(t.tiles - t.whole) * t.slices * t.bc * t.br * 4 : 0;
}

hipError_t fp8_product_launch(const Fp8ProductArgs& a, hipStream_t stream) {
  if (a.rows == 0 || a.cols == 0) return hipSuccess;
  Fp8Params p{};
  p.r = static_cast<const unsigned char*>(a.r.codes); p.rs = static_cast<const unsigned char*>(a.r.scales);
  p.c = static_cast<const unsigned char*>(a.c.codes); p.cs = static_cast<const unsigned char*>(a.c.scales);
  p.rows = a.rows; p.cols = a.cols; p.square = a.square;
  p.steps = static_cast<int>(fp8_blocks(a.k)); p.pitch = fp8_blocks(a.k) * kBlock;
  p.r_lines = fp8_lines(a.rows); p.c_lines = a.square ? fp8_blocks(a.cols) : fp8_lines(a.cols);
  p.out = a.out; p.accumulate = a.accumulate;
  const Tiling t = pick(a);
  p.tiles_c = static_cast<int>((a.cols + t.bc - 1) / t.bc); p.tiles_r = static_cast<int>((a.rows + t.br - 1) / t.br);
  p.whole = t.whole; p.slices = t.slices; p.sums = static_cast<float*>(a.workspace);
  const dim3 sum_grid(static_cast<unsigned>((t.tiles - t.whole) * kShares));
  auto go = [&](auto bc, auto br, auto waves_c, auto waves_r, auto io) {
    constexpr int kBC = decltype(bc)::value, kBR = decltype(br)::value;
    constexpr int kWC = decltype(waves_c)::value, kWR = decltype(waves_r)::value;
    using T = decltype(io);
    tile_product_kernel<kBC, kBR, kWC, kWR, T><<<dim3(t.grid), kWC * kWR * kLanes, 0, stream>>>(p);
    if (t.slices > 1) slices_kernel<kBC, kBR, T><<<sum_grid, 256, 0, stream>>>(p);
  };
  using Two = std::integral_constant<int, 2>;
  using Four = std::integral_constant<int, 4>;
  using Small = std::integral_constant<int, 128>;
  using Large = std::integral_constant<int, 256>;
  if (t.bc == 256 && a.out_io) go(Large{}, Large{}, Two{}, Four{}, uint16_t{});
  else if (t.bc == 256) go(Large{}, Large{}, Two{}, Four{}, float{});
  else if (a.out_io) go(Small{}, Small{}, Two{}, Two{}, uint16_t{});
  else go(Small{}, Small{}, Two{}, Two{}, float{});
  return hipGetLastError();
}

}  // namespace mssm
