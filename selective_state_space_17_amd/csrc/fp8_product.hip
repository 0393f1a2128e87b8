// Product of two matrices in 8 bits (fp8_util.h), for gfx950 (MI355X):
//   out[r, c] (+)= sum_k R[r, k] C[c, k],   R with scales of rows, C with scales of rows or of 128 x 128
// which is a linear layer's output (R: tokens, C: the weight), the gradient of its input (R: the output's gradient,
// C: the weight transposed) and of its weight (both transposed, k over the tokens).
//
// bf16 results: the 8-bit matrix instructions with a scale, 128 k at a time, which is one block: they multiply by the
// two e8m0 scales themselves and sum in fp32.  Within 8 neighbouring k they drop what lies some 14 bits below the
// largest product (measured: 1.2e-5 of the result's 2-norm for normally distributed values, 1 / 300 of bf16's own
// rounding).  fp32 results are to be better than that: the codes are widened to bf16, and the bf16 instructions' sums keep
// fp32's bits, at half the rate.  bf16 holds a code times its scale exactly from 2^-124 on (e4m3 ends at 2^-9 of it, bf16 at
// 2^-133); under the scales 2^-127 to 2^-125 the smallest 24, 16 and 8 magnitudes become multiples of 2^-133, halves to
// even.  (A factor that lifts one operand's smallest values would take as much from its largest.)
//
// Large products are bound by the matrix cores under the power limit, and their time goes with the clock.  32768 x 2560 x
// 10240: 710 us (2.4 PFLOP/s) in a second of nothing else, 740 to 1010 in the first dozen calls after a pause, while the
// clock settles, 677 at best (2.5; matrix cores busy 0.70 of the cycles at some 1.8 GHz).  8192^3: 438, at best 415; with
// fp32 results 848 and 786, where the library's bf16 product of the same values takes 715 and 699.  Few rows are bound by
// latency and the weight's bytes (1 x 2560 x 10240: 7.1 us, 26 MB).  Times below are the best of calls back to back, each
// pair on one GPU.
#include <limits>
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
  int64_t rows, cols, k;
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

// 8 codes times s, as bf16: exact from s = 2^-124 on (above)
__device__ __forceinline__ bf16x8_t wide_codes(uint32_t lo, uint32_t hi, float s) {
  const bf16x2_t a = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(static_cast<int>(lo), s, false);
  const bf16x2_t b = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(static_cast<int>(lo), s, true);
  const bf16x2_t c = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(static_cast<int>(hi), s, false);
  const bf16x2_t d = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(static_cast<int>(hi), s, true);
  return bf16x8_t{a[0], a[1], b[0], b[1], c[0], c[1], d[0], d[1]};
}

// -------------------------------------------------------------------------------------------------- tiles
constexpr int kRow = kBlock / 2;         // bytes of a row of half a step
constexpr int kBand = 4;                 // tiles of R side by side in the order of tiles

__device__ __forceinline__ uint32_t lds_addr(const void* p) {
  return static_cast<uint32_t>(reinterpret_cast<uintptr_t>(p));   // low half of a flat LDS address
}
// Lane l's 16 bytes at base + off + OFF go to LDS offset lds + LDS + 16 l; with fewer bytes each becomes a word at + 4 l
// (base and lds are wave-uniform; the instruction adds its offset to either address).  Written as asm so that the compiler
// does not wait for these loads before the LDS reads of the other halves; they are waited for by count.  No output
// register: nothing can be overwritten while a load is in flight.
template <int BYTES, int LDS, int OFF> __device__ __forceinline__ void dma(const void* base, uint32_t off, uint32_t lds) {
  if constexpr (BYTES == 16)
    asm volatile("s_add_u32 m0, %2, %3\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %0, %1 offset:%4"
                 :: "v"(off), "s"(base), "s"(lds), "n"(LDS - OFF), "n"(OFF) : "memory", "m0", "scc");
  else if constexpr (BYTES == 4)
    asm volatile("s_add_u32 m0, %2, %3\n\ts_nop 0\n\tglobal_load_lds_dword %0, %1 offset:%4"
                 :: "v"(off), "s"(base), "s"(lds), "n"(LDS - OFF), "n"(OFF) : "memory", "m0", "scc");
  else if constexpr (BYTES == 2)
    asm volatile("s_add_u32 m0, %2, %3\n\ts_nop 0\n\tglobal_load_lds_ushort %0, %1 offset:%4"
                 :: "v"(off), "s"(base), "s"(lds), "n"(LDS - OFF), "n"(OFF) : "memory", "m0", "scc");
  else
    asm volatile("s_add_u32 m0, %2, %3\n\ts_nop 0\n\tglobal_load_lds_ubyte %0, %1 offset:%4"
                 :: "v"(off), "s"(base), "s"(lds), "n"(LDS - OFF), "n"(OFF) : "memory", "m0", "scc");
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

// Jobs of a workgroup that stays.  Whole tiles as long as every workgroup gets one; the tiles of the last, partial round
// are cut along k where that fills the chip, each slice with sums of its own that are added afterwards.  Workgroups b,
// b + 8, ... share an XCD and its L2: each XCD takes a contiguous range of an order that walks bands of 4 tiles of R, C
// outer.
struct Job {
  int c0, r0, sum, begin, steps;   // sum: which sums, or -1
};
template <int BC, int BR> struct Jobs {
  const Fp8Params& p;
  int rest, xcd, whole8, cut8, first, end, stride;
  __device__ __forceinline__ explicit Jobs(const Fp8Params& q) : p(q) {
    rest = p.tiles_c * p.tiles_r - p.whole;
    const int cut = rest * p.slices;
    xcd = blockIdx.x % 8;
    stride = gridDim.x / 8;
    whole8 = p.whole / 8;   // of an XCD
    cut8 = (cut + 7) / 8;
    const int mine = cut - xcd * cut8 < cut8 ? cut - xcd * cut8 : cut8;
    first = blockIdx.x / 8;
    end = whole8 + (mine > 0 ? mine : 0);
  }
  __device__ __forceinline__ Job at(int i) const {
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
  }
};

// V neighbouring elements of a row of the output, the first `left` of which exist, to where they belong
template <int V, typename T> __device__ __forceinline__ void put(T* to, float (&v)[V], int64_t left, int accumulate) {
  if (accumulate) {
    float o[V];
    load_row<V>(to, o, left);
#pragma unroll
    for (int e = 0; e < V; ++e) v[e] += o[e];
  }
  store_row<V>(to, v, left);
}

// A tile's, or a slice's, accumulators to where they belong; true where that is the whole tile's kStores stores of a wave.
template <int BC, int BR, int WC, int WR, typename T>
__device__ __forceinline__ bool way_out(const Fp8Params& p, const Job& cur, int lane, int wc, int wr,
                                        f32x16_t (&acc)[BC / WC / 32][BR / WR / 32]) {
  constexpr bool kFine = std::is_same_v<T, float>;
  constexpr int TC = BC / WC / 32, TR = BR / WR / 32;
  // accumulator e = 4 q + f of tile (i, j): R's row TR (8 q + 4 (lane / 32) + f) + j of the wave's share, and row i of
  // C's that are the lane's.  Lanes 16 apart exchange f and f + 1.
  constexpr int kRun = 2 * TC;
  int wave_r = wr * TR * 32 + (lane / 32 * 4 + lane / 16 % 2) * TR;
  asm volatile("" : "+v"(wave_r));   // (known before the loop over jobs, all the rows' places would be registers in it)
  const int c = wc * TC * 32 + lane % 16 * kRun;
  auto each = [&](auto&& to) {   // every pair of f: (row of the tile after wave_r, tile j, first accumulator)
    unrolled<TR * 8>([&](auto i) {
      constexpr int I = decltype(i)::value, J = I / 8, E = I % 8 * 2;
      to(std::integral_constant<int, (E / 4 * 8 + E % 4) * TR + J>{}, std::integral_constant<int, J>{},
         std::integral_constant<int, E>{});
    });
  };
  // (way: which of the three below, so that the compiler does not take what two have in common before the branch, where
  // a second set of accumulators finds no registers)
  auto exchanged = [&](auto way, auto j, auto e, float (&v)[kRun]) {
    constexpr int J = decltype(j)::value, E = decltype(e)::value;
#pragma unroll
    for (int t = 0; t < TC; ++t) {
      float a = acc[t][J][E];
      asm volatile("" : "+v"(a) : "n"(decltype(way)::value));
      const auto x = __builtin_amdgcn_permlane16_swap(__float_as_uint(a), __float_as_uint(acc[t][J][E + 1]), false, false);
      v[t] = __uint_as_float(x[0]);
      v[TC + t] = __uint_as_float(x[1]);
    }
  };
  if (cur.sum >= 0) {
    float* const to = p.sums + static_cast<int64_t>(cur.sum) * BR * BC + wave_r * BC + c;
    const int64_t rows = p.rows - cur.r0 - wave_r;
    each([&](auto r, auto j, auto e) {
      float v[kRun];
      exchanged(std::integral_constant<int, 0>{}, j, e, v);
      if (r < rows) store_row<kRun>(to + r * BC, v);
    });
  } else {
    T* const tile = static_cast<T*>(p.out) + cur.r0 * p.cols + cur.c0;
    const uint32_t at = static_cast<uint32_t>(wave_r * static_cast<int>(p.cols) + c) * sizeof(T);   // (cols <= 2^20)
    auto to = [&](auto r) { return reinterpret_cast<T*>(reinterpret_cast<unsigned char*>(tile + r * p.cols) + at); };
    const int64_t rows = p.rows - cur.r0, cols = p.cols - cur.c0;
    if (rows >= BR && cols >= BC && !p.accumulate) {
      // past the cache: kept there, the output pushes the operands out of it (32768 x 2560 x 10240, which writes 671 MB:
      // 677 us, kept 730)
      each([&](auto r, auto j, auto e) {
        if constexpr (kFine) {
          float v[kRun];
          exchanged(std::integral_constant<int, 1>{}, j, e, v);
          __builtin_nontemporal_store(f32x4_t{v[0], v[1], v[2], v[3]}, reinterpret_cast<f32x4_u*>(to(r)));
        } else {
          constexpr int J = decltype(j)::value, E = decltype(e)::value;
          typedef uint32_t Run __attribute__((ext_vector_type(TC)));
          typedef Run Run_u __attribute__((aligned(2)));
          Run v;
#pragma unroll
          for (int h = 0; h < TC / 2; ++h) {
            const auto x = __builtin_amdgcn_permlane16_swap(pack_bf16(acc[2 * h][J][E], acc[2 * h + 1][J][E]),
                                                            pack_bf16(acc[2 * h][J][E + 1], acc[2 * h + 1][J][E + 1]),
                                                            false, false);
            v[h] = x[0];
            v[TC / 2 + h] = x[1];
          }
          __builtin_nontemporal_store(v, reinterpret_cast<Run_u*>(to(r)));
        }
      });
      return true;
    } else {
      each([&](auto r, auto j, auto e) {
        float v[kRun];
        exchanged(std::integral_constant<int, 2>{}, j, e, v);
        if (r + wave_r < rows) put(to(r), v, cols - c, p.accumulate);
      });
    }
  }
  return false;
}

// A workgroup stays on a CU (two of the small tile) and takes tile after tile, each 128 k (a block) a step, in halves of
// 64 k.  Four halves are in LDS or on their way there.  While a half is multiplied from registers the next one's
// fragments are read, and the place that it was read from before takes the loads of the half four ahead; one barrier
// after each half, before which a wave waits for its loads of the half after the next, by count.  So a load has three
// halves of multiplications to arrive in, and crosses the borders of tiles (with two whole steps in LDS and a barrier a
// step it had two: 497 us at 8192^3, where the ring took 448; a ring of eight halves was no faster).
//
// A wave holds TC x TR tiles of 32 x 32.  Of R, row i of tile t is row TR i + t of its share, of C row 2 TC (i % 16) +
// TC (i / 16) + t: a lane's scales for its tiles are then neighbouring bytes of memory, one word, from which the
// instruction picks a byte.  R's rows are the matrix instructions' rows, so that a lane's accumulators are TC neighbours of
// many output rows.  After lanes 16 apart have exchanged every other row they are 2 TC neighbours, and those of 16 lanes
// are one stretch of a row, 128 bytes or more, which leaves in one store (in pieces of 64 bytes of 16 rows: 712 us for
// 32768 x 2560 x 10240, as here 677; with rows that begin off a line, 10001 columns: 947 and 747).
template <int BC, int BR, int WC, int WR, bool SQUARE>
__global__ __launch_bounds__(WC * WR * 64, 2) void tile_product_kernel(Fp8Params p) {
  constexpr int kW = WC * WR;
  constexpr int TC = BC / WC / 32, TR = BR / WR / 32;      // 32 x 32 tiles of a wave
  constexpr int LC = BC / 16 / kW, LR = BR / 16 / kW;      // 1 KB loads of a wave per half
  constexpr int kLoads = (LC + LR + TC - 1) / TC;          // loads between two rows of multiplications
  constexpr int kReads = (TC + TR + TC - 1) / TC;          // fragments read there
  constexpr int kAhead = 2 * (LC + LR) + 2;                // loads of two neighbouring halves, scales among them
  constexpr int kStores = TR * 8;                          // a whole tile's stores of a wave
  static_assert(LC * 16 * kW == BC && LR * 16 * kW == BR, "loads split evenly over the waves");
  static_assert(TC == 2 || TC == 4, "a lane's scales of C are a word or half of one");
  static_assert(TR == 2, "and those of R half of one");
  static_assert(kAhead + kStores < 64, "what the wait instruction can count");
  constexpr int kC = BC * kRow, kR = BR * kRow;            // bytes of a half
  // LDS: four halves of C, four of R, the scales of two steps, each wave's own (C's, R's).  The ring's two steps lie a power
  // of two apart, so that an exclusive or takes an address from one to the other.
  constexpr int kS = kW * 2 * kLanes * 4;
  __shared__ __attribute__((aligned(4 * kC))) unsigned char lds[4 * kC + 4 * kR + 2 * kS];
  static_assert((kC & (kC - 1)) == 0 && kC == kR && (kS & (kS - 1)) == 0, "powers of two");
  const int lane = threadIdx.x % kLanes;
  const int w = __builtin_amdgcn_readfirstlane(threadIdx.x / kLanes);
  const int wc = w / WR, wr = w % WR;

  const Jobs<BC, BR> jobs(p);
  // ---- loads.  A load is 16 rows x 64 bytes, a lane's part row lane / 4 and the 16-byte chunk lane % 4 as stored.  The
  // chunk it holds is xor-ed with bits 2 and 3 of the row: the reads below, where 32 lanes read one chunk of 32 rows, are
  // served 16 lanes, 256 bytes, at a time, four rows of 64 bytes side by side.  LDS row 32 t + i of a wave's share holds
  // row TC i + t of it.  Rows past the matrix are its last row again.
  const int lrow = lane / 4;
  const uint32_t chunk = static_cast<uint32_t>(((lane % 4) ^ (lane / 16)) * 16);
  int ljob = jobs.first, lleft = 0;           // job of the next loads, and its steps that they have not come to
  const unsigned char *lc = nullptr, *lr = nullptr, *lcs = nullptr, *lrs = nullptr;
  uint32_t oc[LC], orr[LR], ocs = 0, ors = 0;
  const uint32_t pitch = static_cast<uint32_t>(p.pitch);
  auto offsets = [&](int64_t rows, int of, int turned, auto& off) {   // rows: of the matrix, from the tile's first on
    const int last = rows < 256 ? static_cast<int>(rows) - 1 : 255;
#pragma unroll
    for (int i = 0; i < static_cast<int>(sizeof(off) / sizeof(off[0])); ++i) {
      const int at = (i * kW + w) * 16 + lrow;
      const int row = at % 32, t = at / 32 % of;
      const int r = at / (32 * of) * (32 * of) + (turned ? row % 16 * 2 + row / 16 : row) * of + t;
      off[i] = static_cast<uint32_t>(r < last ? r : last) * pitch + chunk;   // (pitch <= 2^22)
    }
  };
  auto start_load = [&]() {   // the next job with steps, if there is one; else the last loads are repeated
    while (ljob < jobs.end) {
      const Job j = jobs.at(ljob);
      if (j.steps > 0) {
        lleft = j.steps;
        offsets(p.cols - j.c0, TC, 1, oc);
        offsets(p.rows - j.r0, TR, 0, orr);
        lc = p.c + static_cast<int64_t>(j.c0) * p.pitch + j.begin * kBlock;
        lr = p.r + static_cast<int64_t>(j.r0) * p.pitch + j.begin * kBlock;
        const int c = wc * (32 * TC) + (lane % 16 * 2 + lane / 16 % 2) * TC, r = wr * (32 * TR) + lane % 32 * TR;
        const int64_t left_c = p.c_lines - j.c0 - TC, left_r = p.r_lines - j.r0 - TR;
        lcs = p.cs + j.begin * p.c_lines + (SQUARE ? j.c0 / kBlock : j.c0);
        lrs = p.rs + j.begin * p.r_lines + j.r0;
        if (SQUARE) ocs = j.c0 / kBlock + wc * (32 * TC) / kBlock < p.c_lines ? wc * (32 * TC) / kBlock : 0;
        else ocs = c < left_c ? c : static_cast<int>(left_c);
        ors = r < left_r ? r : static_cast<int>(left_r);
        return;
      }
      ljob += jobs.stride;
    }
  };
  const uint32_t c_lds = lds_addr(lds), r_lds = c_lds + 4 * kC, s_lds = r_lds + 4 * kR + w * (2 * kLanes * 4);
  // where the ring's step that takes loads lies
  uint32_t c_to = __builtin_amdgcn_readfirstlane(c_lds + w * 1024), r_to = c_to + 4 * kC;
  uint32_t s_to = __builtin_amdgcn_readfirstlane(s_lds);
  // load i of half h of a step
  auto load_one = [&](auto i, auto h) {
    constexpr int I = decltype(i)::value, H = decltype(h)::value;
    if constexpr (I < LC) dma<16, H * kC + I * kW * 1024, H * kRow>(lc, oc[I], c_to);
    else dma<16, H * kR + (I - LC) * kW * 1024, H * kRow>(lr, orr[I - LC], r_to);
  };
  auto load_scales = [&]() {
    dma<SQUARE ? 1 : TC, 0, 0>(lcs, ocs, s_to);
    dma<TR, 4 * kLanes, 0>(lrs, ors, s_to);
  };
  auto loaded = [&]() {   // after a step's last load
    c_to ^= 2 * kC;
    r_to ^= 2 * kR;
    s_to ^= kS;
    if (lleft > 1) {
      --lleft;
      lc += kBlock;
      lr += kBlock;
      lcs += p.c_lines;
      lrs += p.r_lines;
    } else if (ljob < jobs.end) {
      ljob += jobs.stride;
      start_load();
    }
  };

  // ---- fragments: a lane's 32 codes are chunks 2 (lane / 32) and the next of its row
  uint32_t fc_at[2], fr_at[2], fs_at = s_lds + lane * 4;   // by chunk; of the step that is multiplied
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
  auto read_one = [&](auto q, auto h) {   // fragment q of half h into set h
    constexpr int Q = decltype(q)::value, H = decltype(h)::value;
    if constexpr (Q < TR) fr[H][Q] = frag(fr_at, H * kR + Q * 32 * kRow);
    else fc[H][Q - TR] = frag(fc_at, H * kC + (Q - TR) * 32 * kRow);
  };
  struct Scales {
    uint32_t c, r;
  };
  auto read_scales = [&]() {
    return Scales{lds_at<uint32_t>(fs_at) * (SQUARE ? 0x01010101u : 1u), lds_at<uint32_t>(fs_at + 4 * kLanes)};
  };
  auto multiply_row = [&](auto i, int h, const Scales& s) {
    constexpr int I = decltype(i)::value;
    unrolled<TR>([&](auto j) {
      constexpr int J = decltype(j)::value;
      acc[I][J] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(fr[h][J], fc[h][I], acc[I][J], 0, 0, J,
                                                                  static_cast<int>(s.r), I, static_cast<int>(s.c));
      // stays here: the compiler knows of no reason not to move a multiplication to where its result is used
      asm volatile("" : "+v"(acc[I][J]));
    });
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
  using Zero = std::integral_constant<int, 0>;
  start_load();
  Scales now{};
  if (lleft > 0) {   // (no steps at all where k is empty: the tiles are then stored as zeros)
#pragma unroll
    for (int turn = 0; turn < 2; ++turn) {
      load_scales();
      unrolled<2>([&](auto h) { unrolled<LC + LR>([&](auto q) { load_one(q, h); }); });
      loaded();
    }
    turn_over();
    unrolled<TC + TR>([&](auto q) { read_one(q, Zero{}); });
    now = read_scales();
    turn_over();
  }
  for (int job = jobs.first; job < jobs.end; job += jobs.stride) {
    const Job cur = jobs.at(job);
#pragma unroll
    for (int i = 0; i < TC; ++i)
#pragma unroll
      for (int j = 0; j < TR; ++j) acc[i][j] = f32x16_t{};
    for (int s = 0; s < cur.steps; ++s) {
      Scales next;
      fence_schedule();
      unrolled<2>([&](auto h) {
        constexpr int H = decltype(h)::value;
        if constexpr (H == 0) {
          load_scales();
        } else {
          // the next half is the next step's first
#pragma unroll
          for (int q = 0; q < 2; ++q) {
            fc_at[q] ^= 2 * kC;
            fr_at[q] ^= 2 * kR;
          }
          fs_at ^= kS;
          next = read_scales();
        }
        unrolled<TC>([&](auto i) {
          constexpr int I = decltype(i)::value;
          multiply_row(i, H, now);
          fence_schedule();
          unrolled<kLoads>([&](auto q) {
            constexpr int Q = I * kLoads + decltype(q)::value;
            if constexpr (Q < LC + LR) load_one(std::integral_constant<int, Q>{}, h);
          });
          unrolled<kReads>([&](auto q) {
            constexpr int Q = I * kReads + decltype(q)::value;
            if constexpr (Q < TC + TR) read_one(std::integral_constant<int, Q>{}, std::integral_constant<int, H ^ 1>{});
          });
          fence_schedule();
        });
        turn_over();
      });
      now = next;
      loaded();
    }

    if (way_out<BC, BR, WC, WR, uint16_t>(p, cur, lane, wc, wr, acc)) stored = 2;
  }
  // the last loads may still be on their way into this workgroup's LDS
  asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
}

// fp32 results.  Converting two codes takes a SIMD 16 cycles, half of what a matrix instruction of 32 x 32 x 16 does, so a
// code is widened once a workgroup, on its way into LDS: from memory into registers, a half of 64 k ahead, and from there,
// times its scale, into the bf16 half that is multiplied next.  Two halves in LDS and a barrier a half.  (Widened by every
// wave that multiplies it: 1103 us at 8192^3, as here 809, 1.4 PFLOP/s; with tiles of 128 x 128, whose fragments
// are read more often, 1031 to 1057.)
// A thread has 16 codes of two of C's rows and of two of R's; rows lie in LDS as above, 128 bytes each, their chunks of
// 16 bytes xor-ed with a key of the row: bits 1 to 3, so that 16 lanes that read one chunk of 16 rows find them on other
// banks, and bit 0 once more, so that 8 lanes that write every other chunk of two rows do (counter: no conflicts; without
// bit 0 8 cycles for every write, 1 to 4 % of the kernel: dweight of 8192 x 1536 x 768 33.5 us, as here 32.5).
__device__ __forceinline__ int fine_key(int row) { return (row / 2 % 8) ^ (row % 2); }
template <int B, int WC, int WR, bool SQUARE>
__global__ __launch_bounds__(WC * WR * 64, 2) void fine_product_kernel(Fp8Params p) {
  constexpr int TC = B / WC / 32, TR = B / WR / 32;
  constexpr int kRows = WC * WR * kLanes / 4;          // that threads have of either matrix at a time
  static_assert(B == 2 * kRows, "two rows of either a thread");
  constexpr int kLine = kBlock;                        // bytes of a row of half a step in bf16
  constexpr int kMatrix = B * kLine, kBuffer = 2 * kMatrix;
  __shared__ __attribute__((aligned(16))) unsigned char lds[2 * kBuffer];
  const int lane = threadIdx.x % kLanes;
  const int w = __builtin_amdgcn_readfirstlane(threadIdx.x / kLanes);
  const int wc = w / WR, wr = w % WR;
  const Jobs<B, B> jobs(p);

  const int lrow = threadIdx.x / 4, part = threadIdx.x % 4;   // rows lrow and lrow + kRows of either, codes 16 part on
  int ljob = jobs.first, lleft = 0;
  const unsigned char *lc = nullptr, *lr = nullptr, *lcs = nullptr, *lrs = nullptr;
  uint32_t off[4], soff[4];   // C's rows, R's
  auto start_load = [&]() {   // the next job with steps, if there is one; else the last loads are repeated
    while (ljob < jobs.end) {
      const Job j = jobs.at(ljob);
      if (j.steps > 0) {
        lleft = j.steps;
        const int64_t left_c = p.cols - j.c0 - 1, left_r = p.rows - j.r0 - 1;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const int at = h * kRows + lrow, i = at % 32;
          const int c = at / (32 * TC) * (32 * TC) + (i % 16 * 2 + i / 16) * TC + at / 32 % TC;
          const int r = at / (32 * TR) * (32 * TR) + i * TR + at / 32 % TR;
          const int cc = c < left_c ? c : static_cast<int>(left_c), rr = r < left_r ? r : static_cast<int>(left_r);
          off[h] = static_cast<uint32_t>(cc) * static_cast<uint32_t>(p.pitch) + part * 16;       // (pitch <= 2^22)
          off[2 + h] = static_cast<uint32_t>(rr) * static_cast<uint32_t>(p.pitch) + part * 16;
          soff[h] = SQUARE ? cc / kBlock : cc;
          soff[2 + h] = rr;
          asm volatile("" : "+v"(soff[h]));   // (a load known to be the same for all lanes would be waited for at once)
        }
        lc = p.c + static_cast<int64_t>(j.c0) * p.pitch + j.begin * kBlock;
        lr = p.r + static_cast<int64_t>(j.r0) * p.pitch + j.begin * kBlock;
        lcs = p.cs + j.begin * p.c_lines + (SQUARE ? j.c0 / kBlock : j.c0);
        lrs = p.rs + j.begin * p.r_lines + j.r0;
        return;
      }
      ljob += jobs.stride;
    }
  };
  u32x4_t codes[4];
  uint32_t scales[4];
  auto load_one = [&](int m, int h) {
    const unsigned char* const from = m < 2 ? lc : lr;
    codes[m] = *reinterpret_cast<const u32x4_t*>(from + off[m] + h * (kBlock / 2));
  };
  auto load_scale = [&](int m) { scales[m] = (m < 2 ? lcs : lrs)[soff[m]]; };
  auto loaded = [&]() {   // after a step's last load
    if (lleft > 1) {
      --lleft;
      lc += kBlock;
      lr += kBlock;
      lcs += p.c_lines;
      lrs += p.r_lines;
    } else if (ljob < jobs.end) {
      ljob += jobs.stride;
      start_load();
    }
  };
  unsigned char* const put_at = lds + lrow * kLine + (((part * 2) ^ fine_key(lrow)) << 4);
  const int put_next = (((part * 2 + 1) ^ fine_key(lrow)) << 4) - (((part * 2) ^ fine_key(lrow)) << 4);
  auto widen_one = [&](int m, int h) {   // codes[m] to half h
    const float s = fp8_power(scales[m]);
    unsigned char* const to = put_at + h * kBuffer + m / 2 * kMatrix + m % 2 * kRows * kLine;
    *reinterpret_cast<bf16x8_t*>(to) = wide_codes(codes[m][0], codes[m][1], s);
    *reinterpret_cast<bf16x8_t*>(to + put_next) = wide_codes(codes[m][2], codes[m][3], s);
  };
  const unsigned char *fc_at[4], *fr_at[4];   // fragments of 16 k
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    const int at = lane % 32 * kLine + (((2 * q + lane / 32) ^ fine_key(lane)) << 4);
    fc_at[q] = lds + wc * (32 * TC * kLine) + at;
    fr_at[q] = lds + kMatrix + wr * (32 * TR * kLine) + at;
  }
  f32x16_t acc[TC][TR];
  bf16x8_t fc[2][TC], fr[2][TR];
  auto read = [&](int q, int h) {
#pragma unroll
    for (int t = 0; t < TR; ++t) fr[q % 2][t] = *reinterpret_cast<const bf16x8_t*>(fr_at[q] + h * kBuffer + t * 32 * kLine);
#pragma unroll
    for (int t = 0; t < TC; ++t) fc[q % 2][t] = *reinterpret_cast<const bf16x8_t*>(fc_at[q] + h * kBuffer + t * 32 * kLine);
  };
  auto meet = [&]() {
    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
  };

  start_load();
  if (lleft > 0) {
#pragma unroll
    for (int m = 0; m < 4; ++m) {
      load_one(m, 0);
      load_scale(m);
    }
#pragma unroll
    for (int m = 0; m < 4; ++m) {
      widen_one(m, 0);
      load_one(m, 1);
    }
    meet();
  }
  for (int job = jobs.first; job < jobs.end; job += jobs.stride) {
    const Job cur = jobs.at(job);
#pragma unroll
    for (int i = 0; i < TC; ++i)
#pragma unroll
      for (int j = 0; j < TR; ++j) acc[i][j] = f32x16_t{};
    for (int s = 0; s < cur.steps; ++s) {
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        // in registers: step s's second half while its first is multiplied, the next step's first half then
        if (h == 0) loaded();
        read(0, h);
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          if (q < 3) read(q + 1, h);
          widen_one(q, h ^ 1);
          load_one(q, h);
          if (h == 0) load_scale(q);
#pragma unroll
          for (int c = 0; c < TC; ++c)
#pragma unroll
            for (int r = 0; r < TR; ++r)
              acc[c][r] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(fr[q % 2][r], fc[q % 2][c], acc[c][r], 0, 0, 0);
          fence_schedule();
        }
        meet();
      }
    }
    way_out<B, B, WC, WR, float>(p, cur, lane, wc, wr, acc);
  }
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

// ------------------------------------------------------------------------------------------- few rows
// For up to some hundred rows the time goes into C's bytes and into latency, not into multiplications.  A workgroup owns
// a tile of 16 CT x 16 RT; its 8 waves take k's blocks in turn, the operands straight from global memory (C's bytes serve
// once, R's come from the L2), and their sums are added in LDS in the waves' order, a thread 8 neighbouring elements.  No
// barrier and no wait for another wave before that.  What hides a load's latency are the other waves: a wave that had
// several blocks on their way at a time was no faster or slower (8 x 2560 x 20480: 13.5 us, with four blocks, of which the
// last ones are often past the end, 22; 64 x 2560 x 5120: 12.3, two blocks 12.9).
// As above, row i of tile t is row CT i + t of C's 16 CT and RT i + t of R's.
// X: R's type, E4m3 or a plain one for up to 16 rows that fit into LDS in 8 bits: each workgroup rounds them again while
// its first loads of C are on their way, which saves a launch (1 x 2560 x 10240: 7.1 us of the GPU, 26 MB; with each lane
// rounding its own operands 20).
template <int N> __device__ __forceinline__ uint32_t scales_at(const unsigned char* at) {
  if constexpr (N == 4) return *reinterpret_cast<const uint32_t*>(at);
  else if constexpr (N == 2) return *reinterpret_cast<const uint16_t*>(at);
  else return *at;
}
// a lane's 32 codes of a row's block: 16 of either half, so that a load's four lanes of a row read 64 bytes on end (which k
// a lane holds does not matter as long as both sides agree: the scales are the same for all of the block)
__device__ __forceinline__ i32x8_t codes_at(const unsigned char* p) {
  const u32x4_t a = *reinterpret_cast<const u32x4_t*>(p), b = *reinterpret_cast<const u32x4_t*>(p + 64);
  return i32x8_t{static_cast<int>(a[0]), static_cast<int>(a[1]), static_cast<int>(a[2]), static_cast<int>(a[3]),
                 static_cast<int>(b[0]), static_cast<int>(b[1]), static_cast<int>(b[2]), static_cast<int>(b[3])};
}

template <int CT, int RT, int NW> struct FewShared {
  float sums[NW][16 * RT][16 * CT + 4];   // a row off the banks of the next
};

// workgroup `group`
template <int CT, int RT, int NW, typename X, typename T>
__device__ __forceinline__ void few_product(const Fp8Params& p, unsigned group, FewShared<CT, RT, NW>& shared) {
  constexpr bool kFine = std::is_same_v<T, float>, kPlain = !std::is_same_v<X, E4m3>;
  static_assert(!kPlain || RT == 1, "up to 16 plain rows");
  constexpr int kC = 16 * CT, kR = 16 * RT;
  auto& sums = shared.sums;
  extern __shared__ __attribute__((aligned(16))) unsigned char plain[];   // [rows][pitch + 16], [rows][blocks] scales
  const int lane = threadIdx.x % kLanes, w = __builtin_amdgcn_readfirstlane(threadIdx.x / kLanes);
  const int i16 = lane % 16, part = lane / 16;
  const int64_t c0 = static_cast<int64_t>(group % p.tiles_c) * kC, r0 = static_cast<int64_t>(group / p.tiles_c) * kR;
  const unsigned char *ca[CT], *ra[RT];
#pragma unroll
  for (int t = 0; t < CT; ++t) {
    const int64_t c = c0 + i16 * CT + t;
    ca[t] = p.c + (c < p.cols ? c : p.cols - 1) * p.pitch + part * 16;
  }
#pragma unroll
  for (int t = 0; t < RT; ++t) {
    const int64_t r = r0 + i16 * RT + t, row = r < p.rows ? r : p.rows - 1;
    ra[t] = kPlain ? plain + row * (p.pitch + 16) + part * 16 : p.r + row * p.pitch + part * 16;
  }
  const int64_t cs = p.square ? c0 / kBlock : c0 + i16 * CT < p.c_lines - CT ? c0 + i16 * CT : p.c_lines - CT;
  const int64_t rs = r0 + i16 * RT < p.r_lines - RT ? r0 + i16 * RT : p.r_lines - RT;
  struct Step {
    i32x8_t c[CT], r[RT];
    uint32_t sc, sr;
  };
  auto load_c = [&](int s, Step& v) {
#pragma unroll
    for (int t = 0; t < CT; ++t) v.c[t] = codes_at(ca[t] + static_cast<int64_t>(s) * kBlock);
    v.sc = p.square ? p.cs[s * p.c_lines + cs] * 0x01010101u : scales_at<CT>(p.cs + s * p.c_lines + cs);
  };
  auto load_r = [&](int s, Step& v) {
#pragma unroll
    for (int t = 0; t < RT; ++t) v.r[t] = codes_at(ra[t] + static_cast<int64_t>(s) * kBlock);
    if constexpr (kPlain) v.sr = plain[p.rows * (p.pitch + 16) + (i16 < p.rows ? i16 : p.rows - 1) * p.steps + s];
    else v.sr = scales_at<RT>(p.rs + s * p.r_lines + rs);
  };
  f32x4_t acc[CT][RT] = {};
  auto multiply = [&](const Step& v) {
    if constexpr (kFine) {
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        bf16x8_t b[RT];
#pragma unroll
        for (int r = 0; r < RT; ++r) b[r] = wide_codes(v.r[r][2 * q], v.r[r][2 * q + 1], fp8_power((v.sr >> (8 * r)) & 255u));
#pragma unroll
        for (int c = 0; c < CT; ++c) {
          const bf16x8_t a = wide_codes(v.c[c][2 * q], v.c[c][2 * q + 1], fp8_power((v.sc >> (8 * c)) & 255u));
#pragma unroll
          for (int r = 0; r < RT; ++r) acc[c][r] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b[r], acc[c][r], 0, 0, 0);
        }
      }
    } else {
      unrolled<CT>([&](auto c) {
        unrolled<RT>([&](auto r) {
          constexpr int C = decltype(c)::value, R = decltype(r)::value;
          acc[C][R] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(v.c[C], v.r[R], acc[C][R], 0, 0, C,
                                                                       static_cast<int>(v.sc), R, static_cast<int>(v.sr));
        });
      });
    }
  };
  Step v;
  if (w < p.steps) load_c(w, v);
  if constexpr (kPlain) {
    const int work = static_cast<int>(p.rows) * p.steps;
    for (int i = threadIdx.x / 16; i < work; i += NW * 4) {   // 16 lanes a block
      const int r = i / p.steps, b = i - r * p.steps, at = b * kBlock + i16 * 8;
      float x[8];
      load_row<8>(reinterpret_cast<const X*>(p.r) + r * p.k + at, x, p.k - at);
      uint32_t scale;
      *reinterpret_cast<u32x2_t*>(plain + r * (p.pitch + 16) + at) = fp8_block_codes(x, scale);
      if (i16 == 0) plain[p.rows * (p.pitch + 16) + i] = static_cast<unsigned char>(scale);
    }
    __syncthreads();
  }
  for (int s = w; s < p.steps; s += NW) {
    if (s != w) load_c(s, v);
    load_r(s, v);
    multiply(v);
  }
  // accumulator e of tile (i, j): C's row CT (4 part + e) + i and R's row RT i16 + j
#pragma unroll
  for (int j = 0; j < RT; ++j)
#pragma unroll
    for (int q = 0; q < CT; ++q) {
      f32x4_t v;
#pragma unroll
      for (int e = 0; e < 4; ++e) v[e] = acc[(4 * q + e) % CT][j][(4 * q + e) / CT];
      *reinterpret_cast<f32x4_t*>(&sums[w][i16 * RT + j][part * 4 * CT + 4 * q]) = v;
    }
  __syncthreads();
  constexpr int kRuns = kC / 8;
  for (int i = threadIdx.x; i < kR * kRuns; i += NW * kLanes) {
    const int r = i / kRuns, c = i % kRuns * 8;
    const int64_t row = r0 + r, left = p.cols - c0 - c;
    if (row >= p.rows || left <= 0) continue;
    float v[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = sums[0][r][c + e];
#pragma unroll
    for (int k = 1; k < NW; ++k)
#pragma unroll
      for (int e = 0; e < 8; ++e) v[e] += sums[k][r][c + e];
    put(static_cast<T*>(p.out) + row * p.cols + c0 + c, v, left, p.accumulate);
  }
}

template <int CT, int RT, int NW, typename X, typename T>
__global__ __launch_bounds__(NW * 64, CT * RT == 1 ? 4 : 2) void few_product_kernel(Fp8Params p) {
  __shared__ __attribute__((aligned(16))) FewShared<CT, RT, NW> shared;
  few_product<CT, RT, NW, X, T>(p, blockIdx.x, shared);
}
// two products side by side: the first `split` workgroups have the first
template <int CT, int RT, int NW, typename X, typename T>
__global__ __launch_bounds__(NW * 64, CT * RT == 1 ? 4 : 2) void two_products_kernel(Fp8Params p, Fp8Params q, unsigned split) {
  __shared__ __attribute__((aligned(16))) FewShared<CT, RT, NW> shared;
  const bool first = blockIdx.x < split;
  few_product<CT, RT, NW, X, T>(first ? p : q, first ? blockIdx.x : blockIdx.x - split, shared);
}

// ---------------------------------------------------------------------------------------------- plan
enum Kind { kLarge, kSmall, kFew64, kFew64x32, kFew32, kFew16 };   // (few: columns x rows of a tile)

struct Tiling {
  Kind kind;
  int bc, br;              // tile
  int grid;                // workgroups
  int64_t tiles;
  int whole, slices;
  int64_t cost;            // nanoseconds, as the measurements below have it
};

constexpr int kCus = 256;
constexpr int kMostSlices = 32;

// Tiles on workgroups that stay.  one, two: nanoseconds of a step with one and with two workgroups on a CU; round: of a
// tile's way out.  Slices of the last, partial round: those that take the least time, with 3 us for the second launch and
// the sums' way through memory (measured: 0.45 to 0.5 us a MB; 256 x 5120 x 2560 18.8 us in four slices, 21.2 on 64 x
// 64).  At most two rounds of slices, which bounds the sums' memory.
Tiling tiling(const Fp8ProductArgs& a, Kind kind, int side, int grid, int64_t one, int64_t two, int64_t round, int64_t mb) {
  Tiling t{kind, side, side, grid, 0, 0, 1, 0};
  const int64_t tiles_r = (a.rows + side - 1) / side, steps = fp8_blocks(a.k);
  t.tiles = (a.cols + side - 1) / side * tiles_r;
  const int64_t rest = t.tiles % grid, whole = t.tiles / grid;
  const int64_t sums = (a.rows + tiles_r - 1) / tiles_r * side * 4;     // bytes of a slice's sums
  int64_t best = 0;
  for (int64_t s = 1; rest > 0 && s <= kMostSlices && (s == 1 || (rest * s <= 2 * grid && steps / s >= 2)); ++s) {
    const int64_t n = rest * s, each = (steps + s - 1) / s;
    int64_t time = round + (n <= kCus ? each * one : (n + grid - 1) / grid * each * two);
    if (s > 1) time += 3000 + (n * sums * mb >> 20);
    if (s == 1 || time < best) {
      best = time;
      t.slices = static_cast<int>(s);
    }
  }
  t.whole = static_cast<int>(t.tiles - rest);
  t.cost = 3000 + whole * (steps * two + round) + best;
  return t;
}

// Waves of the kernel for few rows (64 x 2560 x 5120 on tiles of 64 x 64: fp32, where widening the codes is most of the
// work, 14.5 us with eight and 19.6 with four; bf16 12.3 and 12.7).
constexpr int kFewWaves = 8;
constexpr int kFewRows = 16;   // up to here one row of tiles of 16 x 16, and rows may be plain

// A workgroup to a tile whose waves share k.  A workgroup on every CU takes one block of each wave in the time that stands
// with each tile: the smaller tiles fill the chip where there are few, the larger ones read less (bf16: 32 x 2560 x 5120
// 9.3, 7.1, 9.3 and 10.9 us on tiles of 16 x 16, 32 x 32, 64 x 32 and 64 x 64; 64 x 2560 x 5120 13.9, 11.5, 9.4 and 12.6;
// 300 x 2560 x 2560 29.5, 19.3, 16.1 and 12.8; fp32 within a twentieth of that).
Tiling few(const Fp8ProductArgs& a, Kind kind) {
  struct Few {
    int bc, br;
    int64_t block;   // nanoseconds
  };
  constexpr Few kFews[] = {{64, 64, 3500}, {64, 32, 2400}, {32, 32, 1600}, {16, 16, 800}};
  const Few& f = kFews[kind - kFew64];
  Tiling t{kind, f.bc, f.br, 0, 0, 0, 1, 0};
  t.tiles = ((a.cols + f.bc - 1) / f.bc) * ((a.rows + f.br - 1) / f.br);
  const int64_t blocks = (fp8_blocks(a.k) + kFewWaves - 1) / kFewWaves;
  t.cost = 2200 + blocks * ((t.tiles + kCus - 1) / kCus) * f.block;
  constexpr int kMostGrid = 1 << 20;   // (more are also slower than on workgroups that stay)
  if (t.tiles > kMostGrid) t.cost = std::numeric_limits<int64_t>::max();
  t.grid = static_cast<int>(t.tiles < kMostGrid ? t.tiles : kMostGrid);
  return t;
}
// go(CT, RT) of a kind's kernel
template <typename F> void with_few(Kind kind, F&& go) {
  using One = std::integral_constant<int, 1>;
  using Two = std::integral_constant<int, 2>;
  using Four = std::integral_constant<int, 4>;
  if (kind == kFew64) go(Four{}, Four{});
  else if (kind == kFew64x32) go(Four{}, Two{});
  else if (kind == kFew32) go(Two{}, Two{});
  else go(One{}, One{});
}

// The least time by what the kernels took (a step of 256 x 256 1.5 us, of 128 x 128 0.6 with one and 1.13 with two
// workgroups on a CU; with fp32 results 3.1, 1.1 and 2.0): for instance, bf16: 8 x 5120 x 2560 5.9 us on tiles of 16 x 16
// (11 on 128 x 128), 1001 x 1000 x 777 7.3 on 64 x 64 (8.5), 128 x 5120 x 2560 15.8 on 128 x 128 in four slices (27.4
// unsliced, 21 on 64 x 64), 16384 x 10240 x 2560 383 on 256 x 256 (530 on 128 x 128); fp32: 4096 x 1536 x 768 17.8 on 128 x
// 128, 34.5 on 256 x 256, and 4096^3 138 and 108.
// No k: zeros, which the workgroups that stay write without a load.
Tiling pick(const Fp8ProductArgs& a) {
  if (a.k == 0) return tiling(a, kSmall, 128, 2 * kCus, 0, 0, 2000, 0);
  Tiling best = few(a, kFew16);
  if (a.rows <= kFewRows) return best;
  auto or_this = [&](const Tiling& t) {
    if (t.cost < best.cost) best = t;
  };
  or_this(few(a, kFew32));
  or_this(few(a, kFew64x32));
  or_this(few(a, kFew64));
  or_this(a.out_io ? tiling(a, kSmall, 128, 2 * kCus, 600, 1130, 2000, 450)
                   : tiling(a, kSmall, 128, 2 * kCus, 1100, 2000, 2000, 450));
  or_this(a.out_io ? tiling(a, kLarge, 256, kCus, 1500, 1600, 4000, 500)
                   : tiling(a, kLarge, 256, kCus, 3000, 3200, 6000, 500));
  return best;
}

}  // namespace

// LDS that plain rows take in 8 bits, and how much of it leaves room for four workgroups on a CU: each rounds all the rows
// again, where a launch of its own rounds them once (bf16, rounded on the way and before: 8 x 2560 x 10240, 21 KB, 10.8 and
// 12.7 us; 16 x 1280 x 10240, 21 KB, 9.4 and 9.8; 16 x 1536 x 10240, 25 KB, 10.8 and 10.7; 16 x 2560 x 10240, 42 KB, 15.5 and
// 13.4; 2560 columns 5.9 and 7.8, 5.0 and 6.5, 5.6 and 6.8, 8.1 and 7.9; fp32 alike)
int64_t plain_bytes(const Fp8ProductArgs& a) { return a.rows * (fp8_blocks(a.k) * (kBlock + 1) + 16); }
constexpr int64_t kMostPlain = 24 << 10;

bool fp8_product_takes_plain(const Fp8ProductArgs& a) { return a.rows <= kFewRows && plain_bytes(a) <= kMostPlain; }

size_t fp8_product_workspace_bytes(const Fp8ProductArgs& a) {
  if (a.rows == 0 || a.cols == 0) return 0;
  const Tiling t = pick(a);
  return t.slices > 1 ? static_cast<size_t>(t.tiles - t.whole) * t.slices * t.bc * t.br * 4 : 0;
}

namespace {
Fp8Params params(const Fp8ProductArgs& a, const Tiling& t) {
  Fp8Params p{};
  p.r = static_cast<const unsigned char*>(a.r.codes); p.rs = static_cast<const unsigned char*>(a.r.scales);
  p.c = static_cast<const unsigned char*>(a.c.codes); p.cs = static_cast<const unsigned char*>(a.c.scales);
  p.rows = a.rows; p.cols = a.cols; p.k = a.k; p.square = a.square;
  p.steps = static_cast<int>(fp8_blocks(a.k)); p.pitch = fp8_blocks(a.k) * kBlock;
  p.r_lines = fp8_lines(a.rows); p.c_lines = a.square ? fp8_blocks(a.cols) : fp8_lines(a.cols);
  p.out = a.out; p.accumulate = a.accumulate;
  p.tiles_c = static_cast<int>((a.cols + t.bc - 1) / t.bc); p.tiles_r = static_cast<int>((a.rows + t.br - 1) / t.br);
  p.whole = t.whole; p.slices = t.slices; p.sums = static_cast<float*>(a.workspace);
  return p;
}
}  // namespace

hipError_t fp8_two_products_launch(const Fp8ProductArgs& a, const Fp8ProductArgs& b, hipStream_t stream) {
  if (a.rows > 0 && a.cols > 0 && b.rows > 0 && b.cols > 0 && a.out_io == b.out_io) {
    const Tiling t = pick(a), u = pick(b);
    if (t.kind == u.kind && t.kind >= kFew64) {
      const Fp8Params p = params(a, t), q = params(b, u);
      auto go = [&](auto out) {
        using T = decltype(out);
        with_few(t.kind, [&](auto ct, auto rt) {
          two_products_kernel<ct, rt, kFewWaves, E4m3, T>
              <<<dim3(static_cast<unsigned>(t.grid + u.grid)), kFewWaves * kLanes, 0, stream>>>(p, q, t.grid);
        });
      };
      if (a.out_io) go(uint16_t{});
      else go(float{});
      return hipGetLastError();
    }
  }
  const hipError_t e = fp8_product_launch(a, stream);
  return e == hipSuccess ? fp8_product_launch(b, stream) : e;
}

hipError_t fp8_product_launch(const Fp8ProductArgs& a, hipStream_t stream) {
  if (a.rows == 0 || a.cols == 0 || (a.k == 0 && a.accumulate)) return hipSuccess;
  const Tiling t = pick(a);
  if (a.plain && (!fp8_product_takes_plain(a) || t.kind != kFew16)) return hipErrorInvalidValue;
  const Fp8Params p = params(a, t);
  const dim3 grid(static_cast<unsigned>(t.grid)), sum_grid(static_cast<unsigned>((t.tiles - t.whole) * kShares));
  auto go = [&](auto out) {
    using T = decltype(out);
    switch (t.kind) {
      case kLarge:
        if constexpr (std::is_same_v<T, uint16_t>) {
          if (p.square) tile_product_kernel<256, 256, 2, 4, true><<<grid, 512, 0, stream>>>(p);
          else tile_product_kernel<256, 256, 2, 4, false><<<grid, 512, 0, stream>>>(p);
        } else {
          if (p.square) fine_product_kernel<256, 4, 2, true><<<grid, 512, 0, stream>>>(p);
          else fine_product_kernel<256, 4, 2, false><<<grid, 512, 0, stream>>>(p);
        }
        if (t.slices > 1) slices_kernel<256, 256, T><<<sum_grid, 256, 0, stream>>>(p);
        break;
      case kSmall:
        if constexpr (std::is_same_v<T, uint16_t>) {
          if (p.square) tile_product_kernel<128, 128, 2, 2, true><<<grid, 256, 0, stream>>>(p);
          else tile_product_kernel<128, 128, 2, 2, false><<<grid, 256, 0, stream>>>(p);
        } else {
          if (p.square) fine_product_kernel<128, 2, 2, true><<<grid, 256, 0, stream>>>(p);
          else fine_product_kernel<128, 2, 2, false><<<grid, 256, 0, stream>>>(p);
        }
        if (t.slices > 1) slices_kernel<128, 128, T><<<sum_grid, 256, 0, stream>>>(p);
        break;
      default:
        if (a.plain) {
          if (a.r_io) few_product_kernel<1, 1, kFewWaves, uint16_t, T><<<grid, kFewWaves * kLanes, plain_bytes(a), stream>>>(p);
          else few_product_kernel<1, 1, kFewWaves, float, T><<<grid, kFewWaves * kLanes, plain_bytes(a), stream>>>(p);
        } else {
          with_few(t.kind, [&](auto ct, auto rt) {
            few_product_kernel<ct, rt, kFewWaves, E4m3, T><<<grid, kFewWaves * kLanes, 0, stream>>>(p);
          });
        }
        break;
    }
  };
  if (a.out_io) go(uint16_t{});
  else go(float{});
  return hipGetLastError();
}

}  // namespace mssm
