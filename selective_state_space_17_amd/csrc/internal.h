// Internal declarations shared by the C-ABI front end and the kernel files.
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace mssm {

// ---------------------------------------------------------------------------
// Mamba-1 selective scan
// ---------------------------------------------------------------------------
struct ScanArgs {
  const void* x;
  const void* delta;
  const float* A;
  const void* B;
  const void* C;
  const float* D;       // nullable
  const void* z;        // nullable
  const float* h0;      // nullable
  void* out;
  float* final_state;   // nullable
  void* workspace;
  int64_t batch, L, dim, N;
  int io;               // 0 fp32, 1 bf16
  int K;                // sequence chunks
  int G;                // lanes per channel
  // optional short causal convolution + SiLU in front of the scan; x is then
  // its input (needs G == 16, N == 16 and 16-byte aligned I/O)
  const float* conv_w = nullptr;     // [dim, conv_width]
  const float* conv_b = nullptr;     // [dim], nullable
  const void* conv_init = nullptr;   // [batch, conv_width - 1, dim], nullable
  int conv_width = 0;
  // optional training-mode output: the state entering every 16-step tile,
  // [batch][ceil(L/16)][16 * ceil(dim/16)][16] fp32 (needs G == 16, N == 16)
  float* ckpt = nullptr;
};

// bytes of the checkpoint array the training-mode forward writes and the gradients read
size_t scan_checkpoint_bytes(int64_t batch, int64_t L, int64_t dim);


// Workspace layout for K > 1 (all fp32 / int32, 256-byte aligned blocks):
//   hend [batch][K][dim][N]  state at each chunk's end (chunk 0: true; others: from zero)
//   hin  [batch][K][dim][N]  true state entering each chunk
//   S    [batch][K][dim]     sum of delta over each chunk
//   neg  [batch][K][dim]     chunk contained a negative delta
size_t scan_workspace_bytes(int64_t batch, int64_t dim, int64_t N, int K);

// Enqueue the scan; returns hipSuccess or the launch error.
hipError_t scan_launch(const ScanArgs& a, hipStream_t stream);

// lanes-per-channel values the kernels are built for
bool scan_supported_G(int G, int64_t N);

// Fixed per-device scratch of the entry point that allocates nothing: its size, and its
// address on the device of `stream` (looked up once per device, then kept).
constexpr size_t kScratchBytes = size_t{32} << 20;
hipError_t scratch_address(hipStream_t stream, void** out);

// ---------------------------------------------------------------------------
// Mamba-2 scalar-A multi-head (SSD) form
// ---------------------------------------------------------------------------
struct SSDArgs {
  const void* x;
  const void* delta;
  const void* lam;   // nullable: the Mamba-2 rule; else the Mamba-3 exponential-trapezoidal rule
  const float* A;
  const void* B;
  const void* C;
  const float* D;
  const void* z;
  const float* h0;
  void* out;
  float* final_state;
  void* workspace;
  int64_t batch, L, H, P, N, G, Q;
  int64_t R = 1;   // inputs and outputs per channel (MIMO); x, z, out [B, L, H, R, P], B, C [B, L, G, R, N]
};

size_t ssd_workspace_bytes(int64_t batch, int64_t L, int64_t H, int64_t P, int64_t N, int64_t G, int64_t Q);
// headdim and dstate the matrix-core block kernel takes (bf16 I/O), and the MIMO ranks
bool ssd_supported(int64_t P, int64_t N);
bool ssd_rank_supported(int64_t R);
hipError_t ssd_launch(const SSDArgs& a, hipStream_t stream);

// ---------------------------------------------------------------------------
// Token-by-token state update (both forms), state read and written in place
// ---------------------------------------------------------------------------
struct UpdateArgs {
  float* state;
  const void* x;
  const void* delta;
  const float* A;
  const void* B;
  const void* C;
  const float* D;       // nullable
  const void* z;        // nullable
  void* out;
  int64_t batch, L, N;
  int64_t dim;          // Mamba-1
  int64_t H, P, G;      // multi-head form
  int io;               // 0 fp32, 1 bf16
  // Mamba-1 only: short causal convolution in front, x being its input
  const float* conv_w = nullptr;   // [dim, conv_width]
  const float* conv_b = nullptr;   // [dim], nullable
  void* conv_state = nullptr;      // [batch, conv_width - 1, dim], read and advanced in place
  const void* conv_in = nullptr;   // with conv_state == nullptr: the window before the first token (nullable)
  void* conv_out = nullptr;        // and the window after the last (nullable: not written)
  int conv_width = 0;
  // multi-head form only: the Mamba-3 exponential-trapezoidal rule
  const void* lam = nullptr;       // [batch, L, H]; nullable = the Mamba-2 rule
  const void* x_prev = nullptr;    // [batch, H, P], the token before the first one; nullable = none
  const void* B_prev = nullptr;    // [batch, G, N], likewise
  const float* omega = nullptr;    // [H, N/2] rotation rates of the state pairs (complex state); nullable
  int64_t rank = 1;                // MIMO inputs and outputs per channel (x, z, out [.., H, rank, P],
                                   // B, C [.., G, rank, N]); > 1 takes no omega
  // with state == nullptr: the state before the first token (nullable: zero) and the one written
  // after the last (nullable: not written), for a whole sequence run through the update kernel
  const float* state_in = nullptr;
  float* state_out = nullptr;
};

hipError_t scan_update_launch(const UpdateArgs& a, hipStream_t stream);
hipError_t ssd_update_launch(const UpdateArgs& a, hipStream_t stream);
// blocks the update kernels launch for `rows` state rows of N states
int64_t update_grid_blocks(int64_t rows, int64_t N);

// ---------------------------------------------------------------------------
// Gradients of the Mamba-1 selective scan (dstate <= 16)
// ---------------------------------------------------------------------------
struct ScanBwdArgs {
  const void* x;
  const void* delta;
  const float* A;
  const void* B;
  const void* C;
  const float* D;       // nullable
  const void* z;        // nullable
  const float* h0;      // nullable
  const void* dout;
  const float* dfinal;  // nullable
  void* dx;
  void* ddelta;
  float* dA;
  float* dB;
  float* dC;
  float* dD;            // written iff D != nullptr
  void* dz;             // written iff z != nullptr
  float* dh0;           // nullable
  const float* ckpt_in = nullptr;   // nullable: checkpoints from the training-mode forward
  void* workspace;
  int64_t batch, L, dim, N;
  int io;
};

// workspace: per-tile state checkpoints, per-block dB/dC partials, per-row dA/dD partials
size_t scan_bwd_workspace_bytes(int64_t batch, int64_t L, int64_t dim, int64_t N);
// blocks of the main gradient kernel
int64_t scan_bwd_grid_blocks(int64_t batch, int64_t dim, int64_t N);
hipError_t scan_bwd_launch(const ScanBwdArgs& a, hipStream_t stream);

// ---------------------------------------------------------------------------
// Around the scan: embedding, norm, loss
// ---------------------------------------------------------------------------
struct EmbedArgs {
  const void* ids;
  int id_bytes;          // 4 or 8
  float scale;
  int64_t tokens, vocab, dim;
  int io;                // 0 fp32, 1 bf16
  const void* weight;    // lookup
  void* out;
  const void* dout;      // gradient
  void* dweight;
  int grad_io;           // dweight in the io type; else fp32
  int accumulate;
  void* workspace;
};

hipError_t embed_fwd_launch(const EmbedArgs& a, hipStream_t stream);
// workspace: the tokens sorted by id (two buffers of pairs), digit counts, sums of runs that cross slices
size_t embed_bwd_workspace_bytes(int64_t tokens, int64_t vocab, int64_t dim);
hipError_t embed_bwd_launch(const EmbedArgs& a, hipStream_t stream);

struct NormArgs {
  int64_t rows, dim;
  float eps;
  int layer;             // 1 layer norm, 0 RMS norm
  int io, res_io;        // 0 fp32, 1 bf16: x, out, dout, dx; residual stream (backward: h, dresidual)
  const void* x;
  const void* residual;  // nullable
  const float* weight;
  const float* bias;     // nullable
  void* out;
  void* residual_out;    // nullable
  float* mean;           // forward: nullable output; backward: input (layer norm)
  float* rstd;           // forward: nullable output; backward: input
  const void* h;
  const void* dout;
  const void* dresidual;   // nullable
  void* dx;                // nullable
  void* dresidual_in;      // nullable
  float* dweight;
  float* dbias;            // nullable
  void* workspace;
  void* codes;             // forward: out in 8 bits instead of `out`, with scales
  void* scales;
};

hipError_t norm_fwd_launch(const NormArgs& a, hipStream_t stream);
// workspace: partial sums of dweight and dbias
size_t norm_bwd_workspace_bytes(int64_t rows, int64_t dim);
hipError_t norm_bwd_launch(const NormArgs& a, hipStream_t stream);

struct XentArgs {
  int64_t tokens, vocab, dim;
  int64_t ignore;
  int io;                // 0 fp32, 1 bf16
  int fine_g;            // bf16: the logits' gradient in two terms whatever the tokens
  int id_bytes;          // 4 or 8
  const void* x;
  const void* weight;
  const void* targets;
  float* loss;           // forward
  float* lse;
  const float* lse_in;   // gradients
  const float* dloss;
  const float* dlse;     // nullable
  void* dx;              // nullable
  void* dweight;         // nullable
  int grad_io;           // dweight in the io type; else fp32
  int accumulate;
  void* workspace;
};

// workspace: the counted tokens' x as the products read it, the forward's partial sums or a piece of the
// logits' gradient, and, where the weight cannot be read in place, a piece of it laid out
size_t xent_workspace_bytes(const XentArgs& a, bool grad);
hipError_t xent_fwd_launch(const XentArgs& a, hipStream_t stream);
hipError_t xent_bwd_launch(const XentArgs& a, hipStream_t stream);

// ---------------------------------------------------------------------------
// 8-bit linear layer
// ---------------------------------------------------------------------------
// a matrix in 8 bits (layout: fp8_util.h)
struct Fp8View {
  void* codes = nullptr;
  void* scales = nullptr;
};

struct Fp8Args {
  int64_t rows, cols;
  int io;                // x or out: 0 fp32, 1 bf16
  int square;            // blocks of 128 x 128 instead of 128 of a row
  const void* x;         // quantize: [rows, cols]
  void* out;             // dequantize: [rows, cols]
  Fp8View m;             // quantize: output, nullable; else input
  Fp8View t;             // the transposed matrix in 8 bits: output, nullable for quantize
};

hipError_t fp8_quantize_launch(const Fp8Args& a, hipStream_t stream);
hipError_t fp8_transpose_launch(const Fp8Args& a, hipStream_t stream);
hipError_t fp8_dequantize_launch(const Fp8Args& a, hipStream_t stream);
// the first to 8 bits and the second, of as many rows, laid out the other way, side by side
hipError_t fp8_both_launch(const Fp8Args& plain, const Fp8Args& packed, hipStream_t stream);

// out[r, c] (+)= sum over k of R[r, k] C[c, k]
struct Fp8ProductArgs {
  int64_t rows, cols, k;
  Fp8View r;             // row scales
  int plain;             // r.codes is a plain matrix (r_io: 0 fp32, 1 bf16) instead: only where fp8_product_takes_plain()
  int r_io;
  Fp8View c;
  int square;            // C's scales
  void* out;             // [rows, cols]
  int out_io;            // 0 fp32, 1 bf16
  int accumulate;
  void* workspace;
};

// whether R may be a plain matrix, which is then rounded on the way (the sizes decide)
bool fp8_product_takes_plain(const Fp8ProductArgs& a);
size_t fp8_product_workspace_bytes(const Fp8ProductArgs& a);
// (of no k: zeros, or with accumulate nothing; operands may then be null)
hipError_t fp8_product_launch(const Fp8ProductArgs& a, hipStream_t stream);
// one after the other (they may share a workspace), or side by side in one launch where either is small
hipError_t fp8_two_products_launch(const Fp8ProductArgs& a, const Fp8ProductArgs& b, hipStream_t stream);

}  // namespace mssm
