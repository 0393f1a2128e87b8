// C-ABI front end of the 8-bit linear layer: matrices in 8 bits, the norm that writes one, the product and its
// gradients.  Every check runs on the host before anything is enqueued.
#include "../../include/mssm.h"

#include "checks.h"
#include "fp8_util.h"
#include "internal.h"

using namespace mssm::checks;
using mssm::Fp8View;
using mssm::fp8_blocks;
using mssm::fp8_lines;

namespace {

// tile offsets are 32-bit: 256 rows of a matrix whose blocks run along the tokens
constexpr int64_t kMostRows = int64_t{1} << 22;
constexpr int64_t kMostCols = int64_t{1} << 20;

int64_t fp8_code_bytes(int64_t rows, int64_t cols) { return rows * fp8_blocks(cols) * mssm::kBlock; }
int64_t fp8_scale_bytes(int64_t rows, int64_t cols, bool square) {
  return fp8_blocks(cols) * (square ? fp8_blocks(rows) : fp8_lines(rows));
}
bool view_aligned(const void* codes, const void* scales) { return aligned(codes, 16) && aligned(scales, 4); }

int validate_matrix(const mssm_fp8_desc* d) {
  if (d == nullptr) return MSSM_ERR_INVALID_ARG;
  if (d->rows < 0 || d->cols <= 0 || d->flags != 0) return MSSM_ERR_INVALID_ARG;
  if (d->kind != MSSM_FP8_ROWS && d->kind != MSSM_FP8_SQUARE) return MSSM_ERR_INVALID_ARG;
  if (!io_ok(d->io_dtype)) return MSSM_ERR_UNSUPPORTED;
  if (d->rows > kMostRows || d->cols > kMostRows) return MSSM_ERR_UNSUPPORTED;
  return MSSM_OK;
}

mssm::Fp8Args matrix_args(const mssm_fp8_desc& d) {
  mssm::Fp8Args a{};
  a.rows = d.rows; a.cols = d.cols; a.io = d.io_dtype; a.square = d.kind == MSSM_FP8_SQUARE;
  return a;
}

int validate_linear(const mssm_fp8_linear_desc* d) {
  if (d == nullptr) return MSSM_ERR_INVALID_ARG;
  if (d->tokens < 0 || d->in_features <= 0 || d->out_features <= 0 || d->flags != 0) return MSSM_ERR_INVALID_ARG;
  if (d->weight_kind != MSSM_FP8_ROWS && d->weight_kind != MSSM_FP8_SQUARE) return MSSM_ERR_INVALID_ARG;
  if (!io_ok(d->io_dtype) || (!io_ok(d->x_dtype) && d->x_dtype != MSSM_E4M3)) return MSSM_ERR_UNSUPPORTED;
  if (d->tokens > kMostRows || d->in_features > kMostCols || d->out_features > kMostCols) return MSSM_ERR_UNSUPPORTED;
  return MSSM_OK;
}

// pieces of a workspace, each 256-byte aligned
struct Pieces {
  unsigned char* at;
  size_t used = 0;
  void* take(int64_t bytes) {
    void* const p = at == nullptr ? nullptr : at + used;
    used += (static_cast<size_t>(bytes) + 255) / 256 * 256;
    return p;
  }
  Fp8View matrix(int64_t rows, int64_t cols) {
    Fp8View v;
    v.codes = take(fp8_code_bytes(rows, cols));
    v.scales = take(fp8_scale_bytes(rows, cols, false));
    return v;
  }
};

struct Fwd {
  mssm::Fp8ProductArgs product{};
  size_t bytes = 0;
  bool rounds = false;   // a plain x goes through
  Fp8View x;
};
Fwd plan_fwd(const mssm_fp8_linear_desc& d, void* workspace) {
  Fwd f;
  Pieces w{static_cast<unsigned char*>(workspace)};
  f.product.rows = d.tokens; f.product.cols = d.out_features; f.product.k = d.in_features;
  f.product.square = d.weight_kind == MSSM_FP8_SQUARE; f.product.out_io = d.io_dtype; f.product.r_io = d.x_dtype;
  f.product.plain = d.x_dtype != MSSM_E4M3 && mssm::fp8_product_takes_plain(f.product);
  f.rounds = d.x_dtype != MSSM_E4M3 && !f.product.plain;
  if (f.rounds) f.x = w.matrix(d.tokens, d.in_features);
  f.product.workspace = w.take(mssm::fp8_product_workspace_bytes(f.product));
  f.bytes = w.used;
  return f;
}

struct Bwd {
  mssm::Fp8ProductArgs dx{}, dw{};
  size_t bytes = 0;
  Fp8View dout, dout_t, x_t;
};
Bwd plan_bwd(const mssm_fp8_linear_desc& d, void* workspace, bool want_dx, bool want_dw, int32_t grad_dtype) {
  Bwd b;
  Pieces w{static_cast<unsigned char*>(workspace)};
  b.dx.rows = d.tokens; b.dx.cols = d.in_features; b.dx.k = d.out_features;
  b.dx.square = d.weight_kind == MSSM_FP8_SQUARE; b.dx.out_io = d.io_dtype;
  b.dw.rows = d.out_features; b.dw.cols = d.in_features; b.dw.k = d.tokens; b.dw.out_io = grad_dtype;
  size_t product = 0;
  if (want_dx) {
    b.dout = w.matrix(d.tokens, d.out_features);
    product = mssm::fp8_product_workspace_bytes(b.dx);
  }
  if (want_dw) {
    b.dout_t = w.matrix(d.out_features, d.tokens);
    b.x_t = w.matrix(d.in_features, d.tokens);
    const size_t p = mssm::fp8_product_workspace_bytes(b.dw);
    product = product < p ? p : product;
  }
  b.dx.workspace = b.dw.workspace = w.take(product);   // one product after the other
  b.bytes = w.used;
  return b;
}

}  // namespace

extern "C" {

int mssm_fp8_quantize(const mssm_fp8_desc* desc, const void* x, void* codes, void* scales, void* codes_t,
                      void* scales_t, void* stream) {
  const int v = validate_matrix(desc);
  if (v != MSSM_OK) return v;
  const mssm_fp8_desc& d = *desc;
  if ((codes == nullptr) != (scales == nullptr) || (codes_t == nullptr) != (scales_t == nullptr))
    return MSSM_ERR_INVALID_ARG;
  if (d.rows == 0) return MSSM_OK;
  if (x == nullptr || (codes == nullptr && codes_t == nullptr)) return MSSM_ERR_INVALID_ARG;
  if (!aligned(x, size_of(d.io_dtype)) || !view_aligned(codes, scales) || !view_aligned(codes_t, scales_t))
    return MSSM_ERR_MISALIGNED;
  const bool square = d.kind == MSSM_FP8_SQUARE;
  const Buf in[] = {{x, d.rows * d.cols * size_of(d.io_dtype)}};
  const Buf outs[] = {{codes, fp8_code_bytes(d.rows, d.cols)}, {scales, fp8_scale_bytes(d.rows, d.cols, square)},
                      {codes_t, fp8_code_bytes(d.cols, d.rows)}, {scales_t, fp8_scale_bytes(d.cols, d.rows, square)}};
  if (!disjoint(in, outs)) return MSSM_ERR_INVALID_ARG;
  mssm::Fp8Args a = matrix_args(d);
  a.x = x; a.m = {codes, scales}; a.t = {codes_t, scales_t};
  return done(mssm::fp8_quantize_launch(a, static_cast<hipStream_t>(stream)));
}

int mssm_fp8_transpose(const mssm_fp8_desc* desc, const void* codes, const void* scales, void* codes_t, void* scales_t,
                       void* stream) {
  const int v = validate_matrix(desc);
  if (v != MSSM_OK) return v;
  const mssm_fp8_desc& d = *desc;
  if (d.kind != MSSM_FP8_ROWS) return MSSM_ERR_UNSUPPORTED;
  if (d.rows == 0) return MSSM_OK;
  if (codes == nullptr || scales == nullptr || codes_t == nullptr || scales_t == nullptr) return MSSM_ERR_INVALID_ARG;
  if (!view_aligned(codes, scales) || !view_aligned(codes_t, scales_t)) return MSSM_ERR_MISALIGNED;
  const Buf in[] = {{codes, fp8_code_bytes(d.rows, d.cols)}, {scales, fp8_scale_bytes(d.rows, d.cols, false)}};
  const Buf outs[] = {{codes_t, fp8_code_bytes(d.cols, d.rows)}, {scales_t, fp8_scale_bytes(d.cols, d.rows, false)}};
  if (!disjoint(in, outs)) return MSSM_ERR_INVALID_ARG;
  mssm::Fp8Args a = matrix_args(d);
  a.m = {const_cast<void*>(codes), const_cast<void*>(scales)}; a.t = {codes_t, scales_t};
  return done(mssm::fp8_transpose_launch(a, static_cast<hipStream_t>(stream)));
}

int mssm_fp8_dequantize(const mssm_fp8_desc* desc, const void* codes, const void* scales, void* out, void* stream) {
  const int v = validate_matrix(desc);
  if (v != MSSM_OK) return v;
  const mssm_fp8_desc& d = *desc;
  if (d.rows == 0) return MSSM_OK;
  if (codes == nullptr || scales == nullptr || out == nullptr) return MSSM_ERR_INVALID_ARG;
  if (!view_aligned(codes, scales) || !aligned(out, size_of(d.io_dtype))) return MSSM_ERR_MISALIGNED;
  const Buf in[] = {{codes, fp8_code_bytes(d.rows, d.cols)},
                    {scales, fp8_scale_bytes(d.rows, d.cols, d.kind == MSSM_FP8_SQUARE)}};
  const Buf outs[] = {{out, d.rows * d.cols * size_of(d.io_dtype)}};
  if (!disjoint(in, outs)) return MSSM_ERR_INVALID_ARG;
  mssm::Fp8Args a = matrix_args(d);
  a.m = {const_cast<void*>(codes), const_cast<void*>(scales)}; a.out = out;
  return done(mssm::fp8_dequantize_launch(a, static_cast<hipStream_t>(stream)));
}

size_t mssm_fp8_linear_fwd_workspace_size(const mssm_fp8_linear_desc* desc) {
  if (validate_linear(desc) != MSSM_OK) return 0;
  return plan_fwd(*desc, nullptr).bytes;
}

int mssm_fp8_linear_fwd(const mssm_fp8_linear_desc* desc, const void* x, const void* x_scales, const void* weight,
                        const void* weight_scales, void* out, void* workspace, size_t workspace_bytes, void* stream) {
  const int v = validate_linear(desc);
  if (v != MSSM_OK) return v;
  const mssm_fp8_linear_desc& d = *desc;
  const bool plain = d.x_dtype != MSSM_E4M3;
  if (plain && x_scales != nullptr) return MSSM_ERR_INVALID_ARG;
  if (d.tokens == 0) return MSSM_OK;
  if (x == nullptr || (!plain && x_scales == nullptr) || weight == nullptr || weight_scales == nullptr || out == nullptr)
    return MSSM_ERR_INVALID_ARG;
  if (!aligned(x, plain ? size_of(d.x_dtype) : 16) || !aligned(x_scales, 4) || !view_aligned(weight, weight_scales) ||
      !aligned(out, size_of(d.io_dtype)))
    return MSSM_ERR_MISALIGNED;
  Fwd f = plan_fwd(d, workspace);
  const int w = workspace_status(workspace, workspace_bytes, f.bytes);
  if (w != MSSM_OK) return w;
  const Buf in[] = {{x, plain ? d.tokens * d.in_features * size_of(d.x_dtype) : fp8_code_bytes(d.tokens, d.in_features)},
                    {x_scales, fp8_scale_bytes(d.tokens, d.in_features, false)},
                    {weight, fp8_code_bytes(d.out_features, d.in_features)},
                    {weight_scales, fp8_scale_bytes(d.out_features, d.in_features, f.product.square)}};
  const Buf outs[] = {{out, d.tokens * d.out_features * size_of(d.io_dtype)},
                      {workspace, static_cast<int64_t>(f.bytes)}};
  if (!disjoint(in, outs)) return MSSM_ERR_INVALID_ARG;
  const hipStream_t s = static_cast<hipStream_t>(stream);
  f.product.r = {const_cast<void*>(x), const_cast<void*>(x_scales)};
  if (f.rounds) {
    mssm::Fp8Args q{};
    q.rows = d.tokens; q.cols = d.in_features; q.io = d.x_dtype; q.x = x; q.m = f.x;
    const int e = done(mssm::fp8_quantize_launch(q, s));
    if (e != MSSM_OK) return e;
    f.product.r = f.x;
  }
  f.product.c = {const_cast<void*>(weight), const_cast<void*>(weight_scales)};
  f.product.out = out;
  return done(mssm::fp8_product_launch(f.product, s));
}

size_t mssm_fp8_linear_bwd_workspace_size(const mssm_fp8_linear_desc* desc, int32_t want_dx, int32_t want_dweight,
                                          int32_t grad_dtype) {
  if (validate_linear(desc) != MSSM_OK || desc->x_dtype != MSSM_E4M3) return 0;
  if (grad_dtype != MSSM_F32 && grad_dtype != desc->io_dtype) return 0;
  return plan_bwd(*desc, nullptr, want_dx != 0, want_dweight != 0, grad_dtype).bytes;
}

int mssm_fp8_linear_bwd(const mssm_fp8_linear_desc* desc, const void* x, const void* x_scales, const void* weight_t,
                        const void* weight_t_scales, const void* dout, void* dx, void* dweight, int32_t grad_dtype,
                        int32_t accumulate, void* workspace, size_t workspace_bytes, void* stream) {
  const int v = validate_linear(desc);
  if (v != MSSM_OK) return v;
  const mssm_fp8_linear_desc& d = *desc;
  if (d.x_dtype != MSSM_E4M3 || (grad_dtype != MSSM_F32 && grad_dtype != d.io_dtype)) return MSSM_ERR_UNSUPPORTED;
  if (dx == nullptr && dweight == nullptr) return MSSM_ERR_INVALID_ARG;
  if (d.tokens > 0) {
    if (dout == nullptr) return MSSM_ERR_INVALID_ARG;
    if (dx != nullptr && (weight_t == nullptr || weight_t_scales == nullptr)) return MSSM_ERR_INVALID_ARG;
    if (dweight != nullptr && (x == nullptr || x_scales == nullptr)) return MSSM_ERR_INVALID_ARG;
  }
  const int64_t es = size_of(d.io_dtype), gs = size_of(grad_dtype);
  if (!view_aligned(x, x_scales) || !view_aligned(weight_t, weight_t_scales) || !aligned(dout, es) || !aligned(dx, es) ||
      !aligned(dweight, gs))
    return MSSM_ERR_MISALIGNED;
  Bwd b = plan_bwd(d, workspace, dx != nullptr, dweight != nullptr, grad_dtype);
  const int w = workspace_status(workspace, workspace_bytes, b.bytes);
  if (w != MSSM_OK) return w;
  const Buf in[] = {{x, fp8_code_bytes(d.tokens, d.in_features)},
                    {x_scales, fp8_scale_bytes(d.tokens, d.in_features, false)},
                    {weight_t, fp8_code_bytes(d.in_features, d.out_features)},
                    {weight_t_scales, fp8_scale_bytes(d.in_features, d.out_features, b.dx.square)},
                    {dout, d.tokens * d.out_features * es}};
  const Buf outs[] = {{dx, d.tokens * d.in_features * es}, {dweight, d.out_features * d.in_features * gs},
                      {workspace, static_cast<int64_t>(b.bytes)}};
  if (!disjoint(in, outs)) return MSSM_ERR_INVALID_ARG;
  const hipStream_t s = static_cast<hipStream_t>(stream);
  mssm::Fp8Args q{}, t{};
  q.rows = d.tokens; q.cols = d.out_features; q.io = d.io_dtype; q.x = dout; q.m = b.dout; q.t = b.dout_t;
  t.rows = d.tokens; t.cols = d.in_features;
  t.m = {const_cast<void*>(x), const_cast<void*>(x_scales)}; t.t = b.x_t;
  const int e = done(dweight != nullptr ? mssm::fp8_both_launch(q, t, s) : mssm::fp8_quantize_launch(q, s));
  if (e != MSSM_OK) return e;
  b.dx.r = b.dout;
  b.dx.c = {const_cast<void*>(weight_t), const_cast<void*>(weight_t_scales)};
  b.dx.out = dx;
  b.dw.r = b.dout_t; b.dw.c = b.x_t; b.dw.out = dweight; b.dw.accumulate = accumulate != 0;
  if (dx != nullptr && dweight != nullptr) return done(mssm::fp8_two_products_launch(b.dx, b.dw, s));
  return done(mssm::fp8_product_launch(dx != nullptr ? b.dx : b.dw, s));
}

}  // extern "C"
