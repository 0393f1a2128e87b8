// C-ABI front end of the operators around the scan: embedding, layer / RMS norm, cross entropy of a linear
// head.  Every check runs on the host before anything is enqueued.
#include "../../include/mssm.h"

#include "checks.h"
#include "internal.h"

using namespace mssm::checks;
using mssm::set_err;

namespace {

constexpr int64_t kMaxTokens = (int64_t{1} << 26) - 1;
constexpr int64_t kMaxWaves = (int64_t{1} << 26) - 4;    // a wave a row, four to a workgroup: a 32-bit work-item count
constexpr int64_t kMaxVocab = int64_t{1} << 30;
constexpr int64_t kMaxDim = int64_t{1} << 20;

bool io_ok(int32_t t) { return t == MSSM_F32 || t == MSSM_BF16; }
int64_t size_of(int32_t t) { return t == MSSM_BF16 ? 2 : 4; }

int done(hipError_t e) {
  if (e == hipSuccess) return MSSM_OK;
  set_err(e);
  return MSSM_ERR_HIP;
}

struct Buf {
  const void* p;
  int64_t bytes;
};
// no output may overlap an input or another output
template <int NI, int NO> bool disjoint(const Buf (&in)[NI], const Buf (&out)[NO]) {
  for (int o = 0; o < NO; ++o) {
    for (int i = 0; i < NI; ++i)
      if (overlap(out[o].p, out[o].bytes, in[i].p, in[i].bytes)) return false;
    for (int k = 0; k < o; ++k)
      if (overlap(out[o].p, out[o].bytes, out[k].p, out[k].bytes)) return false;
  }
  return true;
}

int workspace_status(const void* ws, size_t have, size_t need) {
  if (need == 0) return MSSM_OK;
  if (ws == nullptr || have < need) return MSSM_ERR_WORKSPACE;
  return aligned(ws, 256) ? MSSM_OK : MSSM_ERR_MISALIGNED;
}

int validate_embedding(const mssm_embedding_desc* d) {
  if (d == nullptr) return MSSM_ERR_INVALID_ARG;
  if (d->tokens < 0 || d->vocab <= 0 || d->dim <= 0 || d->flags != 0) return MSSM_ERR_INVALID_ARG;
  if (!(d->scale - d->scale == 0.f)) return MSSM_ERR_INVALID_ARG;   // finite
  int64_t t = 0;
  if (!mul_ok(d->tokens, d->dim, &t) || !mul_ok(t, 16, &t)) return MSSM_ERR_INVALID_ARG;
  if (!mul_ok(d->vocab, d->dim, &t) || !mul_ok(t, 4, &t)) return MSSM_ERR_INVALID_ARG;
  if (!io_ok(d->io_dtype) || (d->id_bytes != 4 && d->id_bytes != 8)) return MSSM_ERR_UNSUPPORTED;
  if (d->tokens > kMaxWaves || d->vocab > kMaxVocab || d->dim > kMaxDim) return MSSM_ERR_UNSUPPORTED;
  return MSSM_OK;
}

mssm::EmbedArgs embed_args(const mssm_embedding_desc& d) {
  mssm::EmbedArgs a{};
  a.tokens = d.tokens; a.vocab = d.vocab; a.dim = d.dim; a.io = d.io_dtype; a.id_bytes = d.id_bytes;
  a.scale = d.scale;
  return a;
}

int validate_norm(const mssm_norm_desc* d) {
  if (d == nullptr) return MSSM_ERR_INVALID_ARG;
  if (d->rows < 0 || d->dim <= 0 || d->flags != 0) return MSSM_ERR_INVALID_ARG;
  if (!(d->eps > 0.f) || !(d->eps - d->eps == 0.f)) return MSSM_ERR_INVALID_ARG;
  if (d->kind != MSSM_LAYER_NORM && d->kind != MSSM_RMS_NORM) return MSSM_ERR_INVALID_ARG;
  int64_t t = 0;
  if (!mul_ok(d->rows, d->dim, &t) || !mul_ok(t, 4, &t)) return MSSM_ERR_INVALID_ARG;
  if (!io_ok(d->io_dtype) || !io_ok(d->res_dtype)) return MSSM_ERR_UNSUPPORTED;
  if (d->io_dtype == MSSM_F32 && d->res_dtype != MSSM_F32) return MSSM_ERR_UNSUPPORTED;
  // a wave per row up to 256 columns, a workgroup of up to 1024 threads above: 32-bit work-item counts
  if (d->rows > (d->dim <= 256 ? kMaxWaves : (int64_t{1} << 22) - 1) || d->dim > kMaxDim) return MSSM_ERR_UNSUPPORTED;
  return MSSM_OK;
}

mssm::NormArgs norm_args(const mssm_norm_desc& d) {
  mssm::NormArgs a{};
  a.rows = d.rows; a.dim = d.dim; a.eps = d.eps; a.layer = d.kind == MSSM_LAYER_NORM;
  a.io = d.io_dtype; a.res_io = d.res_dtype;
  return a;
}

int validate_xent(const mssm_cross_entropy_desc* d) {
  if (d == nullptr) return MSSM_ERR_INVALID_ARG;
  if (d->tokens < 0 || d->vocab <= 0 || d->dim <= 0) return MSSM_ERR_INVALID_ARG;
  if ((d->flags & ~MSSM_CROSS_ENTROPY_FINE_G) != 0) return MSSM_ERR_INVALID_ARG;
  int64_t t = 0;
  // (the workspace holds up to five 16-bit terms of either operand, padded)
  if (!mul_ok(d->tokens, d->dim, &t) || !mul_ok(t, 64, &t)) return MSSM_ERR_INVALID_ARG;
  if (!mul_ok(d->vocab, d->dim, &t) || !mul_ok(t, 64, &t)) return MSSM_ERR_INVALID_ARG;
  if (!io_ok(d->io_dtype) || (d->id_bytes != 4 && d->id_bytes != 8)) return MSSM_ERR_UNSUPPORTED;
  if (d->tokens > kMaxTokens || d->vocab > kMaxVocab || d->dim > kMaxDim) return MSSM_ERR_UNSUPPORTED;
  return MSSM_OK;
}

// bf16 rows of a multiple of 64 are read in place, 16 bytes at a time; any other weight is laid out first
int64_t weight_alignment(const mssm_cross_entropy_desc& d) {
  return d.io_dtype == MSSM_BF16 ? (d.dim % 64 == 0 ? 16 : 2) : 4;
}

mssm::XentArgs xent_args(const mssm_cross_entropy_desc& d, const void* x, const void* weight, const void* targets) {
  mssm::XentArgs a{};
  a.tokens = d.tokens; a.vocab = d.vocab; a.dim = d.dim; a.ignore = d.ignore_id; a.io = d.io_dtype;
  a.id_bytes = d.id_bytes; a.x = x; a.weight = weight; a.targets = targets;
  a.fine_g = (d.flags & MSSM_CROSS_ENTROPY_FINE_G) != 0;
  return a;
}

}  // namespace

extern "C" {

int mssm_embedding_fwd(const mssm_embedding_desc* desc, const void* ids, const void* weight, void* out, void* stream) {
  const int v = validate_embedding(desc);
  if (v != MSSM_OK) return v;
  const mssm_embedding_desc& d = *desc;
  if (d.tokens == 0) return MSSM_OK;
  if (ids == nullptr || weight == nullptr || out == nullptr) return MSSM_ERR_INVALID_ARG;
  const int64_t es = size_of(d.io_dtype);
  if (!aligned(ids, d.id_bytes) || !aligned(weight, es) || !aligned(out, es)) return MSSM_ERR_MISALIGNED;
  const Buf in[] = {{ids, d.tokens * d.id_bytes}, {weight, d.vocab * d.dim * es}};
  const Buf outs[] = {{out, d.tokens * d.dim * es}};
  if (!disjoint(in, outs)) return MSSM_ERR_INVALID_ARG;
  mssm::EmbedArgs a = embed_args(d);
  a.ids = ids; a.weight = weight; a.out = out;
  return done(mssm::embed_fwd_launch(a, static_cast<hipStream_t>(stream)));
}

size_t mssm_embedding_bwd_workspace_size(const mssm_embedding_desc* desc) {
  if (validate_embedding(desc) != MSSM_OK) return 0;
  return mssm::embed_bwd_workspace_bytes(desc->tokens, desc->vocab, desc->dim);
}

int mssm_embedding_bwd(const mssm_embedding_desc* desc, const void* ids, const void* dout, void* dweight,
                       int32_t grad_dtype, int32_t accumulate, void* workspace, size_t workspace_bytes, void* stream) {
  const int v = validate_embedding(desc);
  if (v != MSSM_OK) return v;
  const mssm_embedding_desc& d = *desc;
  if (grad_dtype != MSSM_F32 && grad_dtype != d.io_dtype) return MSSM_ERR_UNSUPPORTED;
  if (dweight == nullptr || (d.tokens > 0 && (ids == nullptr || dout == nullptr))) return MSSM_ERR_INVALID_ARG;
  const int64_t es = size_of(d.io_dtype), gs = size_of(grad_dtype);
  if (!aligned(ids, d.id_bytes) || !aligned(dout, es) || !aligned(dweight, gs)) return MSSM_ERR_MISALIGNED;
  const size_t need = mssm::embed_bwd_workspace_bytes(d.tokens, d.vocab, d.dim);
  const int w = workspace_status(workspace, workspace_bytes, need);
  if (w != MSSM_OK) return w;
  const Buf in[] = {{ids, d.tokens * d.id_bytes}, {dout, d.tokens * d.dim * es}};
  const Buf outs[] = {{dweight, d.vocab * d.dim * gs}, {workspace, static_cast<int64_t>(need)}};
  if (!disjoint(in, outs)) return MSSM_ERR_INVALID_ARG;
  mssm::EmbedArgs a = embed_args(d);
  a.ids = ids; a.dout = dout; a.dweight = dweight; a.grad_io = grad_dtype == MSSM_BF16; a.accumulate = accumulate != 0;
  a.workspace = workspace;
  return done(mssm::embed_bwd_launch(a, static_cast<hipStream_t>(stream)));
}

int mssm_norm_fwd(const mssm_norm_desc* desc, const void* x, const void* residual, const float* weight,
                  const float* bias, void* out, void* residual_out, float* mean, float* rstd, void* stream) {
  const int v = validate_norm(desc);
  if (v != MSSM_OK) return v;
  const mssm_norm_desc& d = *desc;
  if (d.kind == MSSM_RMS_NORM && (bias != nullptr || mean != nullptr)) return MSSM_ERR_INVALID_ARG;
  if (residual != nullptr && residual_out == nullptr) return MSSM_ERR_INVALID_ARG;
  if (d.rows == 0) return MSSM_OK;
  if (x == nullptr || weight == nullptr || out == nullptr) return MSSM_ERR_INVALID_ARG;
  const int64_t es = size_of(d.io_dtype), rs = size_of(d.res_dtype), n = d.rows * d.dim;
  if (!aligned(x, es) || !aligned(out, es) || !aligned(residual, rs) || !aligned(residual_out, rs) ||
      !aligned(weight, 4) || !aligned(bias, 4) || !aligned(mean, 4) || !aligned(rstd, 4))
    return MSSM_ERR_MISALIGNED;
  const Buf in[] = {{x, n * es}, {residual, n * rs}, {weight, d.dim * 4}, {bias, d.dim * 4}};
  const Buf outs[] = {{out, n * es}, {residual_out, n * rs}, {mean, d.rows * 4}, {rstd, d.rows * 4}};
  if (!disjoint(in, outs)) return MSSM_ERR_INVALID_ARG;
  mssm::NormArgs a = norm_args(d);
  a.x = x; a.residual = residual; a.weight = weight; a.bias = bias; a.out = out; a.residual_out = residual_out;
  a.mean = mean; a.rstd = rstd;
  return done(mssm::norm_fwd_launch(a, static_cast<hipStream_t>(stream)));
}

size_t mssm_norm_bwd_workspace_size(const mssm_norm_desc* desc) {
  if (validate_norm(desc) != MSSM_OK) return 0;
  return mssm::norm_bwd_workspace_bytes(desc->rows, desc->dim);
}

int mssm_norm_bwd(const mssm_norm_desc* desc, const void* h, const float* weight, const float* mean, const float* rstd,
                  const void* dout, const void* dresidual, void* dx, void* dresidual_in, float* dweight, float* dbias,
                  void* workspace, size_t workspace_bytes, void* stream) {
  const int v = validate_norm(desc);
  if (v != MSSM_OK) return v;
  const mssm_norm_desc& d = *desc;
  const bool layer = d.kind == MSSM_LAYER_NORM;
  if (!layer && (dbias != nullptr || mean != nullptr)) return MSSM_ERR_INVALID_ARG;
  if (weight == nullptr || dweight == nullptr) return MSSM_ERR_INVALID_ARG;
  if (d.rows > 0 && (h == nullptr || rstd == nullptr || dout == nullptr || (layer && mean == nullptr) ||
                     (dx == nullptr && dresidual_in == nullptr)))
    return MSSM_ERR_INVALID_ARG;
  const int64_t es = size_of(d.io_dtype), rs = size_of(d.res_dtype), n = d.rows * d.dim;
  if (!aligned(h, rs) || !aligned(dout, es) || !aligned(dresidual, rs) || !aligned(dx, es) ||
      !aligned(dresidual_in, rs) || !aligned(weight, 4) || !aligned(mean, 4) || !aligned(rstd, 4) ||
      !aligned(dweight, 4) || !aligned(dbias, 4))
    return MSSM_ERR_MISALIGNED;
  const size_t need = mssm::norm_bwd_workspace_bytes(d.rows, d.dim);
  const int w = workspace_status(workspace, workspace_bytes, need);
  if (w != MSSM_OK) return w;
  const Buf in[] = {{h, n * rs}, {weight, d.dim * 4}, {mean, d.rows * 4}, {rstd, d.rows * 4}, {dout, n * es},
                    {dresidual, n * rs}};
  const Buf outs[] = {{dx, n * es}, {dresidual_in, n * rs}, {dweight, d.dim * 4}, {dbias, d.dim * 4},
                      {workspace, static_cast<int64_t>(need)}};
  if (!disjoint(in, outs)) return MSSM_ERR_INVALID_ARG;
  mssm::NormArgs a = norm_args(d);
  a.h = h; a.weight = weight; a.mean = const_cast<float*>(mean); a.rstd = const_cast<float*>(rstd); a.dout = dout;
  a.dresidual = dresidual; a.dx = dx; a.dresidual_in = dresidual_in; a.dweight = dweight; a.dbias = dbias;
  a.workspace = workspace;
  return done(mssm::norm_bwd_launch(a, static_cast<hipStream_t>(stream)));
}

size_t mssm_linear_cross_entropy_fwd_workspace_size(const mssm_cross_entropy_desc* desc) {
  if (validate_xent(desc) != MSSM_OK) return 0;
  return mssm::xent_workspace_bytes(xent_args(*desc, nullptr, nullptr, nullptr), false);
}

int mssm_linear_cross_entropy_fwd(const mssm_cross_entropy_desc* desc, const void* x, const void* weight,
                                  const void* targets, float* loss, float* lse, void* workspace,
                                  size_t workspace_bytes, void* stream) {
  const int v = validate_xent(desc);
  if (v != MSSM_OK) return v;
  const mssm_cross_entropy_desc& d = *desc;
  if (d.tokens == 0) return MSSM_OK;
  if (x == nullptr || weight == nullptr || targets == nullptr || loss == nullptr || lse == nullptr)
    return MSSM_ERR_INVALID_ARG;
  const int64_t es = size_of(d.io_dtype);
  if (!aligned(x, es) || !aligned(weight, weight_alignment(d)) || !aligned(targets, d.id_bytes) || !aligned(loss, 4) || !aligned(lse, 4))
    return MSSM_ERR_MISALIGNED;
  mssm::XentArgs a = xent_args(d, x, weight, targets);
  const size_t need = mssm::xent_workspace_bytes(a, false);
  const int w = workspace_status(workspace, workspace_bytes, need);
  if (w != MSSM_OK) return w;
  const Buf in[] = {{x, d.tokens * d.dim * es}, {weight, d.vocab * d.dim * es}, {targets, d.tokens * d.id_bytes}};
  const Buf outs[] = {{loss, d.tokens * 4}, {lse, d.tokens * 4}, {workspace, static_cast<int64_t>(need)}};
  if (!disjoint(in, outs)) return MSSM_ERR_INVALID_ARG;
  a.loss = loss; a.lse = lse; a.workspace = workspace;
  return done(mssm::xent_fwd_launch(a, static_cast<hipStream_t>(stream)));
}

size_t mssm_linear_cross_entropy_bwd_workspace_size(const mssm_cross_entropy_desc* desc) {
  if (validate_xent(desc) != MSSM_OK) return 0;
  return mssm::xent_workspace_bytes(xent_args(*desc, nullptr, nullptr, nullptr), true);
}

int mssm_linear_cross_entropy_bwd(const mssm_cross_entropy_desc* desc, const void* x, const void* weight,
                                  const void* targets, const float* lse, const float* dloss, const float* dlse,
                                  void* dx, void* dweight, int32_t grad_dtype, int32_t accumulate, void* workspace,
                                  size_t workspace_bytes, void* stream) {
  const int v = validate_xent(desc);
  if (v != MSSM_OK) return v;
  const mssm_cross_entropy_desc& d = *desc;
  if (grad_dtype != MSSM_F32 && grad_dtype != d.io_dtype) return MSSM_ERR_UNSUPPORTED;
  if (weight == nullptr || (dx == nullptr && dweight == nullptr)) return MSSM_ERR_INVALID_ARG;
  if (d.tokens > 0 && (x == nullptr || targets == nullptr || lse == nullptr || dloss == nullptr))
    return MSSM_ERR_INVALID_ARG;
  const int64_t es = size_of(d.io_dtype), gs = size_of(grad_dtype);
  if (!aligned(x, es) || !aligned(weight, weight_alignment(d)) || !aligned(targets, d.id_bytes) || !aligned(lse, 4) ||
      !aligned(dloss, 4) || !aligned(dlse, 4) || !aligned(dx, es) || !aligned(dweight, gs))
    return MSSM_ERR_MISALIGNED;
  mssm::XentArgs a = xent_args(d, x, weight, targets);
  const size_t need = mssm::xent_workspace_bytes(a, true);
  const int w = workspace_status(workspace, workspace_bytes, need);
  if (w != MSSM_OK) return w;
  const Buf in[] = {{x, d.tokens * d.dim * es}, {weight, d.vocab * d.dim * es}, {targets, d.tokens * d.id_bytes},
                    {lse, d.tokens * 4}, {dloss, d.tokens * 4}, {dlse, d.tokens * 4}};
  const Buf outs[] = {{dx, d.tokens * d.dim * es}, {dweight, d.vocab * d.dim * gs},
                      {workspace, static_cast<int64_t>(need)}};
  if (!disjoint(in, outs)) return MSSM_ERR_INVALID_ARG;
  a.lse_in = lse; a.dloss = dloss; a.dlse = dlse; a.dx = dx; a.dweight = dweight;
  a.grad_io = grad_dtype == d.io_dtype; a.accumulate = accumulate != 0; a.workspace = workspace;
  return done(mssm::xent_bwd_launch(a, static_cast<hipStream_t>(stream)));
}

}  // extern "C"
