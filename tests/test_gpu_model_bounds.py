"""Bounds that follow the kernels' own order of additions and number of bits, tighter than those in model_ops: the
columns' sums of the norms' gradients, and the logits' gradient of a few bf16 tokens."""
import pytest
import torch

import model_ops as R
from gpu_util import say

pytestmark = pytest.mark.gpu
BF16, F32, F64 = torch.bfloat16, torch.float32, torch.float64
U = R.U


@pytest.fixture(scope="module")
def M():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import selective_state_space_17_amd as m
    return m


def column_additions(rows, dim):
    """The most additions that a row's term goes through on its way into a column's sum."""
    groups = min(1024, -(-rows // 4) if dim <= 1024 else rows)
    if dim <= 1024:       # four waves a group, a row each at a time, joined by three additions
        inside = -(-rows // (4 * groups)) + 3
    elif dim <= 16384:    # a row at a time
        inside = -(-rows // groups)
    else:                 # a thread walks over its share of the rows
        groups = min(64, groups)
        inside = -(-rows // groups)
    return inside + -(-groups // 16) + 15     # each of 16 waves adds its groups, then the 16 sums


@pytest.mark.parametrize("rows,dim,io", [(1, 40, F32), (70, 64, BF16), (5000, 72, F32), (9001, 300, BF16), (3001, 1023, F32),
                                         (2500, 1032, BF16), (700, 2050, F32), (40, 16392, F32), (300, 17000, BF16)])
@pytest.mark.parametrize("layer", [True, False], ids=["layer", "rms"])
def test_column_sums(M, rows, dim, io, layer):
    g = torch.Generator().manual_seed(rows + dim)
    h, dout = torch.randn(rows, dim, generator=g).to(io), (torch.randn(rows, dim, generator=g) + 0.5).to(io)
    w = 1 + 0.1 * torch.randn(dim, generator=g)
    mean, rstd = 0.1 * torch.randn(rows, generator=g), 0.5 + torch.rand(rows, generator=g)
    say("column sums", rows, dim, io, layer)
    if layer:
        got = M.layer_norm_bwd(h.cuda(), w.cuda(), mean.cuda(), rstd.cuda(), dout.cuda())
    else:
        got = M.rms_norm_bwd(h.cuda(), w.cuda(), rstd.cuda(), dout.cuda())
    d = dout.to(F64)
    t = d * (h.to(F64) - (mean.to(F64)[:, None] if layer else 0.0)) * rstd.to(F64)[:, None]
    n = column_additions(rows, dim)
    # xh: two roundings (h - mu relative to the difference; times rstd), its product with dout none (a multiply-add)
    # but where the row is wide (db and dw alike there: dout xh rounded too)
    R.check(got["dweight"], (t.sum(0), 1.01 * t.abs().sum(0) * (n + 3) * U), "dweight")
    if layer:
        R.check(got["dbias"], (d.sum(0), 1.01 * d.abs().sum(0) * n * U), "dbias")


def sixteen_bits(M, x, w, y, dl, dz, call):
    """The gradients with G in two bf16 terms: each is the nearest of what is left, so G is right to 2^-8 of 2^-8."""
    loss, lse = M.linear_cross_entropy_fwd(x.cuda(), w.cuda(), y.cuda())
    dw = torch.empty(w.shape, dtype=F32, device="cuda")
    got = call(x.cuda(), w.cuda(), y.cuda(), lse, dl.cuda(), dlse=dz.cuda(), dweight=dw)
    # the same values in fp32: the bounds without G's rounding to bf16
    ref = R.cross_entropy(x.float(), w.float(), y, dloss=dl, dlse=dz, lse_in=lse.cpu())
    keep = ((y >= 0) & (y < w.shape[0])).nonzero()[:, 0]
    xk, w64 = x[keep].to(F64), w.to(F64)
    p = (xk @ w64.T - lse.cpu()[keep].to(F64)[:, None]).exp()
    G = p * (dl + dz)[keep].to(F64)[:, None]
    G[torch.arange(keep.numel()), y[keep]] -= dl[keep].to(F64)
    (dx, e_dx), (dwt, e_dw) = ref["dx"], ref["dweight"]
    e_dx = e_dx + torch.zeros_like(dx).index_copy(0, keep, G.abs() @ w64.abs()) * 2.0 ** -16 + dx.abs() * 2.0 ** -8
    R.check(got["dx"], (dx, e_dx), "dx")
    R.check(got["dweight"], (dwt, e_dw + G.abs().T @ xk.abs() * 2.0 ** -16), "dweight in fp32")


@pytest.mark.parametrize("tokens,vocab,dim", [(1, 300, 64), (16, 2000, 100), (100, 700, 192), (256, 900, 64)])
def test_few_tokens_keep_sixteen_bits_of_g(M, tokens, vocab, dim):
    g = torch.Generator().manual_seed(tokens)
    x, w = torch.randn(tokens, dim, generator=g).to(BF16), (1.5 * dim ** -0.5 * torch.randn(vocab, dim, generator=g)).to(BF16)
    y = torch.randint(0, vocab, (tokens,), generator=g)
    y[1::7] = -100
    dl, dz = torch.rand(tokens, generator=g) + 0.5, 0.1 * torch.randn(tokens, generator=g)
    say("sixteen bits", tokens, vocab, dim)
    sixteen_bits(M, x, w, y, dl, dz, M.linear_cross_entropy_bwd)


@pytest.mark.parametrize("tokens,vocab,dim", [(257, 300, 64), (300, 2049, 100), (2100, 5000, 512)])
def test_more_tokens_keep_sixteen_bits_of_g_on_request(M, tokens, vocab, dim):
    g = torch.Generator().manual_seed(tokens)
    x, w = torch.randn(tokens, dim, generator=g).to(BF16), (1.5 * dim ** -0.5 * torch.randn(vocab, dim, generator=g)).to(BF16)
    y = torch.randint(0, vocab, (tokens,), generator=g)
    y[1::7] = -100
    dl, dz = torch.rand(tokens, generator=g) + 0.5, 0.1 * torch.randn(tokens, generator=g)
    say("sixteen bits on request", tokens, vocab, dim)
    sixteen_bits(M, x, w, y, dl, dz, lambda *a, **kw: M.linear_cross_entropy_bwd(*a, fine=True, **kw))
    need = M.linear_cross_entropy_bwd_workspace_size(tokens, vocab, dim, fine=True)
    assert need > M.linear_cross_entropy_bwd_workspace_size(tokens, vocab, dim)
    with pytest.raises(M.MssmError):
        ws = torch.empty(need - 256, dtype=torch.uint8, device="cuda")
        sixteen_bits(M, x, w, y, dl, dz, lambda *a, **kw: M.linear_cross_entropy_bwd(*a, fine=True, workspace=ws, **kw))
