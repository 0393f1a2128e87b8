"""Cross entropy at sizes where every product takes more than one round of tiles over the chip: workgroups that go from
tile to tile, whole tiles ahead of a last round that is cut along k, several bands of token tiles, and a vocabulary that
the forward pass takes in pieces.  Against the plain 64-bit forms in model_ops, element by element, in 64 bits on the
GPU."""
import pytest
import torch

import model_ops as R
from gpu_util import say

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module")
def M():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import selective_state_space_17_amd as m
    return m


def make(tokens, vocab, dim, io, left_out, seed):
    g = torch.Generator().manual_seed(seed)
    w = torch.randn(vocab, dim, generator=g) * (1.5 * dim ** -0.5)
    y = torch.randint(0, vocab, (tokens,), generator=g)
    x = torch.randn(tokens, dim, generator=g) + 4 * torch.rand(tokens, 1, generator=g) * w[y]
    y[torch.randperm(tokens, generator=g)[:int(tokens * left_out)]] = -100
    dl, dz = torch.rand(tokens, generator=g) + 0.5, 0.1 * torch.randn(tokens, generator=g)
    return [t.cuda() for t in (x.to(io), w.to(io), y, dl, dz)]


def reference(*args, **kw):
    with torch.device("cuda"):
        return {k: (v.cpu(), e.cpu()) for k, (v, e) in R.cross_entropy(*args, **kw).items()}


def check_norms(got, x, w, y, dl, dz, lse):
    """The 2-norm of the gradients' errors.  The bounds per element let every rounding of a long sum go the same way,
    and a slice of it that is missing could hide there; at random they add up to their root.  bf16: G and the result
    are rounded to it, each at most 2^-8 off and evenly spread.  fp32: 2 U of the running sum for each of 6 K additions,
    and 2^-15 for the logits (2 U of each of 3 D additions to a logit of a few units: 1e-5)."""
    keep = (y >= 0).nonzero()[:, 0]
    xk, w64, g = x[keep].double(), w.double(), dl[keep].double()
    G = (xk @ w64.T - lse[keep].double()[:, None]).exp() * (g + dz[keep].double())[:, None]
    G[torch.arange(keep.numel(), device="cuda"), y[keep]] -= g
    for k, a, b, out in (("dx", G, w64, got["dx"][keep]), ("dweight", G.T.contiguous(), xk, got["dweight"])):
        ref = a @ b
        err = float((out.double() - ref).norm())
        if x.dtype == BF16:
            limit = 2.0 ** -8 / 3 ** 0.5 * float(((a * a) @ (b * b)).sum() + (ref * ref).sum()) ** 0.5
        else:
            limit = float(ref.norm()) * (2 * R.U * (6 * a.shape[1]) ** 0.5 + 2.0 ** -15)
        assert err <= limit, (k, err, limit, float(ref.norm()))


def rounds(m, n):
    """Whether an m x n output is more than one round of tiles and no whole number of them, whichever tile is taken."""
    tiles = lambda t: -(-m // t) * -(-n // t)  # noqa: E731
    return tiles(256) > 256 and tiles(256) % 256 and tiles(128) > 512 and tiles(128) % 512


@pytest.mark.parametrize("io", [BF16, F32])
@pytest.mark.parametrize("sizes", [(2100, 40000, 512), (9600, 300, 2100)], ids=["vocabulary", "width"])
def test_more_than_one_round(M, sizes, io):
    """2100 x 40000 x 512: logits, G and dweight; 9600 x 300 x 2100: dx, with a weight that is laid out first."""
    tokens, vocab, dim = sizes
    x, w, y, dl, dz = make(tokens, vocab, dim, io, 0.05, tokens + vocab)
    count = int((y >= 0).sum())
    if vocab > tokens:
        assert rounds(vocab, count) and rounds(dim, vocab)
    else:
        assert rounds(dim, count)
    say("more than one round", sizes, io)
    loss, lse = M.linear_cross_entropy_fwd(x, w, y)
    grads = M.linear_cross_entropy_bwd(x, w, y, lse, dl, dlse=dz)
    ref = reference(x, w, y, dloss=dl, dlse=dz, lse_in=lse)
    for k, got in {"loss": loss, "lse": lse, **grads}.items():
        R.check(got, ref[k], k)
    check_norms(grads, x, w, y, dl, dz, lse)
    again = M.linear_cross_entropy_bwd(x, w, y, lse, dl, dlse=dz)
    assert torch.equal(again["dx"], grads["dx"]) and torch.equal(again["dweight"], grads["dweight"])
    # added to an fp32 table, dx left out
    old = torch.randn(vocab, dim, device="cuda")
    ref = reference(x, w, y, dloss=dl, dlse=dz, lse_in=lse, old=old, grad_dtype=F32)
    got = M.linear_cross_entropy_bwd(x, w, y, lse, dl, dlse=dz, want_dx=False, dweight=old, accumulate=True)
    R.check(got["dweight"], ref["dweight"], "accumulated dweight")


@pytest.mark.parametrize("io", [BF16, F32])
def test_forward_in_pieces(M, io):
    """A million tokens, nearly all left out, and a vocabulary of several pieces in the forward pass: the maximum and sum
    carried between pieces, targets in each of them."""
    T, V, D = 1 << 20, 15000, 8
    need = M.linear_cross_entropy_fwd_workspace_size(T, V, D, M.MSSM_BF16 if io == BF16 else M.MSSM_F32)
    assert need < V // 64 * T * 8, "the partial sums of the whole vocabulary would fit: it is one piece"
    g = torch.Generator().manual_seed(18)
    keep = torch.randperm(T, generator=g)[:300].sort().values
    y = torch.full((T,), -100)
    y[keep] = torch.randint(0, V, (300,), generator=g)
    y[keep[:6]] = torch.tensor([0, V - 1, V // 2, 5119, 5120, 10240])
    x = torch.randn(T, D, generator=g).to(io)
    w = torch.randn(V, D, generator=g)
    w[7000:7010] *= 4.0      # the largest logits of most tokens lie in the middle piece
    w = w.to(io)
    dl = torch.rand(T, generator=g)
    say("forward in pieces", io)
    loss, lse = M.linear_cross_entropy_fwd(x.cuda(), w.cuda(), y.cuda())
    want = R.cross_entropy(x[keep], w, y[keep], dloss=dl[keep], lse_in=lse.cpu()[keep])
    R.check(loss[keep.cuda()], want["loss"], "loss")
    R.check(lse[keep.cuda()], want["lse"], "lse")
    assert int((loss != 0).sum()) <= 300
    grads = M.linear_cross_entropy_bwd(x.cuda(), w.cuda(), y.cuda(), lse, dl.cuda())
    R.check(grads["dx"][keep.cuda()], want["dx"], "dx")
    R.check(grads["dweight"], want["dweight"], "dweight")
    assert int((grads["dx"] != 0).any(1).sum()) <= 300
