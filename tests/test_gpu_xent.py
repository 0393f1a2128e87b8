"""Cross entropy of a linear head and its gradients on the GPU, against the plain 64-bit forms in model_ops."""
import math

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
    drop = torch.randperm(tokens, generator=g)[:int(tokens * left_out)]
    y[drop] = torch.tensor([-100, -1, vocab, vocab + 7])[torch.arange(drop.numel()) % 4]
    return x.to(io), w.to(io), y, torch.rand(tokens, generator=g) + 0.5, 0.1 * torch.randn(tokens, generator=g)


# (tokens, vocab, dim, io, share left out)
CASES = [
    (1, 1, 1, F32, 0.0),
    (1, 2, 64, BF16, 0.0),
    (2, 129, 8, BF16, 0.5),
    (3, 1000, 65, F32, 0.0),
    (16, 255, 64, BF16, 0.0),
    (17, 256, 128, BF16, 0.3),
    (63, 257, 100, BF16, 0.0),
    (64, 513, 192, F32, 0.2),
    (65, 700, 64, BF16, 0.0),
    (130, 1111, 77, BF16, 0.4),
    (200, 600, 320, BF16, 0.1),
    (257, 900, 200, F32, 0.1),
    (300, 2049, 256, BF16, 1.0),
    (513, 1500, 130, BF16, 0.9),
    (16, 33, 256, BF16, 0.1),
    (32, 1000, 640, BF16, 0.0),
    (30, 97, 72, F32, 0.5),
    (9, 500, 512, F32, 1.0),
]


@pytest.mark.parametrize("case", CASES, ids=lambda c: f"t{c[0]}_v{c[1]}_d{c[2]}_{str(c[3])[6:]}_o{c[4]}")
def test_cross_entropy(M, case):
    tokens, vocab, dim, io, left_out = case
    say("cross entropy", case)
    x, w, y, g, gz = make(tokens, vocab, dim, io, left_out, 3 * tokens + vocab)
    loss, lse = M.linear_cross_entropy_fwd(x.cuda(), w.cuda(), y.cuda())
    want = R.cross_entropy(x, w, y)
    R.check(loss, want["loss"], "loss")
    R.check(lse, want["lse"], "lse")
    for dlse in (None, gz):
        say("cross entropy gradients", case, dlse is not None)
        grads = M.linear_cross_entropy_bwd(x.cuda(), w.cuda(), y.cuda(), lse, g.cuda(),
                                           dlse=None if dlse is None else dlse.cuda())
        ref = R.cross_entropy(x, w, y, dloss=g, dlse=dlse, lse_in=lse.cpu())
        R.check(grads["dx"], ref["dx"], "dx")
        R.check(grads["dweight"], ref["dweight"], "dweight")
    again = M.linear_cross_entropy_bwd(x.cuda(), w.cuda(), y.cuda(), lse, g.cuda(), dlse=gz.cuda())
    assert torch.equal(again["dx"], grads["dx"]) and torch.equal(again["dweight"], grads["dweight"])
    # one at a time, and the weight's gradient added to what is there, in both types it may have
    only = M.linear_cross_entropy_bwd(x.cuda(), w.cuda(), y.cuda(), lse, g.cuda(), dlse=gz.cuda(), want_dweight=False)
    assert only["dweight"] is None and torch.equal(only["dx"], grads["dx"])
    for gd in {io, F32}:
        old = torch.randn(vocab, dim, generator=torch.Generator().manual_seed(1)).to(gd)
        got = M.linear_cross_entropy_bwd(x.cuda(), w.cuda(), y.cuda().int(), lse, g.cuda(), dlse=gz.cuda(),
                                         want_dx=False, dweight=old.cuda(), accumulate=True)
        ref = R.cross_entropy(x, w, y, dloss=g, dlse=gz, lse_in=lse.cpu(), old=old, grad_dtype=gd)
        assert got["dx"] is None
        R.check(got["dweight"], ref["dweight"], f"accumulated {gd}")


@pytest.mark.parametrize("io", [BF16, F32])
def test_gradient_against_differences(M, io):
    """d(sum loss * g + lse * gz) along random directions of x and of the weight, against differences of the
    64-bit forward at the same (rounded) point."""
    x, w, y, g, gz = make(12, 90, 24, io, 0.25, 77)
    loss, lse = M.linear_cross_entropy_fwd(x.cuda(), w.cuda(), y.cuda())
    grads = M.linear_cross_entropy_bwd(x.cuda(), w.cuda(), y.cuda(), lse, g.cuda(), dlse=gz.cuda())

    def f(x, w):
        o = R.cross_entropy(x, w, y)
        return float((o["loss"][0] * g.double() + o["lse"][0] * gz.double()).sum())

    torch.manual_seed(3)
    for name, t in (("dx", x), ("dweight", w)):
        for _ in range(5):
            d = torch.randn(t.shape, dtype=torch.float64)
            step = 1e-5
            plus, minus = (x.double(), w.double()), (x.double(), w.double())
            if name == "dx":
                plus, minus = (x.double() + step * d, w.double()), (x.double() - step * d, w.double())
            else:
                plus, minus = (x.double(), w.double() + step * d), (x.double(), w.double() - step * d)
            num = (f(*plus) - f(*minus)) / (2 * step)
            grad = grads[name].cpu().double()
            # the gradients' own rounding (half a step of each element, twice for bf16: G and the result)
            room = float((grad.abs() * d.abs()).sum()) * (2.0 ** -6 if io == BF16 else 2.0 ** -18) + 1e-6
            assert abs(float((grad * d).sum()) - num) <= room, name


def test_fp32_products_carry_24_bits(M):
    """Rows of the identity as weight: the logits are x itself, so the loss sees every bit of x; and the other way
    round, so it sees every bit of the weight."""
    g = torch.Generator().manual_seed(9)
    v = torch.randn(64, 64, generator=g)
    eye = torch.eye(64)
    y = torch.arange(64) % 64
    for x, w, logits in ((v, eye, v.double()), (eye, v.t().contiguous(), v.double())):
        loss, lse = (t.cpu().double() for t in M.linear_cross_entropy_fwd(x.cuda(), w.cuda(), y.cuda()))
        want = torch.logsumexp(logits, 1)
        # exact logits: what is left is the exponentials' sum (64 terms) and the logarithm
        assert (lse - want).abs().max() < 64 * R.U * 8
        hit = logits[torch.arange(64), y]
        assert (lse - loss - hit).abs().max() < 16 * R.U     # one subtraction of values below 8


@pytest.mark.parametrize("ex,ew,eg", [(0, 0, 0), (-70, 66, -90), (90, -92, 100), (-100, -20, 0), (3, -5, -120)])
def test_fp32_ranges(M, ex, ew, eg):
    """fp32 inputs of any size, with outliers 2^12 above the rest in some columns: the products keep fp32's accuracy.
    (The whole tensor's error, in the 2-norm: K roundings of 2^-24 at random add up to sqrt(K) of them; 16 times
    that, and no more than 2e-6.)"""
    g = torch.Generator().manual_seed(31)
    T, V, D = 90, 400, 160
    x = torch.randn(T, D, generator=g)
    w = torch.randn(V, D, generator=g) * 0.1
    x[:, 7] *= 4096.0
    w[:, 7] /= 4096.0
    w[:, 11] *= 64.0
    x[:, 11] /= 64.0
    y = torch.randint(0, V, (T,), generator=g)
    dl = (torch.rand(T, generator=g) + 0.5) * 2.0 ** eg
    x, w = x * 2.0 ** ex, w * 2.0 ** ew
    loss, lse = M.linear_cross_entropy_fwd(x.cuda(), w.cuda(), y.cuda())
    grads = M.linear_cross_entropy_bwd(x.cuda(), w.cuda(), y.cuda(), lse, dl.cuda())
    want = R.cross_entropy(x, w, y, dloss=dl, lse_in=lse.cpu())
    got = {"loss": loss, "lse": lse, **grads}
    for k in ("loss", "lse", "dx", "dweight"):
        ref, out = want[k][0], got[k].cpu().double()
        # (what lies above fp32's largest number, 2^128, comes out as infinity)
        over = ref.abs() >= 2.0 ** 128
        assert torch.equal(out[over], torch.sign(ref[over]) * float("inf")), k
        ref, out = ref[~over], out[~over]
        err = float((out - ref).norm())
        # (what lies below fp32's normal numbers, 2^-126, may come out as 0: at most 2^-126 an element)
        assert err <= 2e-6 * float(ref.norm()) + 2.0 ** -126 * ref.numel() ** 0.5, (k, err, float(ref.norm()))


def test_rows_left_out_are_not_read(M):
    """NaN and infinities in the x of tokens that do not count, and in their dloss, reach nothing."""
    x, w, y, g, gz = make(150, 300, 64, BF16, 0.0, 5)
    y[10:60] = -100
    y[149] = 300
    clean = [t.cuda() for t in (x, w, y, g, gz)]
    loss, lse = M.linear_cross_entropy_fwd(*clean[:3])
    a = M.linear_cross_entropy_bwd(*clean[:3], lse, clean[3], dlse=clean[4])
    x2, g2, gz2, lse2 = x.clone(), g.clone(), gz.clone(), lse.clone()
    out = [*range(10, 60), 149]
    x2[out[:25]] = float("nan")
    x2[out[25:]] = float("inf")
    g2[out] = float("nan")
    gz2[out] = float("inf")
    lse2[out] = float("nan")
    loss2, lse_again = M.linear_cross_entropy_fwd(x2.cuda(), clean[1], clean[2])
    b = M.linear_cross_entropy_bwd(x2.cuda(), clean[1], clean[2], lse2, g2.cuda(), dlse=gz2.cuda())
    assert torch.equal(loss, loss2) and torch.equal(lse, lse_again)
    assert torch.equal(a["dx"], b["dx"]) and torch.equal(a["dweight"], b["dweight"])
    assert float(b["dx"][out].abs().max()) == 0.0 and float(loss2[out].abs().max()) == 0.0


def test_ignore_id_inside_the_vocabulary(M):
    x, w, y, g, _ = make(50, 40, 64, F32, 0.0, 6)
    y[::3] = 0
    loss, lse = M.linear_cross_entropy_fwd(x.cuda(), w.cuda(), y.cuda(), ignore_id=0)
    want = R.cross_entropy(x, w, y, ignore_id=0)
    R.check(loss, want["loss"], "loss")
    grads = M.linear_cross_entropy_bwd(x.cuda(), w.cuda(), y.cuda(), lse, g.cuda(), ignore_id=0)
    ref = R.cross_entropy(x, w, y, ignore_id=0, dloss=g, lse_in=lse.cpu())
    R.check(grads["dx"], ref["dx"], "dx")
    R.check(grads["dweight"], ref["dweight"], "dweight")


def test_large_logits(M):
    """Logits far apart and far from zero: the running maximum keeps the sums finite, certain tokens lose 0."""
    w = torch.zeros(500, 64)
    w[:, 0] = torch.linspace(-3e4, 3e4, 500)
    x = torch.zeros(4, 64)
    x[:, 0] = torch.tensor([1.0, -1.0, 1e3, 0.0])
    y = torch.tensor([499, 0, 0, 7])
    loss, lse = (t.cpu() for t in M.linear_cross_entropy_fwd(x.cuda(), w.cuda(), y.cuda()))
    assert float(loss[0]) == 0.0 and float(loss[1]) == 0.0 and float(loss[2]) == 6e7
    assert abs(float(loss[3]) - math.log(500)) < 1e-5
    g = M.linear_cross_entropy_bwd(x.cuda(), w.cuda(), y.cuda(), lse.cuda(), torch.ones(4).cuda())
    assert torch.isfinite(g["dx"]).all() and torch.isfinite(g["dweight"]).all()
    assert float(g["dx"][0].abs().max()) == 0.0


def test_no_tokens(M):
    w = torch.randn(20, 64).cuda()
    x, y = torch.zeros(0, 64).cuda(), torch.zeros(0, dtype=torch.int64).cuda()
    loss, lse = M.linear_cross_entropy_fwd(x, w, y)
    assert loss.shape == (0,)
    g = M.linear_cross_entropy_bwd(x, w, y, lse, loss, dweight=torch.ones(20, 64).cuda())
    assert g["dx"].shape == (0, 64) and float(g["dweight"].abs().max()) == 0.0


def test_refusals(M):
    x, w, y, g, _ = (t.cuda() for t in make(8, 30, 64, BF16, 0.0, 7))
    with pytest.raises(TypeError):
        M.linear_cross_entropy_fwd(x, w.float(), y)
    with pytest.raises(TypeError):
        M.linear_cross_entropy_fwd(x, w, y.float())
    with pytest.raises(ValueError):
        M.linear_cross_entropy_fwd(x[:, :32].contiguous(), w, y)
    with pytest.raises(ValueError, match="contiguous"):
        M.linear_cross_entropy_fwd(x[:, ::2], w[:, :32].contiguous(), y)
    with pytest.raises(ValueError, match="shape"):
        M.linear_cross_entropy_fwd(x, w, y[:7])
    with pytest.raises(ValueError, match="GPU tensor"):
        M.linear_cross_entropy_fwd(x, w, y.cpu())
    with pytest.raises(M.MssmError):
        M.linear_cross_entropy_fwd(x, w, y, workspace=torch.empty(256, dtype=torch.uint8, device="cuda"))
    buf = torch.zeros(30 * 64 + 1, dtype=BF16).cuda()
    with pytest.raises(M.MssmError) as e:     # weight read in place must be 16-byte aligned
        M.linear_cross_entropy_fwd(x, buf[1:].view(30, 64), y)
    assert e.value.status == M.MSSM_ERR_MISALIGNED
    lse = torch.zeros(8).cuda()
    with pytest.raises(ValueError, match="nothing"):
        M.linear_cross_entropy_bwd(x, w, y, lse, g, want_dx=False, want_dweight=False)
    with pytest.raises(ValueError, match="accumulate"):
        M.linear_cross_entropy_bwd(x, w, y, lse, g, accumulate=True)
    with pytest.raises(M.MssmError):
        M.linear_cross_entropy_bwd(x, w, y, lse, g, dx=x)
