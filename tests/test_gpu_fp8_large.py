"""The 8-bit linear layer at large sizes: every tile kernel with slices and accumulation, offsets beyond 32 bits, the most
tokens.  References in 64 bits on the GPU, from values that fp8_dequantize gives exactly."""
import pytest
import torch

import fp8_ops as Q
import model_ops as R
from gpu_util import say

pytestmark = pytest.mark.gpu
BF16, F32, F64 = torch.bfloat16, torch.float32, torch.float64


@pytest.fixture(scope="module")
def M():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import selective_state_space_17_amd as m
    yield m
    torch.cuda.empty_cache()


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def rnd(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda")


def vals(M, m):
    return M.fp8_dequantize(m, F32).double()


@pytest.mark.parametrize("square", [False, True], ids=["rows", "square"])
@pytest.mark.parametrize("shape", [(2560, 16384, 2560), (9000, 200, 3001), (6000, 1500, 5000), (70, 9000, 3000), (40, 300, 9000)],
                         ids=str)
def test_fwd(M, shape, square):
    tokens, k, n = shape
    say("large fp8 linear", shape, square)
    g = gen(tokens + k)
    x = M.fp8_quantize(rnd(g, tokens, k) * torch.exp(rnd(g, k)))
    w = M.fp8_quantize(rnd(g, n, k) * torch.exp(rnd(g, n, 1)), square=square)
    xv, wv = vals(M, x), vals(M, w)
    for dt in (BF16, F32):
        R.check(M.fp8_linear_fwd(x, w, out_dtype=dt), Q.product_of_values(xv, wv, dt, chunk=256), f"out {dt}")


@pytest.mark.parametrize("dw_dtype", [BF16, F32], ids=str)
def test_bwd(M, dw_dtype):
    """16384 tokens: dx in whole rounds and a last one, dweight cut along its tokens, added to what was there."""
    tokens, k, n = 16384, 2560, 2500
    say("large fp8 linear gradients", dw_dtype)
    g = gen(9)
    x = M.fp8_quantize(rnd(g, tokens, k))
    wt = M.fp8_quantize(rnd(g, k, n) * k ** -0.5, square=True)
    dout = (rnd(g, tokens, n) * 1e-3).to(BF16)
    old = rnd(g, n, k).to(dw_dtype)
    dw = old.clone()
    got = M.fp8_linear_bwd(x, wt, dout, dweight=dw, accumulate=True)
    rows, cols = M.fp8_quantize(dout, both=True)
    R.check(got["dx"], Q.product_of_values(vals(M, rows), vals(M, wt), BF16, chunk=256), "dx")
    want = Q.product_of_values(vals(M, cols), vals(M, M.fp8_transpose(x)), dw_dtype, old=old, chunk=256)
    R.check(dw, want, "dweight")


def test_most_tokens(M):
    """2^22 tokens less a few: outputs and inputs beyond 2^32 bytes, and the longest sums."""
    tokens, k, n = (1 << 22) - 5, 130, 1100
    say("most tokens")
    g = gen(10)
    base, wide = rnd(g, 64, k).to(BF16), rnd(g, 64, n).to(BF16) * 1e-3
    w = M.fp8_quantize(rnd(g, n, k), square=True)
    x = M.fp8_quantize(base.repeat(tokens // 64 + 1, 1)[:tokens])
    out = M.fp8_linear_fwd(x, w)
    assert out.numel() * 2 > 1 << 33
    want = M.fp8_linear_fwd(M.fp8_quantize(base.repeat(4, 1)), w)      # on other tiles: the bounds of either
    few = M.fp8_quantize(base)
    ref, bound = Q.product_of_values(vals(M, few), vals(M, w), BF16)
    R.check(want[:64], (ref, bound), "64 rows")
    for lo in (0, 1 << 21, tokens - 64):
        i = (torch.arange(lo, lo + 64) % 64)
        R.check(out[lo:lo + 64], (ref[i], bound[i]), f"rows from {lo}")
    assert torch.equal(out[:1 << 21][::64], out[:1 << 21][:1].expand(1 << 15, n))
    del out
    dout = wide.repeat(tokens // 64 + 1, 1)[:tokens]
    got = M.fp8_linear_bwd(x, None, dout, want_dx=False, dweight_dtype=F32)["dweight"]
    # the sum over equal groups of 64 tokens, and the last one's first 59: blocks of 128 tokens hold two groups, so that
    # their scales are one group's, but the last block's
    whole = tokens // 128 * 128
    dq, xq = M.fp8_quantize(wide.repeat(2, 1), transposed=True), M.fp8_transpose(M.fp8_quantize(base.repeat(2, 1)))
    dl, xl = M.fp8_quantize(dout[whole:], transposed=True), M.fp8_transpose(M.fp8_quantize(base.repeat(2, 1)[:tokens - whole]))
    many = whole // 128
    ref = (vals(M, dq) @ vals(M, xq).T) * many + vals(M, dl) @ vals(M, xl).T
    mag = (vals(M, dq).abs() @ vals(M, xq).T.abs()) * many + vals(M, dl).abs() @ vals(M, xl).T.abs()
    # fp32 sums over 2^22 products, 32 slices of them at most: every addition may lose 2 u of the running sum, which is at
    # most mag
    bound = mag * 2 * (tokens + 64) * 2.0 ** -24
    err = (got.double() - ref).abs()
    assert bool((err <= bound).all())


@pytest.mark.parametrize("accumulate", [False, True])
def test_no_tokens_many_tiles(M, accumulate):
    """A gradient of more tiles of 64 x 64 than a launch takes, of no tokens: zeros everywhere, or what was there."""
    n, k = 65600, 65600
    say("fp8 weight gradient of no tokens", n, k, accumulate)
    x = M.fp8_quantize(torch.empty(0, k, device="cuda"))
    dw = torch.full((n, k), 1.5, device="cuda", dtype=BF16)
    M.fp8_linear_bwd(x, None, torch.empty(0, n, device="cuda", dtype=BF16), want_dx=False, dweight=dw,
                     accumulate=accumulate)
    want = 1.5 if accumulate else 0.0
    assert dw.min().item() == want and dw.max().item() == want


# one for each tile of the kernel for few rows: 16 x 16, 32 x 32, 64 x 32, 64 x 64
@pytest.mark.parametrize("square", [False, True], ids=["rows", "square"])
@pytest.mark.parametrize("shape", [(33, 1000, 777), (29, 2500, 5003), (61, 2561, 5090), (301, 1000, 2561)], ids=str)
def test_few_rows(M, shape, square):
    tokens, k, n = shape
    say("few rows of fp8 linear", shape, square)
    g = gen(tokens)
    x = M.fp8_quantize(rnd(g, tokens, k) * torch.exp(rnd(g, k)))
    w = M.fp8_quantize(rnd(g, n, k) * torch.exp(rnd(g, n, 1)), square=square)
    xv, wv = vals(M, x), vals(M, w)
    for dt in (BF16, F32):
        R.check(M.fp8_linear_fwd(x, w, out_dtype=dt), Q.product_of_values(xv, wv, dt, chunk=64), f"out {dt}")


@pytest.mark.parametrize("io", [BF16, F32], ids=str)
@pytest.mark.parametrize("shape", [(70, 130, 90), (300, 700, 600), (500, 1000, 1500), (40, 2560, 2000)], ids=str)
def test_gradients_of_few_rows(M, shape, io):
    """Both products small: side by side in one launch where their tiles are the same, else one after the other."""
    tokens, k, n = shape
    say("small gradients of fp8 linear", shape, io)
    g = gen(tokens + n)
    x = M.fp8_quantize(rnd(g, tokens, k))
    wt = M.fp8_quantize(rnd(g, k, n) * k ** -0.5, square=True)
    dout = (rnd(g, tokens, n) * 1e-3).to(io)
    old = rnd(g, n, k).to(io)
    d, dt = M.fp8_quantize(dout, both=True)
    dw_rows, x_rows = vals(M, dt), vals(M, M.fp8_transpose(x))
    for accumulate in (False, True):
        dw = old.clone()
        got = M.fp8_linear_bwd(x, wt, dout, dweight=dw, accumulate=accumulate)
        R.check(got["dx"], Q.product_of_values(vals(M, d), vals(M, wt), io), "dx")
        R.check(dw, Q.product_of_values(dw_rows, x_rows, io, old if accumulate else None), "dweight")
