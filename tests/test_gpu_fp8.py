"""Matrices in 8 bits, the norm that writes one, and the linear layer on them, against the plain 64-bit forms."""
import pytest
import torch

import fp8_ops as Q
import model_ops as R
from gpu_util import say

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32
NAN, INF = float("nan"), float("inf")


@pytest.fixture(scope="module")
def M():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import selective_state_space_17_amd as m
    return m


def gen(seed):
    return torch.Generator().manual_seed(seed)


def spread(g, rows, cols, io):
    """Values whose rows and columns differ in size."""
    return (torch.randn(rows, cols, generator=g) * torch.exp(torch.randn(cols, generator=g)) *
            torch.exp(torch.randn(rows, 1, generator=g))).to(io)


SHAPES = [(1, 1), (1, 128), (1, 129), (2, 7), (3, 127), (4, 130), (5, 256), (127, 64), (128, 128), (129, 257), (130, 1),
          (301, 1000), (64, 5121), (1030, 333)]


# ------------------------------------------------------------------------------------------------- to 8 bits and back
@pytest.mark.parametrize("square", [False, True], ids=["rows", "square"])
@pytest.mark.parametrize("io", [BF16, F32], ids=str)
@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_quantize(M, shape, io, square):
    say("fp8 quantize", shape, io, square)
    x = spread(gen(shape[0] * 7 + shape[1]), *shape, io)
    want, want_t = Q.quantize(x, square), Q.quantize(x.T, square)
    xc = x.cuda()
    a, b = M.fp8_quantize(xc, square=square, both=True)
    Q.same(a, want, "codes of x")
    Q.same(b, want_t, "codes of its transpose")
    Q.same(M.fp8_quantize(xc, square=square), want, "x alone")
    Q.same(M.fp8_quantize(xc, square=square, transposed=True), want_t, "the transpose alone")
    if square:
        assert torch.equal(Q.values(Q.of_gpu(a)), Q.values(Q.of_gpu(b)).T), "a square block has the same values either way"
    for dt in (F32, BF16):
        back = M.fp8_dequantize(a, dt)
        assert back.dtype == dt and torch.equal(back.cpu().double(), Q.values(want))
    if not square:
        back = Q.quantize(Q.values(want).T)
        Q.same(M.fp8_transpose(a), back, "laid out the other way from 8 bits")


@pytest.mark.parametrize("square", [False, True], ids=["rows", "square"])
@pytest.mark.parametrize("io", [BF16, F32], ids=str)
def test_blocks_that_hold_little_or_too_much(M, io, square):
    """Blocks of zeros, of denormals, at the types' ends, at the borders of a scale, and with values that are not finite."""
    tiny, huge = torch.finfo(io).tiny, torch.finfo(io).max
    x = torch.randn(300, 700, generator=gen(3)).to(io)
    x[0, :128] = 0
    x[1, :128] = torch.arange(128).to(io) * (tiny / 64)
    x[2, :128] = huge
    x[3, :128] = torch.linspace(-1, 1, 128).to(io) * huge
    x[4, 5], x[5, 6], x[6, 7] = NAN, INF, -INF
    x[7, 128:256] = NAN
    x[8, 128:256] = INF
    for i, v in enumerate((448.0, 448.0 * 2 ** 5, 450.0, 452.0, 464.0, 256.0, 224.0, 1.75, 1.7578125, 2.0 ** -120)):
        x[10 + i, 256:384] = torch.linspace(-v, v, 128).to(io)
        x[10 + i, 300] = v
    x[150:280, 384:512] = 0
    x[128:256, 512:640] *= 2.0 ** -60
    x = torch.where(x.abs() < tiny / 1024, torch.zeros_like(x), x)
    a, b = M.fp8_quantize(x.cuda(), square=square, both=True)
    Q.same(a, Q.quantize(x, square), "codes")
    Q.same(b, Q.quantize(x.T, square), "transposed codes")


def test_ties_go_to_even(M):
    """Every midpoint between neighbouring e4m3 values, and its fp32 neighbours, under a scale of one."""
    v = torch.arange(127, dtype=torch.uint8).view(torch.float8_e4m3fn).float()
    mid = (v[1:] + v[:-1]) / 2
    x = torch.cat([mid, torch.nextafter(mid, mid + 1), torch.nextafter(mid, mid - 1), -mid])
    x = torch.nn.functional.pad(x, (0, -x.numel() % 127)).reshape(-1, 127)
    x = torch.cat([x, torch.full((x.shape[0], 1), 448.0)], 1)
    got = M.fp8_quantize(x.cuda())
    assert bool((got.scales.view(torch.uint8)[:, :x.shape[0]] == 127).all())
    Q.same(got, Q.quantize(x), "midpoints")


def test_transpose_keeps_values(M):
    """Rows of one size, under any scale: laid out the other way they are what they were, bit for bit."""
    g = gen(5)
    x = (torch.rand(260, 390, generator=g) + 0.5) * 2.0 ** -30
    a = M.fp8_quantize(x.cuda())
    assert torch.equal(M.fp8_dequantize(M.fp8_transpose(a), F32), M.fp8_dequantize(a, F32).T)


def test_matrix_with_nan_and_extreme_scales(M):
    """A matrix that came from elsewhere: scales of 2^-127, 2^127 and NaN."""
    codes = torch.randn(9, 256, generator=gen(6)).to(torch.float8_e4m3fn)
    scales = torch.full((2, 12), 127, dtype=torch.uint8)
    scales[0, 0], scales[0, 1], scales[1, 2], scales[1, 3] = 0, 254, 255, 120
    m = M.Fp8Matrix(codes.cuda(), scales.view(torch.float8_e8m0fnu).cuda(), 256)
    got = M.fp8_dequantize(m, F32).cpu()
    want = codes.float().reshape(9, 2, 128) * scales[:, :9].T.view(torch.float8_e8m0fnu).float()[:, :, None]
    want = want.reshape(9, 256)
    assert torch.equal(got.isnan(), want.isnan()) and got[2, 128:].isnan().all()
    assert torch.equal(got[~want.isnan()], want[~want.isnan()])


def test_many_rows(M):
    """More than 2^32 codes: offsets need 64 bits.  Rows that repeat, so that the result is known without 64-bit copies."""
    rows, cols = (1 << 22) - 3, 1100
    base = torch.randn(8, cols, generator=gen(8)).to(BF16)
    x = base.cuda().repeat(rows // 8 + 1, 1)[:rows]
    m = M.fp8_quantize(x)
    del x
    assert m.codes.numel() > 1 << 32
    want = Q.quantize(base)
    codes = want[0].float().to(torch.float8_e4m3fn).view(torch.uint8).cuda()
    scales = want[1][:, :8].cuda()
    got_s = m.scales.view(torch.uint8)
    for lo in (0, 1 << 20, rows - 4093):
        got = m.codes[lo:lo + 4093].view(torch.uint8)
        i = (torch.arange(lo, lo + 4093, device="cuda") % 8)
        assert torch.equal(got, codes[i]) and torch.equal(got_s[:, lo:lo + 4093], scales[:, i])
    tail = M.fp8_dequantize(m, BF16)[-1].cpu().double()
    assert torch.equal(tail, Q.values(want)[(rows - 1) % 8])


# ------------------------------------------------------------------------------------------------------------- norm
NORMS = [(1, 1, F32, None), (1, 2, BF16, F32), (3, 127, BF16, BF16), (5, 128, F32, F32), (4, 130, BF16, None),
         (130, 250, BF16, F32), (9, 513, F32, None), (66, 512, BF16, BF16), (2101, 72, BF16, None),
         (7, 1000, BF16, F32), (5, 1023, F32, F32), (150, 1032, F32, None), (11, 2560, BF16, F32), (35, 2050, BF16, BF16),
         (4, 5120, BF16, F32), (3, 9000, F32, F32), (2, 16384, BF16, F32), (3, 16392, BF16, BF16), (70, 20001, BF16, F32)]


@pytest.mark.parametrize("kind", ["layer", "rms"])
@pytest.mark.parametrize("case", NORMS, ids=lambda c: f"r{c[0]}_d{c[1]}_{str(c[2])[6:]}_{str(c[3])[6:]}")
def test_norm(M, case, kind):
    rows, dim, io, res = case
    layer = kind == "layer"
    say("norm fp8", kind, case)
    g = gen(31 * rows + dim)
    x = (torch.randn(rows, dim, generator=g) * 0.8 + 0.3).to(io)
    r = None if res is None else (torch.randn(rows, dim, generator=g) * 2).to(res)
    w, b = 1 + 0.2 * torch.randn(dim, generator=g), 0.1 * torch.randn(dim, generator=g)
    args = (x.cuda(), w.cuda()) + ((b.cuda(),) if layer else ())
    rc = None if r is None else r.cuda()
    fwd = M.layer_norm_fp8_fwd if layer else M.rms_norm_fp8_fwd
    got = list(fwd(*args, residual=rc, return_residual=r is not None, return_stats=True))
    plain = list((M.layer_norm_fwd if layer else M.rms_norm_fwd)(*args, residual=rc, return_residual=r is not None,
                                                                 return_stats=True))
    for a, p in zip(got[1:], plain[1:]):
        assert torch.equal(a, p), "the stream and the statistics are those of the plain norm"
    want = R.norm_fwd(x, r, w, b if layer else None, 1e-5, layer, res)
    ref, bound = want["out"]
    bound = bound - ref.abs() * R.half_step(io)      # without the rounding to x's type
    m = Q.of_gpu(got[0])
    codes, scales, cols, _ = m
    assert cols == dim and bool((codes[:, dim:] == 0).all())
    s = scales[:, :rows].to(torch.int64)
    least, most = Q.tops((ref.abs() - bound).clamp(min=0)), Q.tops(ref.abs() + bound)
    assert bool((s >= Q.scale_byte(least).T).all()) and bool((s <= Q.scale_byte(most).T).all()), "scales"
    assert bool((scales[:, rows:] == 127).all())
    step = torch.exp2(s.to(R.F64) - 127).T.repeat_interleave(128, 1)[:, :dim] * 2.0 ** -10
    R.check(Q.values(m), (ref, bound * 1.0625 + torch.maximum(ref.abs() * 2.0 ** -4, step)), "out")


def test_norm_rows_of_nan_stay_alone(M):
    x = torch.randn(6, 300, generator=gen(9))
    clean = Q.of_gpu(M.layer_norm_fp8_fwd(x.cuda(), torch.ones(300).cuda()))
    x[2, 5], x[4, 0] = NAN, INF
    got = Q.of_gpu(M.layer_norm_fp8_fwd(x.cuda(), torch.ones(300).cuda()))
    keep = [0, 1, 3, 5]
    assert torch.equal(got[0][keep], clean[0][keep]) and torch.equal(got[1][:, keep], clean[1][:, keep])
    assert got[0][2, :300].isnan().all() and got[0][4, :300].isnan().any() and bool((got[0][:, 300:] == 0).all())
    zero = Q.of_gpu(M.rms_norm_fp8_fwd(torch.zeros(3, 200).cuda(), torch.ones(200).cuda()))
    assert bool((zero[0] == 0).all()) and bool((zero[1] == 127).all())


# ----------------------------------------------------------------------------------------------------------- product
def operands(g, tokens, k, n, square=True):
    x = Q.quantize(spread(g, tokens, k, F32))
    w = Q.quantize(torch.randn(n, k, generator=g) * k ** -0.5, square)
    return x, w


LINEAR = [(1, 1, 1), (1, 128, 16), (1, 2560, 333), (2, 130, 65), (7, 1000, 777), (8, 5120, 260), (16, 384, 1024),
          (17, 256, 96), (33, 700, 130), (64, 257, 257), (65, 1152, 300), (100, 129, 129), (128, 1000, 256), (200, 320, 513),
          (257, 640, 640), (301, 1000, 777), (513, 2000, 300), (1030, 256, 1030)]


@pytest.mark.parametrize("out_dtype", [BF16, F32], ids=str)
@pytest.mark.parametrize("shape", LINEAR, ids=str)
def test_linear_fwd(M, shape, out_dtype):
    tokens, k, n = shape
    say("fp8 linear", shape, out_dtype)
    x, w = operands(gen(tokens + k + n), *shape)
    xg, wg = Q.to_gpu(M, x), Q.to_gpu(M, w)
    got = M.fp8_linear_fwd(xg, wg, out_dtype=out_dtype)
    assert got.shape == (tokens, n) and got.dtype == out_dtype
    R.check(got, Q.product(x, w, out_dtype), "out")
    assert torch.equal(got, M.fp8_linear_fwd(xg, wg, out_dtype=out_dtype)), "differs between two calls"


# enough tiles for every kernel: whole rounds and a last one, whole or cut along k, ragged on either side
TILES = [(4100, 260, 5000), (9000, 129, 3001), (2048, 1408, 2048), (2300, 1000, 2500), (300, 4096, 520), (5000, 8, 4000),
         (1500, 2900, 1300)]


@pytest.mark.parametrize("square", [False, True], ids=["rows", "square"])
@pytest.mark.parametrize("out_dtype", [BF16, F32], ids=str)
@pytest.mark.parametrize("shape", TILES, ids=str)
def test_linear_fwd_of_many_tiles(M, shape, out_dtype, square):
    tokens, k, n = shape
    say("fp8 linear of many tiles", shape, out_dtype, square)
    x, w = operands(gen(tokens + k + n), tokens, k, n, square)
    got = M.fp8_linear_fwd(Q.to_gpu(M, x), Q.to_gpu(M, w), out_dtype=out_dtype)
    R.check(got, Q.product(x, w, out_dtype, chunk=512, device="cuda"), "out")


@pytest.mark.parametrize("shape", [(3000, 2100, 2400), (20000, 300, 200)], ids=str)
def test_linear_bwd_of_many_tiles(M, shape):
    tokens, k, n = shape
    say("fp8 linear gradients of many tiles", shape)
    g = gen(17)
    x, w = operands(g, *shape)
    wt = Q.quantize(Q.values(w).T, True)
    dout = spread(g, tokens, n, F32).mul(1e-3).to(BF16)
    old = torch.randn(n, k, generator=g).to(BF16)
    got = M.fp8_linear_bwd(Q.to_gpu(M, x), Q.to_gpu(M, wt), dout.cuda(), dweight=old.cuda(), accumulate=True)
    R.check(got["dx"], Q.product(Q.quantize(dout), wt, BF16, chunk=512, device="cuda"), "dx")
    want = Q.product(Q.quantize(dout.T), Q.quantize(Q.values(x).T), BF16, old=old, chunk=512, device="cuda")
    R.check(got["dweight"], want, "dweight")


@pytest.mark.parametrize("io", [BF16, F32], ids=str)
@pytest.mark.parametrize("shape", [(1, 1, 5), (1, 2560, 640), (3, 333, 130), (16, 640, 256), (40, 1000, 96), (300, 384, 200)],
                         ids=str)
def test_linear_fwd_of_a_plain_input(M, shape, io):
    """x in its own type: what fp8_quantize and the product of its result give, bit for bit."""
    tokens, k, n = shape
    say("fp8 linear of a plain input", shape, io)
    g = gen(tokens * k + n)
    x = spread(g, tokens, k, io).cuda()
    w = Q.to_gpu(M, Q.quantize(torch.randn(n, k, generator=g), True))
    for out_dtype in (BF16, F32):
        got = M.fp8_linear_fwd(x, w, out_dtype=out_dtype)
        assert torch.equal(got, M.fp8_linear_fwd(M.fp8_quantize(x), w, out_dtype=out_dtype))
    assert M.fp8_linear_fwd(x.reshape(1, tokens, 1, k), w).shape == (1, tokens, 1, n)


@pytest.mark.parametrize("shape", [(5, 300, 140), (140, 300, 300), (300, 1000, 520)], ids=str)
def test_linear_fwd_with_scales_of_the_weights_rows(M, shape):
    say("fp8 linear, weight with scales of rows", shape)
    g = gen(77)
    x = Q.quantize(spread(g, shape[0], shape[1], F32))
    w = Q.quantize(spread(g, shape[2], shape[1], F32), False)
    for out_dtype in (BF16, F32):
        R.check(M.fp8_linear_fwd(Q.to_gpu(M, x), Q.to_gpu(M, w), out_dtype=out_dtype), Q.product(x, w, out_dtype), "out")


def test_linear_fwd_nan_and_outer_scales(M):
    """NaN stays in its row and its column; blocks many powers of two apart are each taken at their own scale."""
    g = gen(12)
    x, w = spread(g, 70, 300, F32), torch.randn(140, 300, generator=g)
    x[3, 5], x[60, 299] = NAN, INF
    w[7, 0], w[139, 200] = NAN, -INF
    x[10] *= 2.0 ** 90
    x[11] *= 2.0 ** -90
    x[12, :128] *= 2.0 ** 40
    qx, qw = Q.quantize(x), Q.quantize(w, True)
    bad = torch.zeros(70, 140, dtype=torch.bool)
    bad[[3, 60]] = True
    bad[:, [7, 139]] = True
    clean_x, clean_w = (qx[0].nan_to_num(0.0), *qx[1:]), (qw[0].nan_to_num(0.0), *qw[1:])
    for out_dtype in (BF16, F32):
        got = M.fp8_linear_fwd(Q.to_gpu(M, qx), Q.to_gpu(M, qw), out_dtype=out_dtype).cpu()
        assert torch.equal(got.isnan(), bad)
        ref, bound = Q.product(clean_x, clean_w, out_dtype)
        err = (got.double() - ref).abs()
        assert bool((err[~bad] <= bound[~bad]).all())


def test_fp32_results_keep_more(M):
    """A large product next to small ones: whole in fp32."""
    x, w = torch.zeros(20, 128), torch.zeros(30, 128)
    x[:, 0], w[:, 0] = 16.0, 16.0
    x[:, 1:9], w[:, 1:9] = 2.0 ** -4, 1.5 * 2.0 ** -4
    got = M.fp8_linear_fwd(M.fp8_quantize(x.cuda()), M.fp8_quantize(w.cuda(), square=True), out_dtype=F32)
    assert bool((got == 256 + 8 * 1.5 * 2.0 ** -8).all())


# --------------------------------------------------------------------------------------------------------- gradients
GRADS = [(1, 1, 1), (1, 130, 7), (2, 64, 200), (17, 333, 130), (128, 256, 128), (129, 100, 300), (300, 1000, 777),
         (1000, 384, 260), (2100, 129, 64)]


@pytest.mark.parametrize("io,dw_dtype", [(BF16, BF16), (BF16, F32), (F32, F32)], ids=["bf16", "bf16_f32", "f32"])
@pytest.mark.parametrize("shape", GRADS, ids=str)
def test_linear_bwd(M, shape, io, dw_dtype):
    tokens, k, n = shape
    say("fp8 linear gradients", shape, io, dw_dtype)
    g = gen(3 * tokens + k + n)
    x, w = operands(g, *shape)
    wt = Q.quantize(Q.values(w).T, True)
    dout = spread(g, tokens, n, F32).mul(1e-3).to(io)
    xg, wg, dg = Q.to_gpu(M, x), Q.to_gpu(M, wt), dout.cuda()
    got = M.fp8_linear_bwd(xg, wg, dg, dweight_dtype=dw_dtype)
    want_dx = Q.product(Q.quantize(dout), wt, io)
    qd, qx = Q.quantize(dout.T), Q.quantize(Q.values(x).T)
    R.check(got["dx"], want_dx, "dx")
    R.check(got["dweight"], Q.product(qd, qx, dw_dtype), "dweight")
    assert got["dx"].shape == (tokens, k) and got["dweight"].shape == (n, k)
    again = M.fp8_linear_bwd(xg, wg, dg, dweight_dtype=dw_dtype)
    assert all(torch.equal(got[i], again[i]) for i in got), "differs between two calls"
    one = M.fp8_linear_bwd(None, wg, dg, want_dweight=False)
    assert one["dweight"] is None and torch.equal(one["dx"], got["dx"])
    one = M.fp8_linear_bwd(xg, None, dg, want_dx=False, dweight_dtype=dw_dtype)
    assert one["dx"] is None and torch.equal(one["dweight"], got["dweight"])
    old = torch.randn(n, k, generator=g).to(dw_dtype)
    acc = M.fp8_linear_bwd(xg, None, dg, want_dx=False, dweight=old.cuda(), accumulate=True)["dweight"]
    R.check(acc, Q.product(qd, qx, dw_dtype, old=old), "dweight added to what was there")


def test_bwd_against_differences(M):
    """Gradients of sum(out * dout) by central differences of the 64-bit forward in x and in the weight, where dout and
    the transposed x are numbers of 8 bits, so that nothing is rounded."""
    g = gen(21)
    few = torch.tensor([-2.0, -1.5, -1.0, -0.5, 0.5, 1.0, 1.25, 1.75])
    pick = lambda *s: few[torch.randint(0, 8, s, generator=g)]  # noqa: E731
    x, w, dout = pick(9, 13), pick(11, 13), pick(9, 11)
    loss = lambda a, b: float((a.double() @ b.double().T * dout.double()).sum())  # noqa: E731
    got = M.fp8_linear_bwd(M.fp8_quantize(x.cuda()), M.fp8_quantize(w.cuda(), square=True, transposed=True), dout.cuda())
    for which, t, grad in ((0, x, got["dx"]), (1, w, got["dweight"])):
        d = torch.zeros(t.shape, dtype=torch.float64)
        for i in range(t.numel()):
            e = torch.zeros(t.numel(), dtype=torch.float64)
            e[i] = 0.25
            hi, lo = t + e.reshape(t.shape), t - e.reshape(t.shape)
            d.view(-1)[i] = (loss(hi, w) - loss(lo, w) if which == 0 else loss(x, hi) - loss(x, lo)) / 0.5
        # sums of at most 13 products of multiples of 2^-4 below 4: exact in fp32
        assert torch.equal(grad.cpu().double(), d)


def test_no_tokens(M):
    wt = M.fp8_quantize(torch.randn(70, 130).cuda(), square=True)            # [in 70, out 130]
    w = M.fp8_quantize(torch.randn(130, 70).cuda(), square=True)
    x = M.fp8_quantize(torch.zeros(0, 70).cuda())
    assert x.codes.shape == (0, 128) and x.scales.shape == (1, 0)
    assert M.fp8_dequantize(x, F32).shape == (0, 70)
    assert M.rms_norm_fp8_fwd(torch.zeros(0, 70).cuda(), torch.ones(70).cuda()).codes.shape == (0, 128)
    assert M.fp8_linear_fwd(x, w).shape == (0, 130) and M.fp8_linear_fwd(torch.zeros(0, 70).cuda(), w).shape == (0, 130)
    dout = torch.zeros(0, 130).cuda()
    got = M.fp8_linear_bwd(x, wt, dout)
    assert got["dx"].shape == (0, 70) and torch.equal(got["dweight"], torch.zeros(130, 70).cuda())
    old = torch.randn(130, 70).cuda()
    keep = old.clone()
    assert torch.equal(M.fp8_linear_bwd(x, wt, dout, dweight=old, accumulate=True)["dweight"], keep)


# ------------------------------------------------------------------------------------------------ as programs use them
def framed(rows, cols, dtype, value=3.0):
    """A tensor with canaries on both sides, and the buffer it lies in."""
    buf = torch.full((rows * cols + 64,), value, dtype=F32).to(dtype).cuda()
    return buf[32:-32].view(rows, cols), buf


@pytest.mark.parametrize("shape", [(1, 129, 33), (5, 200, 77), (33, 300, 70), (300, 130, 333)], ids=str)
def test_nothing_is_written_beside_the_outputs(M, shape):
    tokens, k, n = shape
    g = gen(tokens)
    x, w = operands(g, *shape)
    xg, wg = Q.to_gpu(M, x), Q.to_gpu(M, w)
    wt = Q.to_gpu(M, Q.quantize(Q.values(w).T, True))
    dout = torch.randn(tokens, n, generator=g).to(BF16).cuda()
    grads = M.fp8_linear_bwd(xg, wt, dout)
    for dt in (BF16, F32):
        view, buf = framed(tokens, n, dt)
        want = M.fp8_linear_fwd(xg, wg, out_dtype=dt)
        assert torch.equal(M.fp8_linear_fwd(xg, wg, out=view), want)
        assert bool((buf[:32] == 3).all()) and bool((buf[-32:] == 3).all())
    dx, bx = framed(tokens, k, BF16)
    dw, bw = framed(n, k, BF16)
    M.fp8_linear_bwd(xg, wt, dout, dx=dx, dweight=dw)
    assert torch.equal(dx, grads["dx"]) and torch.equal(dw, grads["dweight"])
    for b in (bx, bw):
        assert bool((b[:32] == 3).all()) and bool((b[-32:] == 3).all())
    # outputs and plain inputs that start at any element
    buf = torch.zeros(tokens * k + 1, dtype=BF16).cuda()
    plain = buf[1:].view(tokens, k)
    plain.copy_(torch.randn(tokens, k, generator=g))
    odd = torch.zeros(tokens * n + 1, dtype=BF16).cuda()[1:].view(tokens, n)
    assert torch.equal(M.fp8_linear_fwd(plain, wg, out=odd), M.fp8_linear_fwd(plain.clone(), wg))
    Q.same(M.fp8_quantize(plain), Q.quantize(plain.cpu()), "x at any element")
    odd.copy_(dout)
    assert torch.equal(M.fp8_linear_bwd(xg, wt, odd)["dweight"], grads["dweight"])


def block_step(M, s):
    """One training step through a block's norm, input projection and output projection in 8 bits, with the scan
    between them, from held tensors; what it returns is everything that a program would keep."""
    u, h, rstd = M.rms_norm_fp8_fwd(s["x"], s["g"], residual=s["res"], return_residual=True, return_stats=True)
    xz = M.fp8_linear_fwd(u, s["w_in"])
    inner = s["inner"]
    xi, z = (t.contiguous().view(s["b"], -1, inner) for t in xz.split(inner, 1))
    y = M.selective_scan_fwd(xi, s["delta"], s["A"], s["B"], s["C"], s["D"], z)
    y8, x8 = M.fp8_quantize(y.view(-1, inner)), M.fp8_quantize(xi.view(-1, inner))
    out = M.fp8_linear_fwd(y8, s["w_out"])
    last = M.fp8_linear_bwd(y8, s["w_out_t"], s["dout"], dweight_dtype=F32)
    # the scan's gradients from its input as it was kept in 8 bits
    kept = M.fp8_dequantize(x8, BF16).view_as(xi)
    scan = M.selective_scan_bwd(kept, s["delta"], s["A"], s["B"], s["C"], s["D"], z, dout=last["dx"].view_as(y))
    dxz = torch.cat([scan["dx"].view(-1, inner), scan["dz"].view(-1, inner)], 1)
    first = M.fp8_linear_bwd(u, s["w_in_t"], dxz, dweight_dtype=F32)
    norm = M.rms_norm_bwd(h, s["g"], rstd, first["dx"])
    return {"out": out, "dw_out": last["dweight"], "dw_in": first["dweight"], "dx": norm["dx"], "dg": norm["dweight"],
            "u": u.codes, "h": h}


def block_inputs(M, batch, length, dim, inner, seed):
    g = gen(seed)
    t = batch * length
    r = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
    w_in, w_out = (r(2 * inner, dim) * dim ** -0.5).cuda(), (r(dim, inner) * inner ** -0.5).cuda()
    s = {"b": batch, "inner": inner, "x": r(t, dim).to(BF16).cuda(), "res": r(t, dim).cuda(), "g": (1 + 0.1 * r(dim)).cuda(),
         "delta": (0.05 + 0.1 * torch.rand(batch, length, inner, generator=g)).to(BF16).cuda(),
         "A": -(0.5 + torch.rand(inner, 16, generator=g)).cuda(), "B": r(batch, length, 16).to(BF16).cuda(),
         "C": r(batch, length, 16).to(BF16).cuda(), "D": torch.ones(inner).cuda(), "dout": r(t, dim).mul(1e-2).to(BF16).cuda()}
    s["w_in"], s["w_in_t"] = M.fp8_quantize(w_in, square=True, both=True)
    s["w_out"], s["w_out_t"] = M.fp8_quantize(w_out, square=True, both=True)
    return s


def test_block_step(M):
    """The parts in a row, each checked from what it was given."""
    s = block_inputs(M, 2, 75, 200, 160, 40)
    got = block_step(M, s)
    u, h, rstd = M.rms_norm_fp8_fwd(s["x"], s["g"], residual=s["res"], return_residual=True, return_stats=True)
    xz = M.fp8_linear_fwd(u, s["w_in"])
    R.check(xz, Q.product(Q.of_gpu(u), Q.of_gpu(s["w_in"]), BF16), "input projection")
    xi, z = (t.contiguous().view(2, -1, 160) for t in xz.split(160, 1))
    y = M.selective_scan_fwd(xi, s["delta"], s["A"], s["B"], s["C"], s["D"], z).view(-1, 160).cpu()
    R.check(got["out"], Q.product(Q.quantize(y), Q.of_gpu(s["w_out"]), BF16), "output projection")
    d = s["dout"].cpu()
    R.check(got["dw_out"], Q.product(Q.quantize(d.T), Q.quantize(Q.values(Q.quantize(y)).T), F32), "its weight's gradient")
    assert got["dw_in"].shape == (320, 200) and all(bool(t.float().isfinite().all()) for t in got.values())


def test_other_stream_and_graph(M):
    """The step on a stream of its own, and captured and replayed with new inputs in the same buffers, with eager work
    between the replays."""
    s = block_inputs(M, 2, 70, 136, 128, 41)
    want = {k: t.clone() for k, t in block_step(M, s).items()}
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = block_step(M, s)
    torch.cuda.current_stream().wait_stream(side)
    for k in want:
        assert torch.equal(got[k].view(torch.uint8), want[k].view(torch.uint8)), k
    a = M.fp8_quantize(s["res"], stream=side)
    side.synchronize()
    assert torch.equal(a.codes.view(torch.uint8), M.fp8_quantize(s["res"]).codes.view(torch.uint8))
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = block_step(M, s)
    for turn in range(4):
        new = block_inputs(M, 2, 70, 136, 128, 50 + turn)
        for k, t in s.items():
            if isinstance(t, torch.Tensor):
                t.copy_(new[k])
            elif isinstance(t, M.Fp8Matrix):
                t.codes.view(torch.uint8).copy_(new[k].codes.view(torch.uint8))
                t.scales.view(torch.uint8).copy_(new[k].scales.view(torch.uint8))
        graph.replay()
        torch.cuda.synchronize()
        eager = block_step(M, s)
        for k in eager:
            assert torch.equal(held[k].view(torch.uint8), eager[k].view(torch.uint8)), (turn, k)


def test_refusals(M):
    x = torch.randn(6, 200).cuda()
    w = M.fp8_quantize(torch.randn(70, 200).cuda(), square=True)
    q = M.fp8_quantize(x)
    many = torch.randn(300, 200).cuda()      # (a few plain rows need no workspace)
    assert M.fp8_linear_fwd_workspace_size(300, 200, 70, M.MSSM_F32) > 256
    d = torch.randn(6, 70).cuda()
    wt = M.fp8_quantize(torch.randn(200, 70).cuda(), square=True)
    for call in (lambda: M.fp8_quantize(x.half()), lambda: M.fp8_dequantize(q, torch.float16),
                 lambda: M.fp8_linear_fwd(x.half(), w), lambda: M.fp8_linear_fwd(q, x), lambda: M.fp8_transpose(x),
                 lambda: M.fp8_linear_bwd(x, wt, d), lambda: M.fp8_linear_bwd(q, wt, d.half()),
                 lambda: M.fp8_linear_bwd(q, wt, d, dweight_dtype=BF16),
                 lambda: M.fp8_linear_bwd(q, wt, d, dweight=torch.zeros(70, 200).cuda(), dweight_dtype=BF16),
                 lambda: M.fp8_linear_fwd(q._replace(codes=q.codes.view(torch.uint8)), w),
                 lambda: M.fp8_linear_fwd(q._replace(scales=q.scales.view(torch.uint8)), w)):
        with pytest.raises(TypeError):
            call()
    for call in (lambda: M.fp8_quantize(x[0]), lambda: M.fp8_quantize(x[:, ::2]), lambda: M.fp8_quantize(x.cpu()),
                 lambda: M.fp8_transpose(w), lambda: M.fp8_linear_fwd(w, w), lambda: M.fp8_linear_fwd(x[:, :199], w),
                 lambda: M.fp8_linear_fwd(q._replace(cols=199), w), lambda: M.fp8_linear_fwd(q._replace(cols=0), w),
                 lambda: M.fp8_linear_fwd(q._replace(scales=q.scales[:, :4]), w),
                 lambda: M.fp8_linear_fwd(q._replace(codes=q.codes[:, :128]), w),
                 lambda: M.fp8_linear_fwd(q, w._replace(square=False)),
                 lambda: M.fp8_linear_fwd(q, w, out=torch.zeros(6, 71).cuda()),
                 lambda: M.fp8_linear_bwd(q, w, d), lambda: M.fp8_linear_bwd(None, wt, d), lambda: M.fp8_linear_bwd(q, None, d),
                 lambda: M.fp8_linear_bwd(q, wt, d[:5]), lambda: M.fp8_linear_bwd(q, wt, d, accumulate=True),
                 lambda: M.fp8_linear_bwd(q, wt, d, want_dx=False, want_dweight=False),
                 lambda: M.fp8_quantize(torch.zeros(0, 5).cuda(), transposed=True),
                 lambda: M.rms_norm_fp8_fwd(x, torch.ones(200).cuda(), out=w),
                 lambda: M.fp8_linear_fwd(many, w, workspace=torch.zeros(1 << 20, dtype=torch.uint8))):
        with pytest.raises(ValueError):
            call()
    with pytest.raises(M.MssmError):
        M.fp8_linear_fwd(many, w, workspace=torch.zeros(256, dtype=torch.uint8).cuda())
    with pytest.raises(M.MssmError):
        M.fp8_quantize(x, out=M.Fp8Matrix(x.view(torch.float8_e4m3fn).reshape(-1)[:1536].view(6, 256), q.scales, 200))
