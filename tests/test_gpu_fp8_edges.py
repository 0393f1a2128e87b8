"""The 8-bit product with scales at e8m0's ends and plain rows that hold values which are not finite, on each kernel."""
import pytest
import torch

import fp8_ops as Q
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


# sizes for the kernel for few rows and, the larger two, for the kernels with tiles of 128 x 128 and 256 x 256
SHAPES = [(9, 300, 70), (60, 300, 200), (700, 300, 4000), (9000, 129, 3001)]


@pytest.mark.parametrize("square", [False, True], ids=["rows", "square"])
@pytest.mark.parametrize("out_dtype", [BF16, F32], ids=str)
@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_scales_at_their_ends(M, shape, out_dtype, square):
    """2^-127 and 2^127 on one side, met by such powers on the other that results are ordinary numbers; NaN scales.  For
    fp32 results values are fp32 numbers, and 448 x 2^127 is none (2^128 is not): 2^119 there, 448 x 2^119 < 2^128."""
    tokens, k, n = shape
    say("scales at their ends", shape, out_dtype, square)
    g = torch.Generator().manual_seed(tokens)
    x = Q.quantize(torch.randn(tokens, k, generator=g))
    w = Q.quantize(torch.randn(n, k, generator=g), square)
    xs, ws = x[1].clone(), w[1].clone()
    # block 0 of x at the bottom, met by the weight's at the top; block 1 the other way about
    top = 254 if out_dtype == BF16 else 246
    xs[0, :], ws[0, :] = 0, top - 4
    xs[1, :], ws[1, :] = top, 4
    x, w = (x[0], xs, k, False), (w[0], ws, k, square)
    got = M.fp8_linear_fwd(Q.to_gpu(M, x), Q.to_gpu(M, w), out_dtype=out_dtype)
    R.check(got, Q.product(x, w, out_dtype, chunk=512, device="cuda"), "out")
    xs = xs.clone()
    xs[1, 3] = 255
    bad = M.fp8_linear_fwd(Q.to_gpu(M, (x[0], xs, k, False)), Q.to_gpu(M, w), out_dtype=out_dtype)
    assert bool(bad[3].isnan().all())
    keep = [i for i in range(tokens) if i != 3]
    assert torch.equal(bad[keep], got[keep])


@pytest.mark.parametrize("io", [BF16, F32], ids=str)
@pytest.mark.parametrize("rows", [1, 3, 16, 17, 200])
def test_plain_rows_that_are_not_finite(M, rows, io):
    say("plain rows, not finite", rows, io)
    g = torch.Generator().manual_seed(rows)
    x = (torch.randn(rows, 333, generator=g) * torch.exp(3 * torch.randn(rows, 1, generator=g))).to(io)
    x[0, 5], x[0, 130] = float("inf"), float("nan")
    x[rows - 1, 332] = float("-inf")
    x[rows // 2, 128:256] = 0
    w = Q.quantize(torch.randn(90, 333, generator=g), True)
    want_x = Q.quantize(x)
    for dt in (BF16, F32):
        got = M.fp8_linear_fwd(x.cuda(), Q.to_gpu(M, w), out_dtype=dt)
        assert torch.equal(got.view(torch.uint8), M.fp8_linear_fwd(M.fp8_quantize(x.cuda()), Q.to_gpu(M, w),
                                                                  out_dtype=dt).view(torch.uint8))
        bad = torch.zeros(rows, dtype=torch.bool)
        bad[[0, rows - 1]] = True
        assert torch.equal(got.cpu().isnan(), bad[:, None].expand(rows, 90))
        ref, bound = Q.product((want_x[0].nan_to_num(0.0), *want_x[1:]), w, dt)
        if rows > 2:
            R.check(got[1:rows - 1], (ref[1:rows - 1], bound[1:rows - 1]), "rows between")


def test_two_streams_at_once(M):
    """Calls on two streams at once, each with its own buffers: the results of either alone."""
    g = torch.Generator().manual_seed(3)
    sets = []
    for rows in (700, 900):
        x = M.fp8_quantize(torch.randn(rows, 4000, generator=g).cuda())
        w, wt = M.fp8_quantize(torch.randn(500, 4000, generator=g).cuda(), square=True, both=True)
        d = torch.randn(rows, 500, generator=g).cuda()
        sets.append((x, w, wt, d, M.fp8_linear_fwd(x, w), M.fp8_linear_bwd(x, wt, d)))
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in sets]
    got = []
    for _ in range(4):
        for s, (x, w, wt, d, _, _) in zip(streams, sets):
            got.append((M.fp8_linear_fwd(x, w, stream=s), M.fp8_linear_bwd(x, wt, d, stream=s)))
    torch.cuda.synchronize()
    for i, (out, grads) in enumerate(got):
        _, _, _, _, want, wanted = sets[i % 2]
        assert torch.equal(out, want) and all(torch.equal(grads[k], wanted[k]) for k in wanted)


@pytest.mark.parametrize("shape", [(4096, 768, 640), (300, 700, 600)], ids=["slices", "pair"])
def test_gradients_replayed(M, shape):
    """Gradients captured once, with sums of slices in the workspace or both products in one launch, and replayed with new
    inputs and other work on the GPU between: every replay is the eager call's result."""
    tokens, k, n = shape
    say("fp8 gradients in a graph", shape)
    g = torch.Generator(device="cuda").manual_seed(k)

    def rnd(*s):
        return torch.randn(*s, generator=g, device="cuda")

    x, wt = M.fp8_quantize(rnd(tokens, k)), M.fp8_quantize(rnd(k, n), square=True)
    dout = rnd(tokens, n).to(BF16)
    M.fp8_linear_bwd(x, wt, dout, dweight_dtype=F32)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = M.fp8_linear_bwd(x, wt, dout, dweight_dtype=F32)
    for _ in range(4):
        dout.copy_(rnd(tokens, n))
        M.fp8_quantize(rnd(tokens, k), out=x)
        want = M.fp8_linear_bwd(x, wt, dout, dweight_dtype=F32)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(got["dx"], want["dx"]) and torch.equal(got["dweight"], want["dweight"])
