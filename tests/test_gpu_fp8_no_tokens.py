"""The 8-bit layer's weight gradient over no tokens: zeros in every place, or what was there, whatever the weight's sizes."""
import pytest
import torch

from gpu_util import say

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module")
def M():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import selective_state_space_17_amd as m
    yield m
    torch.cuda.empty_cache()


# out_features, in_features: from one place to more than 2^20 tiles of 16 x 16 (the larger ones), and rows whose count alone
# could ask for more LDS than a CU has (10240 x 2560, a layer of the measured ones)
SMALL = [(1, 1), (1, 4097), (16, 40), (17, 300), (777, 1000), (3000, 129)]
LARGE = [(1000, 1 << 20), (4096, 69632), (10240, 2560), (1 << 20, 130)]


@pytest.mark.parametrize("accumulate", [False, True], ids=["over", "add"])
@pytest.mark.parametrize("dtype", [BF16, F32], ids=str)
@pytest.mark.parametrize("shape", SMALL + LARGE, ids=str)
def test_weight_gradient(M, shape, dtype, accumulate):
    n, k = shape
    say("fp8 weight gradient of no tokens", shape, dtype, accumulate)
    x = M.fp8_quantize(torch.empty(0, k, device="cuda"))
    old = -0.0 if accumulate else 1.5            # (what was there stays bit for bit: adding 0 would turn -0 into 0)
    dw = torch.full((n, k), old, device="cuda", dtype=dtype)
    if accumulate:
        dw[n // 2] = float("nan")
        dw[:, k // 2] = 3.0
    keep = dw.clone() if accumulate else torch.zeros_like(dw)
    got = M.fp8_linear_bwd(x, None, torch.empty(0, n, device="cuda", dtype=dtype), want_dx=False, dweight=dw,
                           accumulate=accumulate)
    assert got["dweight"] is dw
    bits = torch.int16 if dtype == BF16 else torch.int32
    assert torch.equal(dw.view(bits), keep.view(bits))


@pytest.mark.parametrize("shape", [(130, 70), (10240, 2560)], ids=str)
def test_both_gradients_and_a_graph(M, shape):
    """With dx of no rows beside it, and captured: every replay clears what was written in between."""
    n, k = shape
    say("fp8 gradients of no tokens", shape)
    x = M.fp8_quantize(torch.empty(0, k, device="cuda"))
    wt = M.fp8_quantize(torch.randn(k, n, device="cuda"), square=True)
    dout = torch.empty(0, n, device="cuda")
    dw = torch.full((n, k), 2.0, device="cuda")
    got = M.fp8_linear_bwd(x, wt, dout, dweight=dw)
    assert got["dx"].shape == (0, k) and not dw.any()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        M.fp8_linear_bwd(x, wt, dout, dweight=dw)
    for _ in range(3):
        dw.fill_(7.0)
        graph.replay()
        torch.cuda.synchronize()
        assert not dw.any()
