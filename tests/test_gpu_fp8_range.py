"""The ends of the range that the 8-bit layer states, code by code, on each kernel."""
import pytest
import torch

from gpu_util import say

pytestmark = pytest.mark.gpu
BF16, F32, F64 = torch.bfloat16, torch.float32, torch.float64
FP8, E8 = torch.float8_e4m3fn, torch.float8_e8m0fnu


@pytest.fixture(scope="module")
def M():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import selective_state_space_17_amd as m
    return m


def alone(M, rows, cols, byte, codes):
    """Row t has codes[t] in its first place and zeros elsewhere, all under the scale 2^(byte - 127)."""
    c = torch.zeros(rows, -(-cols // 128) * 128, dtype=torch.uint8)
    c[:, 0] = codes
    s = torch.full((c.shape[1] // 128, -(-rows // 4) * 4), byte, dtype=torch.uint8)
    return M.Fp8Matrix(c.view(FP8).cuda(), s.view(E8).cuda(), cols)


# rows, k and columns for tiles of 16 x 16, 32 x 32, 64 x 32, 64 x 64, 128 x 128 and 256 x 256
SHAPES = [(127, 130, 8), (2032, 130, 70), (4064, 130, 70), (254, 130, 2990), (2032, 130, 1500), (4064, 1000, 4060)]


@pytest.mark.parametrize("turned", [False, True], ids=["x", "weight"])
@pytest.mark.parametrize("byte", [0, 1, 2, 3])
@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_smallest_values(M, shape, byte, turned):
    """Every magnitude under e8m0's smallest scales, times 2^100: as they are in results in bf16, as bf16 numbers (which end
    at 2^-133) in fp32.  The results, between 2^-36 and 2^-18, are numbers of either type."""
    rows, k, n = shape
    say("smallest values", shape, byte, turned)
    codes = torch.arange(rows) % 127
    x, w = alone(M, rows, k, byte, codes), alone(M, n, k, 227, torch.full((n,), 0x38))       # 0x38: 1
    v = codes.to(torch.uint8).view(FP8).to(F64) * 2.0 ** (byte - 127)
    near = torch.where(v < 2.0 ** -126, torch.round(v * 2.0 ** 133) * 2.0 ** -133, v)      # (round: halves to even)
    assert (near != v).sum() == {0: 24, 1: 16, 2: 8, 3: 0}[byte] * (rows // 127)
    for dtype, want in ((BF16, v), (F32, near)):
        got = M.fp8_linear_fwd(w, x, out_dtype=dtype).T if turned else M.fp8_linear_fwd(x, w, out_dtype=dtype)
        assert torch.equal(got.cpu().to(F64), (want * 2.0 ** 100)[:, None].expand(rows, n)), dtype


def test_values_beyond_fp32(M):
    """2^128 and more, which no fp32 number is: infinite as fp32 or bf16, NaN laid out the other way, and nothing else in
    their rows and columns changes; the smallest such values are what fp8_quantize makes of fp32's largest."""
    g = torch.Generator().manual_seed(4)
    x = torch.randn(9, 300, generator=g)
    border = 248 * 2.0 ** 120                            # between 240 and 256 under the scale 2^120: to the even one, 256
    below = float(torch.nextafter(torch.tensor(border), torch.tensor(0.0)))
    x[2, 5], x[2, 6], x[2, 7], x[2, 8] = torch.finfo(F32).max, border, -border, below
    m = M.fp8_quantize(x.cuda())
    assert int(m.scales.view(torch.uint8)[0, 2]) == 247
    assert m.codes[2, 5:9].cpu().tolist() == [256.0, 256.0, -256.0, 240.0]
    inf = float("inf")
    for dtype in (F32, BF16):
        assert M.fp8_dequantize(m, dtype)[2, 5:9].cpu().tolist() == [inf, inf, -inf, 240 * 2.0 ** 120]
    x[2, 5:8] = 0
    clean = M.fp8_quantize(x.cuda())
    got, want = M.fp8_transpose(m), M.fp8_transpose(clean)
    assert bool(got.codes.float()[5:8, 2].isnan().all())
    a, b = M.fp8_dequantize(got, F32), M.fp8_dequantize(want, F32)
    b[5:8, 2] = a[5:8, 2]
    assert torch.equal(a.view(torch.int32), b.view(torch.int32))
    dout = torch.randn(9, 40, generator=g).cuda()
    dw = M.fp8_linear_bwd(m, None, dout, want_dx=False)["dweight"]
    same = M.fp8_linear_bwd(clean, None, dout, want_dx=False)["dweight"]
    keep = [i for i in range(300) if i not in (5, 6, 7)]
    assert bool(dw[:, 5:8].isnan().all()) and torch.equal(dw[:, keep], same[:, keep])
