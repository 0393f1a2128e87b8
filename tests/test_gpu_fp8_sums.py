"""How exactly the 8-bit product sums, on each of its kernels: sums that fp32 holds exactly in any order have to come out
exactly, so that a block, a slice or a bit that is lost shows however long the sum is."""
import pytest
import torch

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


def whole(g, *shape):
    """-2, -1, 1 or 2, all equally often: numbers of 8 bits under any block's scale, products of at most 4, and within 8
    neighbours all products are within 2^2 of the largest, so that nothing is dropped below it."""
    v = torch.randint(0, 4, shape, generator=g, device="cuda", dtype=torch.int8)
    return torch.where(v < 2, v - 2, v - 1).to(BF16)


def exact(a, b, chunk=1 << 16):
    """sum_k a[k, .] b[k, .] in 64 bits, a chunk of k at a time."""
    s = torch.zeros(a.shape[1], b.shape[1], dtype=F64, device=a.device)
    for lo in range(0, a.shape[0], chunk):
        s += a[lo:lo + chunk].to(F64).T.contiguous() @ b[lo:lo + chunk].to(F64)
    return s


# tokens, k, n.  By the plan: tiles of 16 x 16, 32 x 32, 64 x 32, 64 x 64; 128 x 128, the same in slices (two sizes); 256 x
# 256, in slices after a whole round, in slices alone
KERNELS = [(8, 130, 70), (60, 1000, 2500), (61, 2561, 5090), (254, 130, 2990), (2030, 130, 1500), (1016, 9000, 70),
           (250, 2100, 5000), (4060, 1000, 4060), (4060, 4100, 9000), (1016, 9000, 5000)]


@pytest.mark.parametrize("square", [False, True], ids=["rows", "square"])
@pytest.mark.parametrize("shape", KERNELS, ids=str)
def test_whole_numbers(M, shape, square):
    """All sums are below 4 x 9000, and exact in fp32 in any order; results in bf16 are rounded from them once."""
    tokens, k, n = shape
    say("sums of whole numbers", shape, square)
    g = torch.Generator(device="cuda").manual_seed(k + n)
    x, w = whole(g, tokens, k), whole(g, n, k)
    want = exact(x.T, w.T)
    x8, w8 = M.fp8_quantize(x), M.fp8_quantize(w, square=square)
    for dtype in (F32, BF16):
        assert torch.equal(M.fp8_linear_fwd(x8, w8, out_dtype=dtype), want.to(dtype)), dtype


@pytest.mark.parametrize("square", [False, True], ids=["rows", "square"])
@pytest.mark.parametrize("shape", KERNELS, ids=str)
def test_small_products_beside_large_ones(M, shape, square):
    """In every block of 128 one product of 256 and 8 neighbours of 1.5 x 2^-8, which the 8-bit instructions drop beside it.
    A sum of b blocks is 256 b + 3 b 2^-6, all of its parts multiples of 2^-9 below 2^15: exact in fp32 in any order."""
    tokens, k, n = shape
    say("small products beside large ones", shape, square)
    blocks = (k - 9) // 128 + 1                              # those that hold all nine
    assert 256 * blocks + 1 < 1 << 15
    x, w = torch.zeros(tokens, k), torch.zeros(n, k)
    for b in range(blocks):
        x[:, 128 * b], w[:, 128 * b] = 16.0, 16.0
        x[:, 128 * b + 1:128 * b + 9], w[:, 128 * b + 1:128 * b + 9] = 2.0 ** -4, 1.5 * 2.0 ** -4
    got = M.fp8_linear_fwd(M.fp8_quantize(x.cuda()), M.fp8_quantize(w.cuda(), square=square), out_dtype=F32)
    assert bool((got == blocks * (256 + 3 * 2.0 ** -6)).all())


# tokens, in_features, out_features of gradients in fp32: both products small and side by side; dweight in slices of 128 x
# 128; both on 256 x 256
@pytest.mark.parametrize("shape", [(300, 384, 200), (1000, 900, 700), (8000, 700, 600), (4100, 4000, 4200)], ids=str)
def test_gradients(M, shape):
    tokens, k, n = shape
    say("sums of whole numbers, gradients", shape)
    g = torch.Generator(device="cuda").manual_seed(tokens)
    x, w, dout = whole(g, tokens, k), whole(g, n, k), whole(g, tokens, n)
    x8, wt = M.fp8_quantize(x), M.fp8_quantize(w, square=True, transposed=True)
    dx, dw = exact(dout.T, w), exact(dout, x)
    for dtype in (F32, BF16):
        got = M.fp8_linear_bwd(x8, wt, dout.to(dtype))
        assert torch.equal(got["dx"], dx.to(dtype)) and torch.equal(got["dweight"], dw.to(dtype)), dtype
    old = whole(g, n, k).float()
    got = M.fp8_linear_bwd(x8, None, dout, want_dx=False, dweight=old.clone(), accumulate=True)["dweight"]
    assert torch.equal(got, (dw + old).float())


@pytest.mark.parametrize("sizes", [(1100, 130), (16, 70), (700, 520)], ids=str)
def test_most_tokens(M, sizes):
    """The longest sums, over 2^22 tokens less a few: at most 4 x 2^22 = 2^24, where fp32 still holds every whole number.  A
    block of 128 tokens that is lost changes an element by some 20 or more nearly everywhere."""
    n, k = sizes
    tokens = (1 << 22) - 5
    say("sums of whole numbers over the most tokens", sizes)
    g = torch.Generator(device="cuda").manual_seed(n)
    x, dout = whole(g, tokens, k), whole(g, tokens, n)
    want = exact(dout, x)
    x8 = M.fp8_quantize(x)
    for dtype in (F32, BF16):
        got = M.fp8_linear_bwd(x8, None, dout, want_dx=False, dweight_dtype=dtype)["dweight"]
        assert torch.equal(got, want.to(dtype)), dtype
    # what the comparison sees: any one block of tokens missing from the reference, among them the first and the last
    for lo in (0, 128 * 12345, tokens // 128 * 128):
        less = want - exact(dout[lo:lo + 128], x[lo:lo + 128])
        assert ((less != want).double().mean() > 0.5) and not torch.equal(less.float(), want.float())
