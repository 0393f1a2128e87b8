"""Plain 64-bit implementations of matrices in 8 bits and the linear layer on them, with bounds on what rounding may do.

Matrices are (codes as e4m3 values in 64 bits, scale bytes, cols, square), laid out as include/mssm.h says."""
import torch

from model_ops import F64, U, half_step

BLOCK = 128
LARGEST = 448.0


def e4m3(v):
    """Nearest e4m3 value, halves to even, of |v| <= 448; NaN for what is not finite."""
    a = v.abs()
    e = torch.floor(torch.log2(a.clamp(min=2.0 ** -6)))
    step = torch.exp2(e - 3)
    # log2 may land on the power above for a value just below it: its step must not exceed an eighth of the value's power
    step = torch.where(a.clamp(min=2.0 ** -6) < torch.exp2(e), step / 2, step)
    return torch.where(torch.isfinite(v), torch.round(v / step) * step, torch.full_like(v, float("nan")))


def scale_byte(top):
    """Least power of two that brings top to 448 or less, by comparison; 2^-126 at least, 1 for 0."""
    k = torch.arange(-126, 121, dtype=F64)
    i = torch.searchsorted(LARGEST * torch.exp2(k), top.contiguous())
    return torch.where(top > 0, k[i] + 127, torch.full_like(top, 127.0)).to(torch.uint8)


def quantize(x, square=False):
    """x [rows, cols] (CPU, any type, taken as it is) as (codes [rows, 128 b], scales, cols, square)."""
    rows, cols = x.shape
    b, h = -(-cols // BLOCK), -(-rows // BLOCK) if square else rows
    p = torch.zeros(h * BLOCK if square else h, b * BLOCK, dtype=F64)
    p[:rows, :cols] = x.to(F64)
    p = p.reshape(h, BLOCK if square else 1, b, BLOCK)
    top = torch.where(torch.isfinite(p), p.abs(), torch.zeros_like(p)).amax((1, 3))      # [h, b]
    s = scale_byte(top)
    codes = e4m3(p / torch.exp2(s.to(F64) - 127)[:, None, :, None]).reshape(-1, b * BLOCK)[:rows]
    lines = h if square else -(-rows // 4) * 4
    scales = torch.full((b, lines), 127, dtype=torch.uint8)
    scales[:, :h] = s.T
    return codes, scales, cols, square


def tops(a):
    """Largest of each 128 columns of a row, [rows, blocks]."""
    return torch.nn.functional.pad(a, (0, -a.shape[1] % BLOCK)).reshape(a.shape[0], -1, BLOCK).amax(2)


def values(m):
    codes, scales, cols, square = m
    rows = codes.shape[0]
    s = torch.exp2(scales.to(F64) - 127).T                       # [lines, b]
    s = s.repeat_interleave(BLOCK, 0)[:rows] if square else s[:rows]
    return (codes.reshape(rows, -1, BLOCK) * s[:, :, None]).reshape(rows, -1)[:, :cols]


def to_gpu(M, m):
    codes, scales, cols, square = m
    return M.Fp8Matrix(codes.float().to(torch.float8_e4m3fn).cuda(), scales.view(torch.float8_e8m0fnu).cuda(), cols, square)


def of_gpu(m):
    return (m.codes.cpu().float().to(F64), m.scales.cpu().view(torch.uint8), m.cols, m.square)


def same(got, want, what):
    """Codes and scales equal in every place, NaN where NaN is due."""
    g = of_gpu(got)
    assert g[2] == want[2] and bool(g[3]) == want[3] and g[0].shape == want[0].shape and g[1].shape == want[1].shape, what
    bad = g[1] != want[1]
    assert not bad.any(), f"{what}: {int(bad.sum())} scales differ, the first at {torch.nonzero(bad)[0].tolist()}"
    bad = ~((g[0] == want[0]) | (g[0].isnan() & want[0].isnan()))
    assert not bad.any(), f"{what}: {int(bad.sum())} codes differ, the first at {torch.nonzero(bad)[0].tolist()}"


def product(r, c, out_dtype, old=None, chunk=64, device="cpu"):
    """sum_k r[., k] c[., k] of two matrices in 8 bits, and its bound: see product_of_values."""
    return product_of_values(values(r).to(device), values(c).to(device), out_dtype, old, chunk)


def product_of_values(rv, cv, out_dtype, old=None, chunk=64):
    """fp32: products of e4m3 numbers are exact in fp32 and are summed there; every addition inside the matrix cores may
    lose a whole step, 2 u.  bf16: besides, of 8 neighbouring products each may lose 2^-13 of the largest."""
    device = rv.device
    k = rv.shape[1]
    ref, mag = rv @ cv.T, rv.abs() @ cv.abs().T
    bound = mag * 2 * (k + 64) * U
    if out_dtype == torch.bfloat16 and k:
        pad = -k % 8
        a, b = (torch.nn.functional.pad(v.abs(), (0, pad)).reshape(v.shape[0], -1, 8) for v in (rv, cv))
        lost = torch.zeros_like(ref)
        for i in range(0, ref.shape[0], chunk):
            for j in range(0, ref.shape[1], chunk):
                top = torch.zeros(a[i:i + chunk].shape[0], b[j:j + chunk].shape[0], a.shape[1], dtype=F64, device=device)
                for e in range(8):
                    top = torch.maximum(top, a[i:i + chunk, None, :, e] * b[None, j:j + chunk, :, e])
                lost[i:i + chunk, j:j + chunk] = top.sum(2)
        bound = bound + lost * 8 * 2.0 ** -13
    if old is not None:
        ref = ref + old.to(device, F64)
        bound = bound + U * ref.abs()
    return ref.cpu(), (bound * 1.01 + ref.abs() * half_step(out_dtype)).cpu()
