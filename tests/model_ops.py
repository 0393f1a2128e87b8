"""Plain 64-bit implementations of the operators around the scan, with bounds on what rounding may do to them.

Each function takes CPU tensors holding exactly what the GPU receives and returns {output: (value, bound)}:
the value in 64 bits and, per element, the largest error that the stated roundings allow.  u = 2^-24 is half a
step of fp32; storing in a type T adds eps(T) / 2 of the value."""
import torch

U = 2.0 ** -24
F64 = torch.float64


def half_step(dtype):
    return torch.finfo(dtype).eps / 2


def embedding_fwd(ids, weight, scale):
    ok = (ids >= 0) & (ids < weight.shape[0])
    s = float(torch.tensor(scale, dtype=torch.float32))
    v = weight.to(F64)[ids.clamp(0, weight.shape[0] - 1).long()] * s * ok[..., None]
    # one fp32 product, one store
    return {"out": (v, v.abs() * (U + half_step(weight.dtype)))}


def embedding_bwd(ids, dout, vocab, scale, old=None, out_dtype=None):
    out_dtype = out_dtype or dout.dtype
    s = float(torch.tensor(scale, dtype=torch.float32))
    ids, d = ids.reshape(-1), dout.reshape(-1, dout.shape[-1]).to(F64)
    ok = (ids >= 0) & (ids < vocab)
    n = torch.zeros(vocab, dtype=F64).index_add_(0, ids[ok].long(), torch.ones(int(ok.sum()), dtype=F64))
    v = torch.zeros(vocab, d.shape[1], dtype=F64).index_add_(0, ids[ok].long(), d[ok]) * s
    mag = torch.zeros(vocab, d.shape[1], dtype=F64).index_add_(0, ids[ok].long(), d[ok].abs()) * abs(s)
    if old is not None:
        v, mag = v + old.to(F64), mag + old.to(F64).abs()
    # n - 1 additions, the scale, the addition to the old value, the store
    return {"dweight": (v, mag * (n[:, None] + 2) * U + v.abs() * half_step(out_dtype))}


def norm_fwd(x, residual, weight, bias, eps, layer, res_dtype=None):
    h = x.to(F64)
    o = {}
    if res_dtype is not None:
        s = h if residual is None else h + residual.to(F64)
        o["residual"] = (s, s.abs() * half_step(res_dtype) * 1.01)   # (bf16: the fp32 sum may shift a tie)
        h = (x.float() if residual is None else x.float() + residual.float()).to(res_dtype).to(F64)
    n = h.shape[-1]
    mu = h.mean(-1, keepdim=True) if layer else torch.zeros_like(h[..., :1])
    var = ((h - mu) ** 2).mean(-1, keepdim=True)
    rs = 1 / (var + float(torch.tensor(eps, dtype=torch.float32))).sqrt()
    xh = (h - mu) * rs
    w = weight.to(F64)
    out = xh * w + (bias.to(F64) if bias is not None else 0.0)
    # a row's sums: at most 64 + n / 1024 additions in a chain, plus the tree over lanes and waves (16)
    deep = (80 + n / 1024) * U
    off = deep * h.abs().mean(-1, keepdim=True) if layer else torch.zeros_like(mu)      # of mu
    # of (h - mu): off and a rounding; of the variance relative to itself: twice that, the sum, the square
    rel = 2 * off * rs + deep + 4 * U
    d_rs = rs * (rel / 2 + 4 * U)
    d_xh = rs * (off + U * (h - mu).abs()) + (h - mu).abs() * d_rs + U * xh.abs()
    o["mean"], o["rstd"] = (mu[..., 0], (off + U * mu.abs())[..., 0]), (rs[..., 0], (d_rs + U * rs)[..., 0])
    o["out"] = (out, 1.01 * (w.abs() * (d_xh + U * xh.abs()) + U * out.abs()) + out.abs() * half_step(x.dtype))
    return o


def norm_bwd(h, weight, mean, rstd, dout, dresidual, layer):
    """mean and rstd are inputs: their fp32 values, not the row's exact statistics."""
    hd, w, g = h.to(F64), weight.to(F64), dout.to(F64)
    n, rows = hd.shape[-1], hd.reshape(-1, hd.shape[-1]).shape[0]
    rs = rstd.to(F64)[..., None]
    xh = (hd - (mean.to(F64)[..., None] if layer else 0.0)) * rs
    gw = g * w
    s1 = (gw * xh).mean(-1, keepdim=True)
    s2 = gw.mean(-1, keepdim=True) if layer else torch.zeros_like(s1)
    dh = rs * (gw - xh * s1 - s2) + (dresidual.to(F64) if dresidual is not None else 0.0)
    deep = (80 + n / 1024) * U
    a1 = (gw * xh).abs().mean(-1, keepdim=True)
    a2 = gw.abs().mean(-1, keepdim=True) if layer else torch.zeros_like(a1)
    # xh is two roundings off, gw one; the sums a chain deep; four roundings of the combination
    e = rs * (8 * U * (gw.abs() + (xh * s1).abs() + s2.abs()) + xh.abs() * (deep + 8 * U) * a1 + (deep + 8 * U) * a2)
    if dresidual is not None:
        e = e + U * dh.abs()
    # the column sums: rows of a group one after another, then the groups (2048 at most, four at a time)
    chain = min(rows, rows / 64 + 600) + 8
    col = lambda t: t.reshape(-1, n).sum(0)  # noqa: E731
    o = {"dx": (dh, 1.01 * e + dh.abs() * half_step(dout.dtype)),
         "dresidual": (dh, 1.01 * e + dh.abs() * half_step(h.dtype)),
         "dweight": (col(g * xh), col((g * xh).abs()) * chain * U)}
    if layer:
        o["dbias"] = (col(g), col(g.abs()) * chain * U)
    return o


def cross_entropy(x, weight, targets, ignore_id=-100, dloss=None, dlse=None, lse_in=None, old=None, grad_dtype=None):
    """Loss and lse, and with dloss the gradients (lse_in: the fp32 values the gradient call is given)."""
    vocab, dim = weight.shape
    io = x.dtype
    y = targets.reshape(-1)
    xd, w = x.reshape(-1, dim), weight.to(F64)
    kept = ((y >= 0) & (y < vocab) & (y != ignore_id)).nonzero()[:, 0]
    xk, yk = xd[kept].to(F64), y[kept].long()
    logits = xk @ w.T
    mag = xk.abs() @ w.abs().T
    # bf16 products are exact in fp32; fp32 ones are three products of fp16 terms: either factor may be 2^-23 off and
    # 2^-22 of the product is left out.  Every addition inside the matrix cores may lose a whole step: 2 u each.
    terms = dim * (1 if io == torch.bfloat16 else 3) + 64
    e_l = mag * (2 * terms * U + (0 if io == torch.bfloat16 else 2.0 ** -21))
    top = e_l.max(1).values if kept.numel() else torch.zeros(0, dtype=F64)
    lse = torch.logsumexp(logits, 1)
    # the logits' error, the exponentials (8 u with the argument's rounding: u per unit of the argument) and their sums
    spread = (logits.max(1).values - logits.min(1).values).clamp(max=90) if kept.numel() else top
    e_lse = top + (8 + spread + 40 + vocab / 64) * U + 4 * U * lse.abs()
    hit = logits[torch.arange(kept.numel()), yk]
    full = lambda v, src: torch.zeros(y.numel(), dtype=F64).index_copy(0, kept, src).reshape(targets.shape)  # noqa: E731
    o = {"loss": (full(None, lse - hit), full(None, e_lse + top + U * (lse - hit).abs())),
         "lse": (full(None, lse), full(None, e_lse))}
    if dloss is None:
        return o
    ls = lse_in.reshape(-1)[kept].to(F64)
    g = dloss.reshape(-1)[kept].to(F64)
    gl = g + (dlse.reshape(-1)[kept].to(F64) if dlse is not None else 0.0)
    arg = logits - ls[:, None]
    p = arg.exp()
    one = torch.zeros_like(p)
    one[torch.arange(kept.numel()), yk] = 1.0
    gr = p * gl[:, None] - one * g[:, None]
    e_g = p * gl.abs()[:, None] * (1.01 * e_l + (8 + 2 * arg.abs()) * U + 2 * U) + U * gr.abs() + U * (one * g.abs()[:, None])
    stored = 2.0 ** -8 if io == torch.bfloat16 else 2.0 ** -23    # G as the products read it
    e_g = e_g + gr.abs() * stored
    times = 1 if io == torch.bfloat16 else 3
    split = 0 if io == torch.bfloat16 else 2.0 ** -21
    m_dx, m_dw = gr.abs() @ w.abs(), gr.abs().T @ xk.abs()
    dx = torch.zeros(y.numel(), dim, dtype=F64).index_copy(0, kept, gr @ w)
    e_dx = torch.zeros(y.numel(), dim, dtype=F64).index_copy(
        0, kept, e_g @ w.abs() + m_dx * (2 * (vocab * times + 64) * U + split))
    dw = gr.T @ xk
    e_dw = e_g.T @ xk.abs() + m_dw * (2 * (kept.numel() * times + 64) * U + split)
    if old is not None:
        dw = dw + old.to(F64)
        e_dw = e_dw + U * dw.abs()
    gd = grad_dtype or io
    o["dx"] = (dx.reshape(x.shape), (e_dx + dx.abs() * half_step(io)).reshape(x.shape))
    o["dweight"] = (dw, e_dw + dw.abs() * half_step(gd))
    return o


def check(got, want, what):
    """Every element of the GPU's result within its bound of the 64-bit value."""
    ref, bound = want
    got = got.detach().cpu().to(F64)
    assert got.shape == ref.shape, f"{what}: shape {tuple(got.shape)}, expected {tuple(ref.shape)}"
    err = (got - ref).abs()
    bad = ~(err <= bound + 1e-37)   # (denormal results may be flushed; also catches NaN)
    if bad.any():
        i = tuple(int(k) for k in torch.nonzero(bad)[0])
        raise AssertionError(f"{what}: {int(bad.sum())} of {ref.numel()} outside their bounds, the first at {i}: got "
                             f"{float(got[i])!r}, expected {float(ref[i])!r} +- {float(bound[i])!r}")
