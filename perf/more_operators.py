"""The 8-bit linear layer around the scan, in training and at serving: norm with the residual add and an output in 8 bits,
activations kept in 8 bits in either order, the product with a weight in 8 bits, and its gradients from the input as it
was kept.  Cases, inputs, plain forms and 64-bit values.

A matrix [rows, cols] in 8 bits is its e4m3 codes [rows, 128 * blocks], zeros past cols, and a power of two for each
block of 128 columns of a row, [blocks, rows rounded up to 4] (the weight: for each 128 x 128), as e8m0."""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
BLOCK = 128


# ------------------------------------------------------------------------------------------------------------ cases
def listed():
    return [
        # serving: the pre-norm of a block for 8 new tokens, residual stream in fp32
        {"name": "norm_decode", "op": "norm", "kind": "rms", "rows": 8, "dim": 2560, "io": "bf16", "res": "f32"},
        # training: RMS pre-norm of the 2.8B-like layer, 4 x 8192 tokens, residual stream in fp32
        {"name": "norm_train", "op": "norm", "kind": "rms", "rows": 32768, "dim": 2560, "io": "bf16", "res": "f32"},
        # a ragged batch of an odd width in fp32
        {"name": "norm_odd", "op": "norm", "kind": "layer", "rows": 5001, "dim": 1023, "io": "f32", "res": "f32"},
        # training: the scan's output of the 130M-like model (d_inner 1536) kept in 8 bits, in both orders for the products
        # that take it, and read back for the scan's gradients
        {"name": "keep_train", "op": "keep", "rows": 16384, "cols": 1536, "io": "bf16"},
        # a ragged batch of an odd width in fp32
        {"name": "keep_odd", "op": "keep", "rows": 4999, "cols": 333, "io": "f32"},
        # serving one sequence: a new token through the input projection of the 2.8B-like layer (d_inner 5120, x and z)
        {"name": "linear_token", "op": "linear", "tokens": 1, "in": 2560, "out": 10240, "x": "bf16", "io": "bf16"},
        # serving 8 sequences: a new token of each through its output projection, already in 8 bits
        {"name": "linear_decode", "op": "linear", "tokens": 8, "in": 5120, "out": 2560, "x": "fp8", "io": "bf16"},
        # a short ragged prompt through an odd layer, fp32 out
        {"name": "linear_odd", "op": "linear", "tokens": 301, "in": 1000, "out": 777, "x": "fp8", "io": "f32"},
        # training and long prompts: 4 x 8192 tokens through the input projection of the 2.8B-like layer
        {"name": "linear_train", "op": "linear", "tokens": 32768, "in": 2560, "out": 10240, "x": "fp8", "io": "bf16"},
        # gradients of the output projection of the 130M-like model, 8 x 1024 tokens
        {"name": "grads_train", "op": "grads", "tokens": 8192, "in": 1536, "out": 768, "io": "bf16", "dw": "f32"},
        # gradients of an odd layer over a ragged batch
        {"name": "grads_odd", "op": "grads", "tokens": 1001, "in": 1000, "out": 777, "io": "f32", "dw": "f32"},
        # gradients of the input projection of the 2.8B-like layer, 2 x 8192 tokens
        {"name": "grads_large", "op": "grads", "tokens": 16384, "in": 2560, "out": 10240, "io": "bf16", "dw": "bf16"},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["norm", "keep", "linear", "linear", "grads", "grads"])
    io = rng.choice(["bf16", "bf16", "f32"])

    def width(hi):
        n = _log(rng, 64, hi)
        return n if rng.random() < 0.4 else max(64, n // 64 * 64)

    if op == "norm":
        c = {"op": op, "kind": rng.choice(["layer", "rms"]), "rows": _log(rng, 1, 32768), "dim": width(5120), "io": io,
             "res": rng.choice(["none", io, "f32"])}
        c["rows"] = min(c["rows"], 32768 * 2560 // c["dim"])
        return c
    if op == "keep":
        c = {"op": op, "rows": _log(rng, 1, 32768), "cols": width(5120), "io": io}
        c["rows"] = min(c["rows"], 32768 * 1536 // c["cols"])
        return c
    c = {"op": op, "tokens": _log(rng, 1, 32768), "in": width(5120), "out": width(10240)}
    most = 32768 * 2560 * 10240 // (c["in"] * c["out"])
    if op == "linear":
        return {**c, "tokens": max(1, min(c["tokens"], most)), "x": rng.choice(["fp8", io]), "io": io}
    return {**c, "tokens": max(1, min(c["tokens"], most // 2)), "io": io, "dw": rng.choice([io, "f32"])}


def _size(t):
    return {"bf16": 2, "f32": 4, "fp8": 1, "none": 0}[t]


def work(case):
    s = _size(case["io"])
    if case["op"] == "norm":
        n = case["rows"] * case["dim"]
        return {"bytes": n * (s + 2 * _size(case["res"]) + 1 + 1 / BLOCK) + 8 * case["dim"], "flops": 12 * n}
    if case["op"] == "keep":
        n = case["rows"] * case["cols"]
        return {"bytes": n * (2 * s + 2 + 2 / BLOCK), "flops": 7 * n}
    t, k, n = case["tokens"], case["in"], case["out"]
    if case["op"] == "linear":
        return {"bytes": t * k * _size(case["x"]) + n * k + t * n * s, "flops": 2 * t * k * n}
    return {"bytes": t * n * s + t * k + n * k + t * k * s + n * k * _size(case["dw"]), "flops": 4 * t * k * n}


# ----------------------------------------------------------------------------------------------------------- inputs
def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(int(seed))

    def rnd(*shape):
        return torch.randn(*shape, generator=g, device="cuda")

    st = dict(case)
    if case["op"] == "norm":
        n, d, dt, rdt = case["rows"], case["dim"], DTYPES[case["io"]], DTYPES.get(case["res"])
        st["eps"] = 1e-5
        st["x"] = (rnd(n, d) * 0.8 + 0.1).to(dt)
        st["residual"] = None if rdt is None else (rnd(n, d) * 2.0).to(rdt)
        st["weight"] = 1.0 + 0.2 * rnd(d)
        st["bias"] = 0.1 * rnd(d) if case["kind"] == "layer" else None
        return st
    if case["op"] == "keep":
        # a gated scan's output: channels and tokens of different sizes
        n, d = case["rows"], case["cols"]
        st["x"] = (rnd(n, d) * torch.exp(rnd(d)) * torch.exp(0.5 * rnd(n, 1))).to(DTYPES[case["io"]])
        return st
    t, k, n = case["tokens"], case["in"], case["out"]
    w = rnd(n, k) * k ** -0.5
    x = rnd(t, k) * torch.exp(0.5 * rnd(k))
    if case["op"] == "linear":
        st["weight"] = _pack(w, square=True)
        st["x_in"] = _pack(x) if case["x"] == "fp8" else x.to(DTYPES[case["x"]])
        return st
    st["x_in"] = _pack(x)
    st["weight_t"] = _pack(w.T, square=True)
    st["dout"] = (rnd(t, n) * 1e-3 * torch.exp(0.5 * rnd(t, 1))).to(DTYPES[case["io"]])
    return st


# -------------------------------------------------------------------------------------------------------------- run
def run(st):
    if own:
        return _own(st)
    return {"norm": _plain_norm, "keep": _plain_keep, "linear": _plain_linear, "grads": _plain_grads}[st["op"]](st)


def _own(st):
    import selective_state_space_17_amd as M

    if st["op"] == "norm":
        layer, res = st["kind"] == "layer", st["residual"]
        fwd = M.layer_norm_fp8_fwd if layer else M.rms_norm_fp8_fwd
        args = (st["x"], st["weight"]) + ((st["bias"],) if layer else ())
        got = fwd(*args, residual=res, eps=st["eps"], return_residual=res is not None)
        u, h = got if res is not None else (got, None)
        o = {"codes": u.codes, "scales": u.scales}
        return o if h is None else {**o, "residual": h}
    if st["op"] == "keep":
        a, b = M.fp8_quantize(st["x"], both=True)
        return {"codes": a.codes, "scales": a.scales, "codes_t": b.codes, "scales_t": b.scales,
                "back": M.fp8_dequantize(a, st["x"].dtype)}

    def held(m, square=False):
        codes, scales, cols = m
        return M.Fp8Matrix(codes, scales, cols, square)

    x = held(st["x_in"]) if isinstance(st["x_in"], tuple) else st["x_in"]
    if st["op"] == "linear":
        return {"out": M.fp8_linear_fwd(x, held(st["weight"], True), out_dtype=DTYPES[st["io"]])}
    return M.fp8_linear_bwd(x, held(st["weight_t"], True), st["dout"], dweight_dtype=DTYPES[st["dw"]])


def _blocks(x, square):
    """x padded with zeros to whole blocks, as [rows, 1, blocks, 128] or [row blocks, 128, blocks, 128]."""
    high = BLOCK if square else 1
    rows, cols = x.shape
    x = torch.nn.functional.pad(x, (0, -cols % BLOCK, 0, -rows % high))
    return x.reshape(x.shape[0] // high, high, x.shape[1] // BLOCK, BLOCK)


def _scale(b):
    """The least power of two that brings a block's largest magnitude to 448 or less (fp32; 1 for zeros)."""
    m, e = torch.frexp(b.abs().amax((1, 3), keepdim=True))
    return torch.where(m > 0, torch.ldexp(torch.ones_like(m), torch.clamp(e - 9 + (m > 0.875), min=-126)), torch.ones_like(m))


def _pack(x, square=False):
    """x [rows, cols] in 8 bits, as a program keeps it: codes, scales, cols."""
    rows, cols = x.shape
    b = _blocks(x.float(), square)
    s = _scale(b)
    codes = (b / s).reshape(b.shape[0] * b.shape[1], -1)[:rows].to(torch.float8_e4m3fn)
    e = (torch.frexp(s).exponent + 126)[:, 0, :, 0].T.to(torch.uint8)
    if not square:
        e = torch.nn.functional.pad(e, (0, -rows % 4), value=127)
    return codes.contiguous(), e.contiguous().view(torch.float8_e8m0fnu), cols


def _unpack(m, square=False):
    """The fp32 values that a matrix in 8 bits stands for."""
    codes, scales, cols = m
    rows = codes.shape[0]
    s = torch.ldexp(torch.ones((), device=codes.device), scales.view(torch.uint8).int() - 127).T
    s = s.repeat_interleave(BLOCK, 0)[:rows] if square else s[:rows]
    return (codes.float().reshape(rows, -1, BLOCK) * s[:, :, None]).reshape(rows, -1)[:, :cols]


def _rounded(x):
    """x as it reads back from 8 bits, in fp32."""
    rows, cols = x.shape
    b = _blocks(x.float(), False)
    s = _scale(b)
    return ((b / s).to(torch.float8_e4m3fn).float() * s).reshape(rows, -1)[:, :cols]


def _plain_norm(st):
    x, res, w, layer = st["x"], st["residual"], st["weight"], st["kind"] == "layer"
    o = {}
    h = x.float()
    if res is not None:
        o["residual"] = (h + res.float()).to(res.dtype)
        h = o["residual"].float()
    c = h - h.mean(1, keepdim=True) if layer else h
    xh = c * torch.rsqrt((c * c).mean(1, keepdim=True) + st["eps"])
    codes, scales, _ = _pack(xh * w + st["bias"] if layer else xh * w)
    return {"codes": codes, "scales": scales, **o}


def _plain_keep(st):
    x = st["x"]
    rows, columns = _pack(x), _pack(x.T)
    return {"codes": rows[0], "scales": rows[1], "codes_t": columns[0], "scales_t": columns[1],
            "back": _unpack(rows).to(x.dtype)}


def _plain_linear(st):
    x = _unpack(st["x_in"]) if isinstance(st["x_in"], tuple) else _rounded(st["x_in"])
    return {"out": (x @ _unpack(st["weight"], True).T).to(DTYPES[st["io"]])}


def _plain_grads(st):
    x, wt, dout = _unpack(st["x_in"]), _unpack(st["weight_t"], True), st["dout"]
    dx = _rounded(dout) @ wt.T
    dw = _rounded(dout.T) @ _rounded(x.T).T
    return {"dx": dx.to(dout.dtype), "dweight": dw.to(DTYPES[st["dw"]])}


# ------------------------------------------------------------------------------------------------------------ exact
def _values(m, square):
    """What codes and scales stand for, in 64 bits: each block column by itself."""
    codes, scales, cols = m
    power = torch.pow(torch.tensor(2.0, dtype=torch.float64, device=codes.device), scales.view(torch.uint8).double() - 127)
    v = codes.double()
    row = torch.arange(v.shape[0], device=v.device) // (BLOCK if square else 1)
    for i in range(power.shape[0]):
        v[:, i * BLOCK:(i + 1) * BLOCK] *= power[i][row][:, None]
    return v[:, :cols]


def _split(x, rounded=True):
    """Rows of x in 64 bits as codes (padded to whole blocks; their values before the rounding to 8 bits on request) and
    scales, laid out as a matrix in 8 bits is: the least scale among the powers of two by comparison, a step of an eighth
    of the value's own power of two, of 2^-9 below 2^-6, halves to even."""
    rows, cols = x.shape
    blocks = -(-cols // BLOCK)
    codes = torch.zeros(rows, blocks * BLOCK, dtype=torch.float64, device=x.device)
    codes[:, :cols] = x
    scales = torch.ones(blocks, (rows + 3) // 4 * 4, dtype=torch.float64, device=x.device)
    k = torch.arange(-126, 128, device=x.device, dtype=torch.float64)
    for i in range(blocks):
        v = codes[:, i * BLOCK:(i + 1) * BLOCK]
        top = v.abs().max(1).values
        s = torch.exp2(k[torch.searchsorted(448.0 * torch.exp2(k), top).clamp(max=k.numel() - 1)])
        scales[i, :rows] = torch.where(top > 0, s, torch.ones_like(s))
        v /= scales[i, :rows, None]
        if rounded:
            step = torch.exp2(torch.floor(torch.log2(v.abs().clamp(min=2.0 ** -6))) - 3)
            codes[:, i * BLOCK:(i + 1) * BLOCK] = torch.round(v / step) * step
    return codes, scales


def _to_e4m3(x):
    """Rows of x to 8 bits and back, in 64 bits."""
    codes, scales = _split(x)
    return (codes * scales[:, :x.shape[0]].t().repeat_interleave(BLOCK, 1))[:, :x.shape[1]]


def exact(case, seed):
    """The definitions in 64 bits.  The norm's codes as they are before their rounding to 8 bits, as for any other type."""
    st = prepare(case, seed)
    f64 = torch.float64
    if case["op"] == "norm":
        layer, n = case["kind"] == "layer", case["dim"]
        h = st["x"].to(f64)
        o = {}
        if st["residual"] is not None:
            # the sum is kept rounded to the stream's type, and what is normalised is what is kept
            h = (h + st["residual"].to(f64)).to(st["residual"].dtype).to(f64)
            o["residual"] = h
        mu = h.sum(1, keepdim=True) / n if layer else torch.zeros(h.shape[0], 1, dtype=f64, device=h.device)
        sd = torch.sqrt((h - mu).pow(2).sum(1, keepdim=True) / n + st["eps"])
        u = (h - mu) / sd * st["weight"].to(f64)
        codes, scales = _split(u + st["bias"].to(f64) if layer else u, rounded=False)
        return {"codes": codes, "scales": scales, **o}
    if case["op"] == "keep":
        (a, sa), (b, sb) = _split(st["x"]), _split(st["x"].t())
        return {"codes": a, "scales": sa, "codes_t": b, "scales_t": sb, "back": _to_e4m3(st["x"])}
    x = _values(st["x_in"], False) if isinstance(st["x_in"], tuple) else _to_e4m3(st["x_in"])
    if case["op"] == "linear":
        return {"out": torch.mm(x, _values(st["weight"], True).t())}
    dout = st["dout"]
    dx = torch.mm(_to_e4m3(dout), _values(st["weight_t"], True).t())
    return {"dx": dx, "dweight": torch.mm(_to_e4m3(dout.T.contiguous()), _to_e4m3(x.T.contiguous()).t())}
