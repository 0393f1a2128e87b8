"""The operators around the scan in a language model's training step and at serving: the embedding lookup and its
gradient, layer / RMS norm with the residual add and their gradients, and the softmax cross entropy of a linear head
over a large vocabulary with its gradients.  Cases, inputs, plain forms and 64-bit values."""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


# ------------------------------------------------------------------------------------------------------------ cases
def listed():
    return [
        # serving: one new token for each of 8 sequences, width of the 2.8B-like layer (d_inner 5120)
        {"name": "embed_decode", "op": "embedding", "dir": "fwd", "tokens": 8, "vocab": 50280, "dim": 2560, "io": "bf16"},
        # training: 8 x 2048 tokens of the 130M-like model (d_inner 1536), forward
        {"name": "embed_fwd", "op": "embedding", "dir": "fwd", "tokens": 16384, "vocab": 50280, "dim": 768, "io": "bf16"},
        # its gradient: few ids carry most tokens, most rows of the table none
        {"name": "embed_bwd", "op": "embedding", "dir": "bwd", "tokens": 16384, "vocab": 50280, "dim": 768, "io": "bf16"},
        # gradient of a small odd table in fp32, a ragged batch
        {"name": "embed_bwd_odd", "op": "embedding", "dir": "bwd", "tokens": 4999, "vocab": 32003, "dim": 333, "io": "f32"},
        # serving: the pre-norm of a block for 8 new tokens, residual stream in fp32
        {"name": "norm_decode", "op": "norm", "dir": "fwd", "kind": "rms", "rows": 8, "dim": 2560, "io": "bf16", "res": "f32"},
        # training: RMS pre-norm of the 2.8B-like layer, 4 x 8192 tokens, residual stream in fp32
        {"name": "norm_train", "op": "norm", "dir": "train", "kind": "rms", "rows": 32768, "dim": 2560, "io": "bf16", "res": "f32"},
        # training: plain layer norm, 8 x 2048 tokens of the 130M-like model
        {"name": "norm_train_layer", "op": "norm", "dir": "train", "kind": "layer", "rows": 16384, "dim": 768, "io": "bf16", "res": "none"},
        # a ragged batch of an odd width in fp32
        {"name": "norm_train_odd", "op": "norm", "dir": "train", "kind": "layer", "rows": 5001, "dim": 1023, "io": "f32", "res": "f32"},
        # scoring a few tokens: the head's table is read once
        {"name": "xent_score", "op": "xent", "dir": "fwd", "tokens": 16, "vocab": 50280, "dim": 2560, "io": "bf16", "ignored": 0.0},
        # training step of the 130M-like model, a padded batch
        {"name": "xent_train", "op": "xent", "dir": "train", "tokens": 8192, "vocab": 50280, "dim": 768, "io": "bf16", "ignored": 0.1},
        # fp32 training of a small model, odd sizes
        {"name": "xent_train_f32", "op": "xent", "dir": "train", "tokens": 1001, "vocab": 32003, "dim": 1000, "io": "f32", "ignored": 0.05},
        # training step over a large vocabulary
        {"name": "xent_train_large", "op": "xent", "dir": "train", "tokens": 16384, "vocab": 131072, "dim": 2048, "io": "bf16", "ignored": 0.0},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["embedding", "norm", "xent", "xent"])
    io = rng.choice(["bf16", "bf16", "f32"])
    if op == "embedding":
        c = {"op": op, "dir": rng.choice(["fwd", "bwd"]), "tokens": _log(rng, 1, 65536), "vocab": _log(rng, 1000, 131072),
             "dim": _log(rng, 64, 2560), "io": io}
        c["dim"] = c["dim"] if rng.random() < 0.5 else max(64, c["dim"] // 64 * 64)
        return c
    if op == "norm":
        c = {"op": op, "dir": rng.choice(["fwd", "train"]), "kind": rng.choice(["layer", "rms"]), "rows": _log(rng, 1, 32768),
             "dim": _log(rng, 64, 5120), "io": io, "res": rng.choice(["none", io, "f32"])}
        c["dim"] = c["dim"] if rng.random() < 0.5 else max(64, c["dim"] // 64 * 64)
        c["rows"] = min(c["rows"], 32768 * 2560 // c["dim"])
        return c
    c = {"op": op, "dir": rng.choice(["fwd", "train", "train"]), "tokens": _log(rng, 1, 16384), "vocab": _log(rng, 1000, 131072),
         "dim": _log(rng, 64, 2560), "io": io, "ignored": rng.choice([0.0, 0.1, 0.5])}
    c["dim"] = c["dim"] if rng.random() < 0.4 else max(64, c["dim"] // 64 * 64)
    most = 16384 * 131072 * 2048 // (8 if io == "f32" else 1)
    c["tokens"] = max(1, min(c["tokens"], most // (c["vocab"] * c["dim"])))
    return c


def _left_out(case):
    """Tokens of a loss case that its mask leaves out."""
    return int(case["tokens"] * case["ignored"])


def work(case):
    s = 2 if case["io"] == "bf16" else 4
    if case["op"] == "embedding":
        t, v, d = case["tokens"], case["vocab"], case["dim"]
        if case["dir"] == "fwd":
            return {"bytes": 8 * t + (min(t, v) + t) * d * s, "flops": t * d}
        return {"bytes": 8 * t + (t + v) * d * s, "flops": 2 * t * d}
    if case["op"] == "norm":
        n = case["rows"] * case["dim"]
        r = 0 if case["res"] == "none" else 2 if case["res"] == "bf16" else 4
        b = n * (2 * s + 2 * r)          # x, out, residual in and out
        if case["dir"] == "train":
            b += n * (2 * s + 2 * r)     # dout, dx, the residual's gradient in and out; h is the forward's own
        return {"bytes": b + 8 * case["dim"], "flops": n * (8 if case["dir"] == "fwd" else 22)}
    t, v, d = case["tokens"] - _left_out(case), case["vocab"], case["dim"]
    b = (t + v) * d * s + 16 * case["tokens"]
    if case["dir"] == "fwd":
        return {"bytes": b, "flops": 2 * t * v * d}
    return {"bytes": 2 * b, "flops": 6 * t * v * d}


# ----------------------------------------------------------------------------------------------------------- inputs
def _ids(g, n, vocab):
    """Token ids as text has them: log-uniform ranks (a few ids carry most of the tokens), ranks scattered over the ids."""
    u = torch.rand(n, generator=g, device="cuda", dtype=torch.float64)
    rank = torch.clamp(torch.exp(u * math.log(vocab + 1)).long() - 1, 0, vocab - 1)
    return torch.randperm(vocab, generator=g, device="cuda")[rank]


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(int(seed))
    dt = DTYPES[case["io"]]

    def rnd(*shape):
        return torch.randn(*shape, generator=g, device="cuda")

    st = dict(case)
    if case["op"] == "embedding":
        t, v, d = case["tokens"], case["vocab"], case["dim"]
        st["ids"] = _ids(g, t, v)
        st["scale"] = math.sqrt(d)
        if case["dir"] == "fwd":
            st["weight"] = (rnd(v, d) * d ** -0.5).to(dt)
        else:
            st["dout"] = (rnd(t, d) * 1e-3).to(dt)
        return st
    if case["op"] == "norm":
        n, d = case["rows"], case["dim"]
        rdt = DTYPES.get(case["res"])
        st["eps"] = 1e-5
        st["x"] = (rnd(n, d) * 0.8 + 0.1).to(dt)
        st["residual"] = None if rdt is None else (rnd(n, d) * 2.0).to(rdt)
        st["weight"] = 1.0 + 0.2 * rnd(d)
        st["bias"] = 0.1 * rnd(d) if case["kind"] == "layer" else None
        if case["dir"] == "train":
            st["dout"] = (rnd(n, d) * 1e-2).to(dt)
            st["dresidual"] = None if rdt is None else (rnd(n, d) * 1e-2).to(rdt)
        return st
    t, v, d = case["tokens"], case["vocab"], case["dim"]
    y = _ids(g, t, v)
    w = rnd(v, d) * (1.5 * d ** -0.5)
    # hidden states that lean towards their target's row, more or less, as in training
    lean = 5.0 * torch.rand(t, 1, generator=g, device="cuda")
    x = rnd(t, d) + lean * w[y]
    st["x"], st["weight"] = x.to(dt), w.to(dt)
    out = torch.randperm(t, generator=g, device="cuda")[:_left_out(case)]
    y[out] = -100
    st["targets"] = y
    if case["dir"] == "train":
        # the mean over the tokens that count, each with a weight of its own
        wt = 0.5 + torch.rand(t, generator=g, device="cuda")
        st["dloss"] = wt / max(1, t - _left_out(case))
    return st


# -------------------------------------------------------------------------------------------------------------- run
def run(st):
    if own:
        return _own(st)
    if st["op"] == "embedding":
        return _plain_embedding(st)
    if st["op"] == "norm":
        return _plain_norm(st)
    return _plain_xent(st)


def _own(st):
    import selective_state_space_17_amd as M

    if st["op"] == "embedding":
        if st["dir"] == "fwd":
            return {"out": M.embedding_fwd(st["ids"], st["weight"], scale=st["scale"])}
        return {"dweight": M.embedding_bwd(st["ids"], st["dout"], st["vocab"], scale=st["scale"])}
    if st["op"] == "norm":
        layer, res, train = st["kind"] == "layer", st["residual"], st["dir"] == "train"
        fwd = M.layer_norm_fwd if layer else M.rms_norm_fwd
        args = (st["x"], st["weight"]) + ((st["bias"],) if layer else ())
        got = fwd(*args, residual=res, eps=st["eps"], return_residual=res is not None, return_stats=train)
        got = list(got) if isinstance(got, tuple) else [got]
        o = {"out": got.pop(0)}
        if res is not None:
            o["residual"] = got.pop(0)
        if not train:
            return o
        h = st["x"] if res is None else o["residual"]
        bwd = M.layer_norm_bwd if layer else M.rms_norm_bwd
        grads = bwd(h, st["weight"], *got, st["dout"], dresidual=st["dresidual"], want_dresidual=res is not None)
        return {**o, **{k: t for k, t in grads.items() if t is not None}}
    loss, lse = M.linear_cross_entropy_fwd(st["x"], st["weight"], st["targets"])
    if st["dir"] == "fwd":
        return {"loss": loss, "lse": lse}
    grads = M.linear_cross_entropy_bwd(st["x"], st["weight"], st["targets"], lse, st["dloss"])
    return {"loss": loss, "lse": lse, "dx": grads["dx"], "dweight": grads["dweight"]}


def _plain_embedding(st):
    if st["dir"] == "fwd":
        w = st["weight"]
        return {"out": (w[st["ids"]].float() * st["scale"]).to(w.dtype)}
    dout = st["dout"]
    dw = torch.zeros(st["vocab"], st["dim"], device=dout.device)
    dw.index_add_(0, st["ids"], dout.float() * st["scale"])
    return {"dweight": dw.to(dout.dtype)}


def _plain_norm(st):
    x, res, w, layer = st["x"], st["residual"], st["weight"], st["kind"] == "layer"
    o = {}
    h = x.float()
    if res is not None:
        o["residual"] = (h + res.float()).to(res.dtype)
        h = o["residual"].float()
    c = h - h.mean(1, keepdim=True) if layer else h
    rstd = torch.rsqrt((c * c).mean(1, keepdim=True) + st["eps"])
    xh = c * rstd
    o = {"out": (xh * w + st["bias"] if layer else xh * w).to(x.dtype), **o}
    if st["dir"] == "fwd":
        return o
    dout = st["dout"].float()
    g = dout * w
    dh = g - xh * (g * xh).mean(1, keepdim=True)
    if layer:
        dh = dh - g.mean(1, keepdim=True)
    dh = dh * rstd
    if res is not None:
        dh = dh + st["dresidual"].float()
    o["dx"] = dh.to(x.dtype)
    if res is not None:
        o["dresidual"] = dh.to(res.dtype)
    o["dweight"] = (dout * xh).sum(0)
    if layer:
        o["dbias"] = dout.sum(0)
    return o


def _plain_xent(st):
    y = st["targets"]
    kept = (y >= 0).nonzero()[:, 0]
    x, w, yk = st["x"][kept].float(), st["weight"].float(), y[kept]
    rows = torch.arange(yk.numel(), device=y.device)
    logits = x @ w.T
    top = logits.max(1, keepdim=True).values
    e = torch.exp(logits - top)
    total = e.sum(1, keepdim=True)
    lse_k = (top + torch.log(total))[:, 0]
    zero = torch.zeros(y.numel(), device=y.device)
    o = {"loss": zero.index_copy(0, kept, lse_k - logits[rows, yk]), "lse": zero.index_copy(0, kept, lse_k)}
    if st["dir"] == "fwd":
        return o
    p = e / total
    p[rows, yk] -= 1.0
    p *= st["dloss"][kept][:, None]
    dx = torch.zeros(st["x"].shape, device=y.device).index_copy(0, kept, p @ w)
    return {**o, "dx": dx.to(st["x"].dtype), "dweight": (p.T @ x).to(st["weight"].dtype)}


# ------------------------------------------------------------------------------------------------------------ exact
def exact(case, seed):
    """The definitions in 64 bits, gradients from the sums that define them, row block by row block."""
    st = prepare(case, seed)
    f64 = torch.float64
    if case["op"] == "embedding":
        if case["dir"] == "fwd":
            return {"out": torch.index_select(st["weight"], 0, st["ids"]).to(f64) * st["scale"]}
        order = torch.argsort(st["ids"], stable=True)
        ids = st["ids"][order]
        d = st["dout"][order].to(f64)
        run_sum = torch.cumsum(d, 0)
        last = torch.cat([ids[1:] != ids[:-1], ids.new_ones(1, dtype=torch.bool)]).nonzero()[:, 0]
        upto = run_sum[last]
        upto[1:] = upto[1:] - run_sum[last[:-1]]
        dw = torch.zeros(case["vocab"], case["dim"], dtype=f64, device=d.device)
        dw[ids[last]] = upto * st["scale"]
        return {"dweight": dw}
    if case["op"] == "norm":
        layer, n = case["kind"] == "layer", case["dim"]
        h = st["x"].to(f64)
        o = {"out": None}
        if st["residual"] is not None:
            # the sum is kept rounded to the stream's type, and what is normalised is what is kept
            h = (h + st["residual"].to(f64)).to(st["residual"].dtype).to(f64)
            o["residual"] = h
        mu = h.sum(1, keepdim=True) / n if layer else torch.zeros(h.shape[0], 1, dtype=f64, device=h.device)
        sd = torch.sqrt((h - mu).pow(2).sum(1, keepdim=True) / n + st["eps"])
        w = st["weight"].to(f64)
        xh = (h - mu) / sd
        o["out"] = xh * w + (st["bias"].to(f64) if layer else 0.0)
        if case["dir"] == "fwd":
            return o
        g = st["dout"].to(f64)
        # dh_i = sum_j g_j w_j d(xh_j)/dh_i, d(xh_j)/dh_i = (delta_ij - [layer] 1/n - xh_i xh_j / n) / sd
        gw = g * w
        dh = (gw - xh * ((gw * xh).sum(1, keepdim=True) / n) - (gw.sum(1, keepdim=True) / n if layer else 0.0)) / sd
        if st["residual"] is not None:
            dh = dh + st["dresidual"].to(f64)
        o["dx"] = dh
        if st["residual"] is not None:
            o["dresidual"] = dh
        o["dweight"] = (g * xh).sum(0)
        if layer:
            o["dbias"] = g.sum(0)
        return o
    x, w, y = st["x"].to(f64), st["weight"].to(f64), st["targets"]
    t = y.numel()
    loss, lse = (torch.zeros(t, dtype=f64, device=y.device) for _ in range(2))
    train = case["dir"] == "train"
    dx, dw = (torch.zeros_like(x), torch.zeros_like(w)) if train else (None, None)
    step = max(1, (1 << 28) // w.shape[0])
    for a in range(0, t, step):
        rows = torch.nonzero(y[a:a + step] >= 0)[:, 0] + a
        if rows.numel() == 0:
            continue
        logits = torch.mm(x[rows], w.t())
        z = torch.logsumexp(logits, 1)
        hit = torch.gather(logits, 1, y[rows, None])[:, 0]
        loss[rows], lse[rows] = z - hit, z
        if train:
            gr = torch.exp(logits - z[:, None])
            gr.scatter_add_(1, y[rows, None], torch.full((rows.numel(), 1), -1.0, dtype=f64, device=y.device))
            gr *= st["dloss"][rows].to(f64)[:, None]
            dx[rows] = torch.mm(gr, w)
            dw += torch.mm(gr.t(), x[rows])
    o = {"loss": loss, "lse": lse}
    return {**o, "dx": dx, "dweight": dw} if train else o
