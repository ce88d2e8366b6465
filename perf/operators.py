"""Measured cases of the training-step operators around the tensor-parallel block.

Three operators, each in a plain form (elementary torch operations in 32 bits) and
as the calls that a user of the library makes:

  loss        the output head and its softmax cross-entropy in one call, without
              the logits: loss, log-sum-exp, and the gradients of the hidden
              states and of the vocab-sharded head weight.
  norm_fwd,   the junction of two sublayers: x_out = res_scale * x + gate *
  norm_bwd    Norm_post(f), y = Norm_pre(x_out), and its backward.
  ckpt_fwd,   the MLP's column layer keeping its pre-activation in 8 bits (e4m3
  ckpt_bwd    with a power-of-two scale per 32 columns of a row), and the row
              layer's backward that reads it.
"""
import functools
import math

import torch

own = False

EPS = 1e-5
DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
GROUP = 32  # columns of a row that share a scale


# --------------------------------------------------------------------- cases
def listed():
    return [
        # a handful of tokens on a small head: launches and latency
        {"name": "loss 17 tok v1003", "op": "loss", "dtype": "bf16", "T": 17, "h": 512, "V": 1003, "p": 2, "grad": True},
        # the 12-layer stack's hidden size with a 32k vocab: a training batch
        {"name": "loss 2048 tok v32000 h512", "op": "loss", "dtype": "bf16", "T": 2048, "h": 512, "V": 32000, "p": 4, "grad": True},
        # the 7B-shaped hidden size with a large vocab: the biggest products
        {"name": "loss 4096 tok v131072 h4096", "op": "loss", "dtype": "bf16", "T": 4096, "h": 4096, "V": 131072, "p": 8, "grad": True},
        # the tiny fp32 configuration's type, a ragged vocab
        {"name": "loss fp32 500 tok v8201", "op": "loss", "dtype": "f32", "T": 500, "h": 512, "V": 8201, "p": 2, "grad": True},
        # scoring a few tokens: the loss alone, bound by reading the head weight
        {"name": "score 61 tok v32000 h4096", "op": "loss", "dtype": "bf16", "T": 61, "h": 4096, "V": 32000, "p": 8, "grad": False},
        # one generated token passes the junction
        {"name": "norm fwd 1 row h4096 rms", "op": "norm_fwd", "dtype": "bf16", "kind": "rms", "rows": 1, "h": 4096, "B": 1,
         "post": True, "pre": True, "rs": 1.0},
        # the 7B-shaped training batch, a gate per channel
        {"name": "norm fwd 32768 rows h4096", "op": "norm_fwd", "dtype": "bf16", "kind": "layer", "rows": 32768, "h": 4096, "B": 1,
         "post": True, "pre": True, "rs": 1.0},
        # the sequence-parallel hidden size, a gate per sequence of a batch of 8
        {"name": "norm bwd 8192 rows h8192 B8", "op": "norm_bwd", "dtype": "bf16", "kind": "rms", "rows": 8192, "h": 8192, "B": 8,
         "post": True, "pre": True, "rs": 1.0},
        # fp32, odd sizes, three sequences, a scaled residual
        {"name": "norm bwd fp32 2049 rows h520", "op": "norm_bwd", "dtype": "f32", "kind": "layer", "rows": 2049, "h": 520, "B": 3,
         "post": True, "pre": True, "rs": 0.75},
        # the 7B-shaped SwiGLU MLP over 8 shards
        {"name": "ckpt fwd swiglu 8192 tok 7B", "op": "ckpt_fwd", "act": "swiglu", "T": 8192, "h": 4096, "f": 11008, "p": 8},
        {"name": "ckpt bwd swiglu 8192 tok 7B", "op": "ckpt_bwd", "act": "swiglu", "T": 8192, "h": 4096, "f": 11008, "p": 8},
        # the 12-layer stack's GELU MLP, a ragged token count
        {"name": "ckpt bwd gelu 2011 tok h512", "op": "ckpt_bwd", "act": "gelu", "T": 2011, "h": 512, "f": 2048, "p": 2},
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(("loss", "loss", "norm_fwd", "norm_bwd", "ckpt_fwd", "ckpt_bwd"))
    if op == "loss":
        f32 = rng.random() < 0.2
        p = rng.choice((1, 2, 4, 8))
        h = 8 * p * max(1, _log_int(rng, 64, 1024 if f32 else 4096) // (8 * p))
        V = _log_int(rng, 50, 16384 if f32 else 131072)
        most = (1.2e10 if f32 else 2.0e12) / (V * h)
        T = _log_int(rng, 1, max(2, min(4096, int(most))))
        return {"op": op, "dtype": "f32" if f32 else "bf16", "T": T, "h": h, "V": V, "p": p, "grad": rng.random() < 0.8}
    if op in ("norm_fwd", "norm_bwd"):
        f32 = rng.random() < 0.3
        h = 8 * _log_int(rng, 8, 1024)
        B = rng.choice((0, 1, 1, 2, 5, 8))
        most = max(8, int(5.0e7 // h))
        rows = max(1, _log_int(rng, 1, most) // max(B, 1)) * max(B, 1)
        return {"op": op, "dtype": "f32" if f32 else "bf16", "kind": rng.choice(("layer", "rms")), "rows": rows, "h": h, "B": B,
                "post": rng.random() < 0.8, "pre": rng.random() < 0.8, "rs": rng.choice((1.0, 0.5, 1.25))}
    p = rng.choice((1, 2, 4, 8))
    h = 8 * p * max(1, _log_int(rng, 64, 4096) // (8 * p))
    f = 16 * p * max(1, _log_int(rng, 256, 11008) // (16 * p))
    T = _log_int(rng, 1, max(2, min(8192, int(3.0e11 / (h * f)))))
    return {"op": op, "act": rng.choice(("swiglu", "gelu")), "T": T, "h": h, "f": f, "p": p}


def _padded(V, p):
    return -(-V // (8 * p)) * 8 * p


def _groups(c):
    """Scale groups of a row of one shard: those of each half start anew."""
    fp = c["f"] // c["p"]
    return (2 if c["act"] == "swiglu" else 1) * -(-fp // GROUP)


# -------------------------------------------------------------------- inputs
def _randn(g, *shape, dtype=torch.bfloat16, std=1.0):
    return (torch.randn(*shape, generator=g, device="cuda", dtype=torch.float32) * std).to(dtype)


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return {"loss": _prepare_loss, "norm_fwd": _prepare_norm, "norm_bwd": _prepare_norm,
            "ckpt_fwd": _prepare_ckpt, "ckpt_bwd": _prepare_ckpt}[case["op"]](case, g)


def _prepare_loss(c, g):
    T, h, V, p, dt = c["T"], c["h"], c["V"], c["p"], DTYPES[c["dtype"]]
    Vp = _padded(V, p)
    W = _randn(g, Vp, h, dtype=dt, std=0.02)
    labels = torch.randint(0, V, (T,), generator=g, device="cuda", dtype=torch.int32)
    # half the tokens lean towards their label, as a trained head's do
    lean = (torch.arange(T, device="cuda") % 2 == 0).float()[:, None] * (6.0 / (h * 0.02 ** 2))
    X = (_randn(g, T, h, dtype=torch.float32) + lean * W[labels.long()].float()).to(dt)
    if T > 8:
        labels[T // 3::37] = -1  # padding and prompt tokens are ignored
    new = functools.partial(torch.empty, device="cuda")
    return {"case": c, "X": X, "W": [w.clone() for w in W.chunk(p)], "labels": labels, "scale": 1.0 / T,
            "loss": new(T, dtype=torch.float32), "lse": new(T, dtype=torch.float32),
            "dX": new(T, h, dtype=dt) if c["grad"] else None,
            "dW": [new(Vp // p, h, dtype=dt) for _ in range(p)] if c["grad"] else None}


def _prepare_norm(c, g):
    rows, h, B, dt = c["rows"], c["h"], c["B"], DTYPES[c["dtype"]]
    new = functools.partial(torch.empty, device="cuda")
    s = {"case": c,
         "x": _randn(g, rows, h, dtype=dt), "f": (_randn(g, rows, h, dtype=torch.float32, std=0.5) + 0.05).to(dt),
         "gate": _randn(g, B, h, dtype=dt, std=0.3) if B else None,
         "post": ((1 + _randn(g, h, dtype=torch.float32, std=0.1)).to(dt), _randn(g, h, dtype=dt, std=0.1)) if c["post"] else None,
         "pre": ((1 + _randn(g, h, dtype=torch.float32, std=0.1)).to(dt), _randn(g, h, dtype=dt, std=0.1)) if c["pre"] else None,
         "x_out": new(rows, h, dtype=dt), "y": new(rows, h, dtype=dt) if c["pre"] else None,
         "stats": torch.zeros(4, rows, device="cuda", dtype=torch.float32)}
    if c["op"] == "norm_fwd":
        return s
    f32 = functools.partial(torch.empty, device="cuda", dtype=torch.float32)
    # what the forward left: its output row and its statistics
    x_out, _, stats = _norm_forward(c, s["x"], s["f"], s["gate"], s["post"], s["pre"], torch.float32)
    s |= {"x_out": x_out.to(dt), "stats": stats, "dx_out": _randn(g, rows, h, dtype=dt), "dy": _randn(g, rows, h, dtype=dt) if c["pre"] else None,
          "dx": new(rows, h, dtype=dt), "df": new(rows, h, dtype=dt), "dgate": f32(B, h) if B else None,
          "dpost": (f32(h), f32(h)) if c["post"] else None, "dpre": (f32(h), f32(h)) if c["pre"] else None}
    return s


def _prepare_ckpt(c, g):
    T, h, f, p = c["T"], c["h"], c["f"], c["p"]
    fp = f // p
    n1 = 2 * fp if c["act"] == "swiglu" else fp
    new = functools.partial(torch.empty, device="cuda", dtype=torch.bfloat16)
    s = {"case": c, "H": [new(T, fp) for _ in range(p)]}
    if c["op"] == "ckpt_fwd":
        return s | {"X": _randn(g, T, h), "W": [_randn(g, n1, h, std=h ** -0.5) for _ in range(p)],
                    "bias": [_randn(g, n1, std=0.1) for _ in range(p)] if c["act"] == "gelu" else None,
                    "Zq": [torch.empty(T, n1, device="cuda", dtype=torch.float8_e4m3fn) for _ in range(p)],
                    "Zs": [torch.empty(_groups(c), T, device="cuda", dtype=torch.uint8) for _ in range(p)]}
    packed = [_pack(_randn(g, T, n1, dtype=torch.float32), c) for _ in range(p)]
    return s | {"dY": _randn(g, T, h), "W": [_randn(g, h, fp, std=f ** -0.5) for _ in range(p)],
                "Zq": [q for q, _ in packed], "Zs": [z for _, z in packed],
                "dZ": [new(T, n1) for _ in range(p)], "dW": [new(h, fp) for _ in range(p)],
                "dbias": torch.empty(h, device="cuda", dtype=torch.float32)}


# ---------------------------------------------------------------------- run
def run(state):
    return {"loss": _run_loss, "norm_fwd": _run_norm_fwd, "norm_bwd": _run_norm_bwd,
            "ckpt_fwd": _run_ckpt_fwd, "ckpt_bwd": _run_ckpt_bwd}[state["case"]["op"]](state)


@functools.lru_cache(maxsize=None)
def _plan(hidden, ffn, p, dtype, act, vocab):
    """The plan that a program keeps for its block's sizes."""
    from megatron_tensor_transformer_gemm_b200 import Plan
    plan = Plan(hidden, ffn, 0, p, dtype, act)
    if vocab:
        plan.set_vocab(vocab)
    return plan


def _run_loss(s):
    c = s["case"]
    if own:
        plan = _plan(c["h"], 0, c["p"], c["dtype"], "none", c["V"])
        plan.vocab_linear_cross_entropy(c["T"], s["X"], s["W"], s["labels"], s["scale"], s["loss"], s["lse"], s["dX"], s["dW"])
        return {"loss": s["loss"], "lse": s["lse"], "dX": s["dX"], "dW": s["dW"]}
    V, dt = c["V"], DTYPES[c["dtype"]]
    X = s["X"].float()
    W = torch.cat(s["W"]).float()
    z = X @ W[:V].T
    m = z.amax(1, keepdim=True)
    e = torch.exp(z - m)
    total = e.sum(1, keepdim=True)
    lse = (m + torch.log(total))[:, 0]
    kept = s["labels"] >= 0
    label = s["labels"].long().clamp(min=0)
    rows = torch.arange(c["T"], device=X.device)
    loss = torch.where(kept, lse - z[rows, label], torch.zeros_like(lse))
    if not c["grad"]:
        return {"loss": loss, "lse": lse, "dX": None, "dW": None}
    d = e / total
    d[rows, label] -= 1
    d *= torch.where(kept, s["scale"], 0.0)[:, None]
    dX = (d @ W[:V]).to(dt)
    dW = torch.zeros(W.shape, device=X.device, dtype=dt)
    dW[:V] = (d.T @ X).to(dt)
    return {"loss": loss, "lse": lse, "dX": dX, "dW": list(dW.chunk(c["p"]))}


def _normed(x, kind):
    """(xhat, mean, rstd) of every row."""
    mean = x.mean(1, keepdim=True) if kind == "layer" else torch.zeros_like(x[:, :1])
    rstd = 1 / torch.sqrt(((x - mean) ** 2).mean(1, keepdim=True) + EPS)
    return (x - mean) * rstd, mean, rstd


def _affine(xhat, weights, kind, wide):
    return xhat * weights[0].to(wide) + (weights[1].to(wide) if kind == "layer" else 0)


def _gate_rows(gate, rows, wide):
    """Row r's gate is gate[r % B]: tokens are in sequence-major order."""
    return gate.to(wide)[torch.arange(rows, device=gate.device) % gate.shape[0]] if gate is not None else 1.0


def _norm_forward(c, x, f, gate, post, pre, wide):
    """x_out, y and the statistics [4, rows] in `wide`; y is that of x_out as stored."""
    stats = torch.zeros(4, c["rows"], device=x.device, dtype=wide)
    n = f.to(wide)
    if post is not None:
        xhat, mean, rstd = _normed(n, c["kind"])
        stats[0], stats[1] = mean[:, 0], rstd[:, 0]
        n = _affine(xhat, post, c["kind"], wide)
    x_out = c["rs"] * x.to(wide) + _gate_rows(gate, c["rows"], wide) * n
    y = None
    if pre is not None:
        xhat, mean, rstd = _normed(x_out.to(x.dtype).to(wide), c["kind"])
        stats[2], stats[3] = mean[:, 0], rstd[:, 0]
        y = _affine(xhat, pre, c["kind"], wide)
    return x_out, y, stats


def _run_norm_fwd(s):
    c = s["case"]
    dt = DTYPES[c["dtype"]]
    if own:
        plan = _plan(c["h"], 0, 1, c["dtype"], "none", 0)
        plan.gated_residual_norm_fwd(c["kind"], c["rows"], s["x"], s["f"], s["x_out"], s["y"], res_scale=c["rs"], gate=s["gate"],
                                     post=s["post"], pre=s["pre"], stats=s["stats"])
        return {"x_out": s["x_out"], "y": s["y"], "stats": s["stats"]}
    x_out, y, stats = _norm_forward(c, s["x"], s["f"], s["gate"], s["post"], s["pre"], torch.float32)
    return {"x_out": x_out.to(dt), "y": y.to(dt) if y is not None else None, "stats": stats}


def _norm_input_grad(g, xhat, rstd, kind):
    """Gradient of a norm's input from that of xhat."""
    d = g - xhat * (g * xhat).mean(1, keepdim=True)
    return rstd * (d - g.mean(1, keepdim=True) if kind == "layer" else d)


def _norm_backward(s, wide):
    """The backward's outputs, in `wide`."""
    c = s["case"]
    rows, h, kind, B = c["rows"], c["h"], c["kind"], c["B"]
    f, x_out, stats, D = s["f"].to(wide), s["x_out"].to(wide), s["stats"].to(wide), s["dx_out"].to(wide)
    out = {"dpre": None, "dpost": None, "dgate": None}
    if s["pre"] is not None:
        dy, rstd = s["dy"].to(wide), stats[3][:, None]
        xhat = (x_out - stats[2][:, None]) * rstd
        out["dpre"] = [(dy * xhat).sum(0)] + ([dy.sum(0)] if kind == "layer" else [])
        D = D + _norm_input_grad(dy * s["pre"][0].to(wide), xhat, rstd, kind)
    out["dx"] = c["rs"] * D
    n = f
    if s["post"] is not None:
        rstd = stats[1][:, None]
        xhat = (f - stats[0][:, None]) * rstd
        n = _affine(xhat, s["post"], kind, wide)
    if B:
        out["dgate"] = (D * n).reshape(rows // B, B, h).sum(0)
    dn = D * _gate_rows(s["gate"], rows, wide)
    out["df"] = dn
    if s["post"] is not None:
        out["dpost"] = [(dn * xhat).sum(0)] + ([dn.sum(0)] if kind == "layer" else [])
        out["df"] = _norm_input_grad(dn * s["post"][0].to(wide), xhat, rstd, kind)
    return out


def _run_norm_bwd(s):
    c = s["case"]
    if own:
        plan = _plan(c["h"], 0, 1, c["dtype"], "none", 0)
        plan.gated_residual_norm_bwd(c["kind"], c["rows"], s["f"], s["x_out"], s["stats"], s["dx_out"], s["dy"], s["dx"], s["df"],
                                     res_scale=c["rs"], gate=s["gate"], dgate=s["dgate"], post=s["post"], dpost=s["dpost"],
                                     pre=s["pre"], dpre=s["dpre"])
        n = 2 if c["kind"] == "layer" else 1
        return {"dx": s["dx"], "df": s["df"], "dgate": s["dgate"], "dpost": s["dpost"][:n] if s["dpost"] else None,
                "dpre": s["dpre"][:n] if s["dpre"] else None}
    dt = DTYPES[c["dtype"]]
    out = _norm_backward(s, torch.float32)
    return {"dx": out["dx"].to(dt), "df": out["df"].to(dt), "dgate": out["dgate"], "dpost": out["dpost"], "dpre": out["dpre"]}


# ------------------------------------------------ the 8-bit pre-activations
def _halves(c):
    return 2 if c["act"] == "swiglu" else 1


def _pack(z, c):
    """(q, s) of z [T, n1] in 32 or 64 bits: e4m3 codes [T, n1] and biased scale
    exponents [groups, T]. The scale of 32 columns of a row is the least power
    of two (at least 2^-126) that brings their largest magnitude to at most 448."""
    T, n1 = z.shape
    half = n1 // _halves(c)
    G = -(-half // GROUP)
    a = torch.zeros(T, _halves(c), G * GROUP, device=z.device, dtype=z.dtype)
    a[:, :, :half] = z.reshape(T, _halves(c), half)
    a = a.reshape(T, _halves(c) * G, GROUP)
    mant, expo = torch.frexp(a.abs().amax(2))        # amax = mant * 2^expo, mant in [0.5, 1)
    e = expo - 9 + (mant > 0.875).to(expo.dtype)     # 448 = 0.875 * 2^9
    e = torch.where(mant > 0, e, torch.full_like(e, -126)).clamp(min=-126)
    q = torch.ldexp(a, -e[:, :, None]).float().to(torch.float8_e4m3fn)
    q = q.reshape(T, _halves(c), G * GROUP)[:, :, :half].reshape(T, n1).contiguous()
    return q, (e + 127).to(torch.uint8).T.contiguous()


def _unpack(q, s, c, wide):
    T, n1 = q.shape
    half = n1 // _halves(c)
    G = -(-half // GROUP)
    scale = torch.ldexp(torch.ones((), device=q.device, dtype=wide), s.T.int() - 127)
    scale = scale.reshape(T, _halves(c), G, 1).expand(T, _halves(c), G, GROUP).reshape(T, _halves(c), G * GROUP)[:, :, :half]
    return q.to(wide) * scale.reshape(T, n1)


def _act(z, c):
    """(H, its derivatives' factors): the activation of z [T, n1] and dZ = dH * each."""
    if c["act"] == "swiglu":
        g, u = z.chunk(2, 1)
        sg = 1 / (1 + torch.exp(-g))
        return g * sg * u, [u * sg * (1 + g * (1 - sg)), g * sg]
    phi = 0.5 * (1 + torch.erf(z * 0.5 ** 0.5))
    return z * phi, [phi + z * torch.exp(-0.5 * z * z) * (2 * math.pi) ** -0.5]


def _column_forward(s, wide):
    c = s["case"]
    X = s["X"].to(wide)
    Z = (X @ torch.cat(s["W"]).to(wide).T).chunk(c["p"], 1)
    if s["bias"] is not None:
        Z = [z + b.to(wide) for z, b in zip(Z, s["bias"])]
    packed = [_pack(z, c) for z in Z]
    return [q for q, _ in packed], [z for _, z in packed], [_act(z, c)[0].to(torch.bfloat16) for z in Z]


def _run_ckpt_fwd(s):
    c = s["case"]
    if own:
        plan = _plan(c["h"], c["f"], c["p"], "bf16", c["act"], 0)
        plan.column_fwd_ckpt8(c["T"], s["X"], s["W"], s["bias"], s["Zq"], s["Zs"], s["H"])
        Zq, Zs, H = s["Zq"], s["Zs"], s["H"]
    else:
        Zq, Zs, H = _column_forward(s, torch.float32)
    # the scale's byte is the e8m0 number of its value
    return {"Zq": Zq, "Zs": [z.view(torch.float8_e8m0fnu) for z in Zs], "H": H}


def _row_backward(s, wide):
    """dZ, H, dW and dbias in `wide`; dW is the product with H as stored."""
    c = s["case"]
    dY = s["dY"].to(wide)
    act = [_act(_unpack(q, z, c, wide), c) for q, z in zip(s["Zq"], s["Zs"])]
    H = [a[0].to(torch.bfloat16) for a in act]
    dH = (dY @ torch.cat(s["W"], 1).to(wide)).chunk(c["p"], 1)
    dZ = [torch.cat([d * k for k in a[1]], 1) for d, a in zip(dH, act)]
    dW = (dY.T @ torch.cat(H, 1).to(wide)).chunk(c["p"], 1)
    return dZ, H, dW, dY.sum(0)


def _run_ckpt_bwd(s):
    c = s["case"]
    if own:
        plan = _plan(c["h"], c["f"], c["p"], "bf16", c["act"], 0)
        plan.row_bwd_ckpt8(c["T"], s["dY"], s["W"], s["Zq"], s["Zs"], s["H"], s["dZ"], s["dW"], s["dbias"])
        return {"dZ": s["dZ"], "H": s["H"], "dW": s["dW"], "dbias": s["dbias"]}
    dZ, H, dW, dbias = _row_backward(s, torch.float32)
    return {"dZ": [z.to(torch.bfloat16) for z in dZ], "H": H, "dW": [w.to(torch.bfloat16) for w in dW], "dbias": dbias}


# --------------------------------------------------------------------- work
def work(case):
    c = case
    if c["op"] == "loss":
        size = 2 if c["dtype"] == "bf16" else 4
        T, h, Vp, n = c["T"], c["h"], _padded(c["V"], c["p"]), 2 if c["grad"] else 1
        return {"bytes": n * size * (T * h + Vp * h) + 12 * T, "flops": (6 if c["grad"] else 2) * T * c["V"] * h}
    if c["op"] in ("norm_fwd", "norm_bwd"):
        size, rows, h = 2 if c["dtype"] == "bf16" else 4, c["rows"], c["h"]
        planes = (3 + c["pre"]) if c["op"] == "norm_fwd" else (4 + 2 * c["pre"] if c["pre"] or c["B"] else 3 + c["post"])
        return {"bytes": planes * size * rows * h + (2 + 4 * (c["op"] == "norm_bwd")) * h * (c["B"] + 4), "flops": 20 * rows * h}
    T, h, f, p = c["T"], c["h"], c["f"], c["p"]
    n1 = _halves(c) * f
    packed = T * n1 + p * _groups(c) * T
    if c["op"] == "ckpt_fwd":
        return {"bytes": 2 * (T * h + n1 * h + T * f) + packed, "flops": 2 * T * h * n1}
    return {"bytes": 2 * (T * h + f * h + T * n1 + T * f + f * h) + packed + 4 * h, "flops": 4 * T * h * f}


# -------------------------------------------------------------------- exact
def exact(case, seed):
    """run()'s answer from the definitions in 64 bits."""
    s = prepare(case, seed)
    return {"loss": _exact_loss, "norm_fwd": _exact_norm_fwd, "norm_bwd": _exact_norm_bwd,
            "ckpt_fwd": _exact_ckpt_fwd, "ckpt_bwd": _exact_ckpt_bwd}[case["op"]](case, s)


def _exact_loss(c, s):
    T, V, p, h = c["T"], c["V"], c["p"], c["h"]
    X = s["X"].double()
    W = torch.cat([w.double() for w in s["W"]], 0)
    loss, lse, dX = [], [], []
    dW = torch.zeros_like(W)
    step = max(1, (1 << 28) // V)
    for t in range(0, T, step):  # blocks of tokens bound the memory
        x, y = X[t:t + step], s["labels"][t:t + step].long()
        logp = torch.log_softmax(x @ W[:V].mT, dim=-1)
        some = (y >= 0).nonzero()[:, 0]
        part = torch.zeros(len(y), dtype=torch.float64, device=X.device)
        part[some] = -logp[some, y[some]]
        loss.append(part)
        lse.append((x * W[0]).sum(1) - logp[:, 0])
        if c["grad"]:
            G = torch.zeros_like(logp)
            G[some] = torch.exp(logp[some])
            G[some, y[some]] -= 1.0
            G *= s["scale"]
            dX.append(G @ W[:V])
            dW[:V] += G.mT @ x
    return {"loss": torch.cat(loss), "lse": torch.cat(lse), "dX": torch.cat(dX) if c["grad"] else None,
            "dW": list(torch.split(dW, _padded(V, p) // p)) if c["grad"] else None}


def _exact_rows(x, kind):
    if kind == "layer":
        var, mean = torch.var_mean(x, dim=1, unbiased=False)
    else:
        var, mean = x.pow(2).mean(1), torch.zeros_like(x[:, 0])
    return mean, torch.rsqrt(var + EPS)


def _exact_norm_fwd(c, s):
    x, f, kind, rows = s["x"].double(), s["f"].double(), c["kind"], c["rows"]
    stats = torch.zeros(4, rows, dtype=torch.float64, device=x.device)
    if s["post"] is not None:
        stats[0], stats[1] = _exact_rows(f, kind)
        f = (f - stats[0, :, None]) * stats[1, :, None] * s["post"][0].double()
        f = f + s["post"][1].double() if kind == "layer" else f
    if s["gate"] is not None:
        f = (f.reshape(rows // c["B"], c["B"], -1) * s["gate"].double()).reshape(rows, -1)
    x_out = x * c["rs"] + f
    y = None
    if s["pre"] is not None:
        stored = x_out.to(DTYPES[c["dtype"]]).double()
        stats[2], stats[3] = _exact_rows(stored, kind)
        y = (stored - stats[2, :, None]) * stats[3, :, None] * s["pre"][0].double()
        y = y + s["pre"][1].double() if kind == "layer" else y
    return {"x_out": x_out, "y": y, "stats": stats}


def _exact_norm_bwd(c, s):
    # by automatic differentiation of the definition with the statistics' own
    # dependence on the rows, about the stored f and x_out
    kind, rows, B = c["kind"], c["rows"], c["B"]
    leaf = lambda t: t.double().detach().requires_grad_()  # noqa: E731

    def norm(x, w, b, mean, rstd):
        # the stored statistics as values; their derivatives by the chain rule
        m = x.mean(1, keepdim=True) if kind == "layer" else torch.zeros_like(x[:, :1])
        r = ((x - m) ** 2).mean(1, keepdim=True).add(EPS).rsqrt()
        r = r * (rstd.double()[:, None] / r.detach())
        m = m + (mean.double()[:, None] - m.detach())
        return (x - m) * r * w + (b if kind == "layer" else 0)

    D = s["dx_out"].double()
    out = {"dx": None, "df": None, "dgate": None, "dpost": None, "dpre": None}
    n = 2 if kind == "layer" else 1
    if s["pre"] is not None:
        x, w, b = leaf(s["x_out"]), leaf(s["pre"][0]), leaf(s["pre"][1])
        got = torch.autograd.grad(norm(x, w, b, s["stats"][2], s["stats"][3]), [x, w, b][:n + 1], s["dy"].double())
        D, out["dpre"] = D + got[0], list(got[1:])
    out["dx"] = c["rs"] * D
    f = leaf(s["f"])
    wrt, v = [f], f
    if s["post"] is not None:
        w, b = leaf(s["post"][0]), leaf(s["post"][1])
        wrt += [w, b][:n]
        v = norm(f, w, b, s["stats"][0], s["stats"][1])
    if B:
        gate = leaf(s["gate"])
        wrt.append(gate)
        v = (v.view(rows // B, B, -1) * gate).view(rows, -1)
    else:
        v = v * 1.0
    got = list(torch.autograd.grad(v, wrt, D))
    out["df"] = got.pop(0)
    out["dgate"] = got.pop() if B else None
    out["dpost"] = got if s["post"] is not None else None
    return out


def _exact_pack(z, c):
    parts, scales = [], []
    width = z.shape[1] // _halves(c)
    for part in torch.split(z, width, 1):
        for cols in torch.split(part, GROUP, 1):
            top = cols.abs().amax(1)
            e = torch.ceil(torch.log2(torch.clamp(top, min=1e-300) / 448.0)).clamp(min=-126)
            parts.append((cols / torch.exp2(e)[:, None]).to(torch.float32).to(torch.float8_e4m3fn).double())
            scales.append(torch.exp2(e))
    return torch.cat(parts, 1), torch.stack(scales)


def _exact_ckpt_fwd(c, s):
    Zq, Zs, H = [], [], []
    for i in range(c["p"]):
        z = s["X"].double() @ s["W"][i].double().mT
        if s["bias"] is not None:
            z = z + s["bias"][i].double()
        q, e = _exact_pack(z, c)
        Zq.append(q)
        Zs.append(e)
        if c["act"] == "swiglu":
            half = z.shape[1] // 2
            H.append(torch.nn.functional.silu(z[:, :half]) * z[:, half:])
        else:
            H.append(torch.nn.functional.gelu(z))
    return {"Zq": Zq, "Zs": Zs, "H": H}


def _exact_ckpt_bwd(c, s):
    dY, dZ, Hs, dW = s["dY"].double(), [], [], []
    fp = c["f"] // c["p"]
    G = -(-fp // GROUP)
    for i in range(c["p"]):
        halves = []
        for k in range(_halves(c)):
            z = s["Zq"][i].double()[:, k * fp:(k + 1) * fp].clone()
            for j in range(G):
                z[:, j * GROUP:(j + 1) * GROUP] *= torch.exp2(s["Zs"][i][k * G + j].double() - 127)[:, None]
            halves.append(z.requires_grad_())
        H = torch.nn.functional.silu(halves[0]) * halves[1] if c["act"] == "swiglu" else torch.nn.functional.gelu(halves[0])
        dZ.append(torch.cat(torch.autograd.grad(H, halves, dY @ s["W"][i].double()), 1))
        Hs.append(H.detach())
        dW.append(dY.mT @ H.detach().to(torch.bfloat16).double())
    return {"dZ": dZ, "H": Hs, "dW": dW, "dbias": dY.sum(0)}
