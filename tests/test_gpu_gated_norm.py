"""The junction of two sublayers (norms, gate, scaled residual) against fp64.

Bounds. Both sides read the same stored values. Rounding an output to bf16 is off by
at most 2^-8 of it (fp32: 2^-24). Inside, everything is fp32: a sum of n terms is off by
at most n * 2^-24 of the sum of their magnitudes, and each elementwise operation by 2^-24,
so with e = (hidden + 32) * 2^-24 every quantity made from a row's sums is off by at most
e (or 2e where two such sums combine) of the magnitudes that enter it; sums over rows add
(rows + 32) * 2^-24 of theirs. y is compared with the norm of the device's own x_out,
which is what it is defined on."""
import pytest
import torch

from gpu_helpers import dev

pytestmark = pytest.mark.gpu
EPS = 2.0 ** -24


def _tp():
    from megatron_tensor_transformer_gemm_b200 import tp
    return tp


def _inputs(rows, h, dtype, B, post, pre, seed=0, offset=0.0):
    dt = torch.bfloat16 if dtype == "bf16" else torch.float32
    g = torch.Generator().manual_seed(seed)
    rn = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
    d = {"x": (rn(rows, h) + offset).to(dt), "f": (rn(rows, h) * 0.5 + 0.1 + offset).to(dt),
         "gate": (rn(B, h) * 0.5).to(dt) if B else None,
         "post": ((1 + 0.1 * rn(h)).to(dt), (0.1 * rn(h)).to(dt)) if post else None,
         "pre": ((1 + 0.1 * rn(h)).to(dt), (0.1 * rn(h)).to(dt)) if pre else None,
         "dx_out": rn(rows, h).to(dt), "dy": rn(rows, h).to(dt) if pre else None}
    return d, dt


def _d(t):
    return None if t is None else (tuple(dev(u) for u in t) if isinstance(t, tuple) else dev(t))


def _stats(x, kind):
    mean = x.mean(1) if kind == "layer" else torch.zeros(len(x), dtype=x.dtype)
    return mean, 1 / torch.sqrt(((x - mean[:, None]) ** 2).mean(1) + 1e-5)


def _close(got, ref, lim, what):
    got = got.cpu().double()
    bad = ~((got - ref).abs() <= lim)
    assert not bad.any(), (what, int(bad.sum()), float((got - ref).abs().max()), float(((got - ref).abs() / lim).max()))


def _forward_reference(d, kind, rs):
    """x_out, its magnitude bound, and [4, rows] statistics of the post-norm."""
    x, f = d["x"].double(), d["f"].double()
    rows, h = x.shape
    n, mag = f, f.abs()
    stats = torch.zeros(4, rows, dtype=torch.float64)
    if d["post"] is not None:
        mean, rstd = _stats(f, kind)
        stats[0], stats[1] = mean, rstd
        w, b = (t.double() for t in d["post"])
        n = (f - mean[:, None]) * rstd[:, None] * w + (b if kind == "layer" else 0)
        mag = (f.abs() + f.abs().mean(1, keepdim=True)) * rstd[:, None] * w.abs() + b.abs()
    if d["gate"] is not None:
        g = d["gate"].double()[torch.arange(rows) % d["gate"].shape[0]]
        n, mag = n * g, mag * g.abs()
    return rs * x + n, abs(rs) * x.abs() + mag, stats


CASES = [  # rows, h, B, post, pre, kind, rs
    (1, 8, 1, True, True, "layer", 1.0), (1, 4096, 1, True, True, "rms", 1.0), (3, 64, 3, True, True, "layer", 0.5),
    (7, 520, 0, True, True, "layer", 1.0), (130, 1032, 2, True, True, "rms", -1.25), (64, 2048, 8, True, True, "layer", 1.0),
    (33, 4096, 1, True, True, "layer", 1.0), (37, 8192, 1, True, True, "layer", 1.0), (24, 8192, 8, True, True, "rms", 1.0),
    (600, 256, 1, True, False, "layer", 2.0), (600, 264, 300, True, True, "layer", 1.0), (515, 136, 515, True, True, "rms", 1.0),
    (90, 512, 5, False, True, "layer", 1.0), (90, 512, 5, False, False, "rms", 0.0), (41, 768, 0, False, False, "layer", 1.5),
    (3001, 72, 1, True, True, "layer", 1.0), (2600, 128, 4, True, True, "rms", 1.0), (5, 1024, 1, False, True, "rms", 1.0),
]
WIDE = [(21, 16384, 1, True, True, "layer", 1.0), (18, 12344, 3, True, True, "rms", 0.5)]  # bf16 only: a row over two CTAs


def _params():
    out = [(c, dt) for c in CASES for dt in ("bf16", "f32")] + [(c, "bf16") for c in WIDE]
    out.append(((23, 8188 // 8 * 8 - 8, 1, True, True, "layer", 1.0), "f32"))  # fp32 rows over two CTAs, uneven halves
    return out


@pytest.mark.parametrize("case,dtype", _params())
def test_forward(case, dtype):
    rows, h, B, post, pre, kind, rs = case
    tp = _tp()
    d, dt = _inputs(rows, h, dtype, B, post, pre, seed=rows + h)
    plan = tp.Plan(h, 0, 0, 1, dtype, "none")
    x_out = torch.full((rows, h), 7.0, dtype=dt, device="cuda")
    y = torch.full_like(x_out, 7.0) if pre else None
    stats = torch.full((4, rows), 7.0, device="cuda")
    plan.gated_residual_norm_fwd(kind, rows, _d(d["x"]), _d(d["f"]), x_out, y, res_scale=rs, gate=_d(d["gate"]),
                                 post=_d(d["post"]), pre=_d(d["pre"]), stats=stats)
    ref, mag, rstats = _forward_reference(d, kind, rs)
    half, e = (2.0 ** -8 if dtype == "bf16" else EPS), (h + 32) * EPS
    _close(x_out, ref, half * ref.abs() + 2 * e * mag + 1e-30, "x_out")
    got = stats.cpu().double()
    if pre:
        xo = x_out.cpu().double()
        mean, rstd = _stats(xo, kind)
        w, b = (t.double() for t in d["pre"])
        ry = (xo - mean[:, None]) * rstd[:, None] * w + (b if kind == "layer" else 0)
        mg = (xo.abs() + xo.abs().mean(1, keepdim=True)) * rstd[:, None] * w.abs() + b.abs()
        _close(y, ry, half * ry.abs() + 2 * e * mg + 1e-30, "y")
        rstats[2], rstats[3] = mean, rstd
    mags = [d["f"].double().abs().mean(1), x_out.cpu().double().abs().mean(1)]
    for k, there in ((0, post), (1, pre)):
        if not there:
            assert (got[2 * k:2 * k + 2] == 7).all()  # an absent norm's statistics are left alone
            continue
        # the deviation divides by a rstd that the mean's error moves in second order only
        _close(got[2 * k + 1], rstats[2 * k + 1], 2 * e * rstats[2 * k + 1] + 1e-30, "rstd")
        if kind == "layer":
            _close(got[2 * k], rstats[2 * k], e * mags[k] + 1e-30, "mean")
        else:
            assert (got[2 * k] == 7).all()
    assert tp.device_status() == "TP_OK"


def _backward(plan, kind, rows, d, x_out, stats, rs, sums=True, dx=None, df=None):
    h, dt = plan.hidden, plan.torch_dtype
    f32 = lambda *s: torch.full(s, 7.0, device="cuda")  # noqa: E731
    B = d["gate"].shape[0] if d["gate"] is not None else 0
    out = {"dx": torch.full((rows, h), 7.0, dtype=dt, device="cuda") if dx is None else dx,
           "df": torch.full((rows, h), 7.0, dtype=dt, device="cuda") if df is None else df,
           "dgate": f32(B, h) if B and sums else None,
           "dpost": (f32(h), f32(h) if kind == "layer" else None) if d["post"] is not None and sums else None,
           "dpre": (f32(h), f32(h) if kind == "layer" else None) if d["pre"] is not None and sums else None}
    plan.gated_residual_norm_bwd(kind, rows, _d(d["f"]), x_out, stats, _d(d["dx_out"]), _d(d["dy"]), out["dx"], out["df"],
                                 res_scale=rs, gate=_d(d["gate"]), dgate=out["dgate"], post=_d(d["post"]), dpost=out["dpost"],
                                 pre=_d(d["pre"]), dpre=out["dpre"])
    return out


def _saved(d, kind, rs, dt):
    """x_out as stored and the fp32 statistics, from the fp64 forward."""
    x_out, _, stats = _forward_reference(d, kind, rs)
    x_out = x_out.to(dt)
    stats[2], stats[3] = _stats(x_out.double(), kind)
    return x_out, stats.float()


def _check_backward(out, d, x_out, stats, kind, rs, dtype):
    rows, h = x_out.shape
    half, e = (2.0 ** -8 if dtype == "bf16" else EPS), (h + 32) * EPS
    er = e + (rows + 32) * EPS
    s = stats.double()
    zero = torch.zeros(rows, h, dtype=torch.float64)
    D = d["dx_out"].double() if d["dx_out"] is not None else zero
    M = D.abs()
    avg = lambda t: t.mean(1, keepdim=True)  # noqa: E731
    if d["pre"] is not None and d["dy"] is not None:
        dy, w, r = d["dy"].double(), d["pre"][0].double(), s[3][:, None]
        xh = (x_out.double() - s[2][:, None]) * r
        mh = (x_out.double().abs() + s[2].abs()[:, None]) * r
        g = dy * w
        D = D + r * (g - xh * avg(g * xh) - (avg(g) if kind == "layer" else 0))
        M = M + r * (g.abs() + mh * avg(g.abs() * mh) + avg(g.abs()))
        if out["dpre"]:
            _close(out["dpre"][0], (dy * xh).sum(0), er * (dy.abs() * mh).sum(0) + 1e-30, "dgamma_pre")
            if kind == "layer":
                _close(out["dpre"][1], dy.sum(0), er * dy.abs().sum(0) + 1e-30, "dbeta_pre")
    _close(out["dx"], rs * D, half * (rs * D).abs() + 2 * e * abs(rs) * M + 1e-30, "dx")
    f = d["f"].double()
    n, mn, xh, mh = f, f.abs(), f, f.abs()
    if d["post"] is not None:
        w, b, r = d["post"][0].double(), d["post"][1].double(), s[1][:, None]
        xh = (f - s[0][:, None]) * r
        mh = (f.abs() + s[0].abs()[:, None]) * r
        n, mn = xh * w + (b if kind == "layer" else 0), mh * w.abs() + b.abs()
    a, ma = D, M
    if d["gate"] is not None:
        B = d["gate"].shape[0]
        g = d["gate"].double()[torch.arange(rows) % B]
        a, ma = D * g, M * g.abs()
        if out["dgate"] is not None:
            ref = (D * n).reshape(rows // B, B, h).sum(0)
            # g1 A + b1 S: two sums over rows of D, whose own error is 2e of M
            _close(out["dgate"], ref, 3 * er * (M * mn).reshape(rows // B, B, h).sum(0) + 1e-30, "dgate")
    if d["post"] is not None:
        if out["dpost"]:
            _close(out["dpost"][0], (a * xh).sum(0), 3 * er * (ma * mh).sum(0) + 1e-30, "dgamma_post")
            if kind == "layer":
                _close(out["dpost"][1], a.sum(0), 3 * er * ma.sum(0) + 1e-30, "dbeta_post")
        a, ma = a * w, ma * w.abs()
        a = r * (a - xh * avg(a * xh) - (avg(a) if kind == "layer" else 0))
        ma = r * (ma + mh * avg(ma * mh) + avg(ma))
    _close(out["df"], a, half * a.abs() + 4 * e * ma + 1e-30, "df")


@pytest.mark.parametrize("case,dtype", _params())
def test_backward(case, dtype):
    rows, h, B, post, pre, kind, rs = case
    tp = _tp()
    d, dt = _inputs(rows, h, dtype, B, post, pre, seed=rows + h + 1)
    plan = tp.Plan(h, 0, 0, 1, dtype, "none")
    x_out, stats = _saved(d, kind, rs, dt)
    out = _backward(plan, kind, rows, d, dev(x_out), dev(stats), rs)
    _check_backward(out, d, x_out, stats, kind, rs, dtype)
    again = _backward(plan, kind, rows, d, dev(x_out), dev(stats), rs)  # the sums' order is fixed
    for k in out:
        for a, b in zip(out[k] if isinstance(out[k], tuple) else (out[k],), again[k] if isinstance(again[k], tuple) else (again[k],)):
            assert a is b is None or torch.equal(a, b)
    assert tp.device_status() == "TP_OK"


@pytest.mark.parametrize("which", ["no dx_out", "no dy", "no sums"])
def test_backward_with_parts_missing(which):
    tp = _tp()
    d, dt = _inputs(96, 264, "bf16", 2, True, True, seed=4)
    plan = tp.Plan(264, 0, 0, 1, "bf16", "none")
    x_out, stats = _saved(d, "layer", 1.0, dt)
    if which == "no dx_out":
        d["dx_out"] = None
    if which == "no dy":
        d["dy"] = None
    out = _backward(plan, "layer", 96, d, dev(x_out), dev(stats), 1.0, sums=which != "no sums")
    _check_backward(out, d, x_out, stats, "layer", 1.0, "bf16")
    if which == "no dy":
        assert float(out["dpre"][0].abs().max()) == 0 and float(out["dpre"][1].abs().max()) == 0


@pytest.mark.parametrize("B", [1, 3])
def test_each_sum_alone(B):
    """Any one of the sums can be asked for without the others, with the same bits."""
    tp = _tp()
    d, dt = _inputs(96, 264, "bf16", B, True, True, seed=14)
    plan = tp.Plan(264, 0, 0, 1, "bf16", "none")
    x_out, stats = _saved(d, "layer", 1.0, dt)
    xo, st, args = dev(x_out), dev(stats), {k: _d(v) for k, v in d.items()}
    full = _backward(plan, "layer", 96, d, xo, st, 1.0)
    want = {"dgate": full["dgate"], "dpost0": full["dpost"][0], "dpost1": full["dpost"][1], "dpre0": full["dpre"][0],
            "dpre1": full["dpre"][1]}
    for name, ref in want.items():
        got = torch.full_like(ref, 7.0)
        pair = lambda k: ((got, None) if name == k + "0" else (None, got) if name == k + "1" else None)  # noqa: E731
        dx, df = torch.empty_like(xo), torch.empty_like(xo)
        plan.gated_residual_norm_bwd("layer", 96, args["f"], xo, st, args["dx_out"], args["dy"], dx, df, gate=args["gate"],
                                     dgate=got if name == "dgate" else None, post=args["post"], dpost=pair("dpost"),
                                     pre=args["pre"], dpre=pair("dpre"))
        assert torch.equal(got, ref) and torch.equal(dx, full["dx"]) and torch.equal(df, full["df"]), name


def test_in_place_and_zero_rows():
    tp = _tp()
    d, dt = _inputs(50, 1024, "bf16", 1, True, True, seed=5)
    plan = tp.Plan(1024, 0, 0, 1, "bf16", "none")
    kw = dict(gate=_d(d["gate"]), post=_d(d["post"]), pre=_d(d["pre"]))
    x, f = _d(d["x"]), _d(d["f"])
    st = torch.zeros(4, 50, device="cuda")
    xo, y = torch.empty_like(x), torch.empty_like(x)
    plan.gated_residual_norm_fwd("layer", 50, x, f, xo, y, stats=st, **kw)
    x2, y2 = x.clone(), torch.empty_like(x)
    plan.gated_residual_norm_fwd("layer", 50, x2, f, x2, y2, **kw)
    assert torch.equal(x2, xo) and torch.equal(y2, y)
    a = _backward(plan, "layer", 50, d, xo, st, 1.0)
    dxo, dy = _d(d["dx_out"]), _d(d["dy"])
    plan.gated_residual_norm_bwd("layer", 50, f, xo, st, dxo, dy, dxo, dy, gate=kw["gate"], post=kw["post"], pre=kw["pre"])
    assert torch.equal(dxo, a["dx"]) and torch.equal(dy, a["df"])
    none = torch.empty(0, 1024, dtype=dt, device="cuda")
    plan.gated_residual_norm_fwd("layer", 0, none, none, none, none, **kw)
    dg, dp = torch.full((1, 1024), 3.0, device="cuda"), torch.full((1024,), 3.0, device="cuda")
    plan.gated_residual_norm_bwd("layer", 0, none, none, torch.empty(4, 0, device="cuda"), none, none, none, none, dgate=dg,
                                 dpost=(dp, None), **kw)
    assert float(dg.abs().max()) == 0 and float(dp.abs().max()) == 0


def test_offset_rows_and_constant_rows():
    """Rows far from zero keep their deviation; a constant row has deviation 0 and stays finite."""
    tp = _tp()
    d, dt = _inputs(20, 512, "f32", 1, True, True, seed=6, offset=1000.0)
    d["f"][3] = 5.0
    plan = tp.Plan(512, 0, 0, 1, "f32", "none")
    xo, y = torch.empty(20, 512, device="cuda"), torch.empty(20, 512, device="cuda")
    plan.gated_residual_norm_fwd("layer", 20, _d(d["x"]), _d(d["f"]), xo, y, gate=_d(d["gate"]), post=_d(d["post"]), pre=_d(d["pre"]))
    ref, mag, _ = _forward_reference(d, "layer", 1.0)
    _close(xo, ref, EPS * ref.abs() + 2 * (512 + 32) * EPS * mag, "x_out")
    assert torch.isfinite(xo).all() and torch.isfinite(y).all()


def test_nan_and_inf_stay_in_their_rows():
    tp = _tp()
    d, dt = _inputs(9, 512, "bf16", 1, True, True, seed=7)
    plan = tp.Plan(512, 0, 0, 1, "bf16", "none")
    d["f"][2, 5], d["x"][6, 1] = float("nan"), float("inf")
    xo, y = torch.empty(9, 512, dtype=dt, device="cuda"), torch.empty(9, 512, dtype=dt, device="cuda")
    plan.gated_residual_norm_fwd("rms", 9, _d(d["x"]), _d(d["f"]), xo, y, post=_d(d["post"]), pre=_d(d["pre"]))
    ok = [0, 1, 3, 4, 5, 7, 8]
    assert torch.isfinite(xo[ok]).all() and torch.isfinite(y[ok]).all()
    assert torch.isnan(xo[2]).all() and torch.isnan(y[2]).all()


def test_captured_backward_keeps_its_workspace():
    tp = _tp()
    from megatron_tensor_transformer_gemm_b200.block import CapturedStep
    d, dt = _inputs(64, 512, "bf16", 2, True, True, seed=8)
    plan = tp.Plan(512, 0, 0, 1, "bf16", "none")
    x_out, stats = _saved(d, "layer", 1.0, dt)
    xo, st = dev(x_out), dev(stats)
    f32 = lambda *s: torch.empty(s, device="cuda")  # noqa: E731
    out = {"dx": torch.empty_like(xo), "df": torch.empty_like(xo), "dgate": f32(2, 512), "dpost": (f32(512), f32(512)),
           "dpre": (f32(512), f32(512))}
    args = {k: _d(v) for k, v in d.items()}

    def call():
        plan.gated_residual_norm_bwd("layer", 64, args["f"], xo, st, args["dx_out"], args["dy"], out["dx"], out["df"],
                                     gate=args["gate"], dgate=out["dgate"], post=args["post"], dpost=out["dpost"],
                                     pre=args["pre"], dpre=out["dpre"])

    step = CapturedStep(call)
    big, _ = _inputs(8000, 512, "bf16", 2000, True, True, seed=9)
    xb, sb = _saved(big, "layer", 1.0, dt)
    keep = _backward(plan, "layer", 8000, big, dev(xb), dev(sb), 1.0)
    for t in (out["dx"], out["df"], out["dgate"], *out["dpost"], *out["dpre"]):
        t.zero_()
    step()
    _check_backward(out, d, x_out, stats, "layer", 1.0, "bf16")
    _check_backward(keep, big, xb, sb, "layer", 1.0, "bf16")


@pytest.mark.parametrize("kind", ["layer", "rms"])
def test_gradients_by_differences(kind):
    """fp32: a directional difference of the fp64 forward against all gradients at once."""
    tp = _tp()
    rows, h, B = 12, 64, 3
    d, dt = _inputs(rows, h, "f32", B, True, True, seed=10)
    plan = tp.Plan(h, 0, 0, 1, "f32", "none")
    x_out, stats = _saved(d, kind, 0.75, dt)
    out = _backward(plan, kind, rows, d, dev(x_out), dev(stats), 0.75)
    g = torch.Generator().manual_seed(11)
    U = {k: torch.randn(d[k].shape, generator=g).double() for k in ("x", "f", "gate")}
    U["post"], U["pre"] = (tuple(torch.randn(h, generator=g).double() for _ in range(2)) for _ in range(2))

    def total(t):
        m = {k: d[k].double() + t * U[k] for k in ("x", "f", "gate")}
        for k in ("post", "pre"):
            m[k] = tuple(a.double() + t * b for a, b in zip(d[k], U[k]))
        xo, _, _ = _forward_reference(m, kind, 0.75)
        mean, rstd = _stats(xo, kind)
        y = (xo - mean[:, None]) * rstd[:, None] * m["pre"][0] + (m["pre"][1] if kind == "layer" else 0)
        return float((xo * d["dx_out"].double()).sum() + (y * d["dy"].double()).sum())

    e = 1e-4
    diff = (total(e) - total(-e)) / (2 * e)
    c = lambda t, u: float((t.cpu().double() * u).sum())  # noqa: E731
    got = c(out["dx"], U["x"]) + c(out["df"], U["f"]) + c(out["dgate"], U["gate"])
    for k, o in (("post", out["dpost"]), ("pre", out["dpre"])):
        got += c(o[0], U[k][0]) + (c(o[1], U[k][1]) if kind == "layer" else 0)
    # the central difference is off by e^2 of the third derivative, the sums by about 1e-6
    assert abs(got - diff) <= 1e-4 * max(1.0, abs(diff)) + 1e-3


def test_no_wider_than_the_norms_take():
    tp = _tp()
    plan = tp.Plan(16392, 0, 0, 1, "bf16", "none")
    x = torch.zeros(1, 16392, dtype=torch.bfloat16, device="cuda")
    with pytest.raises(tp.TPError, match="hidden <= 16384"):
        plan.gated_residual_norm_fwd("rms", 1, x, x, x)


