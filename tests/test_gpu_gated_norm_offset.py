"""LayerNorm's backward in the gated junction on rows far from zero, against fp64.

Bounds. The normalised row is xh = (x - mean) * rstd of the stored statistics: the difference
and the product are rounded once each, 2^-24 relative to xh itself, whatever the mean is. A
row's sums are trees: a thread adds at most 16 terms, a warp 5 times, 32 warps' sums 17 times,
so no term passes more than 40 additions, and with the elementwise operations e = 64 * 2^-24
of the magnitudes that enter bounds a row's sum and what is made of it (2e where two
combine). Sums over rows add 2^-24 a row. No magnitude below counts the mean."""
import pytest
import torch

from gpu_helpers import dev
from test_gpu_gated_norm import EPS, _backward, _close, _inputs, _saved, _tp

pytestmark = pytest.mark.gpu


def _check(out, d, x_out, stats, rs, dtype):
    rows, h = x_out.shape
    half, e = (2.0 ** -8 if dtype == "bf16" else EPS), 64 * EPS
    er = e + rows * EPS
    s = stats.double()
    avg = lambda t: t.mean(1, keepdim=True)  # noqa: E731
    D = d["dx_out"].double() if d["dx_out"] is not None else torch.zeros(rows, h, dtype=torch.float64)
    M = D.abs()
    if d["pre"] is not None:
        dy, w, r = d["dy"].double(), d["pre"][0].double(), s[3][:, None]
        xh = (x_out.double() - s[2][:, None]) * r
        g = dy * w
        D = D + r * (g - xh * avg(g * xh) - avg(g))
        M = M + r * (g.abs() + xh.abs() * avg((g * xh).abs()) + avg(g.abs()))
        _close(out["dpre"][0], (dy * xh).sum(0), er * (dy * xh).abs().sum(0) + 1e-30, "dgamma_pre")
        _close(out["dpre"][1], dy.sum(0), er * dy.abs().sum(0) + 1e-30, "dbeta_pre")
    _close(out["dx"], rs * D, half * (rs * D).abs() + 2 * e * abs(rs) * M + 1e-30, "dx")
    w, b, r = d["post"][0].double(), d["post"][1].double(), s[1][:, None]
    xh = (d["f"].double() - s[0][:, None]) * r
    a, ma = D, M
    if d["gate"] is not None:
        B = d["gate"].shape[0]
        g = d["gate"].double()[torch.arange(rows) % B]
        a, ma = D * g, M * g.abs()
        ref = (D * (xh * w + b)).reshape(rows // B, B, h).sum(0)
        _close(out["dgate"], ref, 3 * er * (M * ((xh * w).abs() + b.abs())).reshape(rows // B, B, h).sum(0) + 1e-30, "dgate")
    _close(out["dpost"][0], (a * xh).sum(0), 3 * er * (ma * xh.abs()).sum(0) + 1e-30, "dgamma_post")
    _close(out["dpost"][1], a.sum(0), 3 * er * ma.sum(0) + 1e-30, "dbeta_post")
    a, ma = a * w, ma * w.abs()
    ref = r * (a - xh * avg(a * xh) - avg(a))
    ma = r * (ma + xh.abs() * avg(ma * xh.abs()) + avg(ma))
    _close(out["df"], ref, half * ref.abs() + 4 * e * ma + 1e-30, "df")


CASES = [  # rows, h, gate rows, pre, dx_out
    (1, 64, 1, True, True), (1, 512, 1, True, True), (2, 520, 0, True, True), (3, 1032, 3, True, True), (1, 2048, 1, True, True),
    (2, 4096, 1, True, True), (3, 8184, 1, True, True), (2, 512, 2, False, True), (2, 512, 1, True, False), (600, 264, 300, True, True),
    (1500, 128, 3, True, True),
]


@pytest.mark.parametrize("offset", [100.0, 1000.0])
@pytest.mark.parametrize("case,dtype", [(c, dt) for c in CASES for dt in ("f32", "bf16")] + [((2, 16384, 1, True, True), "bf16")])
def test_layernorm_backward_far_from_zero(case, dtype, offset):
    rows, h, B, pre, has_dx = case
    if dtype == "bf16":
        offset /= 10  # bf16's step at 1000 is 4: rows a hundred deviations away are constant there
    tp = _tp()
    d, dt = _inputs(rows, h, dtype, B, True, pre, seed=rows + h, offset=offset)
    plan = tp.Plan(h, 0, 0, 1, dtype, "none")
    x_out, stats = _saved(d, "layer", 1.0, dt)
    # gradients that lean along the normalised rows: both row sums count
    s = stats.double()
    if pre:
        d["dy"] = (d["dy"].double() + 2 * (x_out.double() - s[2][:, None]) * s[3][:, None]).to(dt)
    d["dx_out"] = (d["dx_out"].double() + 2 * (d["f"].double() - s[0][:, None]) * s[1][:, None]).to(dt) if has_dx else None
    out = _backward(plan, "layer", rows, d, dev(x_out), dev(stats), 1.0)
    _check(out, d, x_out, stats, 1.0, dtype)
    assert tp.device_status() == "TP_OK"
