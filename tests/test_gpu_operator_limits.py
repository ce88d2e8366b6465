"""Calls at the edges of what the fused training operators' descriptions allow: the most shards,
chunks of one token, gradients written over their inputs, a plan used on one stream after
another."""
import pytest
import torch

from gpu_helpers import dev
from test_gpu_ckpt8 import _backward as _ckpt_backward
from test_gpu_ckpt8 import _check_backward as _check_ckpt
from test_gpu_gated_norm import _backward, _d, _inputs, _saved
from test_gpu_loss import _check, _head, _run, _tp

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("T,V,chunk", [(3, 3000, 0), (40, 2000, 0), (300, 5000, 0), (300, 5000, 64), (200, 120, 0)])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_head_over_sixteen_shards(T, V, chunk, dtype):
    plan, Vp, X, W, labels = _head(T, 128, V, 16, dtype, seed=T + V)
    _check(X, W, labels, V, 0.5, _run(plan, Vp, X, W, labels, 0.5, chunk), dtype)
    assert _tp().device_status() == "TP_OK"


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_head_one_token_at_a_time_and_chunks_past_the_batch(dtype):
    plan, Vp, X, W, labels = _head(9, 128, 1003, 2, dtype, seed=31)
    for chunk in (1, 8, 9, 1000):
        _check(X, W, labels, 1003, 0.5, _run(plan, Vp, X, W, labels, 0.5, chunk), dtype)


@pytest.mark.parametrize("act", ["swiglu", "gelu"])
def test_ckpt8_over_sixteen_shards(act):
    _check_ckpt(*_ckpt_backward(200, 256, 768, 16, act, 7), act)
    assert _tp().device_status() == "TP_OK"


@pytest.mark.parametrize("h,dtype", [(264, "bf16"), (1032, "f32"), (12344, "bf16")])
def test_junction_gradients_over_their_inputs(h, dtype):
    """dx over dx_out with df over f, then with df over dy: the bits of separate outputs."""
    rows = 700
    d, dt = _inputs(rows, h, dtype, 4, True, True, seed=h)
    plan = _tp().Plan(h, 0, 0, 1, dtype, "none")
    x_out, stats = _saved(d, "layer", 0.75, dt)
    xo, st = dev(x_out), dev(stats)
    want = _backward(plan, "layer", rows, d, xo, st, 0.75)
    for over in ("f", "dy"):
        a = {k: _d(v) for k, v in d.items()}
        plan.gated_residual_norm_bwd("layer", rows, a["f"], xo, st, a["dx_out"], a["dy"], a["dx_out"], a[over], res_scale=0.75,
                                     gate=a["gate"], post=a["post"], pre=a["pre"])
        assert torch.equal(a["dx_out"], want["dx"]) and torch.equal(a[over], want["df"]), over


def test_one_plan_on_one_stream_after_another():
    """Calls of a plan in turn on three streams, each waiting for the one before, while the workspace
    grows: every call's outputs are its own."""
    plan, Vp, X, W, labels = _head(600, 128, 3001, 2, "bf16", seed=33)
    Ws, streams, outs = [dev(w) for w in W.chunk(2)], [torch.cuda.Stream() for _ in range(3)], []
    torch.cuda.synchronize()
    for k, T in enumerate((30, 200, 600, 70, 600, 1)):
        s = streams[k % 3]
        s.wait_stream(streams[(k - 1) % 3])
        with torch.cuda.stream(s):
            Xd, ld = dev(X[:T]), labels[:T].cuda()
            o = torch.empty(T, device="cuda"), torch.empty(T, device="cuda"), torch.empty_like(Xd), [torch.empty_like(w) for w in Ws]
            plan.vocab_linear_cross_entropy(T, Xd, Ws, ld, 0.5, *o)
            outs.append((T, o, Xd, ld))
    torch.cuda.synchronize()
    for T, o, _, _ in outs:
        _check(X[:T], W, labels[:T], 3001, 0.5, o, "bf16")
