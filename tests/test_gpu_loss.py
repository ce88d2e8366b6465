"""Output head fused with its cross-entropy, without logits, against fp64.

Bounds. Inputs are the same values on both sides. fp32 results (loss, lse): scores
are fp32 sums of h products whose factors are exact, so each is off by at most
h * 2^-24 * sum|x w| <= h * 2^-24 * |x| |w|; the log-sum-exp moves by no more than the
largest score error plus a few 2^-22 of the exponentials, the loss by twice that.
Gradients in bf16: d is rounded once (2^-9 relative to each term, half a step being
2^-9 of the value's binade, 2^-8 of the value at worst), and the result once (2^-8):
|error| <= 2^-8 * sum_k |d_k||b_k| + 2^-8 |result| + the fp32 sum's K * 2^-24 share.
fp32 plans: the products' sums only.
The scores' error: p = 2^(z log2 e - lse2) is off by e = z_err + exp_err relative to p
itself, so d = (p - [v = label]) * scale is off by e * p * scale in absolute terms. Where
p is near 1 at the label that is no small part of d = p - 1, so the term is counted
on p (the softmax), not on |d|: |error| gains e * scale * sum_k p_k |b_k|.
bf16 plans hold the exponentials in 16 bits with 9 of significand before they become d, a
second rounding of 2^-10 on p (the label's is computed apart, in fp32): |error| gains 2^-10 *
scale * sum_k p_k |b_k|, times 1 + 2^-8 where the two roundings meet."""
import numpy as np
import pytest
import torch

from gpu_helpers import dev, host

pytestmark = pytest.mark.gpu


def _tp():
    from megatron_tensor_transformer_gemm_b200 import tp
    return tp


def _head(T, h, V, p, dtype, seed=0, std=0.05, ignored=True):
    tp = _tp()
    dt = torch.bfloat16 if dtype == "bf16" else torch.float32
    plan = tp.Plan(h, 0, 0, p, dtype, "none")
    Vp = plan.set_vocab(V)
    g = torch.Generator().manual_seed(seed)
    X = torch.randn(T, h, generator=g).to(dt)
    W = (torch.randn(Vp, h, generator=g) * std).to(dt)
    labels = torch.randint(0, V, (T,), generator=g, dtype=torch.int32)
    if T > 2:
        labels[0], labels[1] = V - 1, 0
    if ignored and T > 4:
        labels[3::7] = -1
        labels[4] = -100
    return plan, Vp, X, W, labels


def _reference(X, W, labels, V, scale):
    X, W = X.double(), W.double()
    z = X @ W[:V].T
    lse = torch.logsumexp(z, 1)
    keep = labels >= 0
    lab = labels.long().clamp(min=0)
    loss = torch.where(keep, lse - z.gather(1, lab[:, None])[:, 0], torch.zeros_like(lse))
    d = torch.exp(z - lse[:, None])
    pr = d * torch.where(keep, abs(scale), 0.0)[:, None]
    d[torch.arange(len(lab)), lab] -= 1
    d *= torch.where(keep, scale, 0.0)[:, None]
    dW = torch.zeros_like(W)
    dW[:V] = d.T @ X
    bx, px = d.abs() @ W[:V].abs(), pr @ W[:V].abs()
    bw, pw = torch.zeros_like(W), torch.zeros_like(W)
    bw[:V], pw[:V] = d.abs().T @ X.abs(), pr.T @ X.abs()
    return loss, lse, d @ W[:V], dW, bx, bw, px, pw


def _run(plan, Vp, X, W, labels, scale, chunk=0, grad=(True, True), lse=True):
    p, T = plan.p, X.shape[0]
    Xd, Ws, ld = dev(X), [dev(w) for w in W.chunk(p)], labels.cuda()
    loss = torch.full((T,), 7.0, device="cuda")
    ls = torch.full((T,), 7.0, device="cuda") if lse else None
    dX = torch.full_like(Xd, 7.0) if grad[0] else None
    dW = [torch.full_like(w, 7.0) for w in Ws] if grad[1] else None
    plan.vocab_linear_cross_entropy(T, Xd, Ws, ld, scale, loss, ls, dX, dW, chunk)
    return loss, ls, dX, dW


def _check(X, W, labels, V, scale, out, dtype):
    loss, lse, dX, dW = out
    rl, rs, rx, rw, bx, bw, px, pw = _reference(X, W, labels, V, scale)
    h = X.shape[1]
    eps = 2.0 ** -24
    z_err = h * eps * (X.double().norm(dim=1) * W[:V].double().norm(dim=1).max())
    exp_err = 2.0 ** -21 + 4 * eps * (rs.abs() + 8)
    tol = (2 * z_err + 2 * exp_err).numpy()
    assert np.all(np.abs(host(loss) - rl.numpy()) <= tol)
    assert np.all(host(loss)[labels.numpy() < 0] == 0)
    if lse is not None:
        assert np.all(np.abs(host(lse) - rs.numpy()) <= tol)
    rel = float((z_err + exp_err).max())
    half = 2.0 ** -8 if dtype == "bf16" else eps
    rel += 2.0 ** -10 * (1 + half) if dtype == "bf16" else 0.0
    if dX is not None:
        lim = (half + V * eps) * bx + rel * px + half * rx.abs() + 1e-30
        assert np.all(np.abs(host(dX) - rx.numpy()) <= lim.numpy())
    if dW is not None:
        got = np.concatenate([host(w) for w in dW])
        lim = (half + len(X) * eps) * bw + rel * pw + half * rw.abs() + 1e-30
        assert np.all(np.abs(got - rw.numpy()) <= lim.numpy())
        assert np.all(got[V:] == 0)


SHAPES = [  # T, h, V, p, chunk
    (5, 8, 3, 1, 0), (130, 16, 9, 2, 7), (1, 64, 50, 1, 0), (2, 128, 1003, 2, 0), (17, 512, 1003, 2, 0), (129, 72, 3001, 1, 0),
    (300, 256, 777, 4, 0), (640, 512, 4096, 8, 0), (257, 1024, 20011, 4, 0), (513, 128, 260, 2, 0),
    (2500, 64, 131, 1, 0), (300, 256, 777, 4, 100), (1030, 128, 5003, 2, 256), (515, 136, 2048, 1, 513),
]


@pytest.mark.parametrize("T,h,V,p,chunk", SHAPES)
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_loss_and_gradients(T, h, V, p, chunk, dtype):
    plan, Vp, X, W, labels = _head(T, h, V, p, dtype, seed=T + V)
    scale = 1.0 / T
    out = _run(plan, Vp, X, W, labels, scale, chunk)
    _check(X, W, labels, V, scale, out, dtype)
    assert _tp().device_status() == "TP_OK"


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("grad,lse", [((False, False), True), ((False, False), False), ((True, False), True), ((False, True), False)])
def test_parts_of_the_outputs(dtype, grad, lse):
    plan, Vp, X, W, labels = _head(200, 256, 5000, 2, dtype, seed=3)
    out = _run(plan, Vp, X, W, labels, -0.25, 96, grad, lse)
    _check(X, W, labels, 5000, -0.25, out, dtype)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_large_scores_and_sure_tokens(dtype):
    """Scores of several hundred and tokens whose probability is 1 to fp32."""
    plan, Vp, X, W, labels = _head(64, 128, 1003, 2, dtype, seed=9, std=3.0, ignored=False)
    X = X * 4
    labels = (X.double() @ W[:1003].double().T).argmax(1).int()
    out = _run(plan, Vp, X, W, labels, 1.0)
    _check(X, W, labels, 1003, 1.0, out, dtype)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_every_token_ignored_and_no_token(dtype):
    plan, Vp, X, W, labels = _head(130, 128, 1003, 2, dtype, seed=5)
    labels[:] = -1
    loss, lse, dX, dW = _run(plan, Vp, X, W, labels, 1.0)
    assert float(loss.abs().max()) == 0 and float(dX.abs().max()) == 0
    assert all(float(w.abs().max()) == 0 for w in dW)
    assert torch.isfinite(lse).all()
    _, _, _, dW = _run(plan, Vp, X[:0], W, labels[:0], 1.0)
    assert all(float(w.abs().max()) == 0 for w in dW)


def test_label_past_the_vocab_is_ignored_and_reported():
    tp = _tp()
    plan, Vp, X, W, labels = _head(40, 128, 1003, 2, "bf16", seed=6, ignored=False)
    tp.device_status()
    labels[7] = 1003  # a padding row of the head
    loss, _, dX, _ = _run(plan, Vp, X, W, labels, 1.0)
    assert float(loss[7]) == 0 and float(dX[7].abs().max()) == 0
    assert tp.device_status() == "TP_ERR_ARG"
    assert tp.device_status() == "TP_OK"


def test_nan_stays_in_its_row():
    plan, Vp, X, W, labels = _head(40, 128, 1003, 2, "bf16", seed=7, ignored=False)
    X[5, 3] = float("nan")
    loss, lse, dX, _ = _run(plan, Vp, X, W, labels, 1.0, grad=(True, False))
    ok = torch.ones(40, dtype=torch.bool, device="cuda")
    ok[5] = False
    assert torch.isnan(loss[5]) and torch.isnan(lse[5]) and torch.isnan(dX[5]).all()
    assert torch.isfinite(loss[ok]).all() and torch.isfinite(dX[ok]).all()


def test_same_bits_twice_and_rows_alone_agree():
    """Two calls give the same bits; the loss of a row does not depend on the others."""
    plan, Vp, X, W, labels = _head(700, 256, 5003, 4, "bf16", seed=8)
    a = _run(plan, Vp, X, W, labels, 1.0, 256)
    b = _run(plan, Vp, X, W, labels, 1.0, 256)
    for x, y in zip([a[0], a[1], a[2], *a[3]], [b[0], b[1], b[2], *b[3]]):
        assert torch.equal(x, y)


def test_captured_and_replayed_beside_a_larger_eager_call():
    """A captured call keeps its workspace when a later call needs a larger one."""
    tp = _tp()
    plan, Vp, X, W, labels = _head(96, 128, 1003, 2, "bf16", seed=10)
    Xd, Ws, ld = dev(X), [dev(w) for w in W.chunk(2)], labels.cuda()
    loss = torch.empty(96, device="cuda")
    dX, dW = torch.empty_like(Xd), [torch.empty_like(w) for w in Ws]

    def call():
        plan.vocab_linear_cross_entropy(96, Xd, Ws, ld, 0.5, loss, None, dX, dW)

    from megatron_tensor_transformer_gemm_b200.block import CapturedStep
    step = CapturedStep(call)
    big = torch.randn(3000, 128, device="cuda").bfloat16()
    bl = torch.empty(3000, device="cuda")
    plan.vocab_linear_cross_entropy(3000, big, Ws, torch.zeros(3000, dtype=torch.int32, device="cuda"), 1.0, bl, None,
                                    torch.empty_like(big), [torch.empty_like(w) for w in Ws])
    for seed in (11, 12):
        X2 = torch.randn(96, 128, generator=torch.Generator().manual_seed(seed)).bfloat16()
        Xd.copy_(X2)
        loss.zero_()
        step()
        _check(X2, W, labels, 1003, 0.5, (loss, None, dX, dW), "bf16")
    # a call that would have to grow the workspace is refused inside a capture
    fresh = tp.Plan(128, 0, 0, 2, "bf16", "none")
    fresh.set_vocab(1003)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        with pytest.raises(tp.TPError, match="before the stream capture"):
            fresh.vocab_linear_cross_entropy(96, Xd, Ws, ld, 0.5, loss, None, dX, dW)
    torch.cuda.synchronize()
    assert tp.device_status() == "TP_OK"


def test_on_another_stream():
    plan, Vp, X, W, labels = _head(96, 128, 1003, 2, "bf16", seed=13)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        out = _run(plan, Vp, X, W, labels, 0.5)
    torch.cuda.current_stream().wait_stream(s)
    _check(X, W, labels, 1003, 0.5, out, "bf16")


def test_gradient_by_differences():
    """fp32: directional differences of the summed loss against dX and dW."""
    plan, Vp, X, W, labels = _head(12, 64, 203, 2, "f32", seed=14)
    _, _, dX, dW = _run(plan, Vp, X, W, labels, 1.0)
    g = torch.Generator().manual_seed(15)
    U = torch.randn(X.shape, generator=g).double()
    S = torch.zeros(W.shape).double()
    S[:203] = torch.randn(203, 64, generator=g).double()

    def total(e):
        z = (X.double() + e * U) @ (W.double() + e * S)[:203].T
        keep = labels >= 0
        ce = torch.logsumexp(z, 1) - z.gather(1, labels.long().clamp(min=0)[:, None])[:, 0]
        return float(ce[keep].sum())

    e = 1e-4  # the central difference is off by e^2 * third derivative, about 1e-6 of it here
    diff = (total(e) - total(-e)) / (2 * e)
    got = float((torch.from_numpy(host(dX)) * U).sum() + (torch.from_numpy(np.concatenate([host(w) for w in dW])) * S).sum())
    assert abs(got - diff) <= 1e-4 * abs(diff) + 1e-4


@pytest.mark.parametrize("T,chunk", [(40, 0), (515, 0), (515, 200)])
def test_the_scale_is_not_rounded_with_d(T, chunk):
    """A scale halfway between two bf16 values. Rounded with d, every label's entry (near
    -scale where the softmax is small) would be off by nearly the same 2^-8 / (1 + 2^-8) =
    0.0039, and so would dX. With d rounded before the scale, that entry, softmax - 1, is off
    by at most its softmax, 2^-11 in the mean here. What stays is the result's rounding,
    uniform within half a step of at most 2^-8 of the value, so at most 2^-8 / sqrt(3) =
    0.00226 in the mean square, and the other entries' roundings: 2^-8 of terms whose sum
    is below a hundredth of the label's row."""
    V, scale = 4000, (1 + 2.0 ** -8) / 512
    plan, Vp, X, W, labels = _head(T, 256, V, 2, "bf16", seed=T, ignored=False)
    out = _run(plan, Vp, X, W, labels, scale, chunk)
    _check(X, W, labels, V, scale, out, "bf16")
    z = X.double() @ W[:V].double().T
    assert float(torch.softmax(z, 1).gather(1, labels.long()[:, None]).mean()) < 2.0 ** -11
    rx = _reference(X, W, labels, V, scale)[2]
    err = float((torch.from_numpy(host(out[2])) - rx).norm() / rx.norm())
    assert err < 2.0 ** -8 / 3 ** 0.5 + 2.0 ** -11 + 2.0 ** -8 / 100


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("chunk", [0, 100])
def test_streams_and_replays_agree(dtype, chunk, monkeypatch):
    """With and without the side stream, on another stream and replayed: the same bits, ready on
    the caller's stream."""
    plan, Vp, X, W, labels = _head(257, 128, 2003, 2, dtype, seed=21)
    Xd, Ws, ld = dev(X), [dev(w) for w in W.chunk(2)], labels.cuda()

    def new():
        return torch.zeros(257, device="cuda"), torch.zeros_like(Xd), [torch.zeros_like(w) for w in Ws]

    def call(o):
        plan.vocab_linear_cross_entropy(257, Xd, Ws, ld, 0.37, o[0], None, o[1], o[2], chunk)
        return [o[0].clone(), o[1].clone(), *[w.clone() for w in o[2]]]

    want = call(new())
    _check(X, W, labels, 2003, 0.37, (want[0], None, want[1], want[2:]), dtype)
    monkeypatch.setenv("TP_BWD_CONCURRENT", "0")
    assert all(torch.equal(a, b) for a, b in zip(call(new()), want))
    monkeypatch.delenv("TP_BWD_CONCURRENT")
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(st):
        got = call(new())
    st.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    o = new()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = call(o)
    for _ in range(2):
        for t in (o[0], o[1], *o[2]):
            t.fill_(7)
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))
    assert _tp().device_status() == "TP_OK"


@pytest.mark.parametrize("T,V,p,chunk", [(1, 1003, 2, 0), (2, 40000, 8, 0), (17, 3001, 1, 0), (33, 259, 2, 0), (64, 5003, 4, 0),
                                         (200, 1003, 2, 50), (65, 1003, 1, 64), (64, 131, 1, 63)])
def test_few_tokens_carry_d_twice(T, V, p, chunk):
    """Chunks of at most 64 tokens: d is held in two bf16 parts, off by 2^-8 of 2^-8 of it, so
    what is left is the exponentials' 2^-10 of the softmax (the label's own entry is exact),
    the fp32 sums and the result's rounding."""
    plan, Vp, X, W, labels = _head(T, 128, V, p, "bf16", seed=T + p, std=0.3)
    scale = 1.37 / T
    loss, lse, dX, dW = _run(plan, Vp, X, W, labels, scale, chunk)
    _check(X, W, labels, V, scale, (loss, lse, dX, dW), "bf16")
    rl, rs, rx, rw, bx, bw, px, pw = _reference(X, W, labels, V, scale)
    eps = 2.0 ** -24
    z_err = 128 * eps * float((X.double().norm(dim=1) * W[:V].double().norm(dim=1).max()).max())
    rel = z_err + 2.0 ** -21 + 4 * eps * float(rs.abs().max() + 8) + 2.0 ** -10
    lab = labels.long().clamp(min=0)
    keep = (labels >= 0).double()
    pl = torch.exp((X.double() * W.double()[lab]).sum(1) - rs) * scale * keep  # the label's softmax: exact but for z
    for got, ref, b, pr in ((host(dX), rx, bx, px), (np.concatenate([host(w) for w in dW]), rw, bw, pw)):
        lim = (2.0 ** -16 + (V + T) * eps) * b + rel * pr + 2.0 ** -8 * ref.abs() + 1e-30
        assert np.all(np.abs(got - ref.numpy()) <= lim.numpy())
    # the label's row of a token that shares it with none has no 2^-10 either: beyond the
    # result's rounding only the other tokens' softmax in it
    one = [t for t in range(T) if keep[t] > 0 and int((lab == lab[t]).sum()) == 1]
    got = torch.from_numpy(np.concatenate([host(w) for w in dW]))
    for t in one:
        v = int(lab[t])
        others = pw[v] - pl[t] * X[t].double().abs()
        lim = (2.0 ** -16 + T * eps) * bw[v] + (rel - 2.0 ** -10) * pw[v] + 2.0 ** -10 * others.clamp(min=0) + 2.0 ** -8 * rw[v].abs() + 1e-30
        assert bool(((got[v] - rw[v]).abs() <= lim * (1 + 1e-6)).all())
    assert _tp().device_status() == "TP_OK"
