"""8-bit activation checkpoints of the MLP against fp64.

Bounds. Z is an fp32 sum of h products: off by at most e = h * 2^-24 * |x| |w| (row norms),
plus 2^-24 for the bias. A code is the nearest e4m3 value of Z / scale: off by at most 2^-4 of
Z, or half the smallest step, 2^-10 of the scale. The scale is the least power of two s with
448 s >= the group's largest magnitude, which is known to within e. The activations come from
fast exponentials and an erf of absolute error 1.5e-7: their factors (sigmoid, Phi, the
derivatives) are off by at most 2^-20 * (1 + |z|) in all. Rounding to bf16 adds 2^-8 of a value."""
import numpy as np
import pytest
import torch

from gpu_helpers import dev, host

pytestmark = pytest.mark.gpu
EPS = 2.0 ** -24
HALF = 2.0 ** -8


def _tp():
    from megatron_tensor_transformer_gemm_b200 import tp
    return tp


def _halves(act):
    return 2 if act == "swiglu" else 1


def _padded_groups(z, act):
    """[T, groups, 32] of z [T, n1], zeros past the end of each half."""
    T, n1 = z.shape
    k = n1 // _halves(act)
    G = -(-k // 32)
    out = torch.zeros(T, _halves(act), G * 32, dtype=z.dtype)
    out[:, :, :k] = z.reshape(T, _halves(act), k)
    return out.reshape(T, _halves(act) * G, 32)


def _from_groups(a, n1, act):
    T = a.shape[0]
    k = n1 // _halves(act)
    return a.reshape(T, _halves(act), -1)[:, :, :k].reshape(T, n1)


def _encode(z, act):
    """Codes [T, n1] and biased exponents [groups, T] of fp32 or fp64 z, from the definition."""
    a = _padded_groups(z.double(), act)
    top = a.abs().amax(2)
    e = torch.ceil(torch.log2(top.clamp(min=1e-300) / 448))
    e = torch.where(torch.ldexp(torch.full_like(e, 448.0), e.int() - 1) >= top, e - 1, e)  # log2's own rounding
    e = e.clamp(min=-126).int()
    q = torch.ldexp(a, -e[:, :, None]).float().to(torch.float8_e4m3fn)
    return _from_groups(q.float(), z.shape[1], act).to(torch.float8_e4m3fn), (e + 127).to(torch.uint8).T.contiguous()


def _scales(s, n1, act):
    e = s.cpu().T.int() - 127
    sc = torch.ldexp(torch.ones_like(e, dtype=torch.float64), e)
    return _from_groups(sc[:, :, None].expand(*sc.shape, 32), n1, act)


def _decode(q, s, act):
    return q.cpu().double() * _scales(s, q.shape[1], act)


def _act(z, act):
    if act == "swiglu":
        g, u = z.chunk(2, 1)
        sg = torch.sigmoid(g)
        return g * sg * u, torch.cat([u * sg * (1 + g * (1 - sg)), g * sg], 1)
    phi = 0.5 * (1 + torch.erf(z / 2 ** 0.5))
    return z * phi, phi + z * torch.exp(-z * z / 2) / (2 * np.pi) ** 0.5


def _act_error(z, act):
    """Bounds on the error of H and of dZ's factors from the functions alone."""
    if act == "swiglu":
        g, u = z.abs().chunk(2, 1)
        t = 2.0 ** -20 * (1 + g)
        return t * g * u, torch.cat([t * u * (1 + g), t * g], 1)
    t = 2.0 ** -20 * (1 + z.abs())
    return t * z.abs(), t


SHAPES = [  # T, h, f, p
    (5, 8, 16, 1), (1, 64, 16, 1), (3, 128, 96, 2), (17, 512, 272, 1), (130, 256, 2048, 4), (300, 512, 1376, 2), (257, 72, 4096, 8), (641, 1024, 528, 1),
]


def _empty_ckpt(plan, T):
    codes, scales = plan.ckpt8_shapes(T)
    return ([torch.full(codes, 3, dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn) for _ in range(plan.p)],
            [torch.full(scales, 3, dtype=torch.uint8, device="cuda") for _ in range(plan.p)])


def _forward(T, h, f, p, act, seed, bias=True):
    tp = _tp()
    plan = tp.Plan(h, f, 0, p, "bf16", act)
    n1 = _halves(act) * f // p
    g = torch.Generator().manual_seed(seed)
    X = torch.randn(T, h, generator=g).bfloat16()
    W = [(torch.randn(n1, h, generator=g) * (2.0 / h ** 0.5)).bfloat16() for _ in range(p)]
    b = [(torch.randn(n1, generator=g) * 0.3).bfloat16() for _ in range(p)] if act == "gelu" and bias else None
    Zq, Zs = _empty_ckpt(plan, T)
    H = [torch.full((T, f // p), 7.0, dtype=torch.bfloat16, device="cuda") for _ in range(p)]
    plan.column_fwd_ckpt8(T, dev(X), [dev(w) for w in W], [dev(x) for x in b] if b else None, Zq, Zs, H)
    return X, W, b, Zq, Zs, H


@pytest.mark.parametrize("act", ["swiglu", "gelu"])
@pytest.mark.parametrize("T,h,f,p", SHAPES)
def test_forward(T, h, f, p, act):
    X, W, b, Zq, Zs, H = _forward(T, h, f, p, act, T + f, bias=T % 2 == 1)
    for i in range(p):
        z = X.double() @ W[i].double().T + (b[i].double() if b else 0)
        n1 = z.shape[1]
        e = h * EPS * X.double().norm(dim=1, keepdim=True) * W[i].double().norm(dim=1)[None] + 2 * EPS * z.abs() + 1e-30
        sc = _scales(Zs[i], n1, act)
        top = _from_groups(_padded_groups(z.abs(), act).amax(2, keepdim=True).expand(-1, -1, 32), n1, act)
        et = _from_groups(_padded_groups(e, act).amax(2, keepdim=True).expand(-1, -1, 32), n1, act)
        assert (448 * sc >= top - et).all() and (224 * sc < top + et).all(), "scale"
        off = (_decode(Zq[i], Zs[i], act) - z).abs()
        assert (off <= torch.maximum(2.0 ** -4 * z.abs(), 2.0 ** -10 * sc) + 1.1 * e).all(), "codes"
        ref, fac = _act(z, act)
        eh, _ = _act_error(z, act)
        if act == "swiglu":  # dH = d(silu)/dg u eg + silu eu
            moved = fac.abs() * e
            moved = moved[:, :n1 // 2] + moved[:, n1 // 2:]
        else:
            moved = fac.abs() * e
        got = H[i].cpu().double()
        assert ((got - ref).abs() <= HALF * ref.abs() + eh + 2 * moved + 1e-30).all(), "H"
    assert _tp().device_status() == "TP_OK"


@pytest.mark.parametrize("act", ["swiglu", "gelu"])
def test_codes_and_scales_bit_for_bit(act):
    """Small integers and powers of two make every Z exact in fp32, so codes and scales are
    those of the definition: all-zero groups, group maxima at and just over 1.75 * 2^k
    (where the scale steps), tiny and huge magnitudes, a ragged last group."""
    tp = _tp()
    T, h, f = 64, 64, 144
    plan = tp.Plan(h, f, 0, 1, "bf16", act)
    n1 = _halves(act) * f
    g = torch.Generator().manual_seed(1)
    X = torch.zeros(T, h)
    X[:, 0] = torch.ldexp(torch.ones(T), torch.arange(T) * 2 - 64)       # row scales 2^-64 .. 2^62
    W = torch.zeros(n1, h)
    W[:, 0] = torch.randint(-255, 256, (n1,), generator=g).float()       # exact in bf16
    W[5::32, 0] = 224.0                                                  # 1.75 * 2^7: the scale's border
    W[37, 0], W[70, 0] = 225.0, 255.0                                    # just over it
    W[96:128, 0] = 0.0                                                   # a group of zeros
    X[3] = 0.0                                                           # a row of zeros
    z = X @ W.T
    Zq, Zs = _empty_ckpt(plan, T)
    H = [torch.empty(T, f, dtype=torch.bfloat16, device="cuda")]
    plan.column_fwd_ckpt8(T, dev(X.bfloat16()), [dev(W.bfloat16())], None, Zq, Zs, H)
    q, s = _encode(z, act)
    assert torch.equal(Zs[0].cpu(), s)
    assert torch.equal(Zq[0].cpu().float(), q.float())


def test_nan_and_infinity():
    """A NaN decodes to NaN and an infinity to an infinity, and the other rows are untouched."""
    tp = _tp()
    plan = tp.Plan(64, 64, 0, 1, "bf16", "gelu")
    X, W = torch.ones(4, 64), torch.ones(64, 64)
    X[1, 0], X[2, 0] = float("nan"), float("inf")
    Zq, Zs = _empty_ckpt(plan, 4)
    H = [torch.empty(4, 64, dtype=torch.bfloat16, device="cuda")]
    plan.column_fwd_ckpt8(4, dev(X.bfloat16()), [dev(W.bfloat16())], None, Zq, Zs, H)
    z = _decode(Zq[0], Zs[0], "gelu").float()
    assert torch.isnan(z[1]).all() and torch.isinf(z[2]).all()
    assert (z[0] == 64).all() and (z[3] == 64).all()


def _backward(T, h, f, p, act, seed, want_w=True, want_h=True, want_b=True):
    tp = _tp()
    plan = tp.Plan(h, f, 0, p, "bf16", act)
    k, n1 = f // p, _halves(act) * f // p
    g = torch.Generator().manual_seed(seed)
    dY = torch.randn(T, h, generator=g).bfloat16()
    W = [(torch.randn(h, k, generator=g) * f ** -0.5).bfloat16() for _ in range(p)]
    packed = [_encode(torch.randn(T, n1, generator=g) * 2, act) for _ in range(p)]
    bf = lambda *s: torch.full(s, 7.0, dtype=torch.bfloat16, device="cuda")  # noqa: E731
    out = {"H": [bf(T, k) for _ in range(p)] if want_h else None, "dZ": [bf(T, n1) for _ in range(p)],
           "dW": [bf(h, k) for _ in range(p)] if want_w else None,
           "dbias": torch.full((h,), 7.0, device="cuda") if want_b else None}
    plan.row_bwd_ckpt8(T, dev(dY), [dev(w) for w in W], [dev(q) for q, _ in packed], [dev(s) for _, s in packed], out["H"], out["dZ"],
                       out["dW"], out["dbias"])
    return dY, W, packed, out


def _check_backward(dY, W, packed, out, act):
    T, h = dY.shape
    Y = dY.double()
    for i, (q, s) in enumerate(packed):
        z = _decode(q, s, act)
        H, fac = _act(z, act)
        eh, ef = _act_error(z, act)
        w = W[i].double()
        dH, mH = Y @ w, h * EPS * Y.norm(dim=1, keepdim=True) * w.norm(dim=0)[None]
        if act == "swiglu":
            dH, mH = torch.cat([dH, dH], 1), torch.cat([mH, mH], 1)
        ref = dH * fac
        lim = HALF * ref.abs() + 2 * (mH * fac.abs() + (dH.abs() + mH) * ef) + 1e-30
        assert ((out["dZ"][i].cpu().double() - ref).abs() <= lim).all(), "dZ"
        if out["H"] is not None:
            got = out["H"][i].cpu().double()
            assert ((got - H).abs() <= HALF * H.abs() + 2 * eh + 1e-30).all(), "H"
            if out["dW"] is not None:
                ref = Y.T @ got
                lim = HALF * ref.abs() + T * EPS * (Y.abs().T @ got.abs()) + 1e-30
                assert ((out["dW"][i].cpu().double() - ref).abs() <= lim).all(), "dW"
    if out["dbias"] is not None:
        assert ((out["dbias"].cpu().double() - Y.sum(0)).abs() <= T * EPS * Y.abs().sum(0) + 1e-30).all(), "dbias"


@pytest.mark.parametrize("act", ["swiglu", "gelu"])
@pytest.mark.parametrize("T,h,f,p", SHAPES + [(4500, 256, 256, 1)])
def test_backward(T, h, f, p, act):
    _check_backward(*_backward(T, h, f, p, act, T + f + 1), act)
    assert _tp().device_status() == "TP_OK"


@pytest.mark.parametrize("act", ["swiglu", "gelu"])
@pytest.mark.parametrize("want", [(False, False, False), (False, True, False), (True, True, False), (False, False, True)])
def test_backward_parts(act, want):
    _check_backward(*_backward(200, 256, 288, 2, act, 5, *want), act)


@pytest.mark.parametrize("act", ["swiglu", "gelu"])
def test_direct_epilogue_agrees(act, monkeypatch):
    """The epilogue without TMA stores gives the same bits."""
    a = _forward(130, 256, 544, 2, act, 3)
    b = _backward(130, 256, 544, 2, act, 4)
    monkeypatch.setenv("TP_GEMM_TMA_EPI", "0")
    c = _forward(130, 256, 544, 2, act, 3)
    d = _backward(130, 256, 544, 2, act, 4)
    for x, y in zip(a[3] + a[4] + a[5], c[3] + c[4] + c[5]):
        assert torch.equal(x.view(torch.uint8), y.view(torch.uint8))
    for k in ("H", "dZ", "dW"):
        for x, y in zip(b[3][k], d[3][k]):
            assert torch.equal(x, y)


@pytest.mark.parametrize("pair", ["1", "2"])
@pytest.mark.parametrize("act", ["swiglu", "gelu"])
def test_both_tile_layouts(act, pair, monkeypatch):
    monkeypatch.setenv("TP_GEMM_CTA_PAIR", pair)
    for narrow in ("0", "1"):
        monkeypatch.setenv("TP_GEMM_NARROW", narrow)
        _check_backward(*_backward(300, 192, 704, 2, act, 6), act)
        X, W, b, Zq, Zs, H = _forward(300, 192, 704, 2, act, 7)
        for i in range(2):
            z = X.double() @ W[i].double().T + (b[i].double() if b else 0)
            off = (_decode(Zq[i], Zs[i], act) - z).abs()
            assert (off <= torch.maximum(2.0 ** -4 * z.abs(), 2.0 ** -10 * _scales(Zs[i], z.shape[1], act)) + 1e-4).all()


def test_no_token():
    tp = _tp()
    plan = tp.Plan(64, 64, 0, 1, "bf16", "gelu")
    e = lambda *s, **k: torch.empty(*s, device="cuda", **k)  # noqa: E731
    none, w = e(0, 64, dtype=torch.bfloat16), torch.ones(64, 64, dtype=torch.bfloat16, device="cuda")
    q, s = [e(0, 64, dtype=torch.uint8)], [e(2, 0, dtype=torch.uint8)]
    plan.column_fwd_ckpt8(0, none, [w], None, q, s, [none])
    dW, db = [torch.ones_like(w)], torch.ones(64, device="cuda")
    plan.row_bwd_ckpt8(0, none, [w], q, s, [none], [none], dW, db)
    assert float(dW[0].abs().max()) == 0 and float(db.abs().max()) == 0


@pytest.mark.parametrize("defer", [False, True])
@pytest.mark.parametrize("concurrent", ["1", "0"])
def test_backward_on_a_stream_and_replayed(defer, concurrent, monkeypatch):
    """Every output is ready on the caller's stream when the call returns, the bias gradient
    too, which runs beside the products; a replayed graph gives the same bits."""
    monkeypatch.setenv("TP_BWD_CONCURRENT", concurrent)
    T, h, f, p = 515, 256, 1024, 2
    plan = _tp().Plan(h, f, 0, p, "bf16", "gelu")
    plan.set_backward_defer(defer)
    g = torch.Generator().manual_seed(5)
    Z = [(torch.randn(T, f // p, generator=g) * 2).bfloat16() for _ in range(p)]
    packed = [_encode(z.float(), "gelu") for z in Z]
    Zq, Zs = [dev(q.view(torch.uint8)) for q, _ in packed], [dev(s) for _, s in packed]
    dY = dev(torch.randn(T, h, generator=g).bfloat16())
    W = [dev((torch.randn(h, f // p, generator=g) * 0.05).bfloat16()) for _ in range(p)]
    new = lambda: ([torch.zeros(T, f // p, dtype=torch.bfloat16, device="cuda") for _ in range(p)],  # noqa: E731
                   [torch.zeros(T, f // p, dtype=torch.bfloat16, device="cuda") for _ in range(p)],
                   [torch.zeros(h, f // p, dtype=torch.bfloat16, device="cuda") for _ in range(p)], torch.zeros(h, device="cuda"))
    flat = lambda o: [*o[0], *o[1], *o[2], o[3]]  # noqa: E731
    first, side, graphed = new(), new(), new()
    plan.row_bwd_ckpt8(T, dY, W, Zq, Zs, *first)
    want = [host(t).copy() for t in flat(first)]
    db = dY.double().sum(0).cpu().numpy()
    bound = T * EPS * dY.double().abs().sum(0).cpu().numpy()
    assert np.all(np.abs(want[-1] - db) <= bound)
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(st):
        plan.row_bwd_ckpt8(T, dY, W, Zq, Zs, *side)
        copies = [t.clone() for t in flat(side)]
    st.synchronize()
    assert all(np.array_equal(host(a), b) for a, b in zip(copies, want))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        plan.row_bwd_ckpt8(T, dY, W, Zq, Zs, *graphed)
    for _ in range(2):
        for t in flat(graphed):
            t.fill_(7)
        graph.replay()
        torch.cuda.synchronize()
        assert all(np.array_equal(host(a), b) for a, b in zip(flat(graphed), want))
    assert _tp().device_status() == "TP_OK"
