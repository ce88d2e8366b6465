"""Layers with gated residual junctions, 8-bit MLP checkpoints and the fused output head
together, forward and backward, against an fp64 model.

Bounds (row-normalised error, as for the other stacks): one sublayer call in bf16 is within
2e-2, and each bf16 boundary that the values crossed before adds its unit roundoff, 2^-8
(a layer stores a, x1, u1, m, x2, u2: six; the backward as many again). With 8-bit
checkpoints every pre-activation enters the backward with a relative error of at most 2^-4,
on both sides alike but where a rounding falls the other way: 2^-4 more for the gradients."""
import numpy as np
import pytest
import torch

import oracle as O
from gpu_helpers import host
from test_gpu_ckpt8 import _act, _decode, _encode

pytestmark = pytest.mark.gpu
BATCH, SEQ, H_, F_, HEADS, P, V, L = 2, 72, 256, 576, 4, 2, 1003, 2
STEP = 2.0 ** -8


class _Mlp(torch.autograd.Function):
    """act(z) W2^T whose backward sees z through its 8-bit form (per shard), as the layer's does."""

    @staticmethod
    def forward(ctx, z, W2, act, ckpt8):
        # z [T, P, n1], W2 [H, F] by columns of shards
        zs = [z[:, i] for i in range(P)]
        kept = [_decode(*_encode(x.detach(), act), act) if ckpt8 else x for x in zs]
        ctx.save_for_backward(W2, *kept)
        ctx.act = act
        return torch.cat([_act(x, act)[0] for x in zs], 1) @ W2.T

    @staticmethod
    def backward(ctx, dy):
        W2, *kept = ctx.saved_tensors
        pairs = [_act(x, ctx.act) for x in kept]
        dH = (dy @ W2).chunk(P, 1)
        dz = torch.stack([(torch.cat([d, d], 1) if ctx.act == "swiglu" else d) * f for d, (_, f) in zip(dH, pairs)], 1)
        return dz, dy.T @ torch.cat([h for h, _ in pairs], 1), None, None


def _norm(x, g, b, kind):
    m = x.mean(1, keepdim=True) if kind == "layer" else 0.0
    y = (x - m) / torch.sqrt(((x - m) ** 2).mean(1, keepdim=True) + 1e-5) * g
    return y + b if kind == "layer" else y


def _attention(u, Wqkv, Wo):
    d = H_ // HEADS
    q, k, v = (t.reshape(SEQ, BATCH, HEADS, d).permute(1, 2, 0, 3) for t in (u @ Wqkv.T).chunk(3, 1))
    s = q @ k.transpose(2, 3) / d ** 0.5
    s = s.masked_fill(torch.triu(torch.ones(SEQ, SEQ, dtype=torch.bool), 1), -np.inf)
    o = (torch.softmax(s, 3) @ v).permute(2, 0, 1, 3).reshape(SEQ * BATCH, H_)
    return o @ Wo.T


def _build(kind, gate_rows, act, ckpt8, seed=0):
    from megatron_tensor_transformer_gemm_b200.block import TPGatedLayer, TPHead
    g = torch.Generator().manual_seed(seed)
    rn = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
    n1 = 2 * F_ if act == "swiglu" else F_
    scratch = [torch.empty(BATCH * SEQ, F_ // P, dtype=torch.bfloat16, device="cuda") for _ in range(P)]
    layers, prms = [], []
    for _ in range(L):
        prm = {"Wqkv": rn(3 * H_, H_) * 1.5 * H_ ** -0.5, "Wo": rn(H_, H_) * H_ ** -0.5, "W1": rn(n1, H_) * H_ ** -0.5,
               "W2": rn(H_, F_) * F_ ** -0.5}
        for k in range(2):
            prm[f"gate{k}"] = 0.7 + 0.2 * rn(gate_rows, H_)
            for w in ("post", "pre"):
                prm[f"{w}{k}g"], prm[f"{w}{k}b"] = 1 + 0.1 * rn(H_), 0.1 * rn(H_)
        prm = {k: v.bfloat16() for k, v in prm.items()}
        lay = TPGatedLayer(H_, F_, HEADS, P, act, kind, 0.9, gate_rows, ckpt8=ckpt8, H_scratch=scratch if ckpt8 else None)
        lay.attn.load_weights(prm["Wqkv"].cuda(), prm["Wo"].cuda())
        lay.mlp.load_weights(prm["W1"].cuda(), prm["W2"].cuda())
        for k in range(2):
            lay.gate[k].copy_(prm[f"gate{k}"])
            for w in ("post", "pre"):
                for t, n in zip(getattr(lay, w)[k], "gb"):
                    t.copy_(prm[f"{w}{k}{n}"])
        layers.append(lay)
        prms.append(prm)
    head = TPHead(H_, V, P)
    Wv = (rn(V, H_) * 0.1).bfloat16()
    head.load_weight(Wv.cuda())
    x = rn(BATCH * SEQ, H_).bfloat16()
    u = rn(BATCH * SEQ, H_).bfloat16()
    labels = torch.randint(0, V, (BATCH * SEQ,), generator=g, dtype=torch.int32)
    labels[::5] = -1
    return layers, prms, head, Wv, x, u, labels


def _step(layers, head, x, u, labels, scale):
    for lay in layers:
        x, u = lay.forward(x, u, BATCH, SEQ)
    loss = head.loss(u, labels, scale)
    dx, du = None, head.dX
    for lay in reversed(layers):
        dx, du = lay.backward(dx, du, BATCH, SEQ)
    return loss, dx, du


def _reference(prms, Wv, x, u, labels, kind, act, ckpt8, scale):
    leaf = lambda t: t.double().requires_grad_()  # noqa: E731
    P64 = [{k: leaf(v) for k, v in prm.items()} for prm in prms]
    Wv, x0, u0 = leaf(Wv), leaf(x), leaf(u)
    T, fp = len(x), F_ // P
    xs, us = x0, u0
    for q in P64:
        for k in range(2):
            if k == 0:
                f = _attention(us, q["Wqkv"], q["Wo"])
            else:
                z = us @ q["W1"].T
                # shard i: rows i * fp .. of the gate half and of the up half
                z = z.reshape(T, 2 if act == "swiglu" else 1, P, fp).transpose(1, 2).reshape(T, P, -1)
                f = _Mlp.apply(z, q["W2"], act, ckpt8)
            g = q[f"gate{k}"][torch.arange(T) % q[f"gate{k}"].shape[0]]
            xs = 0.9 * xs + g * _norm(f, q[f"post{k}g"], q[f"post{k}b"], kind)
            us = _norm(xs, q[f"pre{k}g"], q[f"pre{k}b"], kind)
    s = us @ Wv.T
    keep = labels >= 0
    loss = (torch.logsumexp(s, 1) - s.gather(1, labels.long().clamp(min=0)[:, None])[:, 0]) * keep
    (loss.sum() * scale).backward()
    return loss.detach(), P64, Wv, x0, u0


@pytest.mark.parametrize("kind,gate_rows,act,ckpt8", [("rms", 1, "swiglu", True), ("layer", BATCH, "gelu", True),
                                                      ("layer", 1, "swiglu", False)])
def test_step_against_fp64(kind, gate_rows, act, ckpt8):
    from megatron_tensor_transformer_gemm_b200 import tp
    layers, prms, head, Wv, x, u, labels = _build(kind, gate_rows, act, ckpt8)
    scale = 1.0 / 64
    loss, dx, du = _step(layers, head, x.cuda(), u.cuda(), labels.cuda(), scale)
    rl, P64, rWv, rx, ru = _reference(prms, Wv, x, u, labels, kind, act, ckpt8, scale)
    fwd = 2e-2 + 6 * L * STEP
    bwd = 2e-2 + 12 * L * STEP + (2.0 ** -4 if ckpt8 else 0.0)
    # a score is a product with a row of u2, each entry within fwd of the row's largest: it moves by
    # at most fwd * max|u2| * sum|w|, the loss by twice that
    with torch.no_grad():
        lim = 2 * fwd * host(layers[-1].us[1]).__abs__().max(1) * float(Wv.double().abs().sum(1).max())
        assert np.all(np.abs(host(loss) - rl.numpy()) <= lim)
        assert np.abs(host(loss) - rl.numpy()).mean() <= fwd * rl.numpy().mean()
    err = lambda got, ref: O.max_row_rel_err(host(got) if isinstance(got, torch.Tensor) else got, ref)  # noqa: E731
    dWv = host(torch.cat(head.dW, 0))
    assert np.all(dWv[V:] == 0)
    errs = {"dx": err(dx, rx.grad.numpy()), "du": err(du, ru.grad.numpy()),
            "dWv": float(np.linalg.norm(dWv[:V] - rWv.grad.numpy()) / np.linalg.norm(rWv.grad.numpy()))}
    for i, (lay, q) in enumerate(zip(layers, P64)):
        W = torch.empty_like(prms[i]["W2"], device="cuda")
        lay.mlp.plan.unshard_row("mlp", lay.mlp.dW2, W)
        errs[f"{i}.dW2"] = err(W, q["W2"].grad.numpy())
        W = torch.empty_like(prms[i]["W1"], device="cuda")
        lay.mlp.plan.unshard_column("mlp", lay.mlp.dW1, W)
        errs[f"{i}.dW1"] = err(W, q["W1"].grad.numpy())
        W = torch.empty_like(prms[i]["Wqkv"], device="cuda")
        lay.attn.plan.unshard_column("qkv", lay.attn.dWqkv, W)
        # all rows together: with random scores single q and k rows are small beside the rest
        errs[f"{i}.dWqkv"] = float(np.linalg.norm(host(W) - q["Wqkv"].grad.numpy()) / np.linalg.norm(q["Wqkv"].grad.numpy()))
        for k in range(2):
            errs[f"{i}.dgate{k}"] = err(lay.dgate[k], q[f"gate{k}"].grad.numpy())
            for w, d in (("post", lay.dpost[k]), ("pre", lay.dpre[k])):
                errs[f"{i}.d{w}{k}g"] = err(d[0][None], q[f"{w}{k}g"].grad.numpy()[None])
                if kind == "layer":
                    errs[f"{i}.d{w}{k}b"] = err(d[1][None], q[f"{w}{k}b"].grad.numpy()[None])
    bad = {k: v for k, v in errs.items() if not v <= bwd}
    assert not bad, (bad, bwd)
    assert tp.device_status() == "TP_OK"


def test_captured_step_gives_the_eager_bits():
    from megatron_tensor_transformer_gemm_b200.block import CapturedStep
    layers, prms, head, Wv, x, u, labels = _build("rms", BATCH, "swiglu", True, seed=3)
    xd, ud, ld = x.cuda(), u.cuda(), labels.cuda()
    step = CapturedStep(lambda: _step(layers, head, xd, ud, ld, 1.0))
    outs = lambda: [head.loss_rows, head.dX, *head.dW, layers[0].dx, *layers[0].mlp.dW2, layers[1].dgate[1], layers[0].dpre[0][0]]  # noqa: E731
    for seed in (4, 5):
        xd.copy_(torch.randn(x.shape, generator=torch.Generator().manual_seed(seed)).bfloat16())
        _step(layers, head, xd, ud, ld, 1.0)
        want = [t.clone() for t in outs()]
        for t in outs():
            t.zero_()
        step()
        torch.cuda.synchronize()
        for a, b in zip(outs(), want):
            assert torch.equal(a, b)


def test_scoring_without_gradients():
    _, _, head, Wv, x, u, labels = _build("rms", 1, "swiglu", True, seed=6)
    loss = head.loss(u.cuda(), labels.cuda())
    s = u.double() @ Wv.double().T
    ref = (torch.logsumexp(s, 1) - s.gather(1, labels.long().clamp(min=0)[:, None])[:, 0]) * (labels >= 0)
    assert head.dX is None and np.abs(host(loss) - ref.numpy()).max() <= 1e-3


def test_two_threads_at_once():
    """Two host threads, each with plans and a stream of its own, through the calls that share the
    device's side stream: the bits of the same calls made one after the other."""
    import threading

    from megatron_tensor_transformer_gemm_b200 import tp
    T, h, V, f = 300, 128, 2003, 512
    n = 30

    def make(seed):
        g = torch.Generator().manual_seed(seed)
        rnd = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
        head, mlp = tp.Plan(h, 0, 0, 1, "f32", "none"), tp.Plan(h, f, 0, 1, "bf16", "gelu")
        Vp = head.set_vocab(V)
        s = {"X": rnd(n, T, h).cuda(), "W": [(rnd(Vp, h) * 0.1).cuda()], "labels": torch.randint(0, V, (T,), generator=g, dtype=torch.int32).cuda(),
             "dY": rnd(n, T, h).bfloat16().cuda(), "W2": [(rnd(h, f) * 0.05).bfloat16().cuda()], "Wc": [rnd(f, h).bfloat16().cuda()]}
        return head, mlp, s

    def run(head, mlp, s, out):
        X16 = s["X"].bfloat16()
        codes, scales = mlp.ckpt8_shapes(T)
        e = lambda *z, dt=torch.float32: torch.empty(*z, dtype=dt, device="cuda")  # noqa: E731
        bf = torch.bfloat16
        for i in range(n):
            loss, dX, dW = e(T), e(T, h), [torch.empty_like(s["W"][0])]
            head.vocab_linear_cross_entropy(T, s["X"][i], s["W"], s["labels"], 0.5, loss, None, dX, dW)
            Zq, Zs, H = [e(*codes, dt=torch.uint8)], [e(*scales, dt=torch.uint8)], [e(T, f, dt=bf)]
            dZ, dW2, db = [e(T, f, dt=bf)], [e(h, f, dt=bf)], e(h)
            mlp.column_fwd_ckpt8(T, X16[i], s["Wc"], None, Zq, Zs, H)
            mlp.row_bwd_ckpt8(T, s["dY"][i], s["W2"], Zq, Zs, H, dZ, dW2, db)
            out.append([loss, dX, dW[0], dZ[0], dW2[0], db])

    sides = [make(31), make(32)]
    want = [[], []]
    for side, w in zip(sides, want):
        run(*side, w)
    torch.cuda.synchronize()
    got, errors = [[], []], []

    def thread(k):
        try:
            st = torch.cuda.Stream()
            with torch.cuda.stream(st):
                run(*sides[k], got[k])
            st.synchronize()
        except Exception as e:  # noqa: BLE001
            errors.append(e)

    threads = [threading.Thread(target=thread, args=(k,)) for k in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not errors, errors
    for w, g in zip(want, got):
        for a, b in zip(w, g):
            assert all(torch.equal(x, y) for x, y in zip(a, b))
    assert tp.device_status() == "TP_OK"
