"""Output head with its cross-entropy: tokens whose label is all but certain, against fp64.

Token t has one feature of its own, so its scores are single products, exact in fp32 and in
the tensor cores, and a column of dW has one token's gradient. What is left to err:
joining two (maximum, sum) pairs multiplies by an exponential good to 2^-22 and adds with
2^-24; a term passes at most 10 joins in its thread, 5 in its warp and 16 across the warps,
say 40 of each with its own. The arguments of a term's exponentials add up to at most 32
where it counts (2^-32 of the largest otherwise), each rounded to 2^-24. So with o the other
columns' share and t the label's, o / t is off by at most 40 * (2^-22 + 2^-24) + 32 * 2^-24 *
ln 2 < 2^-16 of itself, and with a few roundings more so are log1p(o / t), the loss, and
o / (o + t), the label's entry of the gradient, however small they are: 2^-15. bf16 plans add
2^-10 on the other columns' entries (held in 16 bits), 2^-8 where d is rounded (2^-16 in two
parts) and 2^-8 for the result."""
import numpy as np
import pytest
import torch

from gpu_helpers import dev, host
from test_gpu_loss import _check, _head, _reference, _run, _tp

pytestmark = pytest.mark.gpu
REL = 2.0 ** -15


def _sure(T, h, V, p, dtype, seed):
    """Scores of single products: the label's S in [25, 40], a runner-up 5 to 16 below, the rest
    17 and more below; every value exact in bf16."""
    plan, Vp, _, W, _ = _head(T, h, V, p, dtype, seed=seed)
    g = torch.Generator().manual_seed(seed)
    W = (torch.randint(-32, 33, (Vp, h), generator=g) / 8).to(W.dtype)
    X = torch.zeros(T, h, dtype=W.dtype)
    labels = torch.randint(0, V, (T,), generator=g, dtype=torch.int32)
    for t in range(T):
        X[t, t] = float(2 ** int(torch.randint(-1, 2, (1,), generator=g)))
        x, lab = float(X[t, t]), int(labels[t])
        s = 25 + 0.25 * int(torch.randint(0, 61, (1,), generator=g))
        W[lab, t] = s / x
        gap = 5 + 0.25 * int(torch.randint(0, 45, (1,), generator=g))
        W[(lab + 1 + t) % V, t] = (s - gap) / x
    return plan, Vp, X, W, labels


CASES = [(1, 64, 50, 1, 0), (48, 64, 1003, 2, 0), (64, 128, 5003, 4, 0), (200, 256, 777, 4, 0), (200, 256, 1003, 2, 96), (250, 256, 20011, 8, 0)]


@pytest.mark.parametrize("T,h,V,p,chunk", CASES)
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_sure_tokens_keep_their_digits(T, h, V, p, chunk, dtype):
    plan, Vp, X, W, labels = _sure(T, h, V, p, dtype, seed=T + V)
    scale = 1.0 / 4
    loss, lse, dX, dW = _run(plan, Vp, X, W, labels, scale, chunk)
    rl, rs, rx, rw, bx, bw, px, pw = _reference(X, W, labels, V, scale)
    # the reference's own digits: log1p of the others' share of the label's
    z = X.double() @ W[:V].double().T
    lab = labels.long()[:, None]
    o = torch.exp(z - z.gather(1, lab)).scatter(1, lab, 0.0).sum(1)
    rl = torch.log1p(o)
    assert float(rl.min()) < 2e-6 or T < 48
    got = torch.from_numpy(host(loss))
    assert bool((got >= 0).all()) and bool(((got - rl).abs() <= REL * rl).all()), float(((got - rl).abs() / rl).max())
    assert bool(((torch.from_numpy(host(lse)) - rs).abs() <= 2.0 ** -22 * rs.abs()).all())
    d = torch.exp(z - z.gather(1, lab)) / (1 + o)[:, None]
    d = d.scatter(1, lab, (-o / (1 + o))[:, None]) * scale  # [T, V]
    gw = torch.from_numpy(np.concatenate([host(w) for w in dW]))[:V, :T]  # column t: token t alone
    want = (d * X.double().diagonal()[:, None]).T
    rel = torch.full((T, 1), REL).double().expand(T, V).clone()
    if dtype == "bf16":
        rel += 2.0 ** -10
        rel.scatter_(1, lab, REL)
        rel += 2.0 ** -8 + (2.0 ** -16 if T <= 64 else 2.0 ** -8) + 2.0 ** -15  # the last: two roundings' product
    tiny = 2.0 ** -60  # below: what the two parts of d, or their product, cannot hold
    bad = (gw - want).abs() > rel.T * want.abs() + tiny
    assert not bool(bad.any()), float(((gw - want).abs() / (want.abs() + tiny)).max())
    lim = (rel.max() + V * 2.0 ** -24) * (d.abs() @ W[:V].double().abs()) + 2.0 ** -8 * (d @ W[:V].double()).abs() * (dtype == "bf16") + tiny
    assert bool(((torch.from_numpy(host(dX)) - d @ W[:V].double()).abs() <= lim).all())
    assert _tp().device_status() == "TP_OK"


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_a_label_far_below_and_a_vocab_of_one(dtype):
    """A label whose probability is 0 to fp32 (loss = lse - z, gradient -1), and one entry in all."""
    plan, Vp, X, W, labels = _sure(40, 64, 1003, 2, dtype, seed=3)
    labels = (labels + 7) % 1003
    W[labels.long(), torch.arange(40)] = -2.0 ** 9
    z = X.double() @ W[:1003].double().T
    rl = torch.logsumexp(z, 1) - z.gather(1, labels.long()[:, None])[:, 0]
    loss, _, dX, dW = _run(plan, Vp, X, W, labels, 1.0)
    assert bool(((torch.from_numpy(host(loss)) - rl).abs() <= 2.0 ** -22 * rl).all())
    gw = torch.from_numpy(np.concatenate([host(w) for w in dW]))
    assert torch.equal(gw[labels.long(), torch.arange(40)], -X.double().diagonal())
    plan, Vp, X, W, labels = _head(5, 64, 1, 1, dtype, seed=4, ignored=False)
    labels[:] = 0
    loss, lse, dX, dW = _run(plan, Vp, X, W, labels, 1.0)
    assert float(loss.abs().max()) == 0 and float(dX.abs().max()) == 0 and float(dW[0].abs().max()) == 0


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_rows_alone_and_in_a_smaller_batch(dtype):
    """The loss of a row does not depend on the rows beside it: alone, among 5 and among 300 it is
    the same value but for the order of the scores' sums (each h * 2^-24 of |x| |w|)."""
    V, h, T = 3001, 128, 300
    plan, Vp, X, W, labels = _head(T, h, V, 2, dtype, seed=8)
    full = _run(plan, Vp, X, W, labels, 1.0, grad=(True, False))
    eps = 2.0 ** -24
    z_err = float(h * eps * X.double().norm(dim=1).max() * W[:V].double().norm(dim=1).max())
    lim = 2 * (2 * z_err + 2 * (2.0 ** -21 + 4 * eps * (float(full[1].abs().max()) + 8)))
    for rows in ([0], [3], [7], [299], [10, 11, 12, 13, 14]):
        part = _run(plan, Vp, X[rows], W, labels[rows], 1.0, grad=(True, False))
        _check(X[rows], W, labels[rows], V, 1.0, part, dtype)
        for k in (0, 1):
            assert float((part[k] - full[k][rows]).abs().max()) <= lim
