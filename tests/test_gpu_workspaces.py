"""The plan's workspaces around stream captures: what a graph holds is kept, nothing else is."""
import pytest
import torch

from gpu_helpers import dev
from test_gpu_loss import _check, _head, _tp

pytestmark = pytest.mark.gpu
MB = 1 << 20


def _used():
    torch.cuda.synchronize()
    free, total = torch.cuda.mem_get_info()
    return total - free


def test_only_the_block_a_graph_holds_is_kept():
    """After a capture, eager calls of rising sizes replace the plan's block again and again: only
    the one that the graph replays with stays beside the newest."""
    V, h, p, sizes = 16000, 64, 2, [1000 * k for k in range(1, 9)]
    plan, Vp, X, W, labels = _head(96, h, V, p, "bf16", seed=10)
    Xd, Ws, ld = dev(X), [dev(w) for w in W.chunk(p)], labels.cuda()
    loss, dX, dW = torch.empty(96, device="cuda"), torch.empty_like(Xd), [torch.empty_like(w) for w in Ws]

    def call():
        plan.vocab_linear_cross_entropy(96, Xd, Ws, ld, 0.5, loss, None, dX, dW)

    from megatron_tensor_transformer_gemm_b200.block import CapturedStep
    step = CapturedStep(call)
    n = sizes[-1]
    big, bl, bd = torch.randn(n, h, device="cuda").bfloat16(), torch.empty(n, device="cuda"), torch.empty(n, h, device="cuda").bfloat16()
    lab = torch.zeros(n, dtype=torch.int32, device="cuda")
    before = _used()
    for T in sizes:
        plan.vocab_linear_cross_entropy(T, big[:T], Ws, lab[:T], 1.0, bl[:T], None, bd[:T], dW)
    last = n * Vp * 2 + n * (Vp // 128 + p) * 16 + 16 * n * h * 4  # exponentials, statistics, split sums of dX
    assert _used() - before <= last + 24 * MB, (_used() - before, last)  # all of them: 4.5 times that
    for seed in (11, 12):
        X2 = torch.randn(96, h, generator=torch.Generator().manual_seed(seed)).bfloat16()
        Xd.copy_(X2)
        for t in (loss, dX, *dW):
            t.zero_()
        step()
        _check(X2, W, labels, V, 0.5, (loss, None, dX, dW), "bf16")
    assert _tp().device_status() == "TP_OK"


def test_blocks_of_two_graphs_and_the_calls_between():
    """Two graphs captured with blocks of different sizes replay right after both were replaced."""
    from megatron_tensor_transformer_gemm_b200.block import CapturedStep
    V, h, p = 3001, 128, 2
    plan, Vp, X, W, labels = _head(4000, h, V, p, "bf16", seed=20)
    Ws = [dev(w) for w in W.chunk(p)]

    def make(T):
        s = (dev(X[:T]), labels[:T].cuda(), torch.empty(T, device="cuda"), torch.empty(T, h, device="cuda").bfloat16(),
             [torch.empty_like(w) for w in Ws])
        return s, lambda: plan.vocab_linear_cross_entropy(T, s[0], Ws, s[1], 0.5, s[2], None, s[3], s[4])

    small, run_small = make(70)
    g1 = CapturedStep(run_small)
    mid, run_mid = make(900)
    run_mid()
    g2 = CapturedStep(run_mid)
    large, run_large = make(4000)
    run_large()
    for s, g in ((mid, g2), (small, g1), (mid, g2), (small, g1)):
        for t in (s[2], s[3], *s[4]):
            t.zero_()
        g()
        T = len(s[2])
        _check(X[:T], W, labels[:T], V, 0.5, (s[2], None, s[3], s[4]), "bf16")
    run_large()
    _check(X, W, labels, V, 0.5, (large[2], None, large[3], large[4]), "bf16")
