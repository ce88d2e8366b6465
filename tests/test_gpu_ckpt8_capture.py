"""8-bit MLP backward in a stream capture: a call that would have to allocate is refused before it
records anything."""
import pytest
import torch

from gpu_helpers import dev
from test_gpu_ckpt8 import EPS, _encode, _tp

pytestmark = pytest.mark.gpu


def _row_bwd(T=40, h=256, f=64, p=1):
    plan = _tp().Plan(h, f, 0, p, "bf16", "gelu")
    g = torch.Generator().manual_seed(6)
    q, s = _encode(torch.randn(T, f, generator=g), "gelu")
    bf = lambda *z: torch.zeros(*z, dtype=torch.bfloat16, device="cuda")  # noqa: E731
    dY = torch.randn(T, h, generator=g).bfloat16()
    args = (T, dev(dY), [dev((torch.randn(h, f, generator=g) * 0.1).bfloat16())], [dev(q.view(torch.uint8))], [dev(s)],
            [bf(T, f)], [bf(T, f)], [bf(h, f)])
    return plan, dY, args, torch.zeros(h, device="cuda")


def test_a_first_call_with_a_bias_gradient_is_refused_in_a_capture():
    """8-bit backward whose only workspace is the bias sum's: refused with nothing recorded, the
    capture goes on, and after one eager call the same capture works."""
    tp = _tp()
    plan, dY, args, db = _row_bwd()
    graph = torch.cuda.CUDAGraph()
    keep = torch.zeros(8, device="cuda")
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        keep.add_(1.0)
        n = tp.launch_count()
        with pytest.raises(tp.TPError, match="before the stream capture"):
            plan.row_bwd_ckpt8(*args, db)
        assert tp.launch_count() == n
    graph.replay()
    torch.cuda.synchronize()
    assert float(keep[0]) == 1.0 and float(args[6][0].abs().max()) == 0
    plan.row_bwd_ckpt8(*args, db)
    want = [t[0].clone() for t in args[5:]] + [db.clone()]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        plan.row_bwd_ckpt8(*args, db)
    for t in (*args[5], *args[6], *args[7], db):
        t.fill_(7)
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip([t[0] for t in args[5:]] + [db], want))
    Y = dY.double()
    assert bool(((db.cpu().double() - Y.sum(0)).abs() <= 40 * EPS * Y.abs().sum(0) + 1e-30).all())


def test_a_larger_bias_gradient_is_refused_in_a_capture():
    """The counters are there from a small call, the larger sum's partials (1.2 MB) are not."""
    tp = _tp()
    plan, _, args, db = _row_bwd(h=1024)
    plan.row_bwd_ckpt8(*args, db)
    T, h, f = 20000, 1024, 64
    bf = lambda *z: torch.ones(*z, dtype=torch.bfloat16, device="cuda")  # noqa: E731
    u8 = lambda *z: torch.full(z, 127, dtype=torch.uint8, device="cuda")  # noqa: E731
    big = (T, bf(T, h), args[2], [u8(T, f).fill_(0)], [u8(2, T)], None, [bf(T, f)], None, db)
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        args[6][0].add_(0)
        n = tp.launch_count()
        with pytest.raises(tp.TPError, match="before the stream capture"):
            plan.row_bwd_ckpt8(*big)
        assert tp.launch_count() == n
    plan.row_bwd_ckpt8(*big)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        plan.row_bwd_ckpt8(*big)
    db.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert bool((db == T).all())
    assert tp.device_status() == "TP_OK"
