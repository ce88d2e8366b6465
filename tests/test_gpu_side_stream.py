"""Calls that use the device's side stream while another thread captures: a capture has a side
stream of its own, so eager calls beside it, and two captures at once, do not meet."""
import threading

import pytest
import torch

from test_gpu_loss import _tp

pytestmark = pytest.mark.gpu
T, H, F, V = 300, 128, 512, 2003


class Work:
    """Plans, inputs and outputs of one thread; run() is a fp32 head, an 8-bit MLP backward and a
    small MLP's two backward calls, which fork to the side stream."""

    def __init__(self, seed, defer=False):
        tp = _tp()
        g = torch.Generator().manual_seed(seed)
        rnd = lambda *s: torch.randn(*s, generator=g).cuda()  # noqa: E731
        bf = torch.bfloat16
        self.head, self.mlp, self.plain = tp.Plan(H, 0, 0, 1, "f32", "none"), tp.Plan(H, F, 0, 1, "bf16", "gelu"), tp.Plan(H, F, 0, 1, "bf16", "gelu")
        self.defer = defer
        self.plain.set_backward_defer(defer)
        Vp = self.head.set_vocab(V)
        self.X, self.W, self.lab = rnd(T, H), [rnd(Vp, H) * 0.1], torch.randint(0, V, (T,), generator=g, dtype=torch.int32).cuda()
        self.X16, self.dY, self.Wc, self.Wr = rnd(T, H).to(bf), rnd(T, H).to(bf), [(rnd(F, H) * 0.1).to(bf)], [(rnd(H, F) * 0.1).to(bf)]
        codes, scales = self.mlp.ckpt8_shapes(T)
        e = lambda *z, dt=bf: torch.zeros(*z, dtype=dt, device="cuda")  # noqa: E731
        f32 = torch.float32
        self.q, self.s, self.Hh, self.Z = [e(*codes, dt=torch.uint8)], [e(*scales, dt=torch.uint8)], [e(T, F)], [e(T, F)]
        self.mlp.column_fwd_ckpt8(T, self.X16, self.Wc, None, self.q, self.s, self.Hh)
        self.plain.column_fwd("mlp", T, self.X16, self.Wc, None, self.Z, self.Hh)
        self.H2 = [e(T, F)]
        self.loss, self.dX, self.dW = e(T, dt=f32), e(T, H, dt=f32), [torch.zeros_like(self.W[0])]
        self.dZ8, self.dWr8, self.db8 = [e(T, F)], [e(H, F)], e(H, dt=f32)
        self.dZ, self.dWr, self.db, self.dWc, self.dbc, self.dXc = [e(T, F)], [e(H, F)], e(H, dt=f32), [e(F, H)], [e(F, dt=f32)], e(T, H)

    def run(self):
        self.head.vocab_linear_cross_entropy(T, self.X, self.W, self.lab, 0.5, self.loss, None, self.dX, self.dW)
        self.mlp.row_bwd_ckpt8(T, self.dY, self.Wr, self.q, self.s, self.H2, self.dZ8, self.dWr8, self.db8)
        self.plain.row_bwd("mlp", T, self.dY, self.Hh, self.Wr, self.Z, self.dZ, self.dWr, self.db)
        self.plain.column_bwd_reduce("mlp", T, self.X16, self.dZ, self.Wc, self.dWc, self.dbc, self.dXc)
        if self.defer:
            _tp().backward_join()

    def outs(self):
        return [self.loss, self.dX, *self.dW, *self.dZ8, *self.dWr8, self.db8, *self.dZ, *self.dWr, self.db, *self.dWc, *self.dbc, self.dXc]

    def want(self):
        self.run()
        torch.cuda.synchronize()
        w = [t.clone() for t in self.outs()]
        self.clear()
        return w

    def clear(self):
        for t in self.outs():
            t.fill_(7)
        torch.cuda.synchronize()


def _same(work, want):
    torch.cuda.synchronize()
    return all(torch.equal(a, b) for a, b in zip(work.outs(), want))


def _thread(fn):
    errors = []

    def body():
        try:
            fn()
        except Exception as e:  # noqa: BLE001
            errors.append(e)

    t = threading.Thread(target=body)
    t.start()
    return t, errors


@pytest.mark.parametrize("defer", [False, True])
def test_eager_calls_of_another_thread_while_this_one_captures(defer):
    a, b = Work(41, defer), Work(42, defer)
    want_a, want_b = a.want(), b.want()
    sa, sb = torch.cuda.Stream(), torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()

    def eager():
        with torch.cuda.stream(sb):
            for _ in range(3):
                b.run()

    with torch.cuda.stream(sa):
        graph.capture_begin(capture_error_mode="thread_local")
        a.run()
        t, errors = _thread(eager)
        t.join()
        a.run()
        graph.capture_end()
    assert not errors, errors
    assert _same(b, want_b)
    for _ in range(2):
        a.clear()
        graph.replay()
        assert _same(a, want_a)
    assert _tp().device_status() == "TP_OK"


def test_two_threads_capture_at_once_and_replay_together():
    works = [Work(51), Work(52, True)]
    wants = [w.want() for w in works]
    graphs, streams = [torch.cuda.CUDAGraph() for _ in works], [torch.cuda.Stream() for _ in works]
    torch.cuda.synchronize()
    gate = threading.Barrier(2, timeout=60)

    def capture(k):
        with torch.cuda.stream(streams[k]):
            graphs[k].capture_begin(capture_error_mode="thread_local")
            gate.wait()
            for _ in range(3):
                works[k].run()
                gate.wait()
            graphs[k].capture_end()

    threads = [_thread(lambda k=k: capture(k)) for k in range(2)]
    for t, _ in threads:
        t.join()
    assert not threads[0][1] and not threads[1][1], threads
    for _ in range(3):
        for w in works:
            w.clear()
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
        assert all(_same(w, want) for w, want in zip(works, wants))
    # streams of captures that have ended serve the next ones and eager calls go on
    for w, want in zip(works, wants):
        w.clear()
        w.run()
        assert _same(w, want)
    assert _tp().device_status() == "TP_OK"


def test_a_join_without_deferred_work_in_the_capture_is_refused():
    tp = _tp()
    x = torch.zeros(8, device="cuda")
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        x.add_(1.0)
        with pytest.raises(tp.TPError, match="capture"):
            tp.backward_join()
    graph.replay()
    torch.cuda.synchronize()
    assert float(x[0]) == 1.0
