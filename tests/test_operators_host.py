"""Refusals of the fused training operators, on the host before any launch."""
import ctypes

import pytest
import torch

from megatron_tensor_transformer_gemm_b200 import tp

A = 0x10000  # an aligned fake device pointer: validation fails before any use


def _arr(*v):
    return (ctypes.c_void_p * len(v))(*v)


@pytest.fixture()
def head():
    plan = tp.Plan(64, 0, 0, 2, "bf16", "none")
    plan.set_vocab(1000)
    return plan


def _loss(plan, T=4, X=A, W=(A + 16, A + 32), labels=A, loss=A, lse=None, dX=None, dW=None, chunk=0):
    return tp.lib.tp_vocab_linear_cross_entropy(plan.handle, T, X, _arr(*W) if W else None, labels, 1.0, loss, lse, dX,
                                                _arr(*dW) if dW else None, chunk, None)


def test_loss_refusals(head):
    assert _loss(head, T=-1) == 1 and "negative" in tp.last_error()
    assert _loss(head, T=2 ** 31) == 5
    assert _loss(head, chunk=-5) == 1 and "chunk" in tp.last_error()
    assert _loss(head, X=None) == 1 and "X" in tp.last_error()
    assert _loss(head, X=A + 4) == 3
    assert _loss(head, W=None) == 1
    assert _loss(head, W=(A, None)) == 1 and "W[1]" in tp.last_error()
    assert _loss(head, labels=None) == 1
    assert _loss(head, loss=None) == 1
    assert _loss(head, lse=A + 8) == 3
    assert _loss(head, dX=A) == 1 and "alias" in tp.last_error()
    assert _loss(head, dW=(A + 48, A + 16)) == 1 and "alias" in tp.last_error()
    assert _loss(head, dW=(A + 48, A + 50)) == 3
    assert _loss(tp.Plan(64, 0, 0, 2, "bf16", "none")) == 1 and "vocab" in tp.last_error()
    with pytest.raises(ValueError, match="set_vocab"):
        tp.Plan(64, 0, 0, 2, "bf16", "none").vocab_linear_cross_entropy(0, torch.zeros(0, 64).bfloat16(), [], None, 1.0, None)
    assert tp.lib.tp_vocab_linear_cross_entropy(None, 4, A, _arr(A, A), A, 1.0, A, None, None, None, 0, None) == 1
    assert _loss(head, T=0) == 0  # no token, no gradient: nothing to do


def test_loss_binding_checks_shapes_types_and_strides(head):
    X, lab, loss = torch.zeros(4, 64).bfloat16(), torch.zeros(4, dtype=torch.int32), torch.zeros(4)
    W = [torch.zeros(head.vocab_padded // 2, 64).bfloat16() for _ in range(2)]
    call = head.vocab_linear_cross_entropy
    for bad in (X.float(), torch.zeros(4, 128).bfloat16()[:, ::2], torch.zeros(5, 64).bfloat16()):
        with pytest.raises(ValueError, match="X"):
            call(4, bad, W, lab, 1.0, loss)
    with pytest.raises(ValueError, match="labels"):
        call(4, X, W, lab.long(), 1.0, loss)
    with pytest.raises(ValueError, match="loss"):
        call(4, X, W, lab, 1.0, loss.double())
    with pytest.raises(ValueError, match="2 shards"):
        call(4, X, W[:1], lab, 1.0, loss)
    with pytest.raises(ValueError, match=r"dW\[1\]"):
        call(4, X, W, lab, 1.0, loss, dW=[W[0].clone(), W[1][:8].clone()])


def _fwd(plan, kind=0, rows=8, x=A, f=A + 16, gate=None, gate_rows=0, pg=A, pb=A, qg=A, qb=A, xo=A + 32, y=A + 48, stats=None):
    return tp.lib.tp_gated_residual_norm_fwd(plan.handle, kind, rows, x, f, 1.0, gate, gate_rows, pg, pb, qg, qb, xo, y, stats, None)


def _bwd(plan, kind=0, rows=8, f=A, xo=A, stats=A, dxo=A, dy=A, gate=None, gate_rows=0, pg=A, pb=A, qg=A, dx=A + 16, df=A + 32,
         dgate=None, dpg=None, dpb=None, dqg=None, dqb=None):
    return tp.lib.tp_gated_residual_norm_bwd(plan.handle, kind, rows, f, xo, stats, dxo, dy, 1.0, gate, gate_rows, pg, pb, qg,
                                             dx, df, dgate, dpg, dpb, dqg, dqb, None)


def test_gated_norm_refusals():
    plan = tp.Plan(64, 0, 0, 1, "bf16", "none")
    assert _fwd(plan, kind=2) == 1 and "kind" in tp.last_error()
    assert _fwd(plan, rows=-1) == 1
    assert _fwd(plan, x=None) == 1 and _fwd(plan, f=A + 2) == 3 and _fwd(plan, xo=None) == 1
    assert _fwd(plan, y=None) == 1 and "y" in tp.last_error()
    assert _fwd(plan, qg=None) == 1 and "pre-norm" in tp.last_error()
    assert _fwd(plan, pb=None) == 1 and "beta_post" in tp.last_error()
    assert _fwd(plan, qb=None) == 1 and "beta_pre" in tp.last_error()
    assert _fwd(plan, y=A + 32) == 1 and "alias" in tp.last_error()
    assert _fwd(plan, stats=A + 4) == 3
    assert _fwd(plan, gate=A, gate_rows=0) == 1 and "gate_rows" in tp.last_error()
    assert _fwd(plan, gate=A, gate_rows=3) == 2 and "gate_rows = 3" in tp.last_error()
    assert _fwd(plan, rows=0, x=None, f=None, xo=None, y=None) == 0
    assert _fwd(tp.Plan(60, 0, 0, 1, "f32", "none")) == 5
    assert _fwd(tp.Plan(8200, 0, 0, 1, "f32", "none")) == 5 and "hidden <= 8192" in tp.last_error()
    assert _bwd(plan, dxo=None, dy=None) == 1 and "both NULL" in tp.last_error()
    assert _bwd(plan, qg=None) == 1 and "pre-norm" in tp.last_error()
    assert _bwd(plan, dgate=A) == 1 and "gate" in tp.last_error()
    assert _bwd(plan, pg=None, dpg=A) == 1 and _bwd(plan, qg=None, dy=None, dqg=A) == 1
    assert _bwd(plan, kind=1, dpb=A) == 1 and "RMSNorm" in tp.last_error()
    assert _bwd(plan, f=None) == 1 and _bwd(plan, xo=None) == 1 and _bwd(plan, stats=None) == 1
    assert _bwd(plan, dx=None) == 1 and _bwd(plan, df=A + 16) == 1 and "alias" in tp.last_error()
    assert _bwd(plan, rows=131074, gate=A, gate_rows=65537) == 5
    assert _bwd(plan, dqg=A + 4) == 3
    assert _bwd(plan, rows=0, f=None, xo=None, stats=None, dxo=None, dy=None, dx=None, df=None) == 0


def test_gated_norm_binding_checks():
    plan = tp.Plan(64, 0, 0, 1, "bf16", "none")
    x = torch.zeros(8, 64).bfloat16()
    w = torch.ones(64).bfloat16()
    call = plan.gated_residual_norm_fwd
    with pytest.raises(ValueError, match="x_out"):
        call("layer", 8, x, x, x.float())
    with pytest.raises(ValueError, match="post"):
        call("layer", 8, x, x, x, post=(w, None))
    with pytest.raises(ValueError, match="post"):
        call("layer", 8, x, x, x, post=(w.float(), w))
    with pytest.raises(ValueError, match="gate"):
        call("layer", 8, x, x, x, gate=w)
    with pytest.raises(ValueError, match="stats"):
        call("layer", 8, x, x, x, stats=torch.zeros(2, 8))
    with pytest.raises(KeyError):
        call("batch", 8, x, x, x)
    with pytest.raises(ValueError, match="on the CPU"):  # host memory never reaches a kernel
        call("layer", 8, x, x, x)


def _cfwd(plan, T=4, X=A, W=A, bias=None, Zq=A, Zs=A + 1, H=A):
    return tp.lib.tp_column_fwd_ckpt8(plan.handle, T, X, _arr(W), _arr(bias) if bias else None, _arr(Zq), _arr(Zs), _arr(H), None)


def _rbwd(plan, T=4, dY=A, W=A, Zq=A, Zs=A + 1, H=A, dZ=A, dW=None, dbias=None):
    return tp.lib.tp_row_bwd_ckpt8(plan.handle, T, dY, _arr(W), _arr(Zq), _arr(Zs), _arr(H) if H else None, _arr(dZ),
                                   _arr(dW) if dW else None, dbias, None)


def test_ckpt8_refusals():
    gelu = tp.Plan(64, 64, 0, 1, "bf16", "gelu")
    swiglu = tp.Plan(64, 64, 0, 1, "bf16", "swiglu")
    assert _cfwd(tp.Plan(64, 64, 0, 1, "f32", "gelu")) == 4 and "bf16" in tp.last_error()
    assert _cfwd(tp.Plan(64, 64, 0, 1, "bf16", "none")) == 1 and "activation" in tp.last_error()
    assert _cfwd(tp.Plan(64, 0, 0, 1, "bf16", "gelu")) == 1 and "MLP" in tp.last_error()
    assert _cfwd(tp.Plan(64, 72, 0, 1, "bf16", "gelu")) == 3 and "8-bit" in tp.last_error()
    assert _cfwd(swiglu, bias=A) == 1 and "bias" in tp.last_error()
    assert _cfwd(gelu, T=-1) == 1 and _cfwd(gelu, X=None) == 1 and _cfwd(gelu, W=None) == 1
    assert _cfwd(gelu, Zq=A + 8) == 3 and _cfwd(gelu, Zs=None) == 1 and _cfwd(gelu, H=None) == 1
    assert _cfwd(gelu, T=0, X=None, Zq=None, Zs=None, H=None) == 0
    assert _rbwd(gelu, dY=None) == 1 and _rbwd(gelu, dZ=None) == 1 and _rbwd(gelu, Zs=None) == 1
    assert _rbwd(gelu, H=None, dW=A) == 1 and "H" in tp.last_error()
    assert _rbwd(gelu, dbias=A + 4) == 3
    assert _rbwd(gelu, T=0, dY=None, Zq=None, Zs=None, dZ=None) == 0


def test_ckpt8_shapes_and_binding_checks():
    plan = tp.Plan(64, 2 * 1376, 0, 2, "bf16", "swiglu")
    assert plan.ckpt8_shapes(5) == ((5, 2752), (86, 5))
    assert tp.Plan(64, 80, 0, 1, "bf16", "gelu").ckpt8_shapes(7) == ((7, 80), (3, 7))
    X = torch.zeros(5, 64).bfloat16()
    W = [torch.zeros(2752, 64).bfloat16() for _ in range(2)]
    H = [torch.zeros(5, 1376).bfloat16() for _ in range(2)]
    q = [torch.zeros(5, 2752, dtype=torch.uint8) for _ in range(2)]
    s = [torch.zeros(86, 5, dtype=torch.uint8) for _ in range(2)]
    with pytest.raises(ValueError, match="Zs"):
        plan.column_fwd_ckpt8(5, X, W, None, q, [x.T.contiguous() for x in s], H)
    with pytest.raises(ValueError, match="Zq"):
        plan.column_fwd_ckpt8(5, X, W, None, [x.float() for x in q], s, H)
    with pytest.raises(ValueError, match="dZ"):
        plan.row_bwd_ckpt8(5, X, [torch.zeros(64, 1376).bfloat16()] * 2, q, s, H, H)


def test_tensors_of_one_call_are_on_one_device(monkeypatch):
    """With fakes of the device queries: a tensor on another device is refused, and the
    tensors' device is made current for the call when it is not."""
    seen, current = [], [0]

    class Lib:
        @staticmethod
        def f(*args):
            seen.append((current[-1], args))
            return 0

    class Device:
        def __init__(self, d):
            self.d = d

        def __enter__(self):
            current.append(self.d)

        def __exit__(self, *e):
            current.pop()

    monkeypatch.setattr(tp, "lib", Lib)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: current[-1])
    monkeypatch.setattr(torch.cuda, "device", Device)
    tp._on_device(1, "f", 5, "a")
    tp._on_device(0, "f", 5, "b")
    assert seen == [(1, ("a", 5)), (0, ("b", 5))]
    with pytest.raises(ValueError, match="f: the tensors are on the CPU"):
        tp._on_device(-1, "f", 5, "c")
    with pytest.raises(ValueError, match="x: .* on cuda:1, got .* on cpu"):
        tp._use(1, "x", torch.zeros(3), (3,), torch.float32)
    with pytest.raises(ValueError, match=r"W\[0\]: .* on cuda:0, got .* on cpu"):
        tp._use_shards(0, "W", [torch.zeros(3)], 1, (3,), torch.float32)


def test_outputs_that_alias_what_a_call_reads(head):
    assert _loss(head, dX=A + 32) == 1 and "W[1]" in tp.last_error()
    assert _loss(head, dW=(A + 48, A)) == 1 and "dW[1]" in tp.last_error()
    assert _loss(head, dX=A + 48, dW=(A + 48, A + 64)) == 1 and "dW[0]" in tp.last_error()
    plan = tp.Plan(64, 64, 0, 2, "bf16", "gelu")
    call = lambda H: tp.lib.tp_row_bwd_ckpt8(plan.handle, 4, A, _arr(A, A), _arr(A, A), _arr(A, A), H,  # noqa: E731
                                             _arr(A + 16, A + 32), None, None, None)
    assert call(_arr(A + 48, A + 32)) == 1 and "H[1]" in tp.last_error()


def test_a_kept_activation_is_not_shared():
    from megatron_tensor_transformer_gemm_b200.block import TPMLP
    H = [torch.zeros(4, 32).bfloat16() for _ in range(2)]
    with pytest.raises(ValueError, match="ckpt8"):
        TPMLP(64, 64, 2, device="cpu", H_scratch=H)
