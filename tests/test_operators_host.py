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
