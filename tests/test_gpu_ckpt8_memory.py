"""What an MLP with 8-bit checkpoints holds on the device between its passes."""
import gc

import pytest
import torch

from gpu_helpers import dev

pytestmark = pytest.mark.gpu
T, H_, F_, P = 1024, 256, 2048, 2


def _held():
    gc.collect()
    torch.cuda.synchronize()
    return torch.cuda.memory_allocated()


@pytest.mark.parametrize("act", ["swiglu", "gelu"])
def test_only_codes_and_scales_stay_between_the_passes(act):
    """Between the passes and after the backward the layer has the codes and scales (1.03 bytes a
    pre-activation element), Y, dX and the weights' gradients; H and dZ (2 bytes an element each)
    only within a pass. Allocations are whole multiples of 512 bytes."""
    from megatron_tensor_transformer_gemm_b200.block import TPMLP
    n1 = (2 if act == "swiglu" else 1) * F_
    m = TPMLP(H_, F_, P, act, "bf16", fused=True, ckpt8=True)
    g = torch.Generator().manual_seed(1)
    m.load_weights(dev(torch.randn(n1, H_, generator=g).bfloat16() * 0.05), dev(torch.randn(H_, F_, generator=g).bfloat16() * 0.05))
    X, dY = dev(torch.randn(T, H_, generator=g).bfloat16()), dev(torch.randn(T, H_, generator=g).bfloat16())
    before = _held()
    m.forward(X)
    between = _held() - before
    m.backward(dY)
    after = _held() - before
    kept = T * n1 + (T * n1) // 32                        # codes, scales
    rest = 2 * (2 * T * H_ + n1 * H_ + H_ * F_)           # Y, dX, dW1, dW2
    assert between <= kept + rest + 64 * 512, (between, kept, rest)
    assert after <= kept + rest + 64 * 512, (after, kept, rest)
    # the same passes again, and in a graph, give the same bits
    want = [t.clone() for t in (m.Y, m.dX, *m.dW1, *m.dW2)]
    m.forward(X)
    m.backward(dY)
    assert all(torch.equal(a, b) for a, b in zip((m.Y, m.dX, *m.dW1, *m.dW2), want))
    from megatron_tensor_transformer_gemm_b200.block import CapturedStep
    step = CapturedStep(lambda: (m.forward(X), m.backward(dY)))
    other = torch.randn(64 << 20, device="cuda")          # eager allocations beside the graph's own
    for _ in range(2):
        for t in (m.Y, m.dX, *m.dW1, *m.dW2):
            t.zero_()
        step()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip((m.Y, m.dX, *m.dW1, *m.dW2), want))
    assert bool(torch.isfinite(other).all())


@pytest.mark.parametrize("fused,chunks", [(True, 0), (False, 0), (False, 4)])
def test_deferred_weight_gradients_read_what_is_still_there(fused, chunks):
    """With deferred weight gradients dZ is read after backward() has returned: allocations made
    in between do not get its memory."""
    from megatron_tensor_transformer_gemm_b200 import tp
    from megatron_tensor_transformer_gemm_b200.block import TPMLP
    g = torch.Generator().manual_seed(2)
    W1, W2 = dev(torch.randn(2 * F_, H_, generator=g).bfloat16() * 0.05), dev(torch.randn(H_, F_, generator=g).bfloat16() * 0.05)
    X, dY = dev(torch.randn(T, H_, generator=g).bfloat16()), dev(torch.randn(T, H_, generator=g).bfloat16())
    outs = []
    for defer in (False, True):
        m = TPMLP(H_, F_, P, "swiglu", "bf16", fused=fused, overlap_chunks=chunks, ckpt8=True)
        m.load_weights(W1, W2)
        m.plan.set_backward_defer(defer)
        for _ in range(3):
            m.forward(X)
            m.backward(dY)
            junk = [torch.full((T, 2 * F_ // P), 1e4, dtype=torch.bfloat16, device="cuda") for _ in range(4)]
            tp.backward_join()
            del junk
        torch.cuda.synchronize()
        outs.append([t.clone() for t in (m.Y, m.dX, *m.dW1, *m.dW2)])
    # dX and Y in the same order either way; dW1 and dW2 without a K split when deferred
    for a, b in zip(*outs):
        assert float((a.double() - b.double()).norm() / a.double().norm()) <= 2.0 ** -7
    assert all(torch.equal(a, b) for a, b in zip(outs[0][:2], outs[1][:2]))


def test_shared_scratch_is_used():
    from megatron_tensor_transformer_gemm_b200.block import TPMLP
    g = torch.Generator().manual_seed(3)
    H = [torch.full((T, F_ // P), 7.0, dtype=torch.bfloat16, device="cuda") for _ in range(P)]
    m = TPMLP(H_, F_, P, "gelu", "bf16", fused=True, ckpt8=True, H_scratch=H)
    m.load_weights(dev(torch.randn(F_, H_, generator=g).bfloat16() * 0.05), dev(torch.randn(H_, F_, generator=g).bfloat16() * 0.05))
    m.forward(dev(torch.randn(T, H_, generator=g).bfloat16()))
    assert not bool((H[0] == 7).all())
