"""Which buffers the router's training step takes from Python."""
import pytest
import torch

import moe_layer_gating_amd as moe

pytestmark = pytest.mark.gpu


def _batch(T, E, k, seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    logits = torch.randn(T, E, generator=g, device="cuda")
    ids, w = moe.moe_topk_gating(logits, k)
    return logits, ids, w, torch.randn(T, k, generator=g, device="cuda")


def test_a_gradient_over_its_input_is_refused():
    T, E, k = 6, 8, 2
    buf = torch.randn(T * E + 4, device="cuda")
    logits, over = buf[:T * E].view(T, E), buf[4:].view(T, E)
    _, ids, w, gw = _batch(T, E, k)
    _, counts, _, n = moe.moe_balance_loss(logits, ids)
    one = torch.ones(1, device="cuda")
    keep = buf.clone()
    for grad in (over, logits):
        with pytest.raises(moe.MoeError):
            moe.moe_balance_loss_backward(logits, counts, n, k, 1.0, one, grad_logits=grad)
        with pytest.raises(moe.MoeError):
            moe.moe_topk_gating_backward(logits, ids, w, gw, grad_logits=grad)
        with pytest.raises(moe.MoeError):
            moe.moe_router_backward(logits, ids, w, gw, counts, n, 1.0, one, grad_logits=grad)
    assert torch.equal(buf, keep)
    # beside the input is fine
    buf = torch.empty(2 * T * E, device="cuda")
    buf[:T * E] = keep[:T * E]
    logits, grad = buf[:T * E].view(T, E), buf[T * E:].view(T, E)
    moe.moe_router_backward(logits, ids, w, gw, counts, n, 1.0, one, grad_logits=grad)
    want = moe.moe_router_backward(logits, ids, w, gw, counts, n, 1.0, one)
    assert torch.equal(grad, want) and torch.equal(buf[:T * E], keep[:T * E])
