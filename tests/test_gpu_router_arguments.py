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


@pytest.mark.parametrize("E", [61, 64])
@pytest.mark.parametrize("dtype", [torch.uint8, torch.bool])
def test_slices_of_masks_and_of_per_layer_values(E, dtype):
    """A slice of a longer mask, elements of per-layer losses, token counts and
    loss gradients, and rows of per-layer counts and probabilities (of 61
    experts at any 4-byte address) give what buffers of their own give, and
    nothing beside them is written."""
    T, k, layers = 45, 4, 5
    logits, ids, w, gw = _batch(T, E, k)
    long_mask = torch.rand(4 * T, generator=torch.Generator().manual_seed(1)).lt(0.6).to(dtype).cuda()
    losses = torch.full((layers,), 7.0, device="cuda")
    tokens = torch.full((layers,), 7, dtype=torch.int32, device="cuda")
    counts = torch.full((layers, E), 7, dtype=torch.int32, device="cuda")
    probs = torch.full((layers, E), 7.0, device="cuda")
    dl = torch.rand(layers, device="cuda")
    grad = torch.empty(T, E, device="cuda")
    for i, start in ((1, 1), (2, 2), (3, 7), (4, 16)):
        mask = long_mask[start:start + T]
        own = mask.clone()
        want = moe.moe_balance_loss(logits, ids, 0.5, token_mask=own)
        part = slice(i, i + 1)
        got = moe.moe_balance_loss(logits, ids, 0.5, token_mask=mask, loss=losses[part],
                                   expert_counts=counts[i], expert_probs=probs[i],
                                   token_count=tokens[part])
        assert all(torch.equal(a, b) for a, b in zip(got, want))
        args = (counts[i], tokens[part], k, 0.5, dl[part])
        moe.moe_balance_loss_backward(logits, *args, token_mask=mask, grad_logits=grad)
        own_args = (want[1], want[3], k, 0.5, dl[part].clone())
        assert torch.equal(grad, moe.moe_balance_loss_backward(logits, *own_args, token_mask=own))
        for renorm in (True, False):
            for call, more, own_more in (
                    (moe.moe_topk_gating_backward, (), ()),
                    (moe.moe_router_backward, (counts[i], tokens[part], 0.5, dl[part]),
                     (want[1], want[3], 0.5, dl[part].clone()))):
                a = call(logits, ids, w, gw, *more, renormalize=renorm, token_mask=mask)
                b = call(logits, ids, w, gw, *own_more, renormalize=renorm, token_mask=own)
                assert torch.equal(a, b)
    for t in (losses, tokens, counts, probs):
        assert bool((t[0] == 7).all())


def test_a_mask_slice_in_a_captured_graph():
    """The copy of an unaligned mask is part of the graph: replays see the
    mask's present values."""
    T, E, k = 70, 32, 2
    logits, ids, _, _ = _batch(T, E, k)
    base = torch.ones(T + 3, dtype=torch.uint8, device="cuda")
    mask = base[3:]
    ws = moe.balance_loss_workspace(T, k, E)
    out = dict(loss=torch.empty(1, device="cuda"), expert_probs=torch.empty(E, device="cuda"),
               expert_counts=torch.empty(E, dtype=torch.int32, device="cuda"),
               token_count=torch.empty(1, dtype=torch.int32, device="cuda"))
    moe.moe_balance_loss(logits, ids, token_mask=mask, ws=ws, **out)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        moe.moe_balance_loss(logits, ids, token_mask=mask, ws=ws, **out)
    for live in (70, 33, 0, 51):
        base.zero_()
        base[3:3 + live] = 1
        graph.replay()
        torch.cuda.synchronize()
        got = [out[n].clone() for n in ("loss", "expert_counts", "expert_probs", "token_count")]
        want = moe.moe_balance_loss(logits, ids, token_mask=mask.clone())
        assert int(out["token_count"]) == live
        assert all(torch.equal(a, b) for a, b in zip(got, want))
