"""The router kernels over batches whose rows take several rounds of their
pipelined loops, every probability and gradient row against plain64: each lane
width (16, 32, 64), vector and scalar loads, with and without a mask, both
weight rules."""
import numpy as np
import pytest
import torch

import moe_layer_gating_amd as moe
import plain64 as P
from gpu_helpers import say
from test_gpu_router_loss import _dev, _rows_in_a_row, _within

pytestmark = pytest.mark.gpu

# A launch takes 16384, 8192 or 4096 rows of the loss and 32768, 16384 or 8192
# of the gradient at a time (16, 32 and 64 lanes a row): 3 to 5 rounds of the
# one and 2 or 3 of the other, the last of them partly empty.
SHAPES = [(49999, 61, 6), (33001, 64, 8), (66001, 100, 4), (40001, 127, 7), (65600, 256, 8),
          (33001, 255, 3), (33001, 390, 5), (20000, 512, 16), (17001, 1024, 16), (9001, 777, 9)]


@pytest.mark.parametrize("masked", [False, True])
@pytest.mark.parametrize("T,E,k", SHAPES)
def test_every_row(T, E, k, masked):
    say("rows of several rounds", T, E, k, masked)
    g = np.random.default_rng(T + E)
    logits = (2 * g.standard_normal((T, E), dtype=np.float32) +
              g.standard_normal(E, dtype=np.float32))
    ids = ((g.integers(0, E, (T, 1)) + np.arange(k) * max(1, E // 17)) % E).astype(np.int32)
    w = g.random((T, k), dtype=np.float32)
    gw = g.standard_normal((T, k), dtype=np.float32)
    mask = (g.random(T) < 0.7).astype(np.uint8) if masked else None
    coef, gl = float(np.float32(0.25)), 1.5
    dl, di, dw, dg, dm = (_dev(a) for a in (logits, ids, w, gw, mask))
    dgl = torch.full((1,), gl, device="cuda")
    loss, counts, probs, tokens = moe.moe_balance_loss(dl, di, coef, token_mask=dm)
    bal = moe.moe_balance_loss_backward(dl, counts, tokens, k, coef, dgl, token_mask=dm)
    wl, wc, wp, n = P.balance_loss(logits, ids, coef, mask)
    assert np.array_equal(counts.cpu().numpy(), wc) and int(tokens) == n
    pb = P.probs_bound(logits, wp, n, _rows_in_a_row(T))
    _within(probs.cpu().numpy(), wp, pb, "probabilities")
    lb = coef * E * float((wc / (n * k)) @ pb) + abs(wl) * 2 * P.U
    _within(loss.cpu().numpy(), np.array([wl]), lb, "loss")
    b = P.balance_grad(logits, wc, n, k, coef, gl, mask)
    b_bound = P.balance_grad_bound(logits, wc, n, k, coef, gl)
    _within(bal.cpu().numpy(), b, b_bound, "balance gradient")
    for renorm in (True, False):
        args = (dl, di, dw, dg)
        a = P.gating_grad(logits, ids, w, gw, renorm, mask)
        a_bound = P.gating_grad_bound(logits, ids, w, gw, renorm)
        got = moe.moe_topk_gating_backward(*args, renormalize=renorm, token_mask=dm)
        _within(got.cpu().numpy(), a, a_bound, "gating gradient")
        got = moe.moe_router_backward(*args, counts, tokens, coef, dgl, renormalize=renorm,
                                      token_mask=dm)
        # the sum of the two rounds twice more
        bound = a_bound + b_bound + 2 * P.U * (np.abs(a) + np.abs(b))
        _within(got.cpu().numpy(), a + b, bound, "router gradient")


def test_mean_probabilities_of_rows_past_two_to_the_31_bytes():
    """147 rounds of the loss: each expert's mean against a 64-bit softmax."""
    say("rows past 2^31 bytes")
    T, E, k = 600_001, 1000, 2
    gen = torch.Generator(device="cuda").manual_seed(4)
    logits = torch.randn(T, E, generator=gen, device="cuda")
    ids = torch.randint(0, E, (T, k), generator=gen, device="cuda", dtype=torch.int32)
    probs = moe.moe_balance_loss(logits, ids)[2]
    want = torch.zeros(E, dtype=torch.float64, device="cuda")
    for lo in range(0, T, 50_000):
        want += torch.softmax(logits[lo:lo + 50_000].double(), 1).sum(0)
    want = (want / T).cpu().numpy()
    spread = np.zeros((1, E), np.float32)  # a row as far apart as any of them
    spread[0, 0] = float(logits.max() - logits.min())
    _within(probs.cpu().numpy(), want, P.probs_bound(spread, want, T, _rows_in_a_row(T)), "mean")
