"""A logit of +inf in the gradient of the gating weights: its row is NaN under
both weight rules, rows without a finite logit and masked rows stay zero."""
import numpy as np
import pytest
import torch

import moe_layer_gating_amd as moe
from gpu_helpers import say

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("renorm", [True, False])
@pytest.mark.parametrize("E,k", [(4, 1), (16, 2), (61, 6), (256, 8), (300, 5), (390, 16),
                                 (1024, 16)])
def test_rows_with_plus_infinity_are_nan(E, k, renorm):
    """The weights are the gating's own, NaN in every row without a finite
    maximum.  35000 rows: also the rows a lane group reaches in later rounds."""
    say("+inf in the gating gradient", E, k, renorm)
    T = 35000 if E <= 61 else 9000
    g = np.random.default_rng(E)
    logits = g.standard_normal((T, E)).astype(np.float32)
    dev = lambda a: torch.from_numpy(a).cuda()
    gw, mask = dev(g.standard_normal((T, k)).astype(np.float32)), np.ones(T, np.uint8)
    bad = np.array([0, 17, 18, 40, T // 2, T - 1])
    empty, masked = np.array([20, 41, T - 3]), np.array([21, 22, T - 2])
    mask[masked] = 0
    mask = dev(mask)

    def grads(l):
        ids, w = moe.moe_topk_gating(l, k, renormalize=renorm)
        _, counts, _, n = moe.moe_balance_loss(l, ids, 1.0, token_mask=mask)
        one = torch.ones(1, device="cuda")
        return [a.cpu().numpy() for a in (
            moe.moe_topk_gating_backward(l, ids, w, gw, renormalize=renorm, token_mask=mask),
            moe.moe_router_backward(l, ids, w, gw, counts, n, 1.0, one, renormalize=renorm,
                                    token_mask=mask))]

    clean = grads(dev(logits))
    for i, t in enumerate(bad):
        logits[t, (7 * i) % E] = np.inf
    logits[40] = np.inf               # nothing but +inf
    logits[18, : E // 2] = -np.inf    # -inf and NaN beside it
    logits[18, E // 2] = np.nan
    logits[18, E - 1] = np.inf
    logits[empty] = -np.inf
    logits[empty[1], 0] = np.nan
    logits[masked, 0] = np.inf
    got = grads(dev(logits))
    same = np.setdiff1d(np.arange(T), np.r_[bad, empty, masked])
    for a in got:
        assert np.all(np.isnan(a[bad]))
        assert np.all(a[masked] == 0)
    assert np.all(got[0][empty] == 0)
    assert np.all(np.isfinite(got[1][empty]))
    assert np.array_equal(got[0][same], clean[0][same])  # a row's own logits only


def test_without_logits_a_nan_weight_counts_as_zero():
    """The renormalised form may be called without logits, through the C ABI."""
    T, E, k = 5, 12, 3
    ids = torch.arange(T * k, dtype=torch.int32, device="cuda").view(T, k) % E
    w, gw = torch.full((T, k), 0.25, device="cuda"), torch.ones(T, k, device="cuda")
    w[1], w[3, 1] = np.nan, np.nan
    grad = torch.full((T, E), 7.0, device="cuda")
    p = [t.data_ptr() for t in (ids, w, gw)]
    assert moe.lib().moe_topk_gating_backward(None, *p, None, T, E, k, 1, grad.data_ptr(),
                                              torch.cuda.current_stream().cuda_stream) == 0
    ok = torch.nan_to_num(w)
    s = ok.sum(1, keepdim=True)  # quarters: every sum and product below is exact
    want = torch.zeros_like(grad).scatter_(1, ids.long(), ok - ok * s)
    assert torch.equal(grad, want)
