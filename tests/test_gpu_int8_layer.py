"""The INT8 layer holds the down projection's outputs in fp32 until they are
aggregated, however many tokens share the call: the fused call equals the
steps bit for bit and lies within one rounding to bf16 of the 64-bit value,
and a token's output does not depend on the size of its batch."""
import numpy as np
import pytest
import torch

import moe_layer_gating_amd as moe
import plain64 as P
from gpu_helpers import say
from test_gpu_int8 import _dev, _grouping, _layer, _np, _within

pytestmark = pytest.mark.gpu

# T, H, E, k, I: T k H below and above 2^24, 64- and 256-position tiles; the
# last groups its pairs in chunks with k = 8
SIZES = [(2050, 2048, 5, 2, 128), (4100, 2048, 5, 2, 128), (4100, 2048, 5, 2, 1024),
         (1030, 2048, 16, 8, 128), (2100, 1024, 12, 8, 1664)]


@pytest.mark.parametrize("T,H,E,k,I", SIZES)
def test_outputs_are_rounded_once(T, H, E, k, I):
    """Against the 64-bit aggregation of the integer products of the codes of
    h.  y rounds three times (conversion, product of the scales, product with
    it), the aggregation twice per slot, relative to the sum of |w y|; the
    output rounds to bf16 once."""
    say("fused int8 layer", T, H, E, k, I)
    x, logits, w13, s13, w2, s2 = _layer(T, H, E, k, I, 0.3, 8)
    ids, order, offsets, inv = _grouping(logits, k)
    dx, dl, d13, d2, ds13, ds2 = x.cuda(), _dev(logits), _dev(w13), _dev(w2), _dev(s13), _dev(s2)
    h, _ = moe.moe_grouped_gemm_w13_swiglu(dx, d13, ds13, _dev(order), _dev(offsets), k)
    y = moe.moe_grouped_gemm_w2(h, d2, ds2, _dev(offsets), None, k)
    gw = moe.moe_topk_gating(dl, k)[1]
    out = moe.moe_fused_forward(dx, dl, d13, ds13, d2, ds2, k)
    assert torch.equal(out, moe.moe_combine(y, _dev(inv), gw, moe.MOE_INT8, E=E, I=I))
    tokens = np.r_[0:20, T // 2:T // 2 + 20, T - 20:T]
    rows = inv.reshape(T, k)[tokens].reshape(-1)
    e = P.expert_of(offsets, T * k)[rows]
    codes, s = P.quant_i8(_np(h)[rows])
    y64 = np.stack([w2[e[i]].astype(np.float64) @ codes[i].astype(np.float64)
                    for i in range(rows.size)])
    y64 *= s.astype(np.float64)[:, None] * s2.astype(np.float64)[e]
    terms = y64.reshape(tokens.size, k, H) * _np(gw)[tokens][:, :, None]
    want, size = terms.sum(1), np.abs(terms).sum(1)
    bound = np.abs(want) * P.U_BF16 * 1.001 + size * (2 * k + 4) * P.U * 1.01 + 2.0 ** -126
    _within(_np(out)[tokens], want, bound, "out")


@pytest.mark.parametrize("T,H,E,k,I", SIZES[1:])
def test_a_token_does_not_depend_on_its_batch(T, H, E, k, I):
    """The first 700 tokens alone and among all of them (both sizes run in
    tiles, whose formula is one)."""
    say("batches of one int8 layer", T, H, E, k, I)
    x, logits, w13, s13, w2, s2 = _layer(T, H, E, k, I, 0.3, 9)
    w = (_dev(w13), _dev(s13), _dev(w2), _dev(s2), k)
    dx, dl = x.cuda(), _dev(logits)
    few = moe.moe_fused_forward(dx[:700].clone(), dl[:700].clone(), *w)
    assert torch.equal(moe.moe_fused_forward(dx, dl, *w)[:700], few)
