"""Host-side checks of the router-training and INT8 entry points: refused
before anything is enqueued.  CPU only: no call here reaches a launch."""
import ctypes

import pytest
import torch

import moe_layer_gating_amd as moe

GOOD, ODD, WS = ctypes.c_void_p(0x100000), ctypes.c_void_p(0x100004), ctypes.c_void_p(0x200000)


@pytest.fixture(scope="module")
def L():
    return moe.lib()


@pytest.mark.parametrize("shape,want", [
    ((4, 256, 8, 2, 256, 4), 0),
    ((0, 128, 8, 2, 256, 4), 0),
    ((4, 256, 8, 2, 200, 4), -2),
    ((4, 131072, 8, 2, 131072, 4), 0),
    ((4, 131200, 8, 2, 256, 4), -2),   # an int8 sum could overflow
    ((4, 256, 8, 2, 131200, 4), -2),
    ((4, 131200, 8, 2, 256, 1), 0),    # other modes as before
    ((4, 256, 8, 2, 256, 5), -1),
    ((4, 256, 8, 2, 256, -1), -1),
])
def test_int8_shapes(L, shape, want):
    s = moe.make_shape(*shape)
    assert moe.moe_check_shape(s) == want
    assert (moe.moe_workspace_bytes(s) > 0) == (want == 0)


def test_routing_offsets_do_not_depend_on_the_mode(L):
    a, b = (moe.moe_workspace_routing(moe.make_shape(300, 512, 16, 4, 256, m)) for m in (2, 4))
    assert [getattr(a, f) for f, _ in a._fields_] == [getattr(b, f) for f, _ in b._fields_]


def test_int8_products_refuse(L):
    s = moe.make_shape(4, 256, 8, 2, 256, moe.MOE_INT8)
    S, need = ctypes.byref(s), moe.moe_workspace_bytes(s)
    w13, w2 = L.moe_grouped_gemm_w13_swiglu, L.moe_grouped_gemm_w2
    assert w13(S, GOOD, GOOD, None, GOOD, GOOD, GOOD, None, WS, need, None) == -1  # no scales
    assert w13(S, GOOD, GOOD, ODD, GOOD, GOOD, GOOD, None, WS, need, None) == -1
    assert w13(S, GOOD, GOOD, GOOD, GOOD, GOOD, GOOD, None, WS, need - 1, None) == -3
    assert w13(S, None, GOOD, GOOD, GOOD, GOOD, GOOD, None, WS, need, None) == -1
    assert w2(S, GOOD, GOOD, None, GOOD, None, GOOD, WS, need, None) == -1
    assert w2(S, GOOD, GOOD, ODD, GOOD, None, GOOD, WS, need, None) == -1
    assert w2(S, GOOD, GOOD, GOOD, GOOD, None, GOOD, None, need, None) == -3
    assert L.moe_fused_forward(S, GOOD, GOOD, GOOD, GOOD, GOOD, None, GOOD, None, None, WS, need,
                               None) == -1
    assert L.moe_fused_forward(S, GOOD, GOOD, GOOD, None, GOOD, GOOD, GOOD, None, None, WS, need,
                               None) == -1


def test_row_codes_refuse(L):
    f = L.moe_act_quant_i8
    assert f(None, 4, 64, GOOD, GOOD, None) == -1
    assert f(GOOD, 4, 64, None, GOOD, None) == -1
    assert f(GOOD, 4, 64, GOOD, None, None) == -1
    assert f(ODD, 4, 64, GOOD, GOOD, None) == -1
    assert f(GOOD, 4, 64, GOOD, ODD, None) == -1
    assert f(GOOD, 4, 60, GOOD, GOOD, None) == -1
    assert f(GOOD, 4, 0, GOOD, GOOD, None) == -1
    assert f(GOOD, -1, 64, GOOD, GOOD, None) == -1
    assert f(GOOD, 1 << 31, 64, GOOD, GOOD, None) == -1
    assert f(None, 0, 64, None, None, None) == 0


def test_balance_loss_refuses(L):
    f, need = L.moe_balance_loss, moe.moe_balance_loss_workspace_bytes(300, 2, 8)
    assert need > 0 and moe.moe_balance_loss_workspace_bytes(0, 2, 8) > 0
    assert moe.moe_balance_loss_workspace_bytes(300, 9, 8) == 0
    assert moe.moe_balance_loss_workspace_bytes(-1, 2, 8) == 0

    def call(logits=GOOD, ids=GOOD, mask=None, T=300, E=8, k=2, loss=GOOD, counts=GOOD, probs=GOOD,
             tokens=GOOD, ws=WS, n=need):
        return f(logits, ids, mask, T, E, k, 1.0, loss, counts, probs, tokens, ws, n, None)

    for bad in (dict(logits=None), dict(ids=None), dict(loss=None), dict(counts=None),
                dict(probs=None), dict(tokens=None), dict(logits=ODD), dict(mask=ODD),
                dict(probs=ODD), dict(T=-1), dict(E=0), dict(E=1025), dict(k=0), dict(k=9),
                dict(T=0, loss=None)):
        assert call(**bad) == -1, bad
    for bad in (dict(ws=None), dict(ws=ctypes.c_void_p(0x200010)), dict(n=need - 1),
                dict(T=0, ws=None)):
        assert call(**bad) == -3, bad


def test_gradients_refuse(L):
    b, g, r = L.moe_balance_loss_backward, L.moe_topk_gating_backward, L.moe_router_backward
    assert b(GOOD, None, GOOD, GOOD, 4, 8, 2, 1.0, None, GOOD, None) == -1
    assert b(GOOD, None, None, GOOD, 4, 8, 2, 1.0, GOOD, GOOD, None) == -1
    assert b(GOOD, ODD, GOOD, GOOD, 4, 8, 2, 1.0, GOOD, GOOD, None) == -1
    assert b(GOOD, None, GOOD, GOOD, 4, 8, 9, 1.0, GOOD, GOOD, None) == -1
    assert b(None, None, None, None, 0, 8, 2, 1.0, None, None, None) == 0
    assert g(None, GOOD, GOOD, GOOD, None, 4, 8, 2, 0, GOOD, None) == -1  # softmax needs logits
    assert g(GOOD, GOOD, GOOD, GOOD, None, 4, 8, 2, 2, GOOD, None) == -1
    assert g(GOOD, None, GOOD, GOOD, None, 4, 8, 2, 1, GOOD, None) == -1
    assert g(GOOD, GOOD, GOOD, ODD, None, 4, 8, 2, 1, GOOD, None) == -1
    assert g(None, None, None, None, None, 0, 8, 2, 1, None, None) == 0
    assert r(GOOD, GOOD, GOOD, GOOD, None, GOOD, GOOD, 4, 8, 2, 1, 1.0, None, GOOD, None) == -1
    assert r(None, GOOD, GOOD, GOOD, None, GOOD, GOOD, 4, 8, 2, 1, 1.0, GOOD, GOOD, None) == -1
    assert r(GOOD, GOOD, GOOD, GOOD, None, GOOD, GOOD, 4, 8, 2, 1, 1.0, GOOD, ODD, None) == -1
    assert r(GOOD, GOOD, GOOD, GOOD, None, GOOD, GOOD, 4, 8, 2, 3, 1.0, GOOD, GOOD, None) == -1
    assert r(None, None, None, None, None, None, None, 0, 8, 2, 1, 1.0, None, None, None) == 0


def test_binding_refuses_host_tensors(L):
    with pytest.raises(moe.MoeError):
        moe.moe_act_quant_i8(torch.zeros(2, 64, dtype=torch.bfloat16))
    with pytest.raises(moe.MoeError):
        moe.moe_balance_loss(torch.zeros(2, 4), torch.zeros(2, 1, dtype=torch.int32))
    with pytest.raises(moe.MoeError):
        moe.moe_fused_forward(torch.zeros(2, 128).bfloat16(), torch.zeros(2, 4),
                              torch.zeros(4, 256, 128, dtype=torch.int8), torch.zeros(4, 256),
                              torch.zeros(4, 128, 128, dtype=torch.int8), torch.zeros(4, 128), 1)
