"""What the router gradients refuse: grad_logits that shares a byte with an
input, null and misaligned pointers.  CPU only: no call here reaches a launch."""
import ctypes

import pytest

import moe_layer_gating_amd as moe

T, E, k = 5, 8, 2
OUT = 0x1000000
SIZES = dict(logits=T * E * 4, ids=T * k * 4, weights=T * k * 4, grad_weights=T * k * 4, mask=T,
             counts=E * 4, tokens=4, grad_loss=4)
READS = {"balance": ("logits", "mask", "counts", "tokens", "grad_loss"),
         "gating": ("logits", "ids", "weights", "grad_weights", "mask"),
         "router": tuple(SIZES)}


def _call(which, addr, out=OUT):
    L = moe.lib()
    p = {n: ctypes.c_void_p(0x2000000 + 0x10000 * i) for i, n in enumerate(SIZES)}
    p.update({n: ctypes.c_void_p(a) for n, a in addr.items()})
    g = ctypes.c_void_p(out)
    if which == "balance":
        return L.moe_balance_loss_backward(p["logits"], p["mask"], p["counts"], p["tokens"], T, E,
                                           k, 1.0, p["grad_loss"], g, None)
    if which == "gating":
        return L.moe_topk_gating_backward(p["logits"], p["ids"], p["weights"], p["grad_weights"],
                                          p["mask"], T, E, k, 0, g, None)
    return L.moe_router_backward(p["logits"], p["ids"], p["weights"], p["grad_weights"], p["mask"],
                                 p["counts"], p["tokens"], T, E, k, 1, 1.0, p["grad_loss"], g, None)


@pytest.mark.parametrize("which,name", [(w, n) for w, names in READS.items() for n in names])
def test_a_gradient_over_its_input_is_refused(which, name):
    """The input starts in the gradient's last 16 bytes, inside it, with it; and
    the gradient starts in the input's last 16-byte step."""
    nbytes = T * E * 4
    for a in (OUT + nbytes - 16, OUT + 32, OUT):
        assert _call(which, {name: a}) == -1, hex(a)
    last = (SIZES[name] - 1) // 16 * 16
    assert _call(which, {name: OUT - last}) == -1


@pytest.mark.parametrize("which,name", [(w, n) for w, names in READS.items() for n in names])
def test_null_and_misaligned_inputs_are_refused(which, name):
    """With every argument at an address of its own.  E = 8: counts are read 16
    bytes at a time; the one-word values need 4 bytes."""
    at = 0x2000000 + 0x10000 * list(SIZES).index(name)
    if name != "mask":
        assert _call(which, {name: None}) == -1
    for off in (1, 2) if name in ("tokens", "grad_loss") else (1, 4, 8):
        assert _call(which, {name: at + off}) == -1, off
    for out in (None, OUT + 4, OUT + 8):
        assert _call(which, {}, out) == -1
