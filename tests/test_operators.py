"""The measured operators' plain forms and the library's calls against the
64-bit values that perf/operators.py computes apart from both."""
import random

import numpy as np
import pytest
import torch

import perf.operators as O
import plain64 as P
from gpu_helpers import say

SMALL = [dict(kind="balance", T=1, E=1, k=1, mask=False), dict(kind="balance", T=37, E=12, k=3, mask=True),
         dict(kind="balance", T=200, E=64, k=8, mask=False),
         dict(kind="router", T=50, E=16, k=4, mask=True, renorm=True, balance=True),
         dict(kind="router", T=50, E=61, k=6, mask=True, renorm=False, balance=True),
         dict(kind="router", T=9, E=5, k=5, mask=False, renorm=True, balance=False),
         dict(kind="router", T=31, E=20, k=2, mask=False, renorm=False, balance=False),
         dict(kind="w13", T=1, H=128, E=4, k=1, I=128), dict(kind="w13", T=40, H=128, E=3, k=2, I=256),
         dict(kind="w2", T=1, H=128, E=4, k=2, I=128), dict(kind="w2", T=33, H=256, E=5, k=3, I=128),
         dict(kind="layer", T=1, H=128, E=4, k=2, I=128), dict(kind="layer", T=60, H=128, E=6, k=3, I=128)]


def _case(c):
    return dict(dict(mask=False, renorm=True, balance=True), **c) if c["kind"] in ("balance", "router") else c


def _id(c):
    return c.get("name") or "_".join(str(v) for v in c.values())


def _outputs(v):
    return list(v) if isinstance(v, (tuple, list)) else [v]


def _np(t):
    return None if t is None else t.detach().double().cpu().numpy()


def _router_size(s, c):
    """Sum of the magnitudes of the terms of each gradient value."""
    logits = _np(s["logits"])
    T, E = logits.shape
    p, k = P.softmax(logits), c["k"]
    size = np.zeros((T, E))
    if c["kind"] == "balance" or c["balance"]:
        n = max(1, int(s["tokens"]))
        f = _np(s["counts"]) / (n * k)
        size += s["coef"] * E * float(s["grad_loss"]) / n * p * (f + (p @ f)[:, None])
    if c["kind"] == "router":
        w, g, ids = _np(s["weights"]), _np(s["grad_weights"]), s["ids"].cpu().numpy()
        wg = np.abs(w * g)
        own = np.zeros((T, E))
        rows = np.arange(T)[:, None]
        own[rows, ids] = wg + (np.abs(w) * wg.sum(1, keepdims=True) if c["renorm"] else 0)
        size += own if c["renorm"] else own + p * wg.sum(1, keepdims=True)
    return size


def _check(c, seed, own):
    """Runs a case and holds its outputs to the 64-bit values: router values
    within the roundings of their softmax (2 (spread + 4), E additions) and of 8
    products, relative to their terms, twice where a product of two of them
    enters, means over T rows also within T additions (the kernel: 13 and one
    for every 4096 rows, in a lane, wave and block); products within the 4 roundings of
    their scales (sums of codes are exact: integers in the kernels, below 2^24
    in the plain form at K <= 256); h within those of SiLU (432 fp32 steps at
    |g| <= 104) and its rounding to bf16.  A layer's output rounds to bf16 once
    (2^-8), and the values of h that round the other way, at most a share of
    2 * 432 U / 2^-7 of them by 2^-7 each, add less than 2^-10 to its norm."""
    s = O.prepare(c, seed)
    try:
        O.own = own
        got = [_np(t) for t in _outputs(O.run(s))]
    finally:
        O.own = False
    want = [_np(t) for t in _outputs(O.exact(c, seed))]
    assert len(got) == len(want)
    kind = c["kind"]
    if kind in ("balance", "router"):
        logits = _np(s["logits"])
        spread = float(logits.max() - logits.min())
        rel = (2 * (spread + 4) + c["E"] + 8) * P.U * 1.01
        grad = 2 * rel * _router_size(s, c) + 2.0 ** -126
        if kind == "balance":
            assert np.array_equal(got[1], _np(s["counts"])) and got[3] == _np(s["tokens"])
            mean = rel + (13 + c["T"] / 4096 if own else c["T"]) * P.U * 1.01
            bounds = [2 * mean * np.abs(want[0]), None, mean * want[2] + 2.0 ** -126, None, grad]
        else:
            bounds = [grad]
    elif kind == "w2":
        bounds = [np.abs(want[0]) * 4 * P.U + 2.0 ** -126]
    elif kind == "w13":
        bounds = [np.abs(want[0]) * (P.U_BF16 * 1.001 + 432 * P.U) + 2.0 ** -120]
    else:
        assert np.array_equal(got[1], s["ids"].cpu().numpy())
        off = np.linalg.norm(got[0] - want[0]) / np.linalg.norm(want[0])
        assert off <= 2.0 ** -8 + 2.0 ** -10, off
        return
    for g, w, b in zip(got, want, bounds):
        if b is not None:
            worst = float(np.max(np.abs(g - w) / b))
            assert worst <= 1.0, "%.3f of its bound" % worst


@pytest.mark.parametrize("c", SMALL, ids=_id)
def test_plain_forms_against_64_bits(c):
    _check(_case(c), 3, own=False)


def test_drawn_cases_are_of_the_listed_ranges():
    rng = random.Random(1)
    seen = [O.draw(rng) for _ in range(60)]
    assert len({_id(c) for c in seen}) == 60
    assert {c["kind"] for c in seen} == {c["kind"] for c in O.listed()}
    assert all("name" not in c for c in seen)


@pytest.mark.gpu
@pytest.mark.parametrize("c", [_case(c) for c in SMALL] + O.listed(), ids=_id)
def test_library_calls_against_64_bits(c):
    say("operator", _id(c))
    _check(c, 5, own=True)
    torch.cuda.empty_cache()


@pytest.mark.gpu
@pytest.mark.parametrize("draw", range(8))
def test_library_calls_of_drawn_cases(draw):
    c = O.draw(random.Random(100 + draw))
    say("drawn operator", c)
    _check(c, draw, own=True)
    torch.cuda.empty_cache()
