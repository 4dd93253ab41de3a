"""The 64-bit forms the GPU tests compare with, against independent ones:
autograd in float64, central differences, exact rational arithmetic."""
from fractions import Fraction

import numpy as np
import pytest
import torch

import plain64 as P


def _case(T, E, k, seed, masked):
    g = np.random.default_rng(seed)
    logits = g.standard_normal((T, E))
    ids = np.argsort(-logits, 1, kind="stable")[:, :k].astype(np.int32)
    return g, logits, ids, (g.random(T) < 0.6).astype(np.uint8) if masked else None


@pytest.mark.parametrize("masked", [False, True])
@pytest.mark.parametrize("renorm", [False, True])
def test_gradients_match_autograd(renorm, masked):
    T, E, k, coef, gl = 19, 12, 3, 0.4, 1.3
    g, logits, ids, mask = _case(T, E, k, 3, masked)
    gw = g.standard_normal((T, k))
    live = torch.ones(T, dtype=torch.float64) if mask is None else torch.from_numpy(mask).double()
    l = torch.from_numpy(logits).requires_grad_()
    p = torch.softmax(l, 1)
    w = torch.gather(p, 1, torch.from_numpy(ids).long())
    if renorm:
        w = w / w.sum(1, keepdim=True)
    loss, counts, probs, n = P.balance_loss(logits, ids, coef, mask)
    f = torch.from_numpy(counts / (n * k))
    bal = coef * E * (f * (p * live[:, None]).sum(0) / n).sum()
    assert abs(float(bal) - loss) < 1e-14 and abs(probs.sum() - 1) < 1e-14
    assert counts.sum() == n * k
    (bal * gl + (w * torch.from_numpy(gw) * live[:, None]).sum()).backward()
    got = P.balance_grad(logits, counts, n, k, coef, gl, mask) + \
        P.gating_grad(logits, ids, w.detach().numpy(), gw, renorm, mask)
    assert np.abs(got - l.grad.numpy()).max() < 1e-14


def test_balance_gradient_matches_differences():
    T, E, k = 9, 7, 2
    g, logits, ids, mask = _case(T, E, k, 5, True)
    _, counts, _, n = P.balance_loss(logits, ids, 1.0, mask)
    got = P.balance_grad(logits, counts, n, k, 1.0, 1.0, mask)
    h = 1e-5
    for t in range(T):
        for e in range(E):
            up, down = logits.copy(), logits.copy()
            up[t, e] += h
            down[t, e] -= h
            d = (P.balance_loss(up, ids, 1.0, mask)[0] - P.balance_loss(down, ids, 1.0, mask)[0]) / (2 * h)
            assert abs(got[t, e] - d) < 1e-9  # h^2 / 6 and 2^-53 / h, both below


def test_even_load_has_loss_coef_and_no_gradient():
    T, E, k = 8, 4, 2
    ids = np.stack([np.arange(T) % E, (np.arange(T) + 1) % E], 1).astype(np.int32)
    logits = np.random.default_rng(0).standard_normal((T, E))
    loss, counts, _, n = P.balance_loss(logits, ids, 0.7)
    assert abs(loss - 0.7) < 1e-15
    assert np.abs(P.balance_grad(logits, counts, n, k, 0.7, 1.0)).max() < 1e-16


def test_row_codes_match_rational_arithmetic():
    g = np.random.default_rng(2)
    a = torch.from_numpy(g.standard_normal((6, 200))).bfloat16().double().numpy()
    a[0, 3] = np.abs(a[0]).max() / 2
    a[5] = 0
    codes, scale = P.quant_i8(a)
    for r in range(6):
        m = Fraction(float(np.abs(a[r]).max()))
        for c in range(200):
            want = round(127 * Fraction(float(a[r, c])) / m) if m else 0  # ties to even
            assert codes[r, c] == want
        assert scale[r] == (np.float32(float(m)) / np.float32(127) if m else 1)


def test_products_match_a_dense_sum():
    g = np.random.default_rng(4)
    codes = g.integers(-127, 128, (9, 32))
    w = g.integers(-128, 128, (3, 5, 32)).astype(np.int8)
    offsets = np.array([0, 4, 4, 9])
    got = P.grouped_i8(codes, w, offsets)
    e = P.expert_of(offsets, 9)
    assert list(e) == [0] * 4 + [2] * 5
    assert np.array_equal(got, np.einsum("pk,pnk->pn", codes, w[e].astype(np.int64)))
