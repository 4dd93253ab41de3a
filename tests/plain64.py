"""Plain 64-bit forms of the router's loss and gradients and of the int8
expert products, with the error bounds the GPU tests hold the kernels to.

Nothing here is shared with the kernels: NumPy float64 and integers only.
U = 2^-24 is the largest relative error of one fp32 rounding."""
from __future__ import annotations

import numpy as np

U = 2.0 ** -24
U_BF16 = 2.0 ** -8  # half a bf16 step, relative to the value


# ------------------------------------------------------------------ router
def softmax(logits):
    """Row softmax; NaN reads as -inf, a row without a finite logit is zero."""
    l = np.asarray(logits, np.float64)
    l = np.where(np.isnan(l), -np.inf, l)
    m = l.max(1, keepdims=True)
    e = np.exp(l - np.where(np.isneginf(m), 0.0, m))
    s = e.sum(1, keepdims=True)
    return e / np.where(s > 0, s, 1.0)


def live_rows(mask, T):
    return np.ones(T, bool) if mask is None else np.asarray(mask).astype(bool)


def balance_loss(logits, ids, coef, mask=None):
    """(loss, counts, probs, tokens) in float64 / integers."""
    T, E = logits.shape
    k = ids.shape[1]
    live = live_rows(mask, T)
    n = int(live.sum())
    flat = ids[live].reshape(-1)
    counts = np.bincount(flat[(flat >= 0) & (flat < E)], minlength=E)
    if n == 0:
        return 0.0, counts, np.zeros(E), 0
    probs = softmax(logits[live]).sum(0) / n
    return coef * E * float((counts / (n * k)) @ probs), counts, probs, n


def balance_grad(logits, counts, n, k, coef, grad_loss, mask=None):
    T, E = logits.shape
    if n == 0:
        return np.zeros((T, E))
    f = np.asarray(counts, np.float64) / (n * k)
    p = softmax(logits)
    g = coef * E * grad_loss / n * p * (f[None] - (p @ f)[:, None])
    return np.where(live_rows(mask, T)[:, None], g, 0.0)


def gating_grad(logits, ids, weights, grad_weights, renormalize, mask=None):
    T, k = ids.shape
    E = logits.shape[1]
    ok = (ids >= 0) & (ids < E)
    w = np.where(ok & ~np.isnan(weights), weights, 0.0).astype(np.float64)
    wg = w * np.where(ok, grad_weights, 0.0).astype(np.float64)
    S = wg.sum(1, keepdims=True)
    out = np.zeros((T, E)) if renormalize else -softmax(logits) * S
    term = wg - w * S if renormalize else wg
    for j in range(k):
        r = np.nonzero(ok[:, j])[0]
        out[r, ids[r, j]] += term[r, j]
    return np.where(live_rows(mask, T)[:, None], out, 0.0)


def prob_error(logits):
    """Bound on the relative error of an fp32 softmax value: the shift l - m
    (its rounding, U |l - m|, is the exponential's relative error), expf (2
    steps = 4 U), the sum of E terms (E / 16 + 5 additions in a chain of 16
    lanes, each operand with the errors above), the reciprocal (2 U) and the
    product (U).  |l - m| counts up to 104, where the value leaves fp32."""
    l = np.asarray(logits, np.float64)
    l = l[np.isfinite(l)]
    spread = min(104.0, float(l.max() - l.min())) if l.size else 0.0
    E = logits.shape[1]
    return (2 * (spread + 4) + E / 16 + 5 + 3) * U * 1.01


def probs_bound(logits, probs, n, rows_in_a_row):
    """Per expert: the rows' errors, the fp32 additions of the rows that one
    lane sums (rows_in_a_row) and of the wave and block (2 + 8), one rounding.
    2^-120 covers values that underflow."""
    return probs * (prob_error(logits) + (rows_in_a_row + 11) * U * 1.01) + 2.0 ** -120


def balance_grad_bound(logits, counts, n, k, coef, grad_loss):
    """|s p_i (d_i - D)| with d = f - 1/E, D = sum d p: p carries prob_error,
    D carries it once more plus E/16 + 5 additions, each relative to sum |d| p
    <= max |d|; s, d, the difference and two products round once each.  The
    64-bit value is not exact either: its f_i - sum f p cancels (to 0 under an
    even load) between terms of up to max f, each with the errors of E
    additions and three more float64 roundings of 2^-53."""
    T, E = logits.shape
    if n == 0:
        return np.zeros((T, E))
    d = np.abs(np.asarray(counts, np.float64) / (n * k) - 1.0 / E).max()
    rel = 2 * prob_error(logits) + (E / 16 + 5 + 6) * U
    own = np.max(counts) / (n * k) * (E + 3) * 2.0 ** -53
    return abs(coef) * E * abs(grad_loss) / n * softmax(logits) * 2 * (d * rel + own) * 1.01 + 2.0 ** -140


def gating_grad_bound(logits, ids, weights, grad_weights, renormalize):
    """w g rounds once; S adds 16 lanes (4 additions, of sum |w g|); w S, the
    difference and the per-expert sum (k additions) round once each; the plain
    softmax carries prob_error.  Added for every expert that a row names."""
    T, k = ids.shape
    E = logits.shape[1]
    w = np.where(np.isnan(weights), 0.0, np.abs(weights)).astype(np.float64)
    wg = w * np.abs(grad_weights)
    S = wg.sum(1, keepdims=True)
    term = wg * (3 + k) + (w * S * (8 + k) if renormalize else 0.0)
    out = np.zeros((T, E))
    for j in range(k):
        r = np.nonzero((ids[:, j] >= 0) & (ids[:, j] < E))[0]
        out[r, ids[r, j]] += term[r, j] * U
    if not renormalize:
        out += softmax(logits) * S * (prob_error(logits) + 8 * U)
    return out * 1.01 + 2.0 ** -140


# ------------------------------------------------------------------ int8
def quant_i8(a):
    """Codes (int64) and scales (float32) of the rows of `a`, bf16 values as
    float64.  A quotient of two bf16 values times 127 that is no tie is at
    least 2^-17 away from one, so its float64 value rounds to the same
    integer; a tie is exact in float64."""
    a = np.asarray(a, np.float64)
    amax = np.abs(a).max(-1, keepdims=True)
    safe = np.where(amax > 0, amax, 1.0)
    codes = np.rint(127.0 * a / safe).astype(np.int64)
    scale = np.where(amax > 0, amax.astype(np.float32) / np.float32(127.0), np.float32(1.0))
    return codes, scale[..., 0].astype(np.float32)


def grouped_i8(codes, w, offsets):
    """Integer sums [P, channels] of the rows of each expert's group."""
    out = np.zeros((codes.shape[0], w.shape[1]), np.int64)
    for e in range(w.shape[0]):
        lo, hi = offsets[e], offsets[e + 1]
        if hi > lo:  # exact in float64: every sum is below 2^31
            out[lo:hi] = np.rint(codes[lo:hi].astype(np.float64) @ w[e].astype(np.float64).T)
    return out


def expert_of(offsets, n_pairs):
    return np.searchsorted(np.asarray(offsets)[1:], np.arange(n_pairs), side="right")


def w2_i8(h, w2, w2_scale, offsets):
    """y [P,H] float64 and its bound: the integer sum's conversion, the product
    of the scales and the product with it round once each."""
    codes, s = quant_i8(h)
    y = grouped_i8(codes, w2, offsets) * s.astype(np.float64)[:, None]
    y = y * w2_scale.astype(np.float64)[expert_of(offsets, h.shape[0])]
    return y, np.abs(y) * 3.01 * U + 2.0 ** -140


def w13_i8(x, w13, w13_scale, sorted_ids, offsets, k):
    """h [P,I] before its rounding to bf16, and the bound with it: g and u
    carry 3 U; the exponential's argument carries at most 4 U |g| (its factor
    log2 e may round once more), the exponential adds
    4 U, the sum, quotient and product one U each (two for the quotient).
    Past -g = 126 ln 2 the reciprocal of 1 + e^-g is below 2^-126, the least
    normal number, and may become 0 (past 128 ln 2 the exponential is infinite
    and it does), where |h| <= |g u| e^g <= |g u| 2^-126."""
    codes, s = quant_i8(x)
    tok = np.asarray(sorted_ids) // k
    e = expert_of(offsets, tok.size)
    gu = grouped_i8(codes[tok], w13, offsets) * s.astype(np.float64)[tok][:, None]
    gu = gu * w13_scale.astype(np.float64)[e]
    I = gu.shape[1] // 2
    g, u = gu[:, :I], gu[:, I:]
    with np.errstate(over="ignore"):
        h = g / (1.0 + np.exp(-g)) * u
    bound = np.abs(h) * (U_BF16 * 1.001 + (4 * np.minimum(np.abs(g), 104) + 16) * U) + \
        np.abs(g * u) * 2.0 ** -126 + 2.0 ** -120
    return h, bound
