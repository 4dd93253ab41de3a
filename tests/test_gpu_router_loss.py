"""The load-balance loss with its counts, and the router's gradients, on the
GPU against the plain 64-bit forms of plain64 (counts bit for bit, the rest
within bounds that count the kernels' roundings)."""
import numpy as np
import pytest
import torch

import moe_layer_gating_amd as moe
import plain64 as P
from gpu_helpers import say

pytestmark = pytest.mark.gpu

# T, E, k: one token, one expert, k = E, expert counts around the lane and
# load widths (a multiple of 4 or not, 64, 256, 1024), block borders (128 rows
# run in one block, 129 in several), rows that end inside a block
SHAPES = [(1, 1, 1), (1, 64, 8), (3, 2, 2), (16, 8, 8), (33, 61, 6), (64, 64, 16), (127, 128, 2),
          (128, 260, 4), (129, 255, 3), (200, 256, 8), (512, 384, 5), (700, 1024, 16),
          (1000, 1023, 7), (600, 100, 4), (4099, 13, 4), (9001, 256, 8)]


def _inputs(T, E, k, seed, masked, spread=2.0):
    g = np.random.default_rng(seed)
    logits = (g.standard_normal((T, E)) * spread + 0.5 * g.standard_normal(E)).astype(np.float32)
    mask = (g.random(T) < 0.7).astype(np.uint8) if masked else None
    top = np.sort(logits, 1)[:, ::-1][:, :k]
    ids = np.argsort(-logits, 1, kind="stable")[:, :k].astype(np.int32)
    del top
    return g, logits, ids, mask


def _dev(a):
    return None if a is None else torch.from_numpy(np.ascontiguousarray(a)).cuda()


def _rows_in_a_row(T):
    # a block works on 16 to 64 rows at a time, and on more than twice that many
    # only where 256 blocks are not enough
    return max(2, -(-(-(-T // 256)) // 16))


def _within(got, want, bound, what):
    got = np.asarray(got, np.float64)
    off = np.abs(got - want)
    assert np.all(np.isfinite(got)), what
    worst = float(np.max(off / bound)) if off.size else 0.0
    assert worst <= 1.0, "%s: %.2f of its bound" % (what, worst)


@pytest.mark.parametrize("masked", [False, True])
@pytest.mark.parametrize("T,E,k", SHAPES)
def test_loss_counts_and_gradient(T, E, k, masked):
    say("balance loss", T, E, k, masked)
    g, logits, ids, mask = _inputs(T, E, k, T * 7 + E, masked)
    coef, gl = 0.02, np.float32(1.7)
    dl, dm = _dev(logits), _dev(mask)
    loss, counts, probs, tokens = moe.moe_balance_loss(dl, _dev(ids), coef, token_mask=dm)
    grad = moe.moe_balance_loss_backward(dl, counts, tokens, k, coef, _dev(np.array([gl])),
                                         token_mask=dm)
    torch.cuda.synchronize()
    wl, wc, wp, n = P.balance_loss(logits, ids, coef, mask)
    assert np.array_equal(counts.cpu().numpy(), wc) and int(tokens) == n
    pb = P.probs_bound(logits, wp, n, _rows_in_a_row(T))
    _within(probs.cpu().numpy(), wp, pb, "probabilities")
    lb = abs(coef) * E * float((wc / max(1, n * k)) @ pb) + abs(wl) * 2 * P.U + 2.0 ** -140
    _within(loss.cpu().numpy(), np.array([wl]), lb, "loss")
    c32 = float(np.float32(coef))
    _within(grad.cpu().numpy(), P.balance_grad(logits, wc, n, k, c32, float(gl), mask),
            P.balance_grad_bound(logits, wc, n, k, c32, float(gl)), "gradient")
    if masked:
        assert np.all(grad.cpu().numpy()[mask == 0] == 0)


@pytest.mark.parametrize("renorm", [True, False])
@pytest.mark.parametrize("masked", [False, True])
@pytest.mark.parametrize("T,E,k", SHAPES)
def test_gating_and_router_gradients(T, E, k, masked, renorm):
    say("gating gradient", T, E, k, masked, renorm)
    g, logits, ids, mask = _inputs(T, E, k, T * 3 + E, masked)
    dl, di, dm = _dev(logits), _dev(ids), _dev(mask)
    got_ids, w = moe.moe_topk_gating(dl, k, renormalize=renorm)
    assert np.array_equal(got_ids.cpu().numpy(), ids)
    gw = g.standard_normal((T, k)).astype(np.float32)
    coef, gl = 0.3, np.float32(0.8)
    one = moe.moe_topk_gating_backward(dl, di, w, _dev(gw), renormalize=renorm, token_mask=dm)
    _, counts, _, tokens = moe.moe_balance_loss(dl, di, coef, token_mask=dm)
    both = moe.moe_router_backward(dl, di, w, _dev(gw), counts, tokens, coef,
                                   _dev(np.array([gl])), renormalize=renorm, token_mask=dm)
    torch.cuda.synchronize()
    wn = w.cpu().numpy()
    want = P.gating_grad(logits, ids, wn, gw, renorm, mask)
    bound = P.gating_grad_bound(logits, ids, wn, gw, renorm)
    _within(one.cpu().numpy(), want, bound, "gating gradient")
    _, wc, _, n = P.balance_loss(logits, ids, coef, mask)
    c32 = float(np.float32(coef))
    more = P.balance_grad(logits, wc, n, k, c32, float(gl), mask)
    # the sum of the two rounds twice more, relative to both
    bound = bound + P.balance_grad_bound(logits, wc, n, k, c32, float(gl)) + \
        2 * P.U * (np.abs(want) + np.abs(more))
    _within(both.cpu().numpy(), want + more, bound, "router gradient")


@pytest.mark.parametrize("E", [16, 61, 600])
def test_a_logit_of_plus_infinity_is_not_hidden(E):
    """Its row has no softmax: loss and probabilities are NaN, and so is the
    row's gradient where the softmax enters it; the other rows keep theirs."""
    T, k = 40, 2
    g, logits, ids, _ = _inputs(T, E, k, E, False)
    counts = np.bincount(ids.reshape(-1), minlength=E).astype(np.int32)
    w = np.full((T, k), 0.5, np.float32)
    gw = g.standard_normal((T, k)).astype(np.float32)
    one, n = torch.ones(1, device="cuda"), _dev(np.array([T], np.int32))

    def grads(l):
        return [moe.moe_balance_loss_backward(l, _dev(counts), n, k, 1.0, one).cpu().numpy(),
                moe.moe_topk_gating_backward(l, _dev(ids), _dev(w), _dev(gw),
                                             renormalize=False).cpu().numpy()]

    want = grads(_dev(logits))
    logits[17, 3] = np.inf
    dl = _dev(logits)
    loss, c, probs, tokens = moe.moe_balance_loss(dl, _dev(ids), 1.0)
    assert bool(torch.isnan(loss).all()) and bool(torch.isnan(probs).all())
    assert np.array_equal(c.cpu().numpy(), counts) and int(tokens) == T
    for got, ref in zip(grads(dl), want):
        assert np.all(np.isnan(got[17]))
        rest = np.arange(T) != 17
        assert np.array_equal(got[rest], ref[rest])
    mask = np.ones(T, np.uint8)
    mask[17] = 0
    assert bool(torch.isfinite(moe.moe_balance_loss(dl, _dev(ids), 1.0, token_mask=_dev(mask))[0]))


@pytest.mark.parametrize("E", [16, 61, 256])
def test_rows_without_a_finite_logit_nan_and_infinities(E):
    """-inf and NaN logits, rows with nothing left, NaN and infinities in rows
    that the mask leaves out."""
    T, k = 150, 4
    g, logits, ids, _ = _inputs(T, E, k, E, False)
    mask = np.ones(T, np.uint8)
    logits[::7, : E // 2] = -np.inf
    logits[3::11, 1] = np.nan
    logits[5] = -np.inf
    logits[6] = np.nan
    logits[7, 2:] = -np.inf          # two finite logits
    mask[20:40] = 0
    logits[20:30] = np.nan
    logits[30:40] = np.inf
    ids = np.argsort(-np.where(np.isnan(logits), -np.inf, logits), 1, kind="stable")
    ids = ids[:, :k].astype(np.int32)
    ids[20:40] = -77                 # never read
    w = np.exp(g.standard_normal((T, k))).astype(np.float32)
    w /= w.sum(1, keepdims=True)
    w[5] = np.nan                    # what the gating makes of such a row
    w[20:40] = np.nan
    gw = g.standard_normal((T, k)).astype(np.float32)
    gw[20:40] = np.inf
    clean = np.where(mask[:, None] == 0, 0.0, logits).astype(np.float32)
    ok_ids, ok_w, ok_gw = ids.copy(), w.copy(), gw.copy()
    ok_ids[20:40], ok_w[20:40], ok_gw[20:40] = 0, 0, 0
    for mk in (mask, mask.astype(bool)):
        dl, di, dm = _dev(logits), _dev(ids), _dev(mk)
        loss, counts, probs, tokens = moe.moe_balance_loss(dl, di, 1.0, token_mask=dm)
        wl, wc, wp, n = P.balance_loss(clean, ok_ids, 1.0, mask)
        assert np.array_equal(counts.cpu().numpy(), wc) and int(tokens) == n == 130
        pb = P.probs_bound(clean, wp, n, _rows_in_a_row(T))
        _within(probs.cpu().numpy(), wp, pb, "probabilities")
        for renorm in (True, False):
            got = moe.moe_router_backward(dl, di, _dev(w), _dev(gw), counts, tokens, 1.0,
                                          torch.ones(1, device="cuda"), renormalize=renorm,
                                          token_mask=dm).cpu().numpy()
            a = P.gating_grad(clean, ok_ids, ok_w, ok_gw, renorm, mask)
            b = P.balance_grad(clean, wc, n, k, 1.0, 1.0, mask)
            bound = P.gating_grad_bound(clean, ok_ids, ok_w, ok_gw, renorm) + \
                P.balance_grad_bound(clean, wc, n, k, 1.0, 1.0) + 2 * P.U * (np.abs(a) + np.abs(b))
            _within(got, a + b, bound, "gradient")
            assert np.all(got[20:40] == 0)
            if renorm:
                assert np.all(got[5] == 0)


def test_dropped_and_repeated_ids():
    """Ids outside [0, E) are dropped pairs; an expert named twice in a row
    gets both terms."""
    T, E, k = 300, 24, 5
    g, logits, ids, _ = _inputs(T, E, k, 9, False)
    ids[::3, 2] = -1
    ids[1::5, 0] = E
    ids[2::7, 4] = ids[2::7, 1]
    ids[3::11] = 7
    w = g.random((T, k)).astype(np.float32)
    gw = g.standard_normal((T, k)).astype(np.float32)
    _, counts, _, tokens = moe.moe_balance_loss(_dev(logits), _dev(ids))
    _, wc, _, n = P.balance_loss(logits, ids, 1.0)
    assert np.array_equal(counts.cpu().numpy(), wc) and int(tokens) == T
    assert wc.sum() < T * k
    for renorm in (True, False):
        got = moe.moe_topk_gating_backward(_dev(logits), _dev(ids), _dev(w), _dev(gw),
                                           renormalize=renorm).cpu().numpy()
        _within(got, P.gating_grad(logits, ids, w, gw, renorm),
                P.gating_grad_bound(logits, ids, w, gw, renorm), "gradient")


@pytest.mark.parametrize("T", [0, 5, 300])
def test_no_token_counts(T):
    """T = 0 and a mask of zeros: every output is written, and is zero."""
    E, k = 20, 3
    logits = torch.randn(T, E, device="cuda")
    ids = torch.zeros(T, k, dtype=torch.int32, device="cuda")
    mask = torch.zeros(T, dtype=torch.uint8, device="cuda")
    out = dict(loss=torch.full((1,), 7.0, device="cuda"),
               expert_counts=torch.full((E,), 7, dtype=torch.int32, device="cuda"),
               expert_probs=torch.full((E,), 7.0, device="cuda"),
               token_count=torch.full((1,), 7, dtype=torch.int32, device="cuda"))
    loss, counts, probs, tokens = moe.moe_balance_loss(logits, ids, 0.5, token_mask=mask, **out)
    grad = torch.full((T, E), 7.0, device="cuda")
    moe.moe_balance_loss_backward(logits, counts, tokens, k, 0.5, torch.ones(1, device="cuda"),
                                  token_mask=mask, grad_logits=grad)
    torch.cuda.synchronize()
    for t in (loss, counts, probs, tokens, grad):
        assert torch.all(t == 0)


def test_gradient_against_differences():
    """The directional derivative of the 64-bit loss: central differences over
    +-h leave h^2 / 6 times the third derivative, below 1e-6 of the value here
    (both are O(1)); the gradient's own rounding adds its bound."""
    T, E, k = 40, 32, 4
    g, logits, ids, mask = _inputs(T, E, k, 4, True, spread=1.0)
    w64 = None
    for renorm in (True, False):
        gw = g.standard_normal((T, k)).astype(np.float32)

        def value(l):
            p = P.softmax(l)
            w = np.take_along_axis(p, ids, 1)
            if renorm:
                w = w / w.sum(1, keepdims=True)
            f = P.balance_loss(l, ids, 1.0, mask)[0]
            return f + float(((w * gw) * mask[:, None]).sum())

        dl, di, dm = _dev(logits), _dev(ids), _dev(mask)
        w = moe.moe_topk_gating(dl, k, renormalize=renorm)[1]
        _, counts, _, tokens = moe.moe_balance_loss(dl, di, 1.0, token_mask=dm)
        got = moe.moe_router_backward(dl, di, w, _dev(gw), counts, tokens, 1.0,
                                      torch.ones(1, device="cuda"), renormalize=renorm,
                                      token_mask=dm).cpu().numpy().astype(np.float64)
        for _ in range(6):
            v = g.standard_normal((T, E))
            h = 1e-4
            l = logits.astype(np.float64)
            diff = (value(l + h * v) - value(l - h * v)) / (2 * h)
            # an entry's error is at most about 2 prob_error = 80 U < 2^-17 of the
            # terms it is the difference of, themselves at most 4 times larger here
            slack = 1e-6 * max(1.0, abs(diff)) + float(np.abs(got * v).sum()) * 2.0 ** -15
            assert abs(float((got * v).sum()) - diff) <= slack
    del w64


def test_repeated_calls_are_identical():
    T, E, k = 5000, 96, 4
    g, logits, ids, mask = _inputs(T, E, k, 1, True)
    dl, di, dm = _dev(logits), _dev(ids), _dev(mask)
    first = None
    for _ in range(4):
        loss, counts, probs, tokens = moe.moe_balance_loss(dl, di, 0.1, token_mask=dm)
        got = [t.clone() for t in (loss, counts, probs, tokens)]
        if first is None:
            first = got
        assert all(torch.equal(a, b) for a, b in zip(first, got))


def test_logits_past_two_to_the_31_bytes():
    """Row offsets beyond 32 bits: the last rows of a [T,E] tensor of 2.4 GB
    equal the same rows alone."""
    T, E, k = 600_001, 1000, 2
    logits = torch.randn(T, E, device="cuda")
    ids = torch.randint(0, E, (T, k), dtype=torch.int32, device="cuda")
    w, gw = torch.rand(T, k, device="cuda"), torch.randn(T, k, device="cuda")
    loss, counts, probs, tokens = moe.moe_balance_loss(logits, ids, 1.0)
    assert torch.equal(counts.long(), torch.bincount(ids.reshape(-1).long(), minlength=E))
    assert int(tokens) == T and abs(float(probs.sum()) - 1) < 1e-5
    grad = moe.moe_router_backward(logits, ids, w, gw, counts, tokens, 1.0,
                                   torch.ones(1, device="cuda"), renormalize=False)
    t0 = T - 64
    tail = moe.moe_router_backward(logits[t0:].clone(), ids[t0:].clone(), w[t0:].clone(),
                                   gw[t0:].clone(), counts, tokens, 1.0,
                                   torch.ones(1, device="cuda"), renormalize=False)
    assert torch.equal(grad[t0:], tail)


def test_streams_and_graph_replays():
    """A router step on a stream of its own, and two captured graphs that share
    their workspace, replayed in turn with eager work between."""
    E, k, coef = 96, 4, 0.05
    sets = []
    for seed, T in ((1, 300), (2, 90)):
        g, logits, ids, mask = _inputs(T, E, k, seed, True)
        w = moe.moe_topk_gating(_dev(logits), k)[1]
        gw = g.standard_normal((T, k)).astype(np.float32)
        sets.append(dict(l=_dev(logits), i=_dev(ids), m=_dev(mask), w=w, gw=_dev(gw),
                         grad=torch.empty(T, E, device="cuda"), loss=torch.empty(1, device="cuda"),
                         c=torch.empty(E, dtype=torch.int32, device="cuda"),
                         p=torch.empty(E, device="cuda"),
                         n=torch.empty(1, dtype=torch.int32, device="cuda")))
    ws = moe.balance_loss_workspace(300, k, E)
    one = torch.ones(1, device="cuda")

    def step(s):
        moe.moe_balance_loss(s["l"], s["i"], coef, token_mask=s["m"], ws=ws, loss=s["loss"],
                             expert_counts=s["c"], expert_probs=s["p"], token_count=s["n"])
        moe.moe_router_backward(s["l"], s["i"], s["w"], s["gw"], s["c"], s["n"], coef, one,
                                token_mask=s["m"], grad_logits=s["grad"])

    def outputs(s):
        torch.cuda.synchronize()
        return [s[n].clone() for n in ("loss", "c", "p", "n", "grad")]

    want = []
    for s in sets:
        step(s)
        want.append(outputs(s))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        for s in sets:
            step(s)
    torch.cuda.current_stream().wait_stream(side)
    for s, v in zip(sets, want):
        assert all(torch.equal(a, b) for a, b in zip(outputs(s), v))
    graphs = []
    for s in sets:
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr):
            step(s)
        graphs.append(gr)
    for rep in range(4):
        for s, gr, v in zip(sets, graphs, want):
            for n in ("loss", "p", "grad"):
                s[n].fill_(float("nan"))
            s["c"].fill_(-1)
            gr.replay()
            assert all(torch.equal(a, b) for a, b in zip(outputs(s), v)), "replay %d" % rep
        step(sets[rep % 2])
        torch.cuda.synchronize()


def test_refusals_on_the_gpu():
    l, i = torch.randn(4, 8, device="cuda"), torch.zeros(4, 2, dtype=torch.int32, device="cuda")
    w = torch.rand(4, 2, device="cuda")
    with pytest.raises(moe.MoeError):
        moe.moe_balance_loss(l.half(), i)
    with pytest.raises(moe.MoeError):
        moe.moe_balance_loss(l, i.long())
    with pytest.raises(moe.MoeError):
        moe.moe_balance_loss(l, i[:3].contiguous())
    with pytest.raises(moe.MoeError):
        moe.moe_balance_loss(l.t().contiguous().t(), i)
    with pytest.raises(moe.MoeError):
        moe.moe_balance_loss(l, i, token_mask=torch.ones(5, dtype=torch.uint8, device="cuda"))
    with pytest.raises(moe.MoeError):
        moe.moe_balance_loss(l, i, token_mask=torch.ones(4, device="cuda"))
    with pytest.raises(moe.MoeError):
        moe.moe_balance_loss(l, i, ws=torch.empty(1, dtype=torch.uint8, device="cuda"))
    with pytest.raises(moe.MoeError):
        moe.moe_topk_gating_backward(l, i, w, w.cpu())
    with pytest.raises(moe.MoeError):
        moe.moe_topk_gating_backward(l, i, w, w, grad_logits=l)
