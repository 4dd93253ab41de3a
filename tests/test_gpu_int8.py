"""The INT8 mode on the GPU: row codes, the grouped products with a scale per
token and per output channel, and the whole layer on them, against the plain
64-bit forms of plain64.  Codes and scales bit for bit; products within
bounds that count their roundings (the integer sums are exact)."""
import numpy as np
import pytest
import torch

import moe_layer_gating_amd as moe
import plain64 as P
from gpu_helpers import say

pytestmark = pytest.mark.gpu


def _bf16(a):
    return torch.from_numpy(np.ascontiguousarray(a, np.float32)).bfloat16()


def _np(t):
    return t.detach().float().cpu().numpy().astype(np.float64)


def _dev(a):
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


# ------------------------------------------------------------------ row codes
@pytest.mark.parametrize("rows,n", [(1, 8), (3, 128), (5, 2040), (4, 2048), (7, 2056), (3, 4104),
                                    (2, 8192), (3, 16384), (2, 16392), (1, 131072), (1000, 256)])
def test_row_codes(rows, n):
    say("row codes", rows, n)
    g = np.random.default_rng(rows * 31 + n)
    a = _bf16(g.standard_normal((rows, n)) * np.exp(2 * g.standard_normal((rows, 1))))
    a[0, ::5] = a[0].abs().max() / 2  # 63.5 codes: a tie
    codes, scales = moe.moe_act_quant_i8(a.cuda())
    wc, ws = P.quant_i8(_np(a))
    assert np.array_equal(codes.cpu().numpy(), wc)
    assert np.array_equal(scales.cpu().numpy().view(np.uint32), ws.view(np.uint32))
    assert int(codes.max()) == 127 or int(codes.min()) == -127


def test_row_codes_over_the_whole_range():
    """Rows at every binade of bf16, subnormal ones too, zero rows, a row of
    one value, every ratio of two bf16 significands."""
    g = np.random.default_rng(1)
    rows = []
    for e in range(1, 255):
        m = g.integers(0, 128, 256)
        ex = np.maximum(e - g.integers(0, 9, 256), 0)
        ex[0] = e
        rows.append(((g.integers(0, 2, 256) << 15) | (ex << 7) | m).astype(np.uint16))
    rows.append(np.zeros(256, np.uint16))
    rows.append(np.full(256, 0x8000, np.uint16))
    rows.append(np.arange(256, dtype=np.uint16) % 128)  # subnormal values only
    for m in range(128):  # significand m against all others, one binade down
        r = np.concatenate([np.arange(128), np.arange(128)]).astype(np.uint16)
        r[:128] |= 126 << 7
        r[128:] |= 125 << 7
        r[255] = (127 << 7) | m
        rows.append(r)
    bits = np.stack(rows)
    a = torch.from_numpy(bits.view(np.int16)).view(torch.bfloat16)
    codes, scales = moe.moe_act_quant_i8(a.cuda())
    wc, ws = P.quant_i8(_np(a))
    assert np.array_equal(codes.cpu().numpy(), wc)
    assert np.array_equal(scales.cpu().numpy().view(np.uint32), ws.view(np.uint32))


@pytest.mark.parametrize("n", [8, 2048, 20000])
def test_row_codes_of_nan_and_infinity(n):
    a = torch.ones(6, n, dtype=torch.bfloat16)
    for row, bad in ((1, np.nan), (2, np.inf), (3, -np.inf), (4, -np.nan)):
        a[row, n - row] = bad
    scales = moe.moe_act_quant_i8(a.cuda())[1].cpu()
    assert bool(torch.isnan(scales[1:5]).all())
    assert bool((scales[[0, 5]] == np.float32(1) / np.float32(127)).all())


@pytest.mark.parametrize("T,E,k,I", [(3, 8, 2, 256), (200, 4, 2, 128), (2100, 4, 2, 8192)])
def test_nan_and_infinity_in_x_reach_their_tokens_only(T, E, k, I):
    """Few-token kernel, 64- and 256-position tiles: the outputs of two tokens
    are NaN, the others are what they are without those tokens' values."""
    say("NaN and infinity in x", T, E, k, I)
    H = 256
    g = torch.Generator(device="cuda").manual_seed(T)
    x = torch.randn(T, H, generator=g, device="cuda").bfloat16()
    logits = torch.randn(T, E, generator=g, device="cuda")
    w13 = torch.randint(-127, 128, (E, 2 * I, H), generator=g, device="cuda").to(torch.int8)
    w2 = torch.randint(-127, 128, (E, H, I), generator=g, device="cuda").to(torch.int8)
    s13 = torch.rand(E, 2 * I, generator=g, device="cuda") * 1e-3
    s2 = torch.rand(E, H, generator=g, device="cuda") * 1e-3
    want = moe.moe_fused_forward(x, logits, w13, s13, w2, s2, k)
    x[0, 5] = np.nan
    x[T - 1, 255] = -np.inf
    got = moe.moe_fused_forward(x, logits, w13, s13, w2, s2, k)
    assert bool(torch.isnan(got[0]).all()) and bool(torch.isnan(got[T - 1]).all())
    assert torch.equal(got[1:T - 1], want[1:T - 1])


def test_row_codes_of_many_rows():
    """2^24 + 5 rows, and the last of them: a block per row would be 2^32 threads."""
    say("row codes of many rows")
    rows, n = (1 << 24) + 5, 8
    a = torch.zeros(rows, n, dtype=torch.bfloat16, device="cuda")
    a[:, 3] = 2
    a[:, 5] = -1
    a[1::7] *= 3
    codes, scales = moe.moe_act_quant_i8(a)
    want = torch.tensor([0, 0, 0, 127, 0, -64, 0, 0], dtype=torch.int8, device="cuda")
    assert bool((codes == want).all())
    amax = torch.full((rows,), 2.0, device="cuda")
    amax[1::7] *= 3
    # 2 and 6 over 127, rounded once
    assert torch.equal(scales, torch.where(amax == 2, np.float32(2) / np.float32(127),
                                           np.float32(6) / np.float32(127)))


def test_layer_of_many_tokens():
    """More tokens than row blocks (2^20) in the gating, the tile list and the
    down projection; the first and last tokens against the same ones alone."""
    say("layer of many tokens")
    T, H, E, k, I = (1 << 20) + 700, 128, 2, 1, 128
    g = torch.Generator(device="cuda").manual_seed(3)
    x = torch.randn(T, H, generator=g, device="cuda").bfloat16()
    x[1 << 20:] *= 4
    logits = torch.randn(T, E, generator=g, device="cuda")
    w13 = torch.randint(-127, 128, (E, 2 * I, H), generator=g, device="cuda").to(torch.int8)
    w2 = torch.randint(-127, 128, (E, H, I), generator=g, device="cuda").to(torch.int8)
    s13 = torch.rand(E, 2 * I, generator=g, device="cuda") * 1e-3
    s2 = torch.rand(E, H, generator=g, device="cuda") * 1e-3
    out = moe.moe_fused_forward(x, logits, w13, s13, w2, s2, k)
    ids, wts = moe.moe_topk_gating(logits, k)
    _, offsets, sorted_ids, inv = moe.moe_align_sort(ids, E)
    h = moe.moe_grouped_gemm_w13_swiglu(x, w13, s13, sorted_ids, offsets, k)[0]
    y = moe.moe_grouped_gemm_w2(h, w2, s2, offsets, None, k)
    steps = moe.moe_combine(y, inv, wts, moe.MOE_INT8, E)
    for part in (slice(0, 700), slice((1 << 20) - 350, (1 << 20) + 350), slice(T - 700, T)):
        few = moe.moe_fused_forward(x[part].clone(), logits[part].clone(), w13, s13, w2, s2, k)
        # exact: integer sums, one formula in both tile forms, one term (k = 1, weight 1),
        # for which rounding y to bf16 first changes nothing
        assert torch.equal(out[part], few)
        assert torch.equal(steps[part], few)


def test_row_codes_of_no_rows_and_other_shapes():
    codes, scales = moe.moe_act_quant_i8(torch.zeros(0, 64, dtype=torch.bfloat16, device="cuda"))
    assert codes.shape == (0, 64) and scales.shape == (0,)
    a = torch.randn(3, 4, 64, device="cuda").bfloat16()
    codes, scales = moe.moe_act_quant_i8(a)
    assert codes.shape == a.shape and scales.shape == (3, 4)
    c2, s2 = moe.moe_act_quant_i8(a.view(12, 64))
    assert torch.equal(codes.view(12, 64), c2) and torch.equal(scales.view(12), s2)


# ------------------------------------------------------------------ products
# name, T, H, E, k, I, skew: one token, one expert, k = E; few and many pairs
# per expert, tiles that end ragged, experts without a pair, row counts that are
# and are not multiples of 256 channels, reductions of one to many 128-code
# stages, the three groupings
LAYERS = [
    # the few-token kernels (16-position tiles, several per expert in the last)
    ("one_token", 1, 512, 16, 4, 256, 0.0),
    ("one_expert", 5, 128, 1, 1, 128, 0.0),
    ("k_is_E", 6, 256, 4, 4, 128, 0.0),
    ("few_pairs", 16, 640, 16, 4, 384, 0.5),
    ("few_pairs_many_experts", 40, 256, 64, 8, 256, 0.5),
    ("few_blocks", 100, 384, 10, 3, 640, 0.3),
    ("few_blocks_skewed", 211, 256, 8, 2, 256, 2.0),
    # 64-position tiles on 128 rows
    ("small_tiles_9_pairs", 100, 256, 32, 3, 1024, 0.5),
    ("small_tiles", 600, 512, 8, 2, 512, 0.3),
    ("small_tiles_skewed", 1037, 384, 12, 3, 384, 2.0),
    ("small_tiles_odd_rows", 400, 128, 3, 1, 128, 0.5),
    ("small_tiles_chunked", 1100, 256, 16, 8, 128, 1.0),
    ("small_tiles_one_stage", 600, 128, 2, 1, 128, 0.5),
    ("small_tiles_odd_stages", 1100, 384, 3, 2, 640, 1.0),
    ("small_tiles_one_expert", 4100, 256, 1, 1, 256, 0.0),
    # 256-position tiles on 256 rows: every width of the main loop
    ("large_tiles", 1100, 384, 8, 2, 2048, 0.7),
    ("large_tiles_one_stage", 2100, 128, 4, 2, 2560, 0.5),
    ("large_tiles_skewed", 1500, 256, 16, 2, 1920, 2.5),
    ("large_tiles_one_expert", 5000, 256, 1, 1, 2048, 0.0),
    ("large_tiles_prime", 1151, 640, 7, 3, 1664, 1.0),
]


def _layer(T, H, E, k, I, skew, seed):
    g = np.random.default_rng(seed)
    x = _bf16(g.standard_normal((T, H)) * np.exp(g.standard_normal((T, 1))))
    if T > 2:
        x[1] = 0  # a padding row
    logits = (g.standard_normal((T, E)) + skew * g.standard_normal(E)).astype(np.float32)
    w13 = g.integers(-128, 128, (E, 2 * I, H)).astype(np.int8)
    w2 = g.integers(-128, 128, (E, H, I)).astype(np.int8)
    s13 = ((0.5 + g.random((E, 2 * I))) / (64 * H ** 0.5)).astype(np.float32)
    s2 = ((0.5 + g.random((E, H))) / (64 * I ** 0.5)).astype(np.float32)
    s13[0, :3] = 0
    return x, logits, w13, s13, w2, s2


def _grouping(logits, k):
    E = logits.shape[1]
    ids = np.argsort(-logits, 1, kind="stable")[:, :k].astype(np.int32)
    flat = ids.reshape(-1)
    order = np.argsort(flat, kind="stable").astype(np.int32)
    offsets = np.concatenate([[0], np.cumsum(np.bincount(flat, minlength=E))]).astype(np.int32)
    inv = np.empty_like(order)
    inv[order] = np.arange(order.size, dtype=np.int32)
    return ids, order, offsets, inv


def _within(got, want, bound, what):
    got = np.asarray(got, np.float64)
    assert np.all(np.isfinite(got)), what
    worst = float(np.max(np.abs(got - want) / bound))
    assert worst <= 1.0, "%s: %.3f of its bound" % (what, worst)


@pytest.mark.parametrize("c", LAYERS, ids=[c[0] for c in LAYERS])
def test_products_and_layer(c):
    name, T, H, E, k, I, skew = c
    say("int8", name)
    x, logits, w13, s13, w2, s2 = _layer(T, H, E, k, I, skew, len(name) * 7 + T)
    ids, order, offsets, inv = _grouping(logits, k)
    dx, d13, d2 = x.cuda(), _dev(w13), _dev(w2)
    ds13, ds2, doff, dord = _dev(s13), _dev(s2), _dev(offsets), _dev(order)
    # rows behind the last pair stay as they are
    hbuf = torch.full((T * k + 3, I), 5.0, dtype=torch.bfloat16, device="cuda")
    h, _ = moe.moe_grouped_gemm_w13_swiglu(dx, d13, ds13, dord, doff, k, h=hbuf[:T * k])
    want, bound = P.w13_i8(_np(x), w13, s13, order, offsets, k)
    _within(_np(h), want, bound, "h")
    assert torch.all(hbuf[T * k:] == 5.0)
    ybuf = torch.full((T * k + 3, H), 5.0, device="cuda")
    y = moe.moe_grouped_gemm_w2(h, d2, ds2, doff, None, k, y=ybuf[:T * k])
    want, bound = P.w2_i8(_np(h), w2, s2, offsets)
    _within(y.cpu().numpy(), want, bound, "y")
    assert torch.all(ybuf[T * k:] == 5.0)
    # the fused call is the steps in one
    gids, gw = moe.moe_topk_gating(_dev(logits), k)
    assert np.array_equal(gids.cpu().numpy(), ids)
    steps = moe.moe_combine(y, _dev(inv), gw, moe.MOE_INT8, E=E, I=I)
    out = torch.full((T, H), float("nan"), dtype=torch.bfloat16, device="cuda")
    ids_out = torch.empty(T, k, dtype=torch.int32, device="cuda")
    for _ in range(2):
        moe.moe_fused_forward(dx, _dev(logits), d13, ds13, d2, ds2, k, out=out, topk_ids=ids_out)
        assert torch.equal(out, steps), "fused and step results differ"
        assert np.array_equal(ids_out.cpu().numpy(), ids)


@pytest.mark.parametrize("I", [128, 1024])  # 64- and 256-position tiles
def test_layer_with_a_large_y(I):
    """From 2^24 values on the fused call holds y in bf16: the steps' result
    with their fp32 y rounded once, bit for bit."""
    T, H, E, k = 4100, 2048, 5, 2
    assert T * k * H >= 1 << 24
    x, logits, w13, s13, w2, s2 = _layer(T, H, E, k, I, 0.3, 8)
    ids, order, offsets, inv = _grouping(logits, k)
    dx, d13, d2, ds13, ds2 = x.cuda(), _dev(w13), _dev(w2), _dev(s13), _dev(s2)
    h, _ = moe.moe_grouped_gemm_w13_swiglu(dx, d13, ds13, _dev(order), _dev(offsets), k)
    y = moe.moe_grouped_gemm_w2(h, d2, ds2, _dev(offsets), None, k)
    rows = np.r_[0:40, 4000:4060, 8160:8200]  # of the first, a middle and the last expert
    e = P.expert_of(offsets, T * k)[rows]
    codes, s = P.quant_i8(_np(h)[rows])
    want = np.stack([codes[i].astype(np.float64) @ w2[e[i]].astype(np.float64).T for i in range(rows.size)])
    want *= s.astype(np.float64)[:, None] * s2.astype(np.float64)[e]
    _within(y.cpu().numpy()[rows], want, np.abs(want) * 3.01 * P.U + 2.0 ** -140, "y")
    gw = moe.moe_topk_gating(_dev(logits), k)[1]
    steps = moe.moe_combine(y.bfloat16().float(), _dev(inv), gw, moe.MOE_INT8, E=E, I=I)
    out = moe.moe_fused_forward(dx, _dev(logits), d13, ds13, d2, ds2, k)
    assert torch.equal(out, steps)


def test_longest_reduction_of_the_largest_codes():
    """131072 products of 127 and -128: sums of -2 130 706 432, the largest
    that the mode lets occur, in the few-token kernel and both tile forms."""
    I, H = 131072, 128
    w2 = np.full((1, H, I), -128, np.int8)
    w2[0, 5] = 127
    s2 = np.full((1, H), 0.5, np.float32)
    for n in (3, 40, 70):
        h = torch.full((n, I), 3.0, dtype=torch.bfloat16)
        h[1] = -0.75
        offsets = np.array([0, n], np.int32)
        y = moe.moe_grouped_gemm_w2(h.cuda(), _dev(w2), _dev(s2), _dev(offsets), None, 1)
        want, bound = P.w2_i8(_np(h), w2, s2, offsets)
        _within(y.cpu().numpy(), want, bound, "y")


@pytest.mark.parametrize("n", [5, 600, 4300])
def test_weights_past_two_to_the_31_bytes(n):
    """An expert whose codes start 2.1 GB into the tensor (few-token kernel, 64-
    and 256-position tiles)."""
    E, N, K = 66, 8192, 4096
    w2 = torch.zeros(E, N, K, dtype=torch.int8, device="cuda")
    g = torch.Generator(device="cuda").manual_seed(3)
    last = torch.randint(-127, 128, (N, K), generator=g, device="cuda", dtype=torch.int8)
    w2[E - 1] = last
    s2 = torch.rand(E, N, generator=g, device="cuda")
    h = torch.randn(n, K, generator=g, device="cuda").bfloat16()
    offsets = torch.zeros(E + 1, dtype=torch.int32, device="cuda")
    offsets[E] = n
    y = moe.moe_grouped_gemm_w2(h, w2, s2, offsets, None, 1)
    rows = np.unique(np.array([0, 1, n // 2, n - 1]))
    want, bound = P.w2_i8(_np(h)[rows], last.cpu().numpy()[None], s2[E - 1:].cpu().numpy(),
                          np.array([0, rows.size]))
    _within(y.cpu().numpy()[rows], want, bound, "y")


@pytest.mark.parametrize("T", [4, 300])
def test_router_noalloc_events_and_graph(T):
    """The layer's other entry points take int8 weights too: router in front,
    static scratch, stage events, a captured graph replayed between eager
    calls, a stream of its own."""
    H, E, k, I = 256, 32, 4, 256
    x, logits, w13, s13, w2, s2 = _layer(T, H, E, k, I, 0.5, T)
    dx, d13, d2, ds13, ds2 = x.cuda(), _dev(w13), _dev(w2), _dev(s13), _dev(s2)
    wg = _bf16(np.random.default_rng(2).standard_normal((E, H)) * 0.05).cuda()
    lg = torch.empty(T, E, device="cuda")
    out_r = moe.moe_fused_forward_router(dx, wg, d13, ds13, d2, ds2, k, logits=lg)
    out = moe.moe_fused_forward(dx, lg, d13, ds13, d2, ds2, k)
    assert torch.equal(out, out_r)
    out_n = torch.empty_like(out)
    moe.moe_fused_forward_noalloc(dx, lg, d13, ds13, d2, ds2, k, out_n)
    assert torch.equal(out, out_n)
    ev = [torch.cuda.Event(enable_timing=True) for _ in range(moe.NUM_STAGE_EVENTS)]
    for e in ev:
        e.record()
    out_e = moe.moe_fused_forward_events(dx, lg, d13, ds13, d2, ds2, k, [e.cuda_event for e in ev])
    torch.cuda.synchronize()
    assert torch.equal(out, out_e) and ev[0].elapsed_time(ev[8]) >= 0
    ws = moe.workspace(moe.make_shape(T, H, E, k, I, moe.MOE_INT8))
    buf = torch.empty_like(out)

    def step():
        moe.moe_fused_forward(dx, lg, d13, ds13, d2, ds2, k, out=buf, ws=ws)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    assert torch.equal(buf, out)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    for rep in range(4):
        buf.fill_(float("nan"))
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(buf, out), "replay %d" % rep
        step()
        torch.cuda.synchronize()
        assert torch.equal(buf, out)


def test_two_layers_at_once():
    """Two batches on two streams with a workspace each, enqueued alternately."""
    H, E, k, I = 256, 12, 3, 384
    sets = []
    for T in (5, 700):
        x, logits, w13, s13, w2, s2 = _layer(T, H, E, k, I, 0.5, T)
        args = (x.cuda(), _dev(logits), _dev(w13), _dev(s13), _dev(w2), _dev(s2), k)
        want = moe.moe_fused_forward(*args)
        sets.append((args, want, torch.cuda.Stream(), torch.empty_like(want),
                     moe.workspace(moe.make_shape(T, H, E, k, I, moe.MOE_INT8))))
    torch.cuda.synchronize()
    for _ in range(5):
        for args, _, stream, out, ws in sets:
            with torch.cuda.stream(stream):
                moe.moe_fused_forward(*args, out=out, ws=ws)
    torch.cuda.synchronize()
    for _, want, _, out, _ in sets:
        assert torch.equal(out, want)


def test_other_modes_still_refuse_and_take_their_scales():
    """float and FP8 weights keep their paths beside the INT8 one."""
    with pytest.raises(moe.MoeError):
        moe.mode_of(torch.zeros(1, dtype=torch.int16))
    assert moe.mode_of(torch.zeros(1, dtype=torch.int8)) == moe.MOE_INT8
    assert moe.mode_of(torch.zeros(1, dtype=torch.uint8)) == moe.MOE_FP8_E4M3


def test_training_and_serving_steps_together():
    """One batch as a router's training step takes it: the int8 layer, the
    gradient of its gating weights (the derivative of <out, d> by w_tj is
    <d_t, y_tj>), the balance loss and both gradients on the logits."""
    T, H, E, k, I = 200, 256, 16, 4, 256
    x, logits, w13, s13, w2, s2 = _layer(T, H, E, k, I, 0.5, 77)
    mask = np.ones(T, np.uint8)
    mask[150:] = 0
    dl = _dev(logits)
    ids, w = moe.moe_topk_gating(dl, k)
    counts, offsets, order, inv = moe.moe_align_sort(ids, E)
    h, _ = moe.moe_grouped_gemm_w13_swiglu(x.cuda(), _dev(w13), _dev(s13), order, offsets, k)
    y = moe.moe_grouped_gemm_w2(h, _dev(w2), _dev(s2), offsets, None, k)
    d = torch.randn(T, H, device="cuda")
    gw = (y[inv.long()].view(T, k, H) * d[:, None]).sum(-1)
    dm = _dev(mask)
    loss, lcounts, probs, tokens = moe.moe_balance_loss(dl, ids, 0.01, token_mask=dm)
    grad = moe.moe_router_backward(dl, ids, w, gw, lcounts, tokens, 0.01,
                                   torch.ones(1, device="cuda"), token_mask=dm)
    full = moe.moe_balance_loss(dl, ids, 0.01)[1]
    assert torch.equal(full, counts)  # without a mask: the grouping's own counts
    nids, nw, ngw = ids.cpu().numpy(), w.cpu().numpy(), gw.cpu().numpy()
    a = P.gating_grad(logits, nids, nw, ngw, True, mask)
    c32 = float(np.float32(0.01))
    b = P.balance_grad(logits, lcounts.cpu().numpy(), 150, k, c32, 1.0, mask)
    bound = P.gating_grad_bound(logits, nids, nw, ngw, True) + \
        P.balance_grad_bound(logits, lcounts.cpu().numpy(), 150, k, c32, 1.0) + \
        2 * P.U * (np.abs(a) + np.abs(b))
    _within(grad.cpu().numpy(), a + b, bound, "router gradient")


def test_refusals_on_the_gpu():
    x = torch.randn(4, 256, device="cuda").bfloat16()
    lg = torch.randn(4, 8, device="cuda")
    w13 = torch.zeros(8, 512, 256, dtype=torch.int8, device="cuda")
    w2 = torch.zeros(8, 256, 256, dtype=torch.int8, device="cuda")
    s13, s2 = torch.ones(8, 512, device="cuda"), torch.ones(8, 256, device="cuda")
    moe.moe_fused_forward(x, lg, w13, s13, w2, s2, 2)
    for bad in ((x.float(), lg, w13, s13, w2, s2), (x, lg, w13, s13[:, 0].contiguous(), w2, s2),
                (x, lg, w13, s13, w2, s2[:, 0].contiguous()), (x, lg, w13, None, w2, s2),
                (x, lg, w13, s13, w2.view(torch.uint8), s2), (x, lg, w13, s13.double(), w2, s2),
                (x, lg.double(), w13, s13, w2, s2), (x, lg, w13, s13, w2[:4], s2[:4]),
                (x, lg, torch.zeros(8, 513, 256, dtype=torch.int8, device="cuda"),
                 torch.ones(8, 513, device="cuda"), w2, s2)):
        with pytest.raises(moe.MoeError):
            moe.moe_fused_forward(*bad, 2)
    with pytest.raises(moe.MoeError):
        moe.moe_fused_forward(x, lg, w13, s13, w2, s2, 2, ws=torch.empty(1 << 20, device="cuda"))
    with pytest.raises(moe.MoeError):
        moe.moe_act_quant_i8(x.float())
    with pytest.raises(moe.MoeError):
        moe.moe_act_quant_i8(torch.zeros(2, 12, dtype=torch.bfloat16, device="cuda"))
    with pytest.raises(moe.MoeError):
        moe.moe_grouped_gemm_w2(x, w2, s2, torch.zeros(8, dtype=torch.int32, device="cuda"), None, 2)
