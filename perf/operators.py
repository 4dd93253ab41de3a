"""What the router's training step and the 8-bit integer expert products are timed on.

Three operators of the MoE layer, each with its plain form in elementary torch operations:

  balance   the load-balance loss with its per-expert counts, and its gradient on the router logits;
  router    the gradient of the gating weights on the router logits, alone or together with the balance loss's;
  w13, w2   the grouped expert products on int8 codes with one scale per token and one per output channel
            (gate/up with SwiGLU, down), and `layer`, the whole layer on such weights.
"""
import math

import torch

own = False

_KIND = ("balance", "router", "w13", "w2", "layer")


def _router(name, kind, T, E, k, **more):
    return _named(name, dict(kind=kind, T=T, E=E, k=k, mask=False, renorm=True, balance=True) | more)


def _expert(name, kind, T, H, E, k, I, skew=0.5):
    return _named(name, dict(kind=kind, T=T, H=H, E=E, k=k, I=I, skew=skew))


def _named(name, case):
    return dict(name=name, **case) if name else case


def listed():
    return [
        # a decode-sized fine-tuning step: all launch latency
        _router("balance_16_tokens", "balance", 16, 64, 8),
        # one prefill batch of a 256-expert layer
        _router("balance_prefill", "balance", 4096, 256, 8),
        # a padded batch, an expert count that is no multiple of four
        _router("balance_padded_odd", "balance", 16381, 61, 6, mask=True),
        # a global batch of a training step
        _router("balance_global_batch", "balance", 131072, 256, 8),
        # router fine-tuning on a mixed batch, no balance term
        _router("router_gating_only", "router", 512, 128, 8, balance=False),
        # both gradients of a large padded batch, plain softmax weights
        _router("router_both_padded", "router", 65536, 256, 8, mask=True, renorm=False),
        # one token through the whole layer: a stream of eight experts' weights
        _expert("layer_decode_1", "layer", 1, 4096, 64, 8, 8192),
        # sixteen decode tokens: most experts hold one to four pairs
        _expert("w13_decode_16", "w13", 16, 4096, 64, 8, 8192),
        # a mixed batch of prompts and decode tokens
        _expert("w2_mixed", "w2", 509, 6144, 128, 8, 4096),
        # few large experts, thousands of pairs each: bound by the matrix units
        _expert("w13_large_experts", "w13", 8192, 4096, 8, 2, 14336, skew=0.2),
        # a 4096-token prefill of 256 experts
        _expert("layer_prefill", "layer", 4096, 7168, 256, 8, 2048),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    kind = rng.choice(_KIND)
    if kind in ("balance", "router"):
        E = _log(rng, 2, 1024)
        T = max(1, min(_log(rng, 1, 131072), 131072 * 256 // E))
        return _router("", kind, T, E, rng.randint(1, min(16, E)), mask=rng.random() < 0.5,
                       renorm=rng.random() < 0.5, balance=kind == "balance" or rng.random() < 0.5)
    H, I = 128 * _log(rng, 1, 56), 128 * _log(rng, 1, 64)
    E = min(_log(rng, 1, 256), max(1, (3 << 30) // (3 * H * I)))  # at most 3 GiB of weights
    k = rng.randint(1, min(8, E))
    T = max(1, min(_log(rng, 1, 8192), 16384 // k, (1 << 41) // (6 * k * H * I)))
    return _expert("", kind, T, H, E, k, I, skew=round(rng.uniform(0.0, 0.8), 2))


def _device():
    return torch.device("cuda" if torch.cuda.is_available() else "cpu")


def _codes(shape, g):
    """Normal int8 codes, as a symmetric per-channel quantisation of normal weights leaves them."""
    return torch.randn(shape, generator=g, device=g.device).mul_(32).round_().clamp_(-127, 127).to(torch.int8)


def _scales(shape, fan_in, g):
    return (0.5 + torch.rand(shape, generator=g, device=g.device)) / (32 * math.sqrt(fan_in))


def _sorted_pairs(ids, E):
    flat = ids.reshape(-1).long()
    counts = torch.bincount(flat, minlength=E)
    offsets = torch.zeros(E + 1, dtype=torch.int32, device=ids.device)
    offsets[1:] = counts.cumsum(0)
    return torch.sort(flat, stable=True).indices.int(), offsets, int(counts.max())


def prepare(case, seed):
    dev = _device()
    g = torch.Generator(device=dev).manual_seed(seed)
    T, E, k = case["T"], case["E"], case["k"]
    skew = case.get("skew", 0.5)
    logits = torch.randn(T, E, generator=g, device=dev) + skew * torch.randn(E, generator=g, device=dev)
    top, ids = logits.sort(dim=1, descending=True, stable=True)
    top, ids = top[:, :k].contiguous(), ids[:, :k].int().contiguous()
    s = dict(case=case, logits=logits, ids=ids, keep={})
    if case["kind"] in ("balance", "router"):
        mask = None
        if case["mask"]:  # about a third of the tokens is padding
            mask = (torch.rand(T, generator=g, device=dev) < 0.66).to(torch.uint8)
        live = ids if mask is None else ids[mask.bool()]
        counts = torch.bincount(live.reshape(-1).long(), minlength=E).int()
        full = torch.logsumexp(logits if not case["renorm"] else top, 1, keepdim=True)
        s.update(mask=mask, coef=0.01, grad_loss=1 + torch.rand(1, generator=g, device=dev), counts=counts,
                 tokens=torch.tensor([live.shape[0]], dtype=torch.int32, device=dev),
                 weights=torch.exp(top - full), grad_weights=torch.randn(T, k, generator=g, device=dev) / T)
        return s
    H, I, kind = case["H"], case["I"], case["kind"]
    s["sorted_ids"], s["offsets"], s["most"] = _sorted_pairs(ids, E)
    if kind != "w2":
        x = torch.randn(T, H, generator=g, device=dev) * torch.exp(0.5 * torch.randn(T, 1, generator=g, device=dev))
        s["x"] = x.bfloat16()
        s["w13"], s["w13_scale"] = _codes((E, 2 * I, H), g), _scales((E, 2 * I), H, g)
    if kind != "w13":
        s["w2"], s["w2_scale"] = _codes((E, H, I), g), _scales((E, H), I, g)
    if kind == "w2":
        a, b = (torch.randn(T * k, I, generator=g, device=dev) for _ in range(2))
        s["h"] = (a * torch.sigmoid(a) * b).bfloat16()
    return s


# ------------------------------------------------------------------ plain form


def _softmax(l):
    e = torch.exp(l - l.amax(1, keepdim=True))
    return e / e.sum(1, keepdim=True)


def _balance_grad(logits, mask, counts, tokens, k, coef, grad_loss):
    E = logits.shape[1]
    n = tokens.clamp(min=1).to(logits.dtype)
    f = counts.to(logits.dtype) / (n * k)
    p = _softmax(logits)
    grad = p * (f - (p * f).sum(1, keepdim=True)) * (coef * E * grad_loss / n)
    return grad if mask is None else torch.where(mask.bool()[:, None], grad, 0)


def _balance(s, dt):
    """Loss, counts, mean probabilities and the gradient on the logits, in the type `dt`."""
    logits, mask, ids = s["logits"].to(dt), s["mask"], s["ids"].long()
    T, E = logits.shape
    k = ids.shape[1]
    live = torch.ones(T, device=ids.device) if mask is None else mask
    counts = torch.zeros(E, dtype=torch.int32, device=ids.device)
    counts.index_add_(0, ids.reshape(-1), live.int()[:, None].expand(T, k).reshape(-1))
    tokens = live.int().sum(dtype=torch.int32).reshape(1)
    n = tokens.clamp(min=1).to(dt)
    probs = (_softmax(logits) * live.to(dt)[:, None]).sum(0) / n
    loss = s["coef"] * E * (counts.to(dt) / (n * k) * probs).sum().reshape(1)
    grad = _balance_grad(logits, mask, counts, tokens, k, s["coef"], s["grad_loss"].to(dt))
    return loss, counts, probs, tokens, grad


def _router_grad(s, dt):
    case, ids = s["case"], s["ids"].long()
    w, g, logits = (s[n].to(dt) for n in ("weights", "grad_weights", "logits"))
    wg = w * g
    total = wg.sum(1, keepdim=True)
    if case["renorm"]:
        grad = torch.zeros_like(logits).scatter_(1, ids, wg - w * total)
    else:
        grad = (-_softmax(logits) * total).scatter_add_(1, ids, wg)
    if s["mask"] is not None:
        grad = torch.where(s["mask"].bool()[:, None], grad, 0)
    if case["balance"]:
        grad = grad + _balance_grad(logits, s["mask"], s["counts"], s["tokens"], case["k"], s["coef"],
                                    s["grad_loss"].to(dt))
    return grad


def _quant(a):
    a = a.float()
    amax = a.abs().amax(1, keepdim=True)
    codes = torch.round(a * 127 / torch.where(amax > 0, amax, 1))  # 15-bit products: the quotient alone rounds
    return codes, torch.where(amax > 0, amax / 127, 1)


def _grouped(codes, scale, w, w_scale, offsets, most):
    """codes [P,K] in expert order against w [E,N,K]: P x N products with both scales applied."""
    P, K = codes.shape
    E, N, _ = w.shape
    at = torch.arange(P, device=codes.device)
    e = torch.searchsorted(offsets[1:], at, right=True)
    if P < E:  # few pairs: only their experts' weights
        acc = torch.bmm(w[e].float(), codes[:, :, None]).squeeze(2)
    else:
        row = e * most + at - offsets[e]
        full = torch.zeros(E * most, K, device=codes.device).index_copy_(0, row, codes)
        acc = torch.bmm(full.view(E, most, K), w.float().transpose(1, 2)).view(E * most, N)[row]
    return acc * scale * w_scale[e]


def _gate_up(x, sorted_ids, k, w13, w13_scale, offsets, most):
    codes, scale = _quant(x)
    token = sorted_ids.long() // k
    gu = _grouped(codes[token], scale[token], w13, w13_scale, offsets, most)
    gate, up = gu.chunk(2, 1)
    return (gate / (1 + torch.exp(-gate)) * up).bfloat16()


def _layer(s):
    k = s["case"]["k"]
    T, E = s["logits"].shape
    top, ids = s["logits"].sort(dim=1, descending=True, stable=True)
    top, ids = top[:, :k], ids[:, :k]
    weights = _softmax(top)
    flat = ids.reshape(-1)
    order = torch.sort(flat, stable=True).indices
    offsets = torch.zeros(E + 1, dtype=torch.int32, device=flat.device)
    offsets[1:] = torch.zeros(E, dtype=torch.int32, device=flat.device).index_add_(0, flat, torch.ones_like(flat, dtype=torch.int32)).cumsum(0)
    h = _gate_up(s["x"], order, k, s["w13"], s["w13_scale"], offsets, s["most"])
    y = _grouped(*_quant(h), s["w2"], s["w2_scale"], offsets, s["most"])
    pairs = torch.empty_like(y).index_copy_(0, order, y).view(T, k, -1)
    return (pairs * weights[:, :, None]).sum(1).bfloat16(), ids.int()


def _plain(s):
    kind = s["case"]["kind"]
    if kind == "balance":
        return _balance(s, torch.float32)
    if kind == "router":
        return _router_grad(s, torch.float32)
    if kind == "w13":
        return _gate_up(s["x"], s["sorted_ids"], s["case"]["k"], s["w13"], s["w13_scale"], s["offsets"], s["most"])
    if kind == "w2":
        return _grouped(*_quant(s["h"]), s["w2"], s["w2_scale"], s["offsets"], s["most"])
    return _layer(s)


# ------------------------------------------------------------------ the framework's calls


def _buffers(s, moe):
    """What a program keeps between its calls: outputs and the workspace, made at the first one."""
    c, keep, dev = s["case"], s["keep"], s["logits"].device
    T, E, k = c["T"], c["E"], c["k"]
    if c["kind"] in ("balance", "router"):
        keep["grad"] = torch.empty(T, E, device=dev)
        if c["kind"] == "balance":
            keep["ws"] = moe.balance_loss_workspace(T, k, E, dev)
            keep["out"] = dict(loss=torch.empty(1, device=dev), expert_counts=torch.empty(E, dtype=torch.int32, device=dev),
                               expert_probs=torch.empty(E, device=dev),
                               token_count=torch.empty(1, dtype=torch.int32, device=dev))
        return keep
    keep["ws"] = moe.workspace(moe.make_shape(T, c["H"], E, k, c["I"], moe.MOE_INT8), dev)
    if c["kind"] == "w13":
        keep["h"] = torch.empty(T * k, c["I"], dtype=torch.bfloat16, device=dev)
    elif c["kind"] == "w2":
        keep["y"] = torch.empty(T * k, c["H"], device=dev)
    else:
        keep["out"] = torch.empty(T, c["H"], dtype=torch.bfloat16, device=dev)
        keep["ids"] = torch.empty(T, k, dtype=torch.int32, device=dev)
    return keep


def _framework(s):
    import moe_layer_gating_amd as moe

    c, kind, b = s["case"], s["case"]["kind"], s["keep"] or _buffers(s, moe)
    if kind == "balance":
        loss, counts, probs, tokens = moe.moe_balance_loss(s["logits"], s["ids"], s["coef"], token_mask=s["mask"],
                                                           ws=b["ws"], **b["out"])
        grad = moe.moe_balance_loss_backward(s["logits"], counts, tokens, c["k"], s["coef"], s["grad_loss"],
                                             token_mask=s["mask"], grad_logits=b["grad"])
        return loss, counts, probs, tokens, grad
    if kind == "router" and c["balance"]:
        return moe.moe_router_backward(s["logits"], s["ids"], s["weights"], s["grad_weights"], s["counts"], s["tokens"],
                                       s["coef"], s["grad_loss"], renormalize=c["renorm"], token_mask=s["mask"],
                                       grad_logits=b["grad"])
    if kind == "router":
        return moe.moe_topk_gating_backward(s["logits"], s["ids"], s["weights"], s["grad_weights"],
                                            renormalize=c["renorm"], token_mask=s["mask"], grad_logits=b["grad"])
    if kind == "w13":
        return moe.moe_grouped_gemm_w13_swiglu(s["x"], s["w13"], s["w13_scale"], s["sorted_ids"], s["offsets"], c["k"],
                                               ws=b["ws"], h=b["h"])[0]
    if kind == "w2":
        return moe.moe_grouped_gemm_w2(s["h"], s["w2"], s["w2_scale"], s["offsets"], None, c["k"], ws=b["ws"], y=b["y"])
    out = moe.moe_fused_forward(s["x"], s["logits"], s["w13"], s["w13_scale"], s["w2"], s["w2_scale"], c["k"],
                                out=b["out"], ws=b["ws"], topk_ids=b["ids"])
    return out, b["ids"]


def run(state):
    return _framework(state) if own else _plain(state)


# ------------------------------------------------------------------ work and 64-bit values


def work(case):
    T, E, k, kind = case["T"], case["E"], case["k"], case["kind"]
    rows = 4 * T * E
    if kind == "balance":  # logits read by each direction
        return {"bytes": 3 * rows + 4 * T * k + 2 * T * case["mask"] + 16 * E, "flops": 14 * T * E}
    if kind == "router":
        full = case["balance"] or not case["renorm"]
        return {"bytes": (1 + full) * rows + 12 * T * k + T * case["mask"] + 4 * E * case["balance"], "flops": (10 * E if full else 4 * k) * T}
    H, I = case["H"], case["I"]
    active = E * (1 - (1 - k / E) ** T)  # experts that hold a pair, expected
    up, down = active * (2 * I * H + 8 * I), active * (H * I + 4 * H)
    if kind == "w13":
        return {"bytes": up + 2 * T * H + 2 * T * k * I + 4 * T * k, "flops": 4 * T * k * H * I}
    if kind == "w2":
        return {"bytes": down + 2 * T * k * I + 4 * T * k * H, "flops": 2 * T * k * H * I}
    return {"bytes": up + down + rows + 4 * T * H + 4 * T * k, "flops": 6 * T * k * H * I}


def _quant64(a):
    a = a.double()
    amax = a.abs().amax(1, keepdim=True)
    amax = torch.where(amax > 0, amax, torch.full_like(amax, 127.0))
    return torch.round(127.0 * a / amax), amax / 127.0


def exact(case, seed):
    s = prepare(case, seed)
    kind, k, E = case["kind"], case["k"], case["E"]
    if kind in ("balance", "router"):
        logits = s["logits"].double()
        p = torch.softmax(logits, 1)
        live = torch.ones(case["T"], dtype=torch.float64, device=p.device) if s["mask"] is None else s["mask"].double()
        n = float(live.sum())
        hot = torch.zeros_like(p).scatter_(1, s["ids"].long(), 1.0) * live[:, None]
        n = max(n, 1.0)  # without a token every sum below is empty
        f = hot.sum(0) / (n * k)
        scale = s["coef"] * E * float(s["grad_loss"]) / n
        grad = live[:, None] * scale * p * (f[None] - (p @ f)[:, None])
        if kind == "balance":
            mean = (p * live[:, None]).sum(0) / n
            return (s["coef"] * E * (f * mean).sum()).reshape(1), None, mean, None, grad
        if not case["balance"]:
            grad = torch.zeros_like(grad)
        w, g = s["weights"].double(), s["grad_weights"].double()
        inner = (w * g).sum(1)
        own_part = torch.zeros_like(p)
        for j in range(k):
            own_part[torch.arange(case["T"], device=p.device), s["ids"][:, j].long()] += w[:, j] * g[:, j]
        if case["renorm"]:
            taken = torch.zeros_like(p)
            taken.scatter_(1, s["ids"].long(), w)
            own_part -= taken * inner[:, None]
        else:
            own_part -= p * inner[:, None]
        return grad + own_part * live[:, None]
    bounds = s["offsets"].tolist()
    tokens = s["sorted_ids"].long() // k

    def products(codes, scale, w, w_scale):
        y = torch.empty(codes.shape[0], w.shape[1], dtype=torch.float64, device=codes.device)
        for e, (lo, hi) in enumerate(zip(bounds, bounds[1:])):
            if hi > lo:
                y[lo:hi] = torch.mm(codes[lo:hi], w[e].double().t().contiguous()) * scale[lo:hi] * w_scale[e].double()
        return y

    if kind != "w2":
        codes, scale = _quant64(s["x"])
        gu = products(codes[tokens], scale[tokens], s["w13"], s["w13_scale"])
        gate, up = gu[:, :case["I"]], gu[:, case["I"]:]
        h = gate * torch.sigmoid(gate) * up
        if kind == "w13":
            return h
    h = s["h"] if kind == "w2" else h.bfloat16()  # the layer holds h in bf16
    y = products(*_quant64(h), s["w2"], s["w2_scale"])
    if kind == "w2":
        return y
    gates = torch.softmax(torch.gather(s["logits"].double(), 1, s["ids"].long()), 1).reshape(-1)
    out = torch.zeros(case["T"], case["H"], dtype=torch.float64, device=y.device)
    return out.index_add_(0, tokens, y * gates[s["sorted_ids"].long()][:, None]), None
