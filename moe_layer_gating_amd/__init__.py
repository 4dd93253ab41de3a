"""Python binding of the fused MoE library for MI355X (gfx950).

Argument marshalling only: every function passes device pointers, sizes and
the current HIP stream to the C ABI declared in ``include/moe_gfx950.h`` and
raises ``MoeError`` on a non-zero status.  All computation happens in the HIP
kernels of ``libmoe_gfx950.so``; there is no fallback.  PyTorch provides the
device memory and the stream.

Tensor dtypes by mode (taken from the dtype of ``w13``):
  fp32 weights            -> fp32 mode: x, h, out fp32
  bf16 weights            -> bf16 mode: x, h, out bf16
  float8_e4m3fn or uint8  -> FP8 mode: e4m3 codes, fp32 scales [E]; x, h, out bf16
  int8 weights            -> INT8 mode: int8 codes, fp32 scales per output
                             channel (w13_scale [E,2I], w2_scale [E,H]); x, h, out bf16
"""
from __future__ import annotations

import ctypes
import os

import torch

MOE_F32, MOE_BF16, MOE_FP8_E4M3, MOE_INT8 = 0, 1, 2, 4
_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libmoe_gfx950.so")
_lib = None


def _public_raw_stream(dev):
    return torch.cuda.current_stream(dev).cuda_stream


_current_device = torch.cuda.current_device
# the stream's address without a Stream object around it, where torch has it
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", _public_raw_stream)


class MoeError(RuntimeError):
    pass


class moe_shape(ctypes.Structure):
    _fields_ = [("T", ctypes.c_int32), ("H", ctypes.c_int32), ("E", ctypes.c_int32),
                ("k", ctypes.c_int32), ("I", ctypes.c_int32), ("wdtype", ctypes.c_int32),
                ("renormalize", ctypes.c_int32)]


class moe_routing_offsets(ctypes.Structure):
    _fields_ = [(n, ctypes.c_size_t) for n in ("topk_ids", "topk_weights", "expert_counts",
                                                "expert_offsets", "sorted_ids", "inv_perm")]


EXPORTS = ("moe_check_shape", "moe_workspace_bytes", "moe_status_string",
           "moe_align_sort_workspace_bytes", "moe_workspace_routing", "moe_topk_gating",
           "moe_align_sort", "moe_grouped_gemm_w13_swiglu", "moe_grouped_gemm_w2", "moe_combine",
           "moe_act_quant_e4m3", "moe_act_quant_i8", "moe_balance_loss_workspace_bytes",
           "moe_balance_loss", "moe_balance_loss_backward", "moe_topk_gating_backward",
           "moe_router_backward",
           "moe_fused_forward", "moe_fused_forward_events", "moe_router_logits",
           "moe_fused_forward_router", "moe_fused_forward_noalloc", "moe_inv_rope_fp8_quant")
NOALLOC_SCRATCH_BYTES = 64 << 20  # MOE_NOALLOC_SCRATCH_BYTES
# host-only calls whose return type is not a moe_status
_NON_STATUS = ("moe_workspace_bytes", "moe_status_string", "moe_align_sort_workspace_bytes",
               "moe_balance_loss_workspace_bytes")
NUM_STAGE_EVENTS = 9


def lib():
    """Load the HIP library; raises if it has not been built."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise MoeError("libmoe_gfx950.so is not built; run __graft_entry__.build() "
                           "(or python moe_layer_gating_amd/_build.py)")
        L = ctypes.CDLL(LIB_PATH)
        P, i32, sz = ctypes.c_void_p, ctypes.c_int32, ctypes.c_size_t
        S = ctypes.POINTER(moe_shape)
        L.moe_check_shape.argtypes = [S]
        L.moe_check_shape.restype = ctypes.c_int
        L.moe_workspace_bytes.argtypes = [S]
        L.moe_workspace_bytes.restype = sz
        L.moe_status_string.argtypes = [ctypes.c_int]
        L.moe_status_string.restype = ctypes.c_char_p
        L.moe_align_sort_workspace_bytes.argtypes = [i32, i32, i32]
        L.moe_align_sort_workspace_bytes.restype = sz
        L.moe_workspace_routing.argtypes = [S, ctypes.POINTER(moe_routing_offsets)]
        L.moe_topk_gating.argtypes = [P, i32, i32, i32, i32, P, P, P]
        L.moe_align_sort.argtypes = [P, i32, i32, i32, P, P, P, P, P, sz, P]
        L.moe_grouped_gemm_w13_swiglu.argtypes = [S, P, P, P, P, P, P, P, P, sz, P]
        L.moe_grouped_gemm_w2.argtypes = [S, P, P, P, P, P, P, P, sz, P]
        L.moe_combine.argtypes = [S, P, P, P, P, P]
        L.moe_act_quant_e4m3.argtypes = [P, ctypes.c_int64, P, P, P]
        f32 = ctypes.c_float
        L.moe_act_quant_i8.argtypes = [P, ctypes.c_int64, i32, P, P, P]
        L.moe_balance_loss_workspace_bytes.argtypes = [i32, i32, i32]
        L.moe_balance_loss_workspace_bytes.restype = sz
        L.moe_balance_loss.argtypes = [P, P, P, i32, i32, i32, f32, P, P, P, P, P, sz, P]
        L.moe_balance_loss_backward.argtypes = [P, P, P, P, i32, i32, i32, f32, P, P, P]
        L.moe_topk_gating_backward.argtypes = [P, P, P, P, P, i32, i32, i32, i32, P, P]
        L.moe_router_backward.argtypes = [P, P, P, P, P, P, P, i32, i32, i32, i32, f32, P, P, P]
        L.moe_fused_forward.argtypes = [S, P, P, P, P, P, P, P, P, P, P, sz, P]
        L.moe_fused_forward_noalloc.argtypes = [S, P, P, P, P, P, P, P, P, P, P]
        L.moe_inv_rope_fp8_quant.argtypes = [P, P, P, i32, i32, i32, i32, i32, i32, P, P, P]
        L.moe_router_logits.argtypes = [S, P, P, P, P, sz, P]
        L.moe_fused_forward_router.argtypes = [S, P, P, P, P, P, P, P, P, P, P, P, sz, P]
        L.moe_fused_forward_events.argtypes = [S, P, P, P, P, P, P, P, P, P, P, sz, P,
                                               ctypes.POINTER(ctypes.c_void_p), i32]
        for name in EXPORTS:
            if name not in _NON_STATUS:
                getattr(L, name).restype = ctypes.c_int
        _lib = L
    return _lib


def _check(rc, what):
    if rc != 0:
        raise MoeError("%s failed: %d (%s)" % (what, rc, lib().moe_status_string(rc).decode()))


def _ptr(t):
    if t is None:
        return None
    if not t.is_cuda:
        raise MoeError("tensor must live on the GPU")
    if not t.is_contiguous():
        raise MoeError("tensor must be contiguous")
    return ctypes.c_void_p(t.data_ptr())


def _stream():
    return ctypes.c_void_p(torch.cuda.current_stream().cuda_stream)


def _need(ok, what):
    if not ok:
        raise MoeError(what)


def _arg(t, name, dtype, shape, dev):
    """Address of a tensor argument, checked against its declared type, shape
    and device index (the kernels trust all three)."""
    if t.dtype is not dtype or t.shape != shape or t.get_device() != dev or not t.is_contiguous():
        raise MoeError("%s must be a contiguous %s tensor of shape %s on GPU %d, got %s %s on %s%s" % (
            name, dtype, tuple(shape), dev, t.dtype, tuple(t.shape), t.device,
            "" if t.is_contiguous() else " (not contiguous)"))
    return t.data_ptr()


def _aligned_mask(t, T, dev):
    """A token mask the library takes: a slice of a longer one, which may start
    at any byte, is copied to an aligned address."""
    if t is None:
        return None
    _need(t.dtype is torch.uint8 or t.dtype is torch.bool,
          "token_mask must be uint8 or bool, got %s" % t.dtype)
    return t.clone() if _arg(t, "token_mask", t.dtype, (T,), dev) & 15 else t


def _mask_ptr(t):
    return None if t is None else t.data_ptr()


def _gpu(t, name):
    """Device index of the tensor that leads a call."""
    dev = t.get_device()
    if dev < 0:
        raise MoeError("%s must live on the GPU" % name)
    return dev


def _run(what, dev, *args):
    """Calls `what` on GPU `dev`'s current stream, with that GPU current."""
    f = getattr(_lib or lib(), what)
    if dev == _current_device():
        rc = f(*args, _raw_stream(dev))
    else:
        with torch.cuda.device(dev):
            rc = f(*args, _raw_stream(dev))
    if rc != 0:
        _check(rc, what)


def _check_i8(x, x_name, width, w, w_name, scale, ids=()):
    """INT8 mode: operand types and the scale per output channel (a scale of
    another mode's shape would be read out of range)."""
    dev = _gpu(x, x_name)
    _need(dev == _current_device(), "%s must live on the current GPU" % x_name)
    _need(w.dim() == 3 and w.shape[2] == width, "%s must be [E, channels, %d]" % (w_name, width))
    _need(w_name != "w13" or w.shape[1] % 2 == 0, "w13 must hold as many gate as up rows")
    _arg(x, x_name, torch.bfloat16, (x.shape[0], width), dev)
    _arg(w, w_name, torch.int8, w.shape, dev)
    _need(scale is not None, "%s_scale is required in INT8 mode" % w_name)
    _arg(scale, w_name + "_scale", torch.float32, w.shape[:2], dev)
    for name, t, n in ids:
        if t is not None:
            _arg(t, name, torch.int32, (n,), dev)


def mode_of(w):
    if w.dtype == torch.float32:
        return MOE_F32
    if w.dtype == torch.bfloat16:
        return MOE_BF16
    if w.dtype in (torch.float8_e4m3fn, torch.uint8):
        return MOE_FP8_E4M3
    if w.dtype == torch.int8:
        return MOE_INT8
    raise MoeError("unsupported weight dtype %s" % w.dtype)


def act_dtype(mode):
    return torch.float32 if mode == MOE_F32 else torch.bfloat16


def make_shape(T, H, E, k, I, mode, renormalize=True):
    return moe_shape(int(T), int(H), int(E), int(k), int(I), int(mode), int(bool(renormalize)))


def moe_check_shape(shape):
    return lib().moe_check_shape(ctypes.byref(shape))


def moe_workspace_bytes(shape):
    return lib().moe_workspace_bytes(ctypes.byref(shape))


def _workspace_i8(ws, dev):
    """INT8 mode: a caller's workspace is bytes on the tensors' GPU."""
    if ws is not None:
        _arg(ws, "ws", torch.uint8, ws.shape, dev)


def workspace(shape, device=None):
    """Allocate a workspace for `shape` (torch uint8, 256-byte aligned)."""
    n = moe_workspace_bytes(shape)
    if n == 0:
        raise MoeError("invalid shape")
    return torch.empty(n, dtype=torch.uint8, device=device or "cuda")


def moe_topk_gating(logits, k, renormalize=True, topk_ids=None, topk_weights=None):
    T, E = logits.shape
    if topk_ids is None:
        topk_ids = torch.empty((T, k), dtype=torch.int32, device=logits.device)
    if topk_weights is None:
        topk_weights = torch.empty((T, k), dtype=torch.float32, device=logits.device)
    _check(lib().moe_topk_gating(_ptr(logits), T, E, k, int(bool(renormalize)), _ptr(topk_ids),
                                 _ptr(topk_weights), _stream()), "moe_topk_gating")
    return topk_ids, topk_weights


def moe_align_sort_workspace_bytes(T, k, E):
    return lib().moe_align_sort_workspace_bytes(int(T), int(k), int(E))


def moe_align_sort(topk_ids, E, with_inv=True, ws=None):
    T, k = topk_ids.shape
    dev = topk_ids.device
    counts = torch.empty(E, dtype=torch.int32, device=dev)
    offsets = torch.empty(E + 1, dtype=torch.int32, device=dev)
    sorted_ids = torch.empty(T * k, dtype=torch.int32, device=dev)
    inv = torch.empty(T * k, dtype=torch.int32, device=dev) if with_inv else None
    if ws is None:
        n = moe_align_sort_workspace_bytes(T, k, E)
        if n == 0:
            raise MoeError("invalid grouping shape T=%d k=%d E=%d" % (T, k, E))
        ws = torch.empty(n, dtype=torch.uint8, device=dev)
    _check(lib().moe_align_sort(_ptr(topk_ids), T, k, E, _ptr(counts), _ptr(offsets),
                                _ptr(sorted_ids), _ptr(inv), _ptr(ws), ws.numel(), _stream()),
           "moe_align_sort")
    return counts, offsets, sorted_ids, inv


def moe_workspace_routing(shape):
    """Byte offsets of the routing arrays the fused entry points leave in a
    workspace of `shape` (a moe_routing_offsets)."""
    r = moe_routing_offsets()
    _check(lib().moe_workspace_routing(ctypes.byref(shape), ctypes.byref(r)),
           "moe_workspace_routing")
    return r


def routing_from_workspace(ws, T, E, k, H=128, I=128, mode=MOE_BF16):
    """Views (no copies) of the grouping a fused call left in `ws`: counts
    [E], offsets [E+1], sorted_ids [T*k], inv_perm [T*k] (int32), plus the
    ids [T,k] and weights [T,k] slots (filled only when the call kept them in
    the workspace).  H, I and mode must be the call's when they change the
    workspace layout (they place only regions after these)."""
    r = moe_workspace_routing(make_shape(T, H, E, k, I, mode))

    def view(off, n, dt):
        return ws[off:off + 4 * n].view(dt)

    return dict(counts=view(r.expert_counts, E, torch.int32),
                offsets=view(r.expert_offsets, E + 1, torch.int32),
                sorted_ids=view(r.sorted_ids, T * k, torch.int32),
                inv_perm=view(r.inv_perm, T * k, torch.int32),
                topk_ids=view(r.topk_ids, T * k, torch.int32).view(T, k),
                topk_weights=view(r.topk_weights, T * k, torch.float32).view(T, k))


def moe_grouped_gemm_w13_swiglu(x, w13, w13_scale, sorted_ids, expert_offsets, k, ws=None, h=None,
                                act_scales=None):
    mode = mode_of(w13)
    T, H = x.shape
    E, I2, _ = w13.shape
    I = I2 // 2
    shape = make_shape(T, H, E, k, I, mode)
    if mode == MOE_INT8:
        _check_i8(x, "x", H, w13, "w13", w13_scale,
                  (("sorted_ids", sorted_ids, T * k), ("expert_offsets", expert_offsets, E + 1)))
        _workspace_i8(ws, x.get_device())
        if h is not None:
            _arg(h, "h", torch.bfloat16, (T * k, I), x.get_device())
    ws = workspace(shape, x.device) if ws is None else ws
    if h is None:
        h = torch.empty((T * k, I), dtype=act_dtype(mode), device=x.device)
    if act_scales is None and mode != MOE_INT8:  # INT8: a scale per row, kept in the workspace
        act_scales = torch.zeros(4, dtype=torch.float32, device=x.device)
    _check(lib().moe_grouped_gemm_w13_swiglu(ctypes.byref(shape), _ptr(x), _ptr(w13),
                                             _ptr(w13_scale), _ptr(sorted_ids),
                                             _ptr(expert_offsets), _ptr(h), _ptr(act_scales),
                                             _ptr(ws), ws.numel(), _stream()),
           "moe_grouped_gemm_w13_swiglu")
    return h, act_scales


def moe_grouped_gemm_w2(h, w2, w2_scale, expert_offsets, act_scales, k, ws=None, y=None):
    mode = mode_of(w2)
    n_pairs, I = h.shape
    E, H, _ = w2.shape
    T = n_pairs // k
    shape = make_shape(T, H, E, k, I, mode)
    if mode == MOE_INT8:
        _need(n_pairs == T * k, "h must hold a multiple of k rows")
        _check_i8(h, "h", I, w2, "w2", w2_scale, (("expert_offsets", expert_offsets, E + 1),))
        _workspace_i8(ws, h.get_device())
        if y is not None:
            _arg(y, "y", torch.float32, (n_pairs, H), h.get_device())
    ws = workspace(shape, h.device) if ws is None else ws
    if y is None:
        y = torch.empty((n_pairs, H), dtype=torch.float32, device=h.device)
    _check(lib().moe_grouped_gemm_w2(ctypes.byref(shape), _ptr(h), _ptr(w2), _ptr(w2_scale),
                                     _ptr(expert_offsets), _ptr(act_scales), _ptr(y), _ptr(ws),
                                     ws.numel(), _stream()), "moe_grouped_gemm_w2")
    return y


def moe_act_quant_e4m3(a, codes=None, scales=None):
    """Per-tensor e4m3 codes of a bf16 tensor: (codes uint8, scales [s, amax] fp32)."""
    n = a.numel()
    if codes is None:
        codes = torch.empty(a.shape, dtype=torch.uint8, device=a.device)
    if scales is None:
        scales = torch.empty(2, dtype=torch.float32, device=a.device)
    _check(lib().moe_act_quant_e4m3(_ptr(a), n, _ptr(codes), _ptr(scales), _stream()),
           "moe_act_quant_e4m3")
    return codes, scales


def moe_act_quant_i8(a, codes=None, scales=None):
    """Per-row int8 codes of a bf16 tensor [..., n]: (codes int8 like a, scales
    fp32 [...], the value of one code)."""
    dev = _gpu(a, "a")
    _need(a.dim() >= 1, "a must have at least one dimension")
    lead, n = a.shape[:-1], a.shape[-1]
    if codes is None:
        codes = torch.empty(a.shape, dtype=torch.int8, device=dev)
    if scales is None:
        scales = torch.empty(lead, dtype=torch.float32, device=dev)
    _run("moe_act_quant_i8", dev, _arg(a, "a", torch.bfloat16, a.shape, dev),
         scales.numel(), n, _arg(codes, "codes", torch.int8, a.shape, dev),
         _arg(scales, "scales", torch.float32, lead, dev))
    return codes, scales


def moe_balance_loss_workspace_bytes(T, k, E):
    return lib().moe_balance_loss_workspace_bytes(int(T), int(k), int(E))


def balance_loss_workspace(T, k, E, device=None):
    """Allocate a workspace of moe_balance_loss (torch uint8)."""
    n = moe_balance_loss_workspace_bytes(T, k, E)
    _need(n > 0, "invalid router shape T=%d k=%d E=%d" % (T, k, E))
    return torch.empty(n, dtype=torch.uint8, device=device or "cuda")


def moe_balance_loss(logits, topk_ids, coef=1.0, token_mask=None, ws=None, loss=None,
                     expert_counts=None, expert_probs=None, token_count=None):
    """Load-balance loss coef * E * sum_e f_e P_e of the router logits [T,E]
    and the chosen experts topk_ids [T,k].  token_mask [T] (uint8 or bool,
    0 = padding) leaves tokens out.  Returns (loss [1] fp32, expert_counts
    [E] int32, expert_probs [E] fp32, token_count [1] int32).  A mask that is
    not 16-byte aligned is copied first."""
    dev = _gpu(logits, "logits")
    T, E = shape = logits.shape
    token_mask = _aligned_mask(token_mask, T, dev)
    k = topk_ids.shape[-1]
    pairs = (T, k)
    if ws is None:
        ws = balance_loss_workspace(T, k, E, dev)
    if loss is None:
        loss = torch.empty(1, dtype=torch.float32, device=dev)
    if expert_counts is None:
        expert_counts = torch.empty(E, dtype=torch.int32, device=dev)
    if expert_probs is None:
        expert_probs = torch.empty(E, dtype=torch.float32, device=dev)
    if token_count is None:
        token_count = torch.empty(1, dtype=torch.int32, device=dev)
    _run("moe_balance_loss", dev, _arg(logits, "logits", torch.float32, shape, dev),
         _arg(topk_ids, "topk_ids", torch.int32, pairs, dev), _mask_ptr(token_mask), T, E,
         k, coef, _arg(loss, "loss", torch.float32, (1,), dev),
         _arg(expert_counts, "expert_counts", torch.int32, (E,), dev),
         _arg(expert_probs, "expert_probs", torch.float32, (E,), dev),
         _arg(token_count, "token_count", torch.int32, (1,), dev),
         _arg(ws, "ws", torch.uint8, ws.shape, dev), ws.numel())
    return loss, expert_counts, expert_probs, token_count


def moe_balance_loss_backward(logits, expert_counts, token_count, k, coef, grad_loss,
                              token_mask=None, grad_logits=None):
    """Gradient [T,E] of moe_balance_loss on the logits, from the counts it
    returned; grad_loss [1] fp32."""
    dev = _gpu(logits, "logits")
    T, E = shape = logits.shape
    token_mask = _aligned_mask(token_mask, T, dev)
    if grad_logits is None:
        grad_logits = torch.empty(shape, dtype=torch.float32, device=dev)
    _run("moe_balance_loss_backward", dev, _arg(logits, "logits", torch.float32, shape, dev),
         _mask_ptr(token_mask),
         _arg(expert_counts, "expert_counts", torch.int32, (E,), dev),
         _arg(token_count, "token_count", torch.int32, (1,), dev), T, E, k, coef,
         _arg(grad_loss, "grad_loss", torch.float32, (1,), dev),
         _arg(grad_logits, "grad_logits", torch.float32, shape, dev))
    return grad_logits


def moe_topk_gating_backward(logits, topk_ids, topk_weights, grad_weights, renormalize=True,
                             token_mask=None, grad_logits=None):
    """Gradient [T,E] on the logits of the gating weights moe_topk_gating
    returned, from grad_weights [T,k]."""
    dev = _gpu(logits, "logits")
    T, E = shape = logits.shape
    token_mask = _aligned_mask(token_mask, T, dev)
    k = topk_ids.shape[-1]
    pairs = (T, k)
    if grad_logits is None:
        grad_logits = torch.empty(shape, dtype=torch.float32, device=dev)
    _run("moe_topk_gating_backward", dev, _arg(logits, "logits", torch.float32, shape, dev),
         _arg(topk_ids, "topk_ids", torch.int32, pairs, dev),
         _arg(topk_weights, "topk_weights", torch.float32, pairs, dev),
         _arg(grad_weights, "grad_weights", torch.float32, pairs, dev),
         _mask_ptr(token_mask), T, E, k, int(bool(renormalize)),
         _arg(grad_logits, "grad_logits", torch.float32, shape, dev))
    return grad_logits


def moe_router_backward(logits, topk_ids, topk_weights, grad_weights, expert_counts, token_count,
                        coef, grad_loss, renormalize=True, token_mask=None, grad_logits=None):
    """moe_topk_gating_backward plus moe_balance_loss_backward in one pass."""
    dev = _gpu(logits, "logits")
    T, E = shape = logits.shape
    token_mask = _aligned_mask(token_mask, T, dev)
    k = topk_ids.shape[-1]
    pairs = (T, k)
    if grad_logits is None:
        grad_logits = torch.empty(shape, dtype=torch.float32, device=dev)
    _run("moe_router_backward", dev, _arg(logits, "logits", torch.float32, shape, dev),
         _arg(topk_ids, "topk_ids", torch.int32, pairs, dev),
         _arg(topk_weights, "topk_weights", torch.float32, pairs, dev),
         _arg(grad_weights, "grad_weights", torch.float32, pairs, dev),
         _mask_ptr(token_mask),
         _arg(expert_counts, "expert_counts", torch.int32, (E,), dev),
         _arg(token_count, "token_count", torch.int32, (1,), dev), T, E, k,
         int(bool(renormalize)), coef, _arg(grad_loss, "grad_loss", torch.float32, (1,), dev),
         _arg(grad_logits, "grad_logits", torch.float32, shape, dev))
    return grad_logits


def moe_combine(y, inv_perm, topk_weights, mode, E=None, I=128, out=None):
    T, k = topk_weights.shape
    H = y.shape[1]
    shape = make_shape(T, H, E or k, k, I, mode)
    if out is None:
        out = torch.empty((T, H), dtype=act_dtype(mode), device=y.device)
    _check(lib().moe_combine(ctypes.byref(shape), _ptr(y), _ptr(inv_perm), _ptr(topk_weights),
                             _ptr(out), _stream()), "moe_combine")
    return out


def _check_i8_layer(x, w13, w13_scale, w2, w2_scale, T, H, E, I, k, out, logits=None,
                    topk_ids=None, topk_weights=None):
    _check_i8(x, "x", H, w13, "w13", w13_scale)
    dev = x.get_device()
    _arg(w2, "w2", torch.int8, (E, H, I), dev)
    _need(w2_scale is not None, "w2_scale is required in INT8 mode")
    _arg(w2_scale, "w2_scale", torch.float32, (E, H), dev)
    if out is not None:
        _arg(out, "out", torch.bfloat16, (T, H), dev)
    if logits is not None:
        _arg(logits, "logits", torch.float32, (T, E), dev)
    if topk_ids is not None:
        _arg(topk_ids, "topk_ids", torch.int32, (T, k), dev)
    if topk_weights is not None:
        _arg(topk_weights, "topk_weights", torch.float32, (T, k), dev)


def moe_fused_forward(x, logits, w13, w13_scale, w2, w2_scale, k, renormalize=True, out=None,
                      ws=None, topk_ids=None, topk_weights=None):
    mode = mode_of(w13)
    T, H = x.shape
    E, I2, _ = w13.shape
    I = I2 // 2
    if mode == MOE_INT8:
        _check_i8_layer(x, w13, w13_scale, w2, w2_scale, T, H, E, I, k, out, logits, topk_ids,
                        topk_weights)
        _workspace_i8(ws, x.get_device())
    shape = make_shape(T, H, E, k, I, mode, renormalize)
    ws = workspace(shape, x.device) if ws is None else ws
    if out is None:
        out = torch.empty((T, H), dtype=act_dtype(mode), device=x.device)
    _check(lib().moe_fused_forward(ctypes.byref(shape), _ptr(x), _ptr(logits), _ptr(w13),
                                   _ptr(w13_scale), _ptr(w2), _ptr(w2_scale), _ptr(out),
                                   _ptr(topk_ids), _ptr(topk_weights), _ptr(ws), ws.numel(),
                                   _stream()), "moe_fused_forward")
    return out


def moe_fused_forward_noalloc(x, logits, w13, w13_scale, w2, w2_scale, k, out,
                              renormalize=True, topk_ids=None, topk_weights=None):
    """moe_fused_forward on the library's static scratch: no workspace, and
    the caller passes `out` (nothing is allocated here either)."""
    mode = mode_of(w13)
    T, H = x.shape
    E, I2, _ = w13.shape
    if mode == MOE_INT8:
        _check_i8_layer(x, w13, w13_scale, w2, w2_scale, T, H, E, I2 // 2, k, out, logits,
                        topk_ids, topk_weights)
    shape = make_shape(T, H, E, k, I2 // 2, mode, renormalize)
    _check(lib().moe_fused_forward_noalloc(ctypes.byref(shape), _ptr(x), _ptr(logits), _ptr(w13),
                                           _ptr(w13_scale), _ptr(w2), _ptr(w2_scale), _ptr(out),
                                           _ptr(topk_ids), _ptr(topk_weights), _stream()),
           "moe_fused_forward_noalloc")
    return out


def moe_inv_rope_fp8_quant(x, positions, cos_sin, interleaved=False, codes=None, scales=None):
    """Inverse rotary embedding + per-(token, head) e4m3 quantisation.
    x [T, n_heads, head_dim] bf16, positions [T] int32, cos_sin [max_pos,
    rot_dim] fp32 -> (codes uint8 [T, n_heads, head_dim], scales fp32
    [T, n_heads])."""
    T, nh, hd = x.shape
    max_pos, rot = cos_sin.shape
    if codes is None:
        codes = torch.empty((T, nh, hd), dtype=torch.uint8, device=x.device)
    if scales is None:
        scales = torch.empty((T, nh), dtype=torch.float32, device=x.device)
    _check(lib().moe_inv_rope_fp8_quant(_ptr(x), _ptr(positions), _ptr(cos_sin), T, nh, hd, rot,
                                        max_pos, int(bool(interleaved)), _ptr(codes),
                                        _ptr(scales), _stream()), "moe_inv_rope_fp8_quant")
    return codes, scales


def moe_router_logits(x, wg, E=None, k=1, ws=None, logits=None):
    """Router GEMM: logits [T,E] fp32 = x [T,H] . wg [E,H]^T (fp32 or bf16
    operands of the same type, fp32 accumulation)."""
    T, H = x.shape
    E_, H2 = wg.shape
    assert H2 == H and (E is None or E == E_)
    mode = MOE_F32 if x.dtype == torch.float32 else MOE_BF16
    # the workspace depends only on T, H, E here; a minimal expert FFN shape
    shape = make_shape(T, H, E_, min(k, E_), 128, mode)
    ws = workspace(shape, x.device) if ws is None else ws
    if logits is None:
        logits = torch.empty((T, E_), dtype=torch.float32, device=x.device)
    _check(lib().moe_router_logits(ctypes.byref(shape), _ptr(x), _ptr(wg), _ptr(logits), _ptr(ws),
                                   ws.numel(), _stream()), "moe_router_logits")
    return logits


def moe_fused_forward_router(x, wg, w13, w13_scale, w2, w2_scale, k, renormalize=True, out=None,
                             ws=None, logits=None, topk_ids=None, topk_weights=None):
    """The whole layer from x and the router weights wg [E,H] (activation
    type); `logits` (optional [T,E] fp32) receives the router output."""
    mode = mode_of(w13)
    T, H = x.shape
    E, I2, _ = w13.shape
    I = I2 // 2
    assert tuple(wg.shape) == (E, H) and wg.dtype == act_dtype(mode)
    if mode == MOE_INT8:
        _check_i8_layer(x, w13, w13_scale, w2, w2_scale, T, H, E, I, k, out, logits, topk_ids,
                        topk_weights)
        _workspace_i8(ws, x.get_device())
    shape = make_shape(T, H, E, k, I, mode, renormalize)
    ws = workspace(shape, x.device) if ws is None else ws
    if out is None:
        out = torch.empty((T, H), dtype=act_dtype(mode), device=x.device)
    _check(lib().moe_fused_forward_router(ctypes.byref(shape), _ptr(x), _ptr(wg), _ptr(w13),
                                          _ptr(w13_scale), _ptr(w2), _ptr(w2_scale), _ptr(out),
                                          _ptr(logits), _ptr(topk_ids), _ptr(topk_weights),
                                          _ptr(ws), ws.numel(), _stream()),
           "moe_fused_forward_router")
    return out


def moe_fused_forward_events(x, logits, w13, w13_scale, w2, w2_scale, k, events, renormalize=True,
                             out=None, ws=None, topk_ids=None, topk_weights=None):
    """moe_fused_forward that also records the given hipEvent_t handles
    (NUM_STAGE_EVENTS integers, 0 or None to skip a boundary) at the stage
    boundaries."""
    mode = mode_of(w13)
    T, H = x.shape
    E, I2, _ = w13.shape
    I = I2 // 2
    if mode == MOE_INT8:
        _check_i8_layer(x, w13, w13_scale, w2, w2_scale, T, H, E, I, k, out, logits, topk_ids,
                        topk_weights)
        _workspace_i8(ws, x.get_device())
    shape = make_shape(T, H, E, k, I, mode, renormalize)
    ws = workspace(shape, x.device) if ws is None else ws
    if out is None:
        out = torch.empty((T, H), dtype=act_dtype(mode), device=x.device)
    ev = (ctypes.c_void_p * len(events))(*[ctypes.c_void_p(e or None) for e in events])
    _check(lib().moe_fused_forward_events(ctypes.byref(shape), _ptr(x), _ptr(logits), _ptr(w13),
                                          _ptr(w13_scale), _ptr(w2), _ptr(w2_scale), _ptr(out),
                                          _ptr(topk_ids), _ptr(topk_weights), _ptr(ws), ws.numel(),
                                          _stream(), ev, len(events)), "moe_fused_forward_events")
    return out
