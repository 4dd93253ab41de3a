"""The modes beside INT8 keep their scales' shapes and meaning."""
import pytest
import torch

import moe_layer_gating_amd as moe

pytestmark = pytest.mark.gpu


def _layer(T, dtype, seed=0):
    H, E, k, I = 256, 8, 2, 256
    g = torch.Generator(device="cuda").manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=g, device="cuda")
    x, logits = r(T, H), r(T, E)
    w13, w2 = r(E, 2 * I, H) / 16, r(E, H, I) / 16
    x = x if dtype == torch.float32 else x.bfloat16()
    return x, logits, w13.to(dtype), w2.to(dtype), k, E


@pytest.mark.parametrize("T", [3, 300])  # few-token and tiled kernels
def test_fp8_takes_one_scale_per_expert(T):
    """Powers of two pass through exactly: doubling w2's scales doubles the
    output, an expert's scale reaches its tokens only, and a call without
    scales is refused."""
    x, logits, w13, w2, k, E = _layer(T, torch.float8_e4m3fn)
    s13, s2 = torch.full((E,), 0.5, device="cuda"), torch.full((E,), 0.25, device="cuda")
    out = moe.moe_fused_forward(x, logits, w13, s13, w2, s2, k)
    assert bool(torch.isfinite(out).all()) and float(out.float().abs().max()) > 0
    assert torch.equal(moe.moe_fused_forward(x, logits, w13, s13, w2, 2 * s2, k), 2 * out)
    ids = moe.moe_topk_gating(logits, k)[0]
    s2[3] *= 4
    changed = (moe.moe_fused_forward(x, logits, w13, s13, w2, s2, k) != out).any(1)
    assert torch.equal(changed, (ids == 3).any(1))
    for bad in ((None, s2), (s13, None)):
        with pytest.raises(moe.MoeError):
            moe.moe_fused_forward(x, logits, w13, bad[0], w2, bad[1], k)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("T", [3, 300])
def test_float_weights_take_no_scales(T, dtype):
    """Scales beside fp32 or bf16 weights are ignored, int8-shaped ones too."""
    x, logits, w13, w2, k, E = _layer(T, dtype)
    out = moe.moe_fused_forward(x, logits, w13, None, w2, None, k)
    assert out.dtype == moe.act_dtype(moe.mode_of(w13)) and bool(torch.isfinite(out).all())
    s13, s2 = (torch.full(w.shape[:2], 9.0, device="cuda") for w in (w13, w2))
    assert torch.equal(moe.moe_fused_forward(x, logits, w13, s13, w2, s2, k), out)
