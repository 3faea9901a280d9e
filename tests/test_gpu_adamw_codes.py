"""The 8-bit states of kg_adamw bit for bit: the codes and scales that include/kgwgrad.h states,
from the states that the same step leaves in fp32."""
import numpy as np
import pytest
import torch

import fp8_grouped_gemm_tn_amd as kg

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
f32 = np.float32


def stated(x, up):
    """(codes, scales) of fp32 numpy x."""
    n = x.size
    b = np.zeros((-(-n // 128), 128), f32)
    b.reshape(-1)[:n] = x
    amax = np.abs(b).max(1)
    kept = amax >= f32(2.0 ** -118)
    with np.errstate(divide="ignore", invalid="ignore", over="ignore"):
        y = b * np.where(kept, f32(448) * (f32(1) / amax), f32(0))[:, None]
    y = y.astype(f32)
    if up:
        y = np.where((y > 0) & (y < f32(2.0 ** -9)), f32(2.0 ** -9), y)
    q = torch.from_numpy(y.reshape(-1)[:n].copy()).to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    return q, np.where(kept, (amax * (f32(1) / f32(448))).astype(f32), f32(0))


@pytest.mark.parametrize("spread", [0, 30, 60])
def test_codes_and_scales(spread):
    """Gradients of one size, and over up to 2^60: blocks below 2^-118, ties, far smaller elements
    than their block's largest."""
    n = 128 * 300 + 77
    g = torch.Generator(DEV).manual_seed(spread)
    grad = torch.randn(n, generator=g, device=DEV) * torch.exp2(
        -torch.rand(n, generator=g, device=DEV) * spread)
    scale = torch.exp2(torch.linspace(20, -125, 301, device=DEV).floor()).repeat_interleave(128)[:n]
    grad = grad * scale
    grad[500:600] = 0
    z = lambda *s, **kw: torch.zeros(*s, device=DEV, **kw)
    p, q = z(n), z(n)
    m, v = z(n), z(n)
    m8, v8 = z(n, dtype=torch.uint8), z(n, dtype=torch.uint8)
    ms, vs = z(301), z(301)
    kg.kg_adamw(kg.AdamWTable([p], [grad], [m], [v]), 1e-3)
    kg.kg_adamw(kg.AdamWTable([q], [grad], [m8], [v8], [ms], [vs]), 1e-3)
    assert torch.equal(p, q)  # the step sees the unrounded states
    for codes, scales, x, up in ((m8, ms, m.cpu().numpy(), False),
                                 (v8, vs, np.sqrt(v.cpu().numpy()), True)):
        want_q, want_s = stated(x, up)
        assert np.array_equal(scales.cpu().numpy().view(np.uint32), want_s.view(np.uint32))
        got = codes.cpu().numpy()
        # (a negative element that rounds to zero keeps its sign, in either)
        assert np.array_equal(got, want_q)
