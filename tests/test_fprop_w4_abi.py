"""Host-side checks of kg_fprop_w4: bad arguments are refused before anything is enqueued (no HIP
call is made here); the helpers that make 4-bit weights."""
import pytest
import torch

import fp8_grouped_gemm_tn_amd as kg
from fp8_grouped_gemm_tn_amd import _binding as B
from fp8_grouped_gemm_tn_amd import inputs

GB = 1 << 30
FAKE = [(i + 1) * 64 * GB for i in range(12)]  # aligned, far apart, never dereferenced


def w4(A=FAKE[0], lda=256, W=FAKE[1], sw=FAKE[2], zp=FAKE[3], D=FAKE[4], ldd=64, ms=FAKE[5], G=3,
       N=64, K=256, M=100, group=128, kind=B.KG_W4_INT_F32, flags=0):
    return B.lib().kg_fprop_w4(A, lda, W, sw, zp, D, ldd, ms, G, N, K, M, group, kind, flags, None)


@pytest.mark.parametrize("kw,code", [
    (dict(kind=3), B.KG_ERR_DTYPE),
    (dict(kind=-1), B.KG_ERR_DTYPE),
    (dict(flags=kg.KG_FLAG_FP8_MFMA), B.KG_ERR_DTYPE),
    (dict(kind=B.KG_W4_E2M1, group=32), B.KG_ERR_DTYPE),  # with zero points
    (dict(G=-1), B.KG_ERR_SHAPE),
    (dict(M=-1), B.KG_ERR_SHAPE),
    (dict(lda=248), B.KG_ERR_SHAPE),
    (dict(ldd=63), B.KG_ERR_SHAPE),
    (dict(group=16), B.KG_ERR_GRAN),
    (dict(group=0), B.KG_ERR_GRAN),
    (dict(group=256), B.KG_ERR_GRAN),
    (dict(kind=B.KG_W4_E2M1, zp=None, group=64), B.KG_ERR_GRAN),
    (dict(G=1025), B.KG_ERR_UNSUPPORTED),
    (dict(lda=(1 << 22) + 8), B.KG_ERR_UNSUPPORTED),
    (dict(N=(1 << 24) + 1, ldd=(1 << 24) + 1), B.KG_ERR_UNSUPPORTED),
    (dict(K=192), B.KG_ERR_ALIGN),
    (dict(lda=260), B.KG_ERR_ALIGN),
    (dict(A=None), B.KG_ERR_NULL),
    (dict(W=None), B.KG_ERR_NULL),
    (dict(sw=None), B.KG_ERR_NULL),
    (dict(D=None), B.KG_ERR_NULL),
    (dict(ms=None), B.KG_ERR_NULL),
    (dict(A=FAKE[0] + 8), B.KG_ERR_ALIGN),
    (dict(W=FAKE[1] + 8), B.KG_ERR_ALIGN),
    (dict(sw=FAKE[2] + 2), B.KG_ERR_ALIGN),
    (dict(sw=FAKE[2] + 1, kind=B.KG_W4_INT_BF16), B.KG_ERR_ALIGN),
    (dict(D=FAKE[4] + 2), B.KG_ERR_ALIGN),
    (dict(ms=FAKE[5] + 2), B.KG_ERR_ALIGN),
    (dict(D=FAKE[0]), B.KG_ERR_ALIAS),
    (dict(D=FAKE[1] + 3 * 64 * 128 - 4), B.KG_ERR_ALIAS),
    (dict(D=FAKE[2] + 3 * 64 * 2 * 4 - 4), B.KG_ERR_ALIAS),
    (dict(D=FAKE[3] + 3 * 64 * 2 - 4), B.KG_ERR_ALIAS),
    (dict(ms=FAKE[4] + 4 * 64 * 99), B.KG_ERR_ALIAS),
    (dict(G=0), B.KG_OK),
    (dict(N=0, ldd=0), B.KG_OK),
    (dict(M=0), B.KG_OK),
])
def test_refusals(kw, code):
    assert w4(**kw) == code


def tensors(**kw):
    t = dict(A=torch.zeros(4, 256, dtype=torch.bfloat16), W=torch.zeros(2, 8, 128, dtype=torch.uint8),
             sw=torch.zeros(2, 8, 2), D=torch.zeros(4, 8), ms=torch.zeros(2, dtype=torch.int32))
    t.update(kw)
    return t


@pytest.mark.parametrize("kw", [
    dict(A=torch.zeros(4, 256)),
    dict(A=torch.zeros(4, 128, dtype=torch.bfloat16)),
    dict(W=torch.zeros(2, 8, 128)),
    dict(W=torch.zeros(2, 8, 256, dtype=torch.uint8)[:, :, ::2]),
    dict(sw=torch.zeros(2, 8, 2, dtype=torch.float16)),
    dict(sw=torch.zeros(2, 9, 2)),
    dict(sw=torch.zeros(2, 8, 3)),
    dict(zp=torch.zeros(2, 8, 2)),
    dict(zp=torch.zeros(2, 8, 4, dtype=torch.uint8)),
    dict(D=torch.zeros(4, 8, dtype=torch.float16)),
    dict(D=torch.zeros(5, 8)),
    dict(ms=torch.zeros(3, dtype=torch.int32)),
    dict(ms=torch.zeros(2)),
    dict(),  # not on a GPU
])
def test_binding_refuses(kw):
    with pytest.raises(ValueError):
        kg.kg_fprop_w4(**tensors(**kw))


def codes_of(W):
    return torch.stack((W & 15, W >> 4), 3).flatten(2).long()


@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("zero", [True, False])
def test_quantised_weights_are_half_a_step_off(group, zero):
    w = torch.randn((2, 5, 256), generator=torch.Generator().manual_seed(group))
    w[0, 0, :group] = 0
    W, s, z = inputs.quantize_w4(w, group, zero, torch.float32)
    s = s.repeat_interleave(group, 2)
    z = 8.0 if z is None else z.float().repeat_interleave(group, 2)
    back = (codes_of(W) - z) * s
    # half a step, and with zero points half a step more where the point's rounding cuts off an end
    assert bool(((back - w).abs() <= (1.0 if zero else 0.5) * s * (1 + 1e-5)).all())
    assert bool((back[0, 0, :group] == 0).all())


def test_e2m1_weights_are_the_nearest_codes():
    w = torch.randn((1, 7, 96), generator=torch.Generator().manual_seed(1))
    w[0, 0, :32] = 0
    W, e = inputs.quantize_e2m1(w)
    values = torch.tensor([0.0, 0.5, 1, 1.5, 2, 3, 4, 6])
    values = torch.cat((values, -values))
    scale = torch.exp2(e.float() - 127).repeat_interleave(32, 2)
    off = (values[codes_of(W)] * scale - w).abs()
    best = (values * scale[..., None] - w[..., None]).abs().amin(-1)
    assert torch.equal(off, best)
    assert bool((w.abs().unflatten(2, (-1, 32)).amax(3) < 8 * torch.exp2(e.float() - 127) + (e == 0)).all())
