"""kg_fprop_w4 at sizes that are chosen for the kernel that takes them, which each test asserts."""
import pytest
import torch

import fp8_grouped_gemm_tn_amd as kg
import test_gpu_fprop_w4 as base
import w4_plan

pytestmark = pytest.mark.gpu


def plan(M, G, N, K, kind, group, zp):
    return w4_plan.Plan(M, G, N, K, kind, group, zp, torch.cuda.get_device_properties(0).multi_processor_count)


def check(ms, N, K, group, kind, seed, zero=True, some=None):
    """Against the definition in 64 bits: outputs `some` (None: all)."""
    A, W, sw, zp, m = base.make(ms, N, K, group, kind, seed, zero=zero)
    if some is None:
        return base.check(A, W, sw, zp, m, group, torch.float32)
    D = torch.full((sum(ms), N), float("nan"), device="cuda")
    kg.kg_fprop_w4(A, W, sw, D, m, zp)
    assert kg.kg_status() == kg.KG_OK and D.isfinite().all()
    w, size = base.weights64(W[:, some], sw[:, some], None if zp is None else zp[:, some], group)
    a, at = A.cpu().double(), 0
    for g, n in enumerate(ms):
        want, mag = a[at:at + n] @ w[g].t(), a[at:at + n].abs() @ size[g].t()
        tol = (K / 32 + 3 * K / group + 16) * 2.0 ** -24 * mag
        assert bool(((D[at:at + n, some].cpu().double() - want).abs() <= tol).all()), g
        at += n


@pytest.mark.parametrize("ms,N,K,group,zero", [([1] * 8, 4096, 6656, 32, True), ([1], 5120, 13312, 32, True),
                                               ([1] * 4, 4096, 13216, 32, True), ([1] * 16, 2048, 13312, 64, True)])
def test_scales_that_fill_the_lds(ms, N, K, group, zero):
    """fp32 scales (and zero points) of few channels each and long rows: with 16 waves the tokens or the
    closing sums would no longer fit beside them."""
    p = plan(sum(ms), len(ms), N, K, "f32", group, zero)
    assert not p.streams or p.lds <= p.limit
    check(ms, N, K, group, "f32", 1, zero, some=torch.tensor([0, 1, 15, 16, 31, 32, N // 2 + 3, N - 17, N - 1]))


@pytest.mark.parametrize("kind,dtype", [("bf16", torch.bfloat16), ("f32", torch.float32), ("e2m1", torch.uint8)])
@pytest.mark.parametrize("rows", [1, 16, 100])
def test_no_channels(kind, dtype, rows):
    """K = 0: zeros, from as many rows as a workgroup takes at a time too."""
    D = torch.full((rows, 40), 3.0, device="cuda")
    empty = lambda *s, dtype: torch.empty(s, dtype=dtype, device="cuda")
    kg.kg_fprop_w4(empty(rows, 0, dtype=torch.bfloat16), empty(1, 40, 0, dtype=torch.uint8),
                   empty(1, 40, 0, dtype=dtype), D, torch.tensor([rows], dtype=torch.int32, device="cuda"))
    assert kg.kg_status() == kg.KG_OK and (D == 0).all()
