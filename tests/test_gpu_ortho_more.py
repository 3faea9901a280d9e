"""kg_orthogonalize's own error, apart from its result's rounding to bf16, which test_gpu_ortho's bound
contains three times over.

The result is o = y + r, with y within b of the 64-bit steps' w (relative to the norm) and r the
rounding to bf16. The rounding of N elements by amounts that do not depend on y - w adds in
quadrature: |o - w|^2 = |y - w|^2 + |r|^2 up to 2 <y - w, r>, whose deviation is at most
2 |y - w| |r| / sqrt(N). |r| is that of w's own rounding, up to 1 / sqrt(N) of itself. Six deviations
are left for both."""
import math

import pytest
import torch

import fp8_grouped_gemm_tn_amd as kg
import test_gpu_ortho as base

pytestmark = pytest.mark.gpu
BOUND = {1: 2e-3, 2: 2e-3, 3: 2e-3, 5: 2e-3, 8: 4e-3}  # by steps, as the header has it


def own_error(o, w, bound):
    o, w = o.detach().cpu().double(), w.cpu().double()
    assert o.isfinite().all()
    n = w.numel()
    off, size = float((o - w).norm()), float(w.norm())
    r = float((w.to(torch.bfloat16).double() - w).norm())
    most = (bound * size) ** 2 + r * r + 6 / math.sqrt(n) * (2 * bound * size * r + r * r)
    assert off * off <= most, (off / size, r / size)


@pytest.mark.parametrize("steps", sorted(BOUND))
@pytest.mark.parametrize("kind", ["noise", "low", "decay", "channels"])
@pytest.mark.parametrize("R,C", [(24, 40), (150, 100), (64, 256), (300, 77), (256, 384), (777, 1000)])
def test_own_error(R, C, kind, steps):
    u = base.update(R, C, R + steps, kind)
    own_error(kg.kg_orthogonalize(u, steps=steps), base.steps64(u, steps), BOUND[steps])


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("G,R,C", [(3, 2100, 1900), (2, 700, 4200), (8, 384, 256)])
def test_own_error_of_larger_ones(G, R, C, dtype):
    gen = torch.Generator("cuda").manual_seed(R)
    us = torch.randn((G, R, C), generator=gen, device="cuda").to(dtype)
    o = kg.kg_orthogonalize(us)
    for g in range(G):
        x = us[g].double()
        x = x / x.norm()
        x = x.t().contiguous() if R > C else x
        for _ in range(5):
            a = x @ x.t().contiguous()
            x = base.NS_A * x + (base.NS_B * a + base.NS_C * (a @ a)) @ x
        own_error(o[g], x.t() if R > C else x, 2e-3)


@pytest.mark.parametrize("steps", [8, 16, 64])
@pytest.mark.parametrize("R,C", [(40, 60), (300, 77), (200, 256)])
def test_many_steps_keep_the_singular_vectors(R, C, steps):
    """However many steps: with U = p s q the result is p t q with every t in 0.68 .. 1.27. Taken into
    p's and q's coordinates it is that diagonal, up to roundings of 5e-2 of the norm in all, of which one
    direction may have most, and to 2^-9 a direction of the result's own."""
    u = base.update(R, C, steps, "decay")
    p, s, q = torch.linalg.svd(u.cpu().double(), full_matrices=False)
    o = kg.kg_orthogonalize(u, steps=steps).cpu().double()
    t = p.t() @ o @ q.t()
    away = 5e-2 * float(o.norm())
    d = torch.diagonal(t)
    assert float((t - torch.diag(d)).norm()) <= away + 2.0 ** -8 * float(o.norm())
    assert float((o - (p * d) @ q).norm()) <= away + 2.0 ** -8 * float(o.norm())
    values = torch.linalg.svdvals(o)
    assert 0.68 - 0.02 <= float(values.min()) and float(values.max()) <= 1.27 + 0.02


@pytest.mark.parametrize("G,R,C,dtype", [(8, 384, 256, torch.float32), (3, 777, 1000, torch.bfloat16),
                                         (4, 60, 300, torch.float32), (17, 1100, 800, torch.bfloat16)])
def test_the_same_in_every_run(G, R, C, dtype):
    """Bit for bit, whatever the workspace held before."""
    gen = torch.Generator("cuda").manual_seed(R)
    u = torch.randn((G, R, C), generator=gen, device="cuda").to(dtype)
    ws = kg.new_orthogonalize_workspace(G, R, C, "cuda")
    outs = []
    for fill in (0, 255, 60, 0):
        ws.fill_(fill)
        outs.append(kg.kg_orthogonalize(u, ws=ws))
    assert all(torch.equal(outs[0], o) for o in outs[1:])


@pytest.mark.parametrize("G,R,C", [(600, 2048, 2048), (50_000, 100, 500)])
def test_many_matrices_past_32_bit_offsets(G, R, C):
    """More than 2^31 elements: the matrices behind that are right (their inputs repeat, so do they)."""
    assert G * R * C > 2 ** 31
    gen = torch.Generator("cuda").manual_seed(G)
    some = torch.randn((10, R, C), generator=gen, device="cuda").to(torch.bfloat16)
    us = some.repeat(G // 10, 1, 1)
    o = kg.kg_orthogonalize(us, us)
    for g in (0, 7):
        x = some[g].double()
        x = x / x.norm()
        for _ in range(5):
            a = x @ x.t().contiguous()
            x = base.NS_A * x + (base.NS_B * a + base.NS_C * (a @ a)) @ x
        own_error(o[G - 10 + g], x, 2e-3)
    o = o.view(G // 10, 10, -1)
    for i in range(1, G // 10):
        # (tiles are chosen by all matrices together, and a rounding that falls otherwise is multiplied by
        # the steps: two results may each be 2e-3 off, and rounded by half a step)
        off = (o[i].float() - o[0].float()).norm(dim=1) / o[0].float().norm(dim=1)
        assert float(off.max()) <= 4e-3 + 2 * 2.0 ** -8, i
