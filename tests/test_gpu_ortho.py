"""kg_orthogonalize against the same Newton-Schulz steps in 64 bits.

Tolerance. fp16 rounds an operand by 2^-11 of itself at most, 2^-11 / sqrt(12) in the mean square.
In a step X's rounding enters through B X, with |B| <= 2.9, and A's and B's through their off-diagonal
parts (the diagonals are carried beside them), together at most about 2.9 + 4.8 + 1 times that of a
unit. The state is carried exactly up to the last step, so what counts are the last three steps' or
so, the later steps multiplying errors by 1 or less where singular values are near 1: sqrt(3) * 8.7 *
2^-11 / sqrt(12) = 2e-3 of the result's norm. The rounding to bf16 adds at most 2^-8 of each
element."""
import pytest
import torch

import fp8_grouped_gemm_tn_amd as kg

pytestmark = pytest.mark.gpu
TOL = 2e-3 + 2.0 ** -8
NS_A, NS_B, NS_C = 3.4445, -4.7750, 2.0315


def steps64(u, steps=5):
    x = u.detach().cpu().double()
    size = x.norm()
    x = x / size if size > 0 else x
    turn = x.shape[0] > x.shape[1]
    x = x.t() if turn else x
    for _ in range(steps):
        a = x @ x.t()
        x = NS_A * x + (NS_B * a + NS_C * (a @ a)) @ x
    return x.t() if turn else x


def near(got, want):
    got = got.detach().cpu().double()
    assert got.isfinite().all()
    off = float((got - want).norm() / want.norm())
    assert off <= TOL, off
    return off


def update(R, C, seed, kind="noise", dtype=torch.float32):
    gen = torch.Generator("cuda").manual_seed(seed)
    r = lambda *s: torch.randn(s, generator=gen, device="cuda")
    u = r(R, C)
    if kind == "low":  # few directions that stand out by far
        u = 0.01 * u + r(R, 4) @ r(4, C)
    elif kind == "decay":  # singular values over three decades
        k = min(R, C)
        p, _ = torch.linalg.qr(r(max(R, C), k).cpu().double())
        q, _ = torch.linalg.qr(r(k, k).cpu().double())
        u = (p * torch.logspace(0, -3, k, dtype=torch.float64)) @ q
        u = (u if R >= C else u.t()).float().cuda()
    elif kind == "channels":
        u = u * torch.exp(r(1, C)) * torch.exp(r(R, 1))
    return u.to(dtype).contiguous()


@pytest.mark.parametrize("R,C", [(1, 1), (1, 9), (9, 1), (7, 5), (64, 64), (63, 65), (65, 200), (128, 128),
                                 (129, 127), (300, 77), (256, 512), (511, 260), (640, 640), (777, 1000)])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_sizes(R, C, dtype):
    u = update(R, C, R + C, dtype=dtype)
    o = kg.kg_orthogonalize(u)
    assert o.dtype == torch.bfloat16 and o.shape == u.shape
    near(o, steps64(u))


@pytest.mark.parametrize("kind", ["low", "decay", "channels"])
@pytest.mark.parametrize("R,C", [(128, 256), (500, 300), (512, 1024)])
def test_spectra(kind, R, C):
    u = update(R, C, R, kind)
    near(kg.kg_orthogonalize(u), steps64(u))


@pytest.mark.parametrize("G", [1, 3, 40])
def test_batches(G):
    us = torch.stack([update(96, 160, i) * 10.0 ** (i % 7 - 3) for i in range(G)])
    o = kg.kg_orthogonalize(us)
    for i in range(G):
        near(o[i], steps64(us[i]))
        assert torch.equal(o[i], kg.kg_orthogonalize(us[i]))


@pytest.mark.parametrize("G,R,C", [(70, 300, 400), (70, 400, 300), (3, 2100, 1900), (2, 1500, 4200), (1, 4096, 2112)])
def test_large_tiles(G, R, C):
    """Sizes at which products take the larger tiles; every matrix against 64 bits on the GPU."""
    gen = torch.Generator("cuda").manual_seed(G)
    us = torch.randn((G, R, C), generator=gen, device="cuda")
    o = kg.kg_orthogonalize(us)
    for g in range(0, G, max(1, G // 3)):
        x = us[g].double()
        x = x / x.norm()
        x = x.t() if R > C else x
        for _ in range(5):
            a = x @ x.t()
            x = NS_A * x + (NS_B * a + NS_C * (a @ a)) @ x
        near(o[g], (x.t() if R > C else x).cpu())


@pytest.mark.parametrize("G,R,C", [(30, 800, 1000), (26, 1000, 800), (17, 800, 1100), (17, 1100, 800), (101, 500, 700)])
def test_last_rounds(G, R, C):
    """Numbers of tiles a little above a multiple of the compute units, whose last ones are done as smaller
    ones; every matrix."""
    gen = torch.Generator("cuda").manual_seed(G)
    us = torch.randn((G, R, C), generator=gen, device="cuda").to(torch.bfloat16)
    o = kg.kg_orthogonalize(us)
    for g in range(G):
        x = us[g].double()
        x = x / x.norm()
        x = x.t() if R > C else x
        for _ in range(5):
            a = x @ x.t()
            x = NS_A * x + (NS_B * a + NS_C * (a @ a)) @ x
        near(o[g], (x.t() if R > C else x).cpu())


@pytest.mark.parametrize("G,n,m", [(3, 1, 2048), (2, 7, 30), (5, 32, 32), (2, 32, 2048), (2, 32, 2049),
                                   (2, 33, 100), (40, 64, 1024), (2, 64, 1025), (3, 50, 999), (2, 65, 66),
                                   (3, 128, 384), (2, 128, 385), (300, 100, 380), (2, 129, 300)])
@pytest.mark.parametrize("tall", [False, True])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_small(G, n, m, tall, dtype):
    """Matrices of a workgroup each, and the first ones past that."""
    R, C = (m, n) if tall else (n, m)
    us = torch.stack([update(R, C, 7 * G + g, "channels" if g % 2 else "noise", dtype) for g in range(min(G, 4))])
    us = us.repeat(-(-G // 4), 1, 1)[:G].contiguous() if G > 4 else us
    guard = torch.full((G * R * C + 64,), 7.0, dtype=torch.bfloat16, device="cuda")
    o = guard[32:-32].view(G, R, C)
    kg.kg_orthogonalize(us, o)
    assert (guard[:32] == 7).all() and (guard[-32:] == 7).all()
    for g in range(min(G, 4)):
        near(o[g], steps64(us[g]))
    for g in range(4, G):
        assert torch.equal(o[g], o[g % 4])


def test_small_shifted_over_its_inputs():
    """The result lies over the inputs of other matrices."""
    us = torch.stack([update(40, 96, g) for g in range(6)])
    want = kg.kg_orthogonalize(us)
    for shift in (0, 40 * 96 * 3 + 8):
        space = torch.zeros(us.numel() * 4 + 64 * 1024, dtype=torch.uint8, device="cuda")
        u = space[1024:1024 + us.numel() * 4].view(torch.float32).view(us.shape)
        u.copy_(us)
        o = space[1024 + 2 * shift:][:us.numel() * 2].view(torch.bfloat16).view(us.shape)
        kg.kg_orthogonalize(u, o)
        for g in range(6):
            near(o[g], steps64(us[g]))
            assert (o[g].float() - want[g].float()).abs().max() <= 2.0 ** -6


@pytest.mark.parametrize("steps", [1, 2, 3, 8])
def test_steps(steps):
    u = update(150, 100, steps)
    near(kg.kg_orthogonalize(u, steps=steps), steps64(u, steps))


def test_singular_values():
    o = kg.kg_orthogonalize(update(300, 500, 1))
    s = torch.linalg.svdvals(o.cpu().double())
    assert 0.6 < float(s.min()) and float(s.max()) < 1.3


@pytest.mark.parametrize("scale", [1e-30, 1e-12, 1e12, 1e30])
def test_any_size_of_update(scale):
    """The result does not depend on the update's size, where its squares leave fp32's range too."""
    u = update(100, 130, 3) * scale
    near(kg.kg_orthogonalize(u), steps64(u))


def test_few_directions():
    """Rank one, one element, a zero matrix and a zero row among others."""
    us = torch.zeros((4, 70, 90), device="cuda")
    us[0] = update(70, 1, 1) @ update(1, 90, 2)
    us[1, 3, 5] = -2.0
    us[3] = update(70, 90, 3)
    us[3, 10], us[3, :, 20] = 0, 0
    o = kg.kg_orthogonalize(us)
    near(o[0], steps64(us[0]))
    near(o[1], steps64(us[1]))
    assert (o[2] == 0).all() and (o[3, 10] == 0).all() and (o[3, :, 20] == 0).all()
    near(o[3], steps64(us[3]))


def test_not_finite_matrices_stay_apart():
    us = torch.stack([update(80, 70, i) for i in range(4)])
    want = kg.kg_orthogonalize(us)
    us[1, 3, 3], us[2, 0, 0] = float("nan"), float("inf")
    o = kg.kg_orthogonalize(us)
    assert torch.equal(o[0], want[0]) and torch.equal(o[3], want[3])
    assert o[1].isnan().any() and o[2].isnan().any()


def test_in_place_and_around():
    """O may be U; nothing around it is written."""
    store = torch.full((3 * 50 * 37 + 20,), 7.0, dtype=torch.bfloat16, device="cuda")
    u = store[9:9 + 3 * 50 * 37].view(3, 50, 37)
    u.copy_(torch.stack([update(50, 37, i) for i in range(3)]))
    want = kg.kg_orthogonalize(u.clone())
    assert kg.kg_orthogonalize(u, u) is u
    assert torch.equal(u, want)
    assert (store[:9] == 7).all() and (store[9 + 3 * 50 * 37:] == 7).all()


def test_workspace_of_the_exact_size():
    """A workspace between guard bytes, filled with NaN patterns before the call."""
    n = kg.new_orthogonalize_workspace(2, 130, 200, "cuda").numel()
    store = torch.full((n + 512,), 255, dtype=torch.uint8, device="cuda")
    u = torch.stack([update(130, 200, i) for i in range(2)])
    o = kg.kg_orthogonalize(u, ws=store[256:256 + n])
    assert (store[:256] == 255).all() and (store[256 + n:] == 255).all()
    assert torch.equal(o, kg.kg_orthogonalize(u))


def test_empty():
    for shape in ((0, 3, 4), (2, 0, 4), (2, 3, 0), (0, 5)):
        assert kg.kg_orthogonalize(torch.empty(shape, device="cuda")).shape == shape


def test_on_a_stream_and_in_a_graph():
    u = torch.stack([update(200, 140, i) for i in range(3)])
    want = kg.kg_orthogonalize(u)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    o = kg.kg_orthogonalize(u, stream=s)
    torch.cuda.current_stream().wait_stream(s)
    assert torch.equal(o, want)
    ws, got = kg.new_orthogonalize_workspace(3, 200, 140, "cuda"), torch.empty_like(want)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        kg.kg_orthogonalize(u, got, ws=ws)
    for seed in range(3):
        u.copy_(torch.stack([update(200, 140, 10 * seed + i) for i in range(3)]))
        got.zero_()
        g.replay()
        assert torch.equal(got, kg.kg_orthogonalize(u))


def test_small_ones_in_a_graph_and_on_two_streams():
    """One launch each: in a captured graph whose workspace eager calls share, in turn, and at once on two streams."""
    us = torch.stack([update(60, 300, i, dtype=torch.bfloat16) for i in range(5)])
    want = kg.kg_orthogonalize(us)
    for g in range(5):
        near(want[g], steps64(us[g]))
    ws, got = kg.new_orthogonalize_workspace(5, 60, 300, "cuda"), torch.empty_like(want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        kg.kg_orthogonalize(us, got, ws=ws)
    for _ in range(3):
        got.zero_()
        graph.replay()
        assert torch.equal(got, want)
        assert torch.equal(kg.kg_orthogonalize(us, ws=ws), want)
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    outs = [[kg.kg_orthogonalize(us, stream=s) for s in streams] for _ in range(10)]
    torch.cuda.synchronize()
    assert all(torch.equal(o, want) for two in outs for o in two)
    # in place
    same = us.clone()
    kg.kg_orthogonalize(same, same)
    assert torch.equal(same, want)


def test_a_step_on_expert_gradients():
    """kg_wgrad's gradient of a layer's weights made orthogonal: against 64 bits, and along the
    gradient."""
    G, M, N, T = 3, 128, 256, 300
    gen = torch.Generator("cuda").manual_seed(1)
    x = torch.randn((T, N), generator=gen, device="cuda").to(torch.bfloat16)
    dy = torch.randn((T, M), generator=gen, device="cuda").to(torch.bfloat16)
    ks = torch.tensor([100, 0, 200], dtype=torch.int32, device="cuda")
    D = torch.empty((G, M, N), device="cuda")
    kg.kg_wgrad(dy, None, x, None, None, D, ks, 128, kg.KG_BF16)
    assert kg.kg_status() == kg.KG_OK
    o = kg.kg_orthogonalize(D)
    assert (o[1] == 0).all()
    for g, (a, b) in ((0, (0, 100)), (2, (100, 300))):
        grad = dy[a:b].cpu().double().t() @ x[a:b].cpu().double()
        near(o[g], steps64(grad))
        assert float((grad * o[g].cpu().double()).sum()) > 0
