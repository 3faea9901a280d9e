"""kg_fprop_w4 against the definition in 64 bits.

Tolerance. Products are exact; fp32 rounds each running sum by 2^-24 of its size at most: after every
MFMA of 32 channels (K / 32), and for whole-number codes three times per group when a group's sum
is corrected, scaled and added (the correction's own sum among them). With S the sum of
magnitudes that pass through those sums (|a| s (16 + q + 16 + z), or |a w|) a result is off by at
most (K / 32 + 3 K / group + 16) 2^-24 S; a bf16 result by half a step more, 2^-8 of itself."""
import math

import pytest
import torch

import fp8_grouped_gemm_tn_amd as kg
from fp8_grouped_gemm_tn_amd import inputs

pytestmark = pytest.mark.gpu
E2M1 = torch.tensor([0.0, 0.5, 1, 1.5, 2, 3, 4, 6, -0.0, -0.5, -1, -1.5, -2, -3, -4, -6]).double()


def make(ms, N, K, group, kind, seed, pad=0, zero=True):
    gen = torch.Generator("cuda").manual_seed(seed)
    G, M = len(ms), sum(ms)
    rand = lambda lo, hi, *s: torch.randint(lo, hi, s, generator=gen, device="cuda", dtype=torch.uint8)
    W = rand(0, 256, G, N, K // 2)
    zp = None
    if kind == "e2m1":
        sw = rand(110, 130, G, N, K // 32)
    else:
        sw = (torch.rand((G, N, K // group), generator=gen, device="cuda") - 0.3).to(
            torch.bfloat16 if kind == "bf16" else torch.float32)
        if zero:
            zp = rand(0, 16, G, N, K // group)
    A = torch.full((M, K + pad), math.nan, dtype=torch.bfloat16, device="cuda")[:, :K]
    A.copy_(torch.randn((M, K), generator=gen, device="cuda"))
    return A, W, sw, zp, torch.tensor(ms, dtype=torch.int32, device="cuda")


def weights64(W, sw, zp, group):
    """The weights and the magnitudes that pass through the sums, [G, N, K] in 64 bits."""
    W, sw = W.cpu(), sw.cpu()
    q = torch.stack((W & 15, W >> 4), 3).flatten(2).long()
    if sw.dtype == torch.uint8:
        w = E2M1[q] * torch.exp2(sw.double() - 127).repeat_interleave(32, 2)
        return w, w.abs()
    z = 8.0 if zp is None else zp.cpu().double().repeat_interleave(group, 2)
    s = sw.double().repeat_interleave(group, 2)
    return (q - z) * s, (32 + q + z) * s.abs()


def check(A, W, sw, zp, ms, group, out, ldd=0):
    M, (G, N, K) = A.shape[0], (W.shape[0], W.shape[1], W.shape[2] * 2)
    wide = torch.full((M + 2, N + ldd), -77.0, dtype=out, device="cuda")
    D = wide[1:M + 1, :N]
    kg.kg_fprop_w4(A, W, sw, D, ms, zp)
    assert kg.kg_status() == kg.KG_OK
    assert (wide[0] == -77).all() and (wide[M + 1] == -77).all() and (wide[:, N:] == -77).all()
    w, size = weights64(W, sw, zp, group)
    a, at = A.cpu().double(), 0
    for g, n in enumerate(ms.tolist()):
        want, mag = a[at:at + n] @ w[g].t(), a[at:at + n].abs() @ size[g].t()
        tol = (K / 32 + 3 * K / group + 16) * 2.0 ** -24 * mag
        if out == torch.bfloat16:
            tol = tol + 2.0 ** -8 * want.abs()
        got = D[at:at + n].cpu().double()
        assert got.isfinite().all() and bool(((got - want).abs() <= tol).all()), (g, n)
        at += n
    return D


KINDS = [("bf16", 128), ("bf16", 64), ("bf16", 32), ("f32", 128), ("f32", 64), ("f32", 32), ("e2m1", 32)]
ROWS = [[1], [16], [3, 0, 1, 7], [17], [0, 40, 0, 64, 1, 0], [65, 200], [128], [129, 0, 3]]


@pytest.mark.parametrize("kind,group", KINDS)
@pytest.mark.parametrize("ms", ROWS, ids=str)
@pytest.mark.parametrize("out", [torch.bfloat16, torch.float32])
def test_rows(kind, group, ms, out):
    for N, K in ((33, 3 * group), (272, 1024 + group), (64, 2048)):
        A, W, sw, zp, m = make(ms, N, K, group, kind, N)
        check(A, W, sw, zp, m, group, out)


@pytest.mark.parametrize("kind,group", KINDS)
@pytest.mark.parametrize("rows", [2, 33, 200])
def test_odd(kind, group, rows):
    """Odd numbers of outputs, one group, wider matrices, no zero points."""
    for N, K, pad, ldd in ((1, group, 8, 1), (257, 5 * group, 40, 0), (31, 11 * group, 0, 7), (513, 128, 8, 3)):
        A, W, sw, zp, m = make([rows, 0, 5], N, K, group, kind, N + rows, pad, zero=N == 257)
        check(A, W, sw, zp, m, group, torch.bfloat16 if N % 4 == 1 else torch.float32, ldd)


@pytest.mark.parametrize("kind,group", [("bf16", 128), ("f32", 32), ("e2m1", 32)])
def test_many_experts(kind, group):
    gen = torch.Generator().manual_seed(1)
    for total in (40, 700, 3000):
        ms = torch.bincount(torch.randint(0, 200, (total,), generator=gen), minlength=256).tolist()
        A, W, sw, zp, m = make(ms, 96, 256, group, kind, total)
        check(A, W, sw, zp, m, group, torch.bfloat16)


@pytest.mark.parametrize("kind,group", [("bf16", 128), ("e2m1", 32)])
@pytest.mark.parametrize("G,M", [(1, 1), (2, 20), (1, 300)])
def test_one_row_of_long_ones(kind, group, G, M):
    ms = [M - (G - 1)] + [1] * (G - 1)
    A, W, sw, zp, m = make(ms, 160, 8192, group, kind, M)
    check(A, W, sw, zp, m, group, torch.float32)


@pytest.mark.parametrize("kind,group", KINDS)
@pytest.mark.parametrize("G,N,K,total", [(60, 2080, 256, 80), (70, 4200, 128, 300), (33, 4100, 640, 33), (200, 1030, 128, 1500)])
def test_many_workgroups(kind, group, G, N, K, total):
    """More workgroups than compute units hold at once, in which several sets of outputs share rows."""
    gen = torch.Generator().manual_seed(G)
    ms = torch.bincount(torch.randint(0, G, (total,), generator=gen), minlength=G).tolist()
    A, W, sw, zp, m = make(ms, N, K, group, kind, G)
    check(A, W, sw, zp, m, group, torch.bfloat16 if kind == "bf16" else torch.float32)


def test_zero_points_past_fifteen():
    A, W, sw, zp, m = make([5, 70], 40, 256, 64, "f32", 1)
    zp.copy_(torch.arange(zp.numel(), device="cuda").view(zp.shape) % 256)
    check(A, W, sw, zp, m, 64, torch.float32)


@pytest.mark.parametrize("rows", [1, 100])
def test_exponents(rows):
    """Every exponent byte from 2 to 252, one at a time; 255 is NaN; 0 and 1 next to nothing."""
    K = 32
    A = torch.zeros((rows, K), dtype=torch.bfloat16, device="cuda")
    A[:, 3], A[:, 4] = 1, 0.5
    W = torch.zeros((1, 256, K // 2), dtype=torch.uint8, device="cuda")
    W[0, :, 1], W[0, :, 2] = 0x90, 0x07  # channel 3: -0.5; channel 4: 6
    sw = torch.arange(256, dtype=torch.int32, device="cuda").to(torch.uint8).view(1, 256, 1)
    D = torch.empty((rows, 256), device="cuda")
    kg.kg_fprop_w4(A, W, sw, D, torch.tensor([rows], dtype=torch.int32, device="cuda"))
    want = 2.5 * torch.exp2(torch.arange(256).double() - 127)
    got = D.cpu().double()
    assert torch.equal(got[:, 2:253], want[2:253].expand(rows, -1))
    assert (got[:, :2].abs() <= 2.0 ** -124).all() and got[:, 255].isnan().all()
    assert (got[:, 253] == want[253]).all() or got[:, 253].isinf().all()


def test_every_code():
    """All 256 bytes of codes, alone in their channels: exact."""
    W = torch.zeros((1, 256, 16), dtype=torch.uint8, device="cuda")
    W[0, :, 5] = torch.arange(256, device="cuda").to(torch.uint8)
    A = torch.zeros((2, 32), dtype=torch.bfloat16, device="cuda")
    A[0, 10], A[1, 11] = 1, 1
    m = torch.tensor([2], dtype=torch.int32, device="cuda")
    D = torch.empty((2, 256), device="cuda")
    b = torch.arange(256)
    kg.kg_fprop_w4(A, W, torch.full((1, 256, 1), 127, dtype=torch.uint8, device="cuda"), D, m)
    assert torch.equal(D.cpu(), torch.stack((E2M1[b & 15], E2M1[b >> 4])).float())
    kg.kg_fprop_w4(A, W, torch.ones((1, 256, 1), device="cuda"), D, m)
    assert torch.equal(D.cpu(), torch.stack((b & 15, b >> 4)).float() - 8)


def test_not_finite_rows_stay_apart():
    for rows in (4, 90):
        A, W, sw, zp, m = make([rows, 30], 50, 256, 128, "bf16", rows)
        D = torch.empty((rows + 30, 50), device="cuda")
        kg.kg_fprop_w4(A, W, sw, D, m, zp)
        bad = A.clone()
        bad[1, 7], bad[2, 200] = math.nan, math.inf
        E = torch.empty_like(D)
        kg.kg_fprop_w4(bad, W, sw, E, m, zp)
        keep = [t for t in range(rows + 30) if t not in (1, 2)]
        assert torch.equal(D[keep], E[keep]) and not E[1].isfinite().any() and not E[2].isfinite().any()


def test_inconsistent_counts_write_nothing():
    for rows in (5, 60, 300):
        A, W, sw, zp, m = make([rows, 3], 40, 128, 128, "bf16", 1)
        D = torch.full((rows + 3, 40), 3.0, device="cuda")
        kg.kg_fprop_w4(A, W, sw, D, m + 1, zp)
        assert kg.kg_status() == kg.KG_ERR_KSUM and (D == 3).all()
        kg.kg_fprop_w4(A, W, sw, D, m, zp)
        assert kg.kg_status() == kg.KG_OK and (D != 3).any()


def test_no_channels_and_no_rows():
    m = torch.tensor([4], dtype=torch.int32, device="cuda")
    empty = lambda *s, dtype=torch.uint8: torch.empty(s, dtype=dtype, device="cuda")
    D = torch.full((4, 8), 3.0, device="cuda")
    kg.kg_fprop_w4(empty(4, 0, dtype=torch.bfloat16), empty(1, 8, 0), empty(1, 8, 0), D, m)
    assert (D == 0).all()
    A, W, sw, zp, m = make([0, 0], 8, 64, 64, "f32", 1)
    kg.kg_fprop_w4(A, W, sw, empty(0, 8, dtype=torch.float32), m, zp)
    assert kg.kg_status() == kg.KG_OK


@pytest.mark.parametrize("kind", ["f32", "e2m1"])
def test_past_32_bit_offsets(kind):
    """Weights of more than 2^32 bytes, results past 2^32: whole-number results that are exact."""
    G, N, K = 5, 65536, 28672
    gen = torch.Generator("cuda").manual_seed(3)
    W = torch.randint(0, 256, (G, N, K // 2), generator=gen, device="cuda", dtype=torch.uint8)
    assert W.numel() > 2 ** 32
    group = 32 if kind == "e2m1" else 128
    sw = torch.full((G, N, K // group), 128 if kind == "e2m1" else 2, device="cuda",
                    dtype=torch.uint8 if kind == "e2m1" else torch.float32)
    for ms in ([1, 0, 2, 1, 3], [20, 40, 0, 30, 50]):
        M = sum(ms)
        A = torch.randint(-1, 2, (M, K), generator=gen, device="cuda").to(torch.bfloat16)
        D = torch.empty((M, (1 << 24) + 8 if M > 100 else N), device="cuda")[:, :N]
        kg.kg_fprop_w4(A, W, sw, D, torch.tensor(ms, dtype=torch.int32, device="cuda"))
        assert kg.kg_status() == kg.KG_OK
        at = 0
        for g, n in enumerate(ms):
            for o in (0, 1, N // 2 + 5, N - 1):
                q = torch.stack((W[g, o] & 15, W[g, o] >> 4), 1).flatten().cpu().long()
                w = 2 * (E2M1[q] if kind == "e2m1" else q.double() - 8)
                want = A[at:at + n].cpu().double() @ w
                assert torch.equal(D[at:at + n, o].cpu().double(), want), (ms, g, o)
            at += n
        del D


def test_in_a_graph_and_on_a_stream():
    for rows in (3, 50, 200):
        A, W, sw, zp, m = make([rows, 2, 9], 300, 512, 128, "bf16", rows)
        D, E = (torch.empty((rows + 11, 300), device="cuda") for _ in range(2))
        kg.kg_fprop_w4(A, W, sw, D, m, zp)
        torch.cuda.synchronize()
        s = torch.cuda.Stream()
        kg.kg_fprop_w4(A, W, sw, E, m, zp, stream=s)
        torch.cuda.current_stream().wait_stream(s)
        assert torch.equal(D, E)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            kg.kg_fprop_w4(A, W, sw, E, m, zp)
        for seed in range(3):
            A.copy_(torch.randn(A.shape, device="cuda"))
            E.fill_(0)
            g.replay()
            kg.kg_fprop_w4(A, W, sw, D, m, zp)
            assert torch.equal(D, E)


def test_served_layer():
    """kg_gate, kg_route, kg_dispatch, kg_fprop_w4 and kg_combine, with weights quantised by the
    library's own helpers, against the same layer of those weights in 64 bits."""
    T, G, k, K, N = 60, 12, 3, 256, 192
    gen = torch.Generator("cuda").manual_seed(7)
    w = torch.randn((G, N, K), generator=gen, device="cuda") * K ** -0.5
    x = torch.randn((T, K), generator=gen, device="cuda").to(torch.bfloat16)
    router = torch.randn((G, K), generator=gen, device="cuda") * K ** -0.5
    idx, p = kg.kg_gate(x.float() @ router.t(), k, None, kg.KG_GATE_NORM)
    ks = torch.empty(G, dtype=torch.int32, device="cuda")
    pos, _ = kg.kg_route(idx, ks)
    rows = kg.kg_dispatch(x, pos)
    for zero, group, e2m1 in ((True, 64, False), (False, 128, False), (False, 32, True)):
        W, sw, zp = (*inputs.quantize_e2m1(w), None) if e2m1 else inputs.quantize_w4(w, group, zero)
        y = torch.empty((T * k, N), dtype=torch.bfloat16, device="cuda")
        kg.kg_fprop_w4(rows, W, sw, y, ks, zp)
        out = kg.kg_combine(y, pos, p)
        wq = weights64(W, sw, zp, group)[0]
        # half a step of 15 (or of e2m1's 2 significant bits) off the weights
        assert float((wq - w.cpu().double()).norm()) <= (0.25 if e2m1 else 0.12) * float(w.norm())
        one = torch.bmm(wq[idx.cpu().long().flatten()], x.cpu().double().repeat_interleave(k, 0)[:, :, None])
        want = (one.view(T, k, N) * p.cpu().double()[..., None]).sum(1)
        # two roundings to bf16
        assert float((out.cpu().double() - want).norm()) <= 2 * 2.0 ** -8 * float(want.norm())
