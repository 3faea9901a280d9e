"""kg_fprop against its definition in 64 bits.

Tolerances, with S = sum of |a w| over a result's products (scales included): a block's fp32 sum
of up to 128 exact products is off by at most 128 2^-24 of its share of S, its two scales and
the sum over nk blocks add (nk + 3) 2^-24 S; bf16 results are rounded by 2^-8 |y| more. The fp8
MFMA mode is held to 2^-10 S and 1e-4 of the whole result's norm, as kg_dgrad's."""
import numpy as np
import pytest
import torch

import fp8_grouped_gemm_tn_amd as kg

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
BF16, F32 = torch.bfloat16, torch.float32
FAST = kg.KG_FLAG_FP8_MFMA
E4M3 = torch.float8_e4m3fn


def make(ms, N, K, seed=0, pad=0):
    g = torch.Generator(DEV).manual_seed(seed)
    M, G, nk, nb = sum(ms), len(ms), -(-K // 128), -(-N // 128)
    codes = lambda *s: torch.randn(s, generator=g, device=DEV).mul(60).clamp(-448, 448).to(E4M3).view(torch.uint8)
    A = torch.full((M, K + pad), 0x7F, dtype=torch.uint8, device=DEV)  # NaN next to the rows
    A[:, :K] = codes(M, K)
    A = A[:, :K]
    W = codes(G, N, K)
    sa = torch.exp(torch.randn((nk, M), generator=g, device=DEV)) * 1e-2
    sw = torch.exp(torch.randn((G, nb, nk), generator=g, device=DEV)) * 1e-2
    return A, sa, W, sw, torch.tensor(ms, dtype=torch.int32, device=DEV)


def ref(A, sa, W, sw, ms):
    """(y, S) in 64 bits on the CPU."""
    N, K = W.shape[1:]
    val = lambda t: t.contiguous().view(E4M3).float().cpu().double()
    a = val(A) * sa.cpu().double().t().repeat_interleave(128, 1)[:, :K]
    w = val(W) * sw.cpu().double().repeat_interleave(128, 1)[:, :N].repeat_interleave(128, 2)[:, :, :K]
    y, S, at = [], [], 0
    for g, n in enumerate(ms.tolist()):
        y.append(a[at:at + n] @ w[g].t())
        S.append(a[at:at + n].abs() @ w[g].abs().t())
        at += n
    return torch.cat(y), torch.cat(S)


def check(D, A, sa, W, sw, ms, flags):
    y, S = ref(A, sa, W, sw, ms)
    got = D.double().cpu()
    half = 2.0 ** -8 if D.dtype == BF16 else 2.0 ** -24
    nk = sa.shape[0]
    if flags & FAST:
        tol = 2.0 ** -10 * S
        frob = 1e-4 + (half if D.dtype == BF16 else 0)
        assert (got - y).norm() <= frob * y.norm()
    else:
        tol = (128 + nk + 3) * 2.0 ** -24 * S
    assert torch.isfinite(got).all()
    assert ((got - y).abs() <= tol * (1 + half) + half * y.abs()).all()


def run(ms, N, K, dt, flags, seed=0, pad=0):
    A, sa, W, sw, m = make(ms, N, K, seed, pad)
    D = torch.full((sum(ms), N), float("nan"), dtype=dt, device=DEV)
    kg.kg_fprop(A, sa, W, sw, D, m, flags)
    assert kg.kg_status() == kg.KG_OK
    check(D, A, sa, W, sw, m, flags)


SHAPES = [
    ([1], 1, 16), ([1], 64, 128), ([1], 100, 144), ([3], 33, 1040), ([17], 130, 256), ([40], 256, 512),
    ([64], 200, 384),
    ([0, 1, 0, 2, 5], 96, 272), ([16, 0, 33, 1], 160, 400), ([100, 0, 0, 3], 65, 128), ([0, 0, 7], 32, 16),
    ([65], 1, 16), ([200], 128, 128), ([257], 300, 1040), ([300, 0, 1, 511], 264, 656),
    ([1000, 256, 0, 2], 520, 240), ([700], 1, 272), ([0, 0, 900], 257, 128),
]


@pytest.mark.parametrize("ms,N,K", SHAPES)
@pytest.mark.parametrize("dt", [F32, BF16])
@pytest.mark.parametrize("flags", [0, FAST])
def test_small(ms, N, K, dt, flags):
    run(ms, N, K, dt, flags, seed=N + K)


@pytest.mark.parametrize("ms,N,K", [([30, 2], 96, 400), ([500, 90], 200, 272)])
@pytest.mark.parametrize("flags", [0, FAST])
def test_row_stride(ms, N, K, flags):
    run(ms, N, K, F32, flags, seed=1, pad=48)


@pytest.mark.parametrize("flags", [0, FAST])
@pytest.mark.parametrize("dt,off,pad", [(F32, 1, 5), (BF16, 3, 7), (BF16, 8, 8)])
@pytest.mark.parametrize("ms", [[20, 5], [300, 140]])
def test_output_stride_and_alignment(ms, dt, off, pad, flags):
    """D a part of a wider matrix: nothing outside it is written."""
    N = 72
    A, sa, W, sw, m = make(ms, N, 256, 3)
    wide = torch.full((sum(ms), N + off + pad), 5.0, dtype=dt, device=DEV)
    D = wide[:, off:off + N]
    kg.kg_fprop(A, sa, W, sw, D, m, flags)
    check(D, A, sa, W, sw, m, flags)
    assert (wide[:, :off] == 5).all() and (wide[:, off + N:] == 5).all()


@pytest.mark.parametrize("avg", [4, 30, 60, 90, 200])
@pytest.mark.parametrize("flags", [0, FAST])
def test_many_experts(avg, flags):
    rng = np.random.default_rng(avg)
    ms = rng.poisson(avg * rng.dirichlet(np.ones(150)) * 150).tolist()
    run(ms, 136, 384, BF16, flags, seed=avg)


def test_1024_experts():
    rng = np.random.default_rng(0)
    for lam in (1, 70):
        run(rng.poisson(lam, 1024).tolist(), 32, 128, F32, FAST, seed=lam)
        run(rng.poisson(lam, 1024).tolist(), 32, 128, F32, 0, seed=lam)


def test_random_configurations():
    rng = np.random.default_rng(11)
    for i in range(40):
        G = int(rng.integers(1, 20))
        ms = np.floor(np.exp(rng.uniform(0, np.log(600), G))).astype(int) * (rng.random(G) < 0.8)
        if ms.sum() == 0:
            ms[0] = 3
        N, K = int(rng.integers(1, 700)), 16 * int(rng.integers(1, 80))
        flags = FAST if rng.random() < 0.5 else 0
        print(f"[case] {i}: ms {ms.tolist()} N {N} K {K} flags {flags}", flush=True)
        run(ms.tolist(), N, K, BF16 if rng.random() < 0.5 else F32, flags, seed=i)


@pytest.mark.parametrize("ms", [[5, 3], [400, 100]])
def test_no_channels_gives_zeros(ms):
    D = torch.full((sum(ms), 40), float("nan"), device=DEV)
    z = lambda *s: torch.zeros(s, device=DEV)
    kg.kg_fprop(z(sum(ms), 0).to(torch.uint8), z(0, sum(ms)), z(2, 40, 0).to(torch.uint8), z(2, 1, 0),
                D, torch.tensor(ms, dtype=torch.int32, device=DEV))
    assert (D == 0).all()


@pytest.mark.parametrize("ms,M", [([5, 4], 10), ([5, -1, 6], 10), ([200, 300], 501), ([400, -2, 103], 501)])
def test_counts_that_do_not_add_up(ms, M):
    A, sa, W, sw, _ = make([M] + [0] * (len(ms) - 1), 64, 128)
    D = torch.full((M, 64), 5.0, device=DEV)
    kg.kg_fprop(A, sa, W, sw, D, torch.tensor(ms, dtype=torch.int32, device=DEV))
    assert kg.kg_status() == kg.KG_ERR_KSUM
    assert (D == 5).all()
    assert kg.kg_status() == kg.KG_OK


@pytest.mark.parametrize("flags", [0, FAST])
@pytest.mark.parametrize("ms", [[3, 0, 9], [300, 0, 257]])
def test_special_values_stay_in_their_rows(ms, flags):
    """A NaN code or an infinite scale reaches its own row (or output column) alone."""
    A, sa, W, sw, m = make(ms, 70, 256)
    A[1, 7] = 0x7F
    sa[1, 2] = float("inf")
    W[2, 11, 3] = 0xFF
    D = torch.empty((sum(ms), 70), device=DEV)
    kg.kg_fprop(A, sa, W, sw, D, m, flags)
    bad = ~torch.isfinite(D)
    want = torch.zeros_like(bad)
    want[1], want[2], want[ms[0]:, 11] = True, True, True
    assert torch.equal(bad, want)


@pytest.mark.parametrize("ms", [[4, 0, 3], [150, 0, 120]])
def test_gradients_against_differences(ms):
    """With whole-number codes and scales of 1 every sum is exact, so differences of kg_fprop
    equal what kg_dgrad (rows) and kg_wgrad (weights) give as its gradients."""
    N, K, G, M = 128, 256, len(ms), sum(ms)
    g = torch.Generator(DEV).manual_seed(4)
    whole = lambda lo, hi, *s: torch.randint(lo, hi + 1, s, generator=g, device=DEV).float()
    enc = lambda t: t.to(E4M3).view(torch.uint8)
    ones = lambda *s: torch.ones(s, device=DEV)
    a, w, dy, ea, ew = whole(-3, 3, M, K), whole(-3, 3, G, N, K), whole(-3, 3, M, N), \
        whole(-2, 2, M, K), whole(-2, 2, G, N, K)
    m = torch.tensor(ms, dtype=torch.int32, device=DEV)

    def y(a, w):
        D = torch.empty((M, N), device=DEV)
        return kg.kg_fprop(enc(a), ones(2, M), enc(w), ones(G, 1, 2), D, m)

    dx = kg.kg_dgrad(enc(dy), ones(1, M), enc(w), ones(G, 1, 2), torch.empty((M, K), device=DEV), m)
    nblk = sum(-(-x // 128) for x in ms)
    dw = torch.empty((G, N, K), device=DEV)
    kg.kg_wgrad(enc(dy), ones(nblk, N), enc(a), ones(nblk, K), None, dw, m, 128, kg.KG_E4M3_F32SCALE)
    assert kg.kg_status() == kg.KG_OK
    base = y(a, w)
    assert ((y(a + ea, w) - base).double() * dy).sum() == (dx.double() * ea).sum()
    assert ((y(a, w + ew) - base).double() * dy).sum() == (dw.double() * ew).sum()


def test_rows_and_weights_past_32_bit_offsets():
    g = torch.Generator(DEV).manual_seed(6)
    big = lambda *s: torch.randint(0, 0x40, s, generator=g, device=DEV, dtype=torch.uint8)
    # rows: 620000 x 7168 bytes; weights: 150 x 4096 x 7168 bytes
    for ms, N, K in (([300000, 320000], 32, 7168), ([0] * 148 + [7, 300], 4096, 7168)):
        M, G = sum(ms), len(ms)
        A, W = big(M, K), big(G, N, K)
        sa, sw = torch.rand((K // 128, M), device=DEV), torch.rand((G, -(-N // 128), K // 128), device=DEV)
        m = torch.tensor(ms, dtype=torch.int32, device=DEV)
        for flags in (0, FAST):
            D = torch.empty((M, N), device=DEV)
            kg.kg_fprop(A, sa, W, sw, D, m, flags)
            assert kg.kg_status() == kg.KG_OK
            n = ms[-1]
            last = torch.tensor([0] * (G - 1) + [min(n, 40)], dtype=torch.int32)[-1:]
            r = slice(M - int(last[0]), M)
            check(D[r], A[r], sa[:, r], W[-1:], sw[-1:], last, flags)


def test_many_outputs_of_few_rows():
    """2^24 outputs of 40 experts with a row each: more workgroups than the streaming kernel's
    launch would hold."""
    G, N, K = 40, 1 << 24, 16
    W = torch.randint(0, 0x40, (G, N, K), dtype=torch.uint8, device=DEV)
    A = torch.randint(0, 0x40, (G, K), dtype=torch.uint8, device=DEV)
    sa, sw = torch.rand((1, G), device=DEV), torch.rand((G, N // 128, 1), device=DEV)
    m = torch.ones(G, dtype=torch.int32, device=DEV)
    D = torch.full((G, N), float("nan"), dtype=BF16, device=DEV)
    kg.kg_fprop(A, sa, W, sw, D, m, FAST)
    assert kg.kg_status() == kg.KG_OK
    for g in (0, 17, 39):
        n = slice(N - 4096, N)
        check(D[g:g + 1, n], A[g:g + 1], sa[:, g:g + 1], W[g:g + 1, n], sw[g:g + 1, -32:],
              torch.ones(1, dtype=torch.int32), FAST)
    assert torch.isfinite(D.float().sum())


def test_other_stream_and_graph():
    A, sa, W, sw, m = make([200, 0, 150], 200, 512, 9)
    A = A.contiguous()
    small = make([3, 0, 4], 200, 512, 10)
    D, Ds = torch.empty((350, 200), dtype=BF16, device=DEV), torch.empty((7, 200), device=DEV)

    def step():
        kg.kg_fprop(A, sa, W, sw, D, m, FAST)
        kg.kg_fprop(small[0], *small[1:4], Ds, small[4])

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for i in range(4):
        sa.mul_(1.5)
        small[3].mul_(0.7)
        step()
        want, want_s = D.clone(), Ds.clone()
        D.zero_(), Ds.zero_()
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(D, want) and torch.equal(Ds, want_s)
    check(D, A, sa, W, sw, m, FAST)


@pytest.mark.parametrize("G,N,K,avg", [(140, 130, 4096, 2), (140, 130, 4096, 40), (129, 257, 8192, 3)])
@pytest.mark.parametrize("dt,flags", [(BF16, 0), (F32, FAST)])
def test_rows_a_multiple_of_4096_bytes_apart(G, N, K, avg, dt, flags):
    """Many experts with few rows: a tile's blocks are added from a start of its own, round the end."""
    rng = np.random.default_rng(G + K)
    ms = rng.poisson(avg * rng.dirichlet(np.ones(G)) * G).tolist()
    run(ms, N, K, dt, flags, seed=avg)


@pytest.mark.parametrize("ms,N,K", [([5], 37, 3600), ([16], 16, 1168), ([33], 50, 2064), ([64], 130, 7184),
                                    ([49], 4000, 1936), ([2, 0, 9], 90, 3088), ([30, 34], 70, 2320),
                                    ([1] * 40, 3000, 3600), ([16], 33000, 272), ([3], 34000, 4096)])
@pytest.mark.parametrize("dt", [F32, BF16])
@pytest.mark.parametrize("flags", [0, FAST])
def test_few_rows(ms, N, K, dt, flags):
    """Streaming: several blocks per wave, 16 or 32 outputs per workgroup, passes over the rows."""
    run(ms, N, K, dt, flags, seed=K)
