"""kg_fprop where byte and element offsets pass 2^31 and 2^32: in the rows, in the weights, and in
the results' rows. Every result is looked at for having been written, and rows on both sides of
the borders are compared with the definition in 64 bits (tolerances as in test_gpu_fprop:
S = sum |a w|, 128 exact products and nk + 3 more roundings of 2^-24 S in the exact mode, 2^-10 S
with the fp8 MFMA, half a step of the result's type)."""
import pytest
import torch

import fp8_grouped_gemm_tn_amd as kg

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
BF16, F32 = torch.bfloat16, torch.float32
E4M3 = torch.float8_e4m3fn


def near(D, A, sa, W, sw, flags):
    """Rows D [n, N] of one expert: A [n, K], sa [nk, n], W [N, K], sw [ceil(N / 128), nk]."""
    N, K = W.shape
    val = lambda t: t.contiguous().view(E4M3).float().cpu().double()
    a = val(A) * sa.cpu().double().t().repeat_interleave(128, 1)[:, :K]
    w = val(W) * sw.cpu().double().repeat_interleave(128, 0)[:N].repeat_interleave(128, 1)[:, :K]
    y, S = a @ w.t(), a.abs() @ w.abs().t()
    half = 2.0 ** -8 if D.dtype == BF16 else 2.0 ** -24
    tol = (2.0 ** -10 if flags else (128 + sa.shape[0] + 3) * 2.0 ** -24) * S
    assert ((D.cpu().double() - y).abs() <= tol * (1 + half) + half * y.abs()).all()


def codes(gen, *shape):
    """Normal values of either sign (no NaN among the codes)."""
    t = torch.randint(0x10, 0x50, shape, generator=gen, device=DEV, dtype=torch.uint8)
    return t.bitwise_or_(torch.randint(0, 2, shape, generator=gen, device=DEV, dtype=torch.uint8).mul_(0x80))


@pytest.mark.parametrize("flags", [0, kg.KG_FLAG_FP8_MFMA])
def test_rows(flags):
    """620000 rows of 7168 bytes, two experts: rows around the offsets of 2^31 and 2^32 bytes and
    around the experts' border."""
    g = torch.Generator(DEV).manual_seed(1)
    ms, N, K = [300000, 320000], 32, 7168
    M = sum(ms)
    A, W = codes(g, M, K), codes(g, 2, N, K)
    sa = torch.rand((K // 128, M), generator=g, device=DEV) + 0.5
    sw = torch.rand((2, 1, K // 128), generator=g, device=DEV) + 0.5
    D = torch.full((M, N), float("nan"), device=DEV)
    kg.kg_fprop(A, sa, W, sw, D, torch.tensor(ms, dtype=torch.int32, device=DEV), flags)
    assert kg.kg_status() == kg.KG_OK
    assert torch.isfinite(D).all()
    for at in (0, 2 ** 31 // K, ms[0], 2 ** 32 // K, M):
        for e, lo, hi in ((0, 0, ms[0]), (1, ms[0], M)):
            r = slice(max(lo, at - 40), min(hi, at + 40))
            if r.start < r.stop:
                near(D[r], A[r], sa[:, r], W[e], sw[e], flags)


@pytest.mark.parametrize("flags", [0, kg.KG_FLAG_FP8_MFMA])
@pytest.mark.parametrize("each", [2, 70])
def test_weights(flags, each):
    """150 experts' weights of 4096 x 7168 bytes: those that 2^31 and 2^32 lie in, the last one and
    the first, with few rows and with more."""
    g = torch.Generator(DEV).manual_seed(2)
    G, N, K = 150, 4096, 7168
    live = [0, 2 ** 31 // (N * K), 2 ** 32 // (N * K), G - 1]
    ms = [each if e in live else 0 for e in range(G)]
    M = sum(ms)
    A, W = codes(g, M, K), codes(g, G, N, K)
    sa = torch.rand((K // 128, M), generator=g, device=DEV) + 0.5
    sw = torch.rand((G, N // 128, K // 128), generator=g, device=DEV) + 0.5
    D = torch.full((M, N), float("nan"), device=DEV)
    kg.kg_fprop(A, sa, W, sw, D, torch.tensor(ms, dtype=torch.int32, device=DEV), flags)
    assert kg.kg_status() == kg.KG_OK
    assert torch.isfinite(D).all()
    for i, e in enumerate(live):
        r = slice(i * each, (i + 1) * each)
        near(D[r], A[r], sa[:, r], W[e], sw[e], flags)


@pytest.mark.parametrize("flags", [0, kg.KG_FLAG_FP8_MFMA])
@pytest.mark.parametrize("dt", [F32, BF16])
@pytest.mark.parametrize("ms,ldd", [([4], 2 ** 30), ([2, 0, 3], 2 ** 30 - 56), ([70, 80], 2 ** 25 + 24)])
def test_results(ms, ldd, dt, flags):
    """Rows of the results so far apart that the last ones lie past 2^31 elements; what lies
    between the rows is not written."""
    g = torch.Generator(DEV).manual_seed(3)
    G, M, N, K = len(ms), sum(ms), 136, 400
    A, W = codes(g, M, K), codes(g, G, N, K)
    sa = torch.rand((4, M), generator=g, device=DEV) + 0.5
    sw = torch.rand((G, 2, 4), generator=g, device=DEV) + 0.5
    assert (M - 1) * ldd > 2 ** 31
    flat = torch.empty((M - 1) * ldd + N + 64, dtype=dt, device=DEV)
    D = flat[:(M - 1) * ldd + N].as_strided((M, N), (ldd, 1))
    past = flat.as_strided((M, N + 64), (ldd, 1))
    past.fill_(5.0)
    kg.kg_fprop(A, sa, W, sw, D, torch.tensor(ms, dtype=torch.int32, device=DEV), flags)
    assert kg.kg_status() == kg.KG_OK
    assert (past[:, N:] == 5).all()
    at = 0
    for e, n in enumerate(ms):
        near(D[at:at + n], A[at:at + n], sa[:, at:at + n], W[e], sw[e], flags)
        at += n
