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


def ends(N):
    """The first outputs, some of the middle, and those of the last workgroup and the one before."""
    return torch.tensor(sorted(set(range(min(N, 40))) | {N // 2} | set(range(max(0, N - 200), N))))


# waves, waves that share an output, tiles of a set: experts, rows of each, channels, outputs of whole
# workgroups, outputs of one
FORMS = {(8, 8, 1): (1, 5, 256, 32, 16), (16, 8, 1): (1, 12, 4096, 64, 32), (8, 8, 2): (70, 2, 256, 64, 32),
         (16, 8, 2): (70, 8, 4096, 64, 64), (8, 4, 2): (70, 2, 640, 512, 64), (16, 4, 2): (16, 8, 4096, 2048, 128)}


@pytest.mark.parametrize("kind,group", [("bf16", 128), ("bf16", 64), ("f32", 32), ("e2m1", 32)])
@pytest.mark.parametrize("form", sorted(FORMS), ids=str)
def test_streaming_forms(form, kind, group):
    """Every number of waves and way to share outputs, with last workgroups that are full, whose last set
    is partial, and whose last sets have no outputs; rows that are not even."""
    G, each, K, whole, per = FORMS[form]
    if form[1] == 4 and group == 32 and kind == "f32":
        each, K = (4, K) if form[0] == 16 else (1, 1024)  # (with more rows the tiles take the call)
    ms = [2 * each if g % 4 == 0 else 0 if g % 4 == 1 else each for g in range(G)] if G > 1 else [each]
    for more in sorted({0, 5, per // 2 + 1, per - 3}):
        N = whole + more
        p = plan(sum(ms), G, N, K, kind, group, kind != "e2m1")
        assert p.streams and (p.waves, p.split, p.nj) == form, (N, vars(p))
        assert 16 * p.nj * p.waves // p.split == per
        check(ms, N, K, group, kind, N, some=ends(N))


def test_many_experts_without_rows():
    """Workgroups of experts that have no rows, first, last and between: they load and store nothing."""
    ms = [0] * 100
    ms[3], ms[40], ms[98] = 30, 1, 5
    p = plan(36, 100, 300, 512, "bf16", 64, True)
    assert p.streams
    check(ms, 300, 512, 64, "bf16", 2)


@pytest.mark.parametrize("kind,group", [("bf16", 128), ("e2m1", 32)])
def test_streaming_past_32_bit_offsets(kind, group):
    """Weights of more than 2^32 bytes, a few rows for each of many experts."""
    G, N, K = 70, 65536, 2048
    assert G * N * K // 2 > 2 ** 32
    assert plan(G, G, N, K, kind, group, False).streams
    gen = torch.Generator("cuda").manual_seed(5)
    W = torch.randint(0, 256, (G, N, K // 2), generator=gen, device="cuda", dtype=torch.uint8)
    sw = torch.full((G, N, K // group), 128 if kind == "e2m1" else 2, device="cuda",
                    dtype=torch.uint8 if kind == "e2m1" else torch.bfloat16)
    ms = torch.ones(G, dtype=torch.int32, device="cuda")
    ms[5], ms[6], ms[69], ms[68] = 0, 2, 2, 0
    A = torch.randint(-1, 2, (G, K), generator=gen, device="cuda").to(torch.bfloat16)
    D = torch.empty((G, N), device="cuda")
    kg.kg_fprop_w4(A, W, sw, D, ms)
    assert kg.kg_status() == kg.KG_OK
    at = 0
    for g, n in enumerate(ms.tolist()):
        for o in (0, 17, N // 2 + 5, N - 1):
            q = torch.stack((W[g, o] & 15, W[g, o] >> 4), 1).flatten().cpu().long()
            w = 2 * (base.E2M1[q] if kind == "e2m1" else q.double() - 8)
            # sums of whole (e2m1: half) numbers below 2^24: exact
            assert torch.equal(D[at:at + n, o].cpu().double(), A[at:at + n].cpu().double() @ w), (g, o)
        at += n


TILES = {(32, 128): (3, 40, 400), (64, 128): (5, 400, 400), (128, 128): (8, 128, 1540), (128, 256): (8, 100, 4100),
         (256, 256): (8, 200, 4100)}  # experts, rows of each, outputs


@pytest.mark.parametrize("tile,kind,group", [
    (t, *k) for t in sorted(TILES) for k in (("bf16", 128), ("bf16", 64), ("f32", 32), ("e2m1", 32))
    if k[0] == "e2m1" or t != (256, 256)], ids=str)  # (whole numbers have no tile of 256 x 256)
def test_tiles(tile, kind, group):
    """Every tile, with partial tiles of rows and outputs and last blocks that are not whole."""
    G, each, N = TILES[tile]
    ms = [each + 13, 0, 2 * each - 13] + [each] * (G - 3)
    for K in (640, 608) if group == 32 else (640, 704) if group == 64 else (640,):
        p = plan(sum(ms), G, N, K, kind, group, kind != "e2m1")
        assert not p.streams and (p.bt, p.bn) == tile, vars(p)
        check(ms, N, K, group, kind, N, some=ends(N))
