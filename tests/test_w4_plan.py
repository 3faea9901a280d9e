"""kg_fprop_w4's host-side arithmetic: what its launches read and hold, without a GPU."""
import pytest

import w4_plan

FORMS = [(8, 8, 1), (16, 8, 1), (8, 8, 2), (16, 8, 2), (8, 4, 2), (16, 4, 2)]  # waves, split, nj


@pytest.mark.parametrize("waves,split,nj", FORMS)
@pytest.mark.parametrize("K", [32, 128, 160, 640, 1056, 7168])
def test_streaming_reads_end_with_the_weights(waves, split, nj, K):
    """Every wave's buffer of codes ends with the last output of its set at the latest, whatever
    part of the last workgroup's outputs exists: also where a set has none. (A load's 16 bytes are
    bounded by the buffer, so this bounds every address.)"""
    L = w4_plan.lib()
    n0, kbytes, nk = 16 * nj, K // 2, -(-K // 128)
    sets = waves // split
    for outs_there in range(1, n0 * sets + 1):  # of the last workgroup
        for side in range(sets):
            m0 = side * n0
            outs = L.set_outs(outs_there, m0, n0)
            assert outs == max(0, min(n0, outs_there - m0))
            base = (m0 if outs else 0) * kbytes
            for part in range(split):
                first, to = part * nk // split, (part + 1) * nk // split
                for kb in range(first, to + 8):  # and the blocks asked for behind the last one
                    left = L.codes_left(outs, kbytes, kb, to)
                    if kb >= to or outs == 0:
                        assert left == 0
                    else:
                        assert left > 0 and base + 64 * kb + left == (m0 + outs) * kbytes
                        assert base + 64 * kb + left <= outs_there * kbytes


def forms():
    for kind, group in (("bf16", 128), ("bf16", 64), ("bf16", 32), ("f32", 128), ("f32", 64), ("f32", 32),
                        ("e2m1", 32)):
        for zp in (0, 1) if kind != "e2m1" else (0,):
            yield kind, group, zp


@pytest.mark.parametrize("kind,group,zp", list(forms()))
def test_streaming_fits_in_lds(kind, group, zp):
    """What a streaming launch asks for is what a workgroup may have: over widths, experts and
    rows, every K of whole groups up to 16384."""
    for G, M in ((1, 1), (1, 16), (8, 8), (8, 100), (64, 64), (256, 40)):
        for N in (1, 33, 4096, 5120):
            for K in range(group, 16385, group):
                p = w4_plan.Plan(M, G, N, K, kind, group, zp)
                assert not p.streams or p.lds <= p.limit, (M, G, N, K, p.waves, p.lds)


@pytest.mark.parametrize("kind,group,zp", list(forms()))
def test_a_launch_holds_its_rows(kind, group, zp):
    """The LDS set aside for tokens holds as many rows as the kernel loads at a time, without any
    channels too, and the closing sums of every wave; scales and zero points follow."""
    L, bytes_of = w4_plan.lib(), {"bf16": 2, "f32": 4, "e2m1": 1}[kind]
    for G, M in ((1, 1), (1, 5), (1, 16), (1, 100), (8, 8), (64, 64), (256, 40), (16, 512)):
        for N in (1, 33, 700, 4096):
            for K in (0, group, 4 * group, 512, 640, 1024, 2048, 4096, 7168, 8192, 14336):
                p = w4_plan.Plan(M, G, N, K, kind, group, zp)
                if not p.rows:
                    continue
                outs = 16 * p.nj * p.waves // p.split
                assert p.rows * 1024 * L.pieces(-(-K // 128)) <= p.tokens
                assert 1024 * p.waves * p.nj <= p.tokens
                assert outs * (K // group) * bytes_of <= p.scales
                assert p.tokens + p.scales + (outs * (K // group) if zp else 0) <= p.lds <= p.limit
