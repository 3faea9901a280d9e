"""Tokens into expert order and back (kg_route, kg_dispatch, kg_dispatch_fp8, kg_combine,
kg_combine_bwd) against their definitions, computed on the CPU in 64 bits.

Tolerances: the plan, the copied rows, the codes and their scales are exact. A weighted sum of
k rows in fp32 is off by at most (k + 1) 2^-24 sum |w y|, a dot product over H channels by at
most (H + 1) 2^-24 sum |g y|; a result rounded to bf16 is off by 2^-8 |y| more (half a step, relative
to the value, is eps / 2 = 2^-8)."""
import numpy as np
import pytest
import torch

import fp8_grouped_gemm_tn_amd as kg

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
BF16, F32 = torch.bfloat16, torch.float32


def plan_of(idx, G):
    """(ks, pos, src) of numpy int32 [T, k]."""
    key = idx.reshape(-1).astype(np.int64)
    kept = (key >= 0) & (key < G)
    key = np.where(kept, key, G)
    order = np.argsort(key, kind="stable")
    row = np.empty_like(order)
    row[order] = np.arange(order.size)
    ks = np.bincount(key, minlength=G + 1)[:G]
    return ks, np.where(kept, row, ~row).reshape(idx.shape), np.where(kept[order], order, ~order)


def make_idx(T, k, G, kind, seed=0):
    rng = np.random.default_rng(seed)
    if kind == "uniform":
        idx = rng.integers(0, G, (T, k))
    elif kind == "one":
        idx = np.full((T, k), G - 1)
    elif kind == "none":
        idx = np.full((T, k), -1)
    elif kind == "wild":  # values far outside [0, G) are dropped slots too
        idx = rng.integers(0, G, (T, k))
        idx = np.where(rng.random((T, k)) < 0.3, rng.choice([-1, G, 2**31 - 1, -2**31], (T, k)), idx)
    else:  # sorted: long runs of one expert
        idx = np.sort(rng.integers(0, G, T * k)).reshape(T, k)
    return idx.astype(np.int32)


def route(idx, G):
    d = torch.from_numpy(idx).to(DEV)
    ks = torch.full((G,), -7, dtype=torch.int32, device=DEV)
    pos, src = kg.kg_route(d, ks)
    return ks, pos, src


@pytest.mark.parametrize("T,k,G", [(1, 1, 1), (1, 8, 256), (8, 8, 256), (7, 3, 1024), (63, 1, 5),
                                   (65, 2, 2), (1000, 4, 64), (512, 8, 256), (513, 8, 256),
                                   (4097, 1, 37), (20000, 8, 1024), (70000, 3, 255), (0, 4, 8),
                                   (300, 0, 8)])
@pytest.mark.parametrize("kind", ["uniform", "one", "none", "wild", "sorted"])
def test_plan(T, k, G, kind):
    idx = make_idx(T, k, G, kind, seed=T + G)
    ks, pos, src = route(idx, G)
    want = plan_of(idx, G)
    assert np.array_equal(ks.cpu().numpy(), want[0])
    assert np.array_equal(pos.cpu().numpy(), want[1])
    assert np.array_equal(src.cpu().numpy(), want[2])


def test_plan_without_src_and_with_kept_workspace():
    ws = kg.new_route_workspace(5000, 4, 100, DEV)
    ks = torch.empty(100, dtype=torch.int32, device=DEV)
    for seed, T in enumerate((5000, 4000, 10)):  # a workspace serves every smaller plan
        idx = make_idx(T, 4, 100, "wild", seed)
        pos, src = kg.kg_route(torch.from_numpy(idx).to(DEV), ks, ws=ws)
        want = plan_of(idx, 100)
        assert np.array_equal(pos.cpu().numpy(), want[1])
        assert np.array_equal(ks.cpu().numpy(), want[0])
    d = torch.from_numpy(make_idx(50, 2, 100, "uniform")).to(DEV)
    pos = torch.empty_like(d)
    stream = torch.cuda.current_stream().cuda_stream
    rc = kg.layer.lib().kg_route(d.data_ptr(), 50, 2, 100, ks.data_ptr(), pos.data_ptr(), None,
                                 None, 0, stream)
    assert rc == kg.KG_OK
    assert np.array_equal(pos.cpu().numpy(), plan_of(d.cpu().numpy(), 100)[1])


def rows64(x):
    return x.double().cpu().numpy()


SHAPES = [(1, 1, 1, 1), (1, 8, 16, 7168), (5, 3, 4, 7), (33, 2, 8, 129), (64, 8, 256, 1000),
          (17, 9, 12, 1235), (300, 4, 32, 2048), (9, 17, 20, 40), (130, 1, 3, 4100)]


@pytest.mark.parametrize("T,k,G,H", SHAPES)
@pytest.mark.parametrize("dt", [BF16, F32])
@pytest.mark.parametrize("kind", ["uniform", "wild", "none"])
def test_dispatch_combine_and_gradients(T, k, G, H, dt, kind):
    g = torch.Generator(DEV).manual_seed(T * 31 + H)
    idx = make_idx(T, k, G, kind, seed=H)
    _, pos, _ = route(idx, G)
    _, want_pos, want_src = plan_of(idx, G)
    R = T * k
    X = torch.randn((T, H), generator=g, device=DEV).to(dt)
    Y = torch.randn((R, H), generator=g, device=DEV).to(dt)
    w = torch.rand((T, k), generator=g, device=DEV) - 0.3
    dropped = torch.from_numpy(want_pos < 0).to(DEV)
    # what dropped slots hold must not show: NaN in their weights and rows
    w[dropped] = float("nan")
    Y[torch.from_numpy(want_src < 0).to(DEV)] = float("nan")

    Xp = kg.kg_dispatch(X, pos, torch.full((R, H), 3.0, device=DEV, dtype=dt))
    kept = want_src >= 0
    want = rows64(X)[np.where(kept, want_src, ~want_src) // k] * kept[:, None]
    assert np.array_equal(rows64(Xp), want)

    half = 2.0 ** -8 if dt == BF16 else 2.0 ** -24
    y, wt = np.nan_to_num(rows64(Y)), np.nan_to_num(rows64(w))
    at = np.where(want_pos < 0, ~want_pos, want_pos)
    on = want_pos >= 0
    for weights in (w, None):
        wj = (wt if weights is not None else np.ones((T, k))) * on
        out = kg.kg_combine(Y, pos, weights, torch.full((T, H), 5.0, device=DEV, dtype=dt))
        terms = wj[..., None] * y[at]
        tol = half * np.abs(terms.sum(1)) + (k + 1) * 2.0 ** -24 * np.abs(terms).sum(1) * (1 + half)
        assert (np.abs(rows64(out) - terms.sum(1)) <= tol).all()

        dY, dw = kg.kg_combine_bwd(X, Y, pos, weights,
                                   torch.full((R, H), 7.0, device=DEV, dtype=dt))
        gx = rows64(X)
        full = np.zeros((R, H))
        full[at.reshape(-1)] = (wj[..., None] * gx[:, None]).reshape(R, H)
        assert (np.abs(rows64(dY) - full) <= half * np.abs(full)).all()
        prod = gx[:, None] * y[at] * on[..., None]
        assert (np.abs(rows64(dw) - prod.sum(2)) <=
                (H + 1) * 2.0 ** -24 * np.abs(prod).sum(2)).all()
        dY2, none = kg.kg_combine_bwd(X, None, pos, weights, need_dw=False)
        assert none is None and torch.equal(dY2.view(torch.uint8), dY.view(torch.uint8))


def e4m3_of(x):
    """(codes as values, scales) of fp32 numpy rows, one scale per 128 channels, binary32."""
    T, H = x.shape
    xb = np.zeros((T, -(-H // 128) * 128), np.float32)
    xb[:, :H] = x
    xb = xb.reshape(T, -1, 128)
    amax = np.abs(np.where(np.isnan(xb), 0, xb)).max(2)
    s = np.where(amax == 0, np.float32(1), amax / np.float32(448)).astype(np.float32)
    with np.errstate(invalid="ignore"):
        q = torch.from_numpy((xb / s[..., None]).reshape(T, -1)[:, :H].copy())
    return q.to(torch.float8_e4m3fn), s


@pytest.mark.parametrize("T,k,G,H", [(1, 8, 16, 7168), (3, 2, 4, 16), (40, 3, 8, 144), (65, 8, 32, 2000),
                                     (200, 2, 5, 128), (10, 1, 2, 4112), (60000, 8, 40, 656),
                                     (250000, 1, 7, 1040)])
@pytest.mark.parametrize("kind", ["uniform", "wild"])
def test_dispatch_fp8(T, k, G, H, kind):
    g = torch.Generator(DEV).manual_seed(H)
    idx = make_idx(T, k, G, kind, seed=T)
    _, pos, _ = route(idx, G)
    _, _, src = plan_of(idx, G)
    X = (torch.randn((T, H), generator=g, device=DEV) *
         torch.exp2(torch.randint(-20, 20, (T, 1), generator=g, device=DEV))).to(BF16)
    X[0, : H // 2] = 0
    X[T // 2, 3] = float("nan")
    X[T - 1, 5] = 1e-38
    X[T - 1, 6:] = 0
    Q, sa = kg.kg_dispatch_fp8(X, pos)
    q, s = e4m3_of(X.float().cpu().numpy())
    kept = src >= 0
    tok = np.where(kept, src, ~src) // k
    want = q.view(torch.uint8).numpy()[tok] * kept[:, None].astype(np.uint8)
    got = Q.cpu().numpy()
    nan = (want & 0x7F) == 0x7F
    assert np.array_equal(np.where(nan, 0x7F, want), got)
    want_s = np.where(kept[:, None], s[tok], np.float32(1)).T
    assert np.array_equal(sa.cpu().numpy().view(np.uint32), want_s.astype(np.float32).view(np.uint32))


def test_fp8_scales_in_two_steps_and_in_one():
    """With and without the workspace: the same bits, and rows that no slot names are left alone
    whatever the workspace held."""
    T, k, H = 60000, 4, 1168  # 10 blocks: 2.4 M scales
    pos = torch.randperm(T * k, device=DEV).to(torch.int32).view(T, k)
    pos[::3, 1] = ~pos[::3, 1]
    pos[5, 0], pos[6, 2], pos[7, 3] = T * k, -2**31, 2**31 - 1
    X = torch.randn((T, H), device=DEV).to(BF16)
    L = kg.layer.lib()
    n = L.kg_dispatch_fp8_workspace_bytes(T, k, H)
    assert n > 0
    got = []
    for fill in (None, 0, 1, 0xFF):
        Q = torch.full((T * k, H), 0x55, dtype=torch.uint8, device=DEV)
        sa = torch.full((10, T * k), 9.0, device=DEV)
        if fill is None:
            st = torch.cuda.current_stream().cuda_stream
            assert L.kg_dispatch_fp8(X.data_ptr(), H, pos.data_ptr(), T, k, H, Q.data_ptr(),
                                     sa.data_ptr(), None, 0, st) == kg.KG_OK
        else:
            kg.kg_dispatch_fp8(X, pos, Q, sa, torch.full((n,), fill, dtype=torch.uint8, device=DEV))
        got.append((Q, sa))
    for Q, sa in got[1:]:
        assert torch.equal(Q, got[0][0]) and torch.equal(sa, got[0][1])
    assert int((got[0][1] == 9).all(0).sum()) == 3


def test_special_values():
    """Infinities pass, an infinity in a block makes its scale infinite as kg_requant's."""
    idx = np.array([[1, 0], [0, 2]], np.int32)
    _, pos, _ = route(idx, 3)
    X = torch.ones((2, 256), dtype=BF16, device=DEV)
    X[0, 3], X[1, 200] = float("inf"), float("-inf")
    Q, sa = kg.kg_dispatch_fp8(X, pos)
    r = pos.cpu().numpy()
    q, s = Q.cpu().numpy(), sa.cpu().numpy()
    assert np.isinf(s[0, r[0, 0]]) and s[1, r[0, 0]] == np.float32(1) / np.float32(448)
    assert q[r[0, 0], 3] == 0x7F and (q[r[0, 0], 4:128] == 0).all() and (q[r[0, 0], 128:] == 0x7E).all()
    assert np.isinf(s[1, r[1, 1]]) and q[r[1, 1], 200] == 0x7F
    Y = torch.ones((4, 256), device=DEV)
    Y[int(r[0, 1]), 7] = float("inf")
    out = kg.kg_combine(Y, pos, torch.full((2, 2), 0.5, device=DEV))
    assert torch.isinf(out[0, 7]) and (out[1] == 1).all() and (out[0, 8:] == 1).all()


@pytest.mark.parametrize("dt", [BF16, F32])
def test_strides_and_unaligned_views(dt):
    T, k, G, H = 37, 3, 6, 203
    idx = make_idx(T, k, G, "uniform", 3)
    _, pos, _ = route(idx, G)
    wide = torch.randn((T, H + 30), device=DEV).to(dt)
    flat = torch.randn(T * k * H + 1, device=DEV).to(dt)
    X, Y = wide[:, 5:5 + H], flat[1:].view(T * k, H)
    same = lambda a, b: torch.equal(a.contiguous().view(torch.uint8), b.contiguous().view(torch.uint8))
    assert same(kg.kg_dispatch(X, pos), kg.kg_dispatch(X.contiguous(), pos))
    out = torch.full((T, H + 9), 2.0, device=DEV, dtype=dt)
    kg.kg_combine(Y, pos, None, out[:, 4:4 + H])
    assert same(out[:, 4:4 + H], kg.kg_combine(Y.clone(), pos))
    assert (out[:, :4] == 2).all() and (out[:, 4 + H:] == 2).all()
    a = kg.kg_combine_bwd(X, Y, pos)
    b = kg.kg_combine_bwd(X.contiguous(), Y.clone(), pos)
    assert same(a[0], b[0]) and same(a[1], b[1])
    if dt == BF16:
        X16 = wide[:, 3:3 + 192]
        a, b = kg.kg_dispatch_fp8(X16, pos), kg.kg_dispatch_fp8(X16.contiguous(), pos)
        assert same(a[0], b[0]) and same(a[1], b[1])


def test_a_plan_that_names_no_row_touches_nothing():
    """pos values outside [0, T * k) (either sign) are passed over by every row kernel."""
    T, k, H = 6, 2, 64
    pos = torch.arange(T * k, dtype=torch.int32, device=DEV).view(T, k)
    bad = pos.clone()
    bad[1, 0], bad[2, 1], bad[3, 0], bad[4, 1] = T * k, 2**31 - 1, -2**31, ~(T * k)
    ok = (bad == pos).cpu()
    X = torch.randn((T, H), device=DEV)
    Xp = kg.kg_dispatch(X, bad, torch.full((T * k, H), 9.0, device=DEV))
    assert torch.equal(Xp.cpu(), torch.where(ok.view(-1, 1), X.cpu().repeat_interleave(k, 0), 9.0))
    Q = torch.full((T * k, H), 77, dtype=torch.uint8, device=DEV)
    sa = torch.full((1, T * k), 9.0, device=DEV)
    kg.kg_dispatch_fp8(X.to(BF16), bad, Q, sa)
    off = ~ok.view(-1).to(DEV)
    assert (Q[off] == 77).all() and (sa[0][off] == 9).all() and (sa[0][~off] != 9).all()
    Y = torch.randn((T * k, H), device=DEV)
    out = kg.kg_combine(Y, bad)
    assert torch.allclose(out.cpu(), torch.where(ok.view(-1, 1), Y.cpu(), 0.0).view(T, k, H).sum(1))
    dY, dw = kg.kg_combine_bwd(X, Y, bad, None, torch.full((T * k, H), 9.0, device=DEV))
    assert (dY[off] == 9).all() and (dw.view(-1)[off] == 0).all()
    assert torch.equal(dY[~off].cpu(), X.cpu().repeat_interleave(k, 0)[ok.view(-1)])


def test_gradients_against_differences():
    """combine and dispatch are linear in their rows and weights: with small whole numbers
    the differences of their values are exact, and equal what the gradients say."""
    T, k, G, H = 30, 3, 7, 66
    g = torch.Generator(DEV).manual_seed(1)
    whole = lambda *s: torch.randint(-3, 4, s, generator=g, device=DEV).float()
    _, pos, _ = route(make_idx(T, k, G, "wild", 5), G)
    Y, w, dOut, eY, ew = whole(T * k, H), whole(T, k), whole(T, H), whole(T * k, H), whole(T, k)
    dY, dw = kg.kg_combine_bwd(dOut, Y, pos, w)
    out = kg.kg_combine(Y, pos, w)
    assert ((kg.kg_combine(Y + eY, pos, w) - out) * dOut).sum() == (dY * eY).sum()
    assert ((kg.kg_combine(Y, pos, w + ew) - out) * dOut).sum() == (dw * ew).sum()
    X, eX, dXp = whole(T, H), whole(T, H), whole(T * k, H)
    dX = kg.kg_combine(dXp, pos)
    assert ((kg.kg_dispatch(X + eX, pos) - kg.kg_dispatch(X, pos)) * dXp).sum() == (dX * eX).sum()


def test_rows_past_32_bit_offsets():
    """8 slots of 40000 tokens at 8192 channels: the row tensors hold over 2^32 bytes."""
    T, k, G, H = 40000, 8, 64, 8192
    g = torch.Generator(DEV).manual_seed(2)
    idx = make_idx(T, k, G, "uniform", 9)
    _, pos, src = route(idx, G)
    X = torch.randn((T, H), generator=g, device=DEV).to(BF16)
    Xp = kg.kg_dispatch(X, pos)
    for a in range(0, T * k, 80000):
        assert torch.equal(Xp[a:a + 80000], X[src[a:a + 80000].long() // k])
    out = kg.kg_combine(Xp, pos)  # k equal rows: exact in fp32
    assert torch.equal(out, (X.float() * k).to(BF16))
    dY, dw = kg.kg_combine_bwd(X, Xp, pos)
    assert torch.equal(dY.view(torch.int16), Xp.view(torch.int16))
    want = X.double().square().sum(1)
    assert ((dw.double() - want[:, None]).abs() <= (H + 1) * 2.0 ** -24 * want[:, None]).all()


def test_other_stream_and_graph():
    """On a stream of its own, and captured: every replay follows the inputs it finds."""
    T, k, G, H = 600, 8, 64, 512
    g = torch.Generator(DEV).manual_seed(3)
    idx = torch.from_numpy(make_idx(T, k, G, "uniform", 1)).to(DEV)
    X = torch.randn((T, H), generator=g, device=DEV).to(BF16)
    w = torch.rand((T, k), generator=g, device=DEV)
    ks = torch.empty(G, dtype=torch.int32, device=DEV)
    ws = kg.new_route_workspace(T, k, G, DEV)
    pos, src = torch.empty_like(idx), torch.empty(T * k, dtype=torch.int32, device=DEV)
    Xp, out = torch.empty((T * k, H), dtype=BF16, device=DEV), torch.empty_like(X)
    Q, sa = torch.empty((T * k, H), dtype=torch.uint8, device=DEV), torch.empty((4, T * k), device=DEV)

    def step():
        kg.kg_route(idx, ks, pos, src, ws)
        kg.kg_dispatch(X, pos, Xp)
        kg.kg_dispatch_fp8(X, pos, Q, sa)
        kg.kg_combine(Xp, pos, w, out)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for seed in range(4):
        idx.copy_(torch.from_numpy(make_idx(T, k, G, "wild", 20 + seed)))
        X.copy_(torch.randn((T, H), generator=g, device=DEV))
        step()
        want = [t.clone() for t in (ks, pos, src, Xp, Q, sa, out)]
        for t in (ks, pos, src, Xp, Q, sa, out):
            t.zero_()
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(want, (ks, pos, src, Xp, Q, sa, out)):
            assert torch.equal(a, b)
        assert np.array_equal(pos.cpu().numpy(), plan_of(idx.cpu().numpy(), G)[1])


def test_tensors_made_for_a_stream():
    """With `stream` given, what a call makes (outputs, the plan's workspace) stays untouched by
    later allocations of the current stream until that stream is done with it."""
    T, k, G, H = 3000, 8, 64, 256
    idx = torch.from_numpy(make_idx(T, k, G, "uniform", 4)).to(DEV)
    X = torch.randn((T, H), device=DEV).to(BF16)
    ks = torch.empty(G, dtype=torch.int32, device=DEV)
    want = plan_of(idx.cpu().numpy(), G)
    side = torch.cuda.Stream()
    busy = torch.randn((4096, 4096), device=DEV)
    torch.cuda.synchronize()
    for _ in range(3):
        with torch.cuda.stream(side):
            for _ in range(4):
                busy @ busy  # the side stream's work is late
        pos, src = kg.kg_route(idx, ks, stream=side)
        Xp = kg.kg_dispatch(X, pos, stream=side)
        out = kg.kg_combine(Xp, pos, stream=side)
        for _ in range(50):  # would land in memory that was freed too early
            torch.full((2 ** 18,), 77, dtype=torch.int32, device=DEV)
        side.synchronize()
        assert np.array_equal(pos.cpu().numpy(), want[1]) and np.array_equal(src.cpu().numpy(), want[2])
        assert torch.equal(out, (X.float() * k).to(BF16))


def test_more_workgroups_than_a_line_holds():
    """300 million tokens of one slot: the launches need over 2^24 workgroups."""
    T, H = 300_000_000, 8
    pos = torch.arange(T - 1, -1, -1, dtype=torch.int32, device=DEV).view(T, 1)
    X = (torch.arange(T * H, device=DEV) & 0xFF).to(BF16).view(T, H)
    Xp = kg.kg_dispatch(X, pos)
    assert torch.equal(Xp.view(torch.int32), X.flip(0).view(torch.int32))
    out = kg.kg_combine(Xp, pos)
    assert torch.equal(out.view(torch.int32), X.view(torch.int32))
    dY, dw = kg.kg_combine_bwd(X, Xp, pos)
    assert torch.equal(dY.view(torch.int32), Xp.view(torch.int32))
    want = X.float().square().sum(1)
    assert torch.equal(dw.view(-1), want)  # whole numbers below 2^24


@pytest.mark.parametrize("T,k,G,H", [(400, 3, 20, 7), (200, 9, 12, 1235), (90, 17, 20, 40), (1100, 1, 3, 100),
                                     (900, 2, 8, 129), (130, 8, 16, 2500), (128, 8, 16, 520), (1, 1025, 9, 66)])
@pytest.mark.parametrize("dt", [BF16, F32])
@pytest.mark.parametrize("kind", ["uniform", "wild"])
def test_gradients_on_both_sides_of_the_slots_taken_one_by_one(T, k, G, H, dt, kind):
    test_dispatch_combine_and_gradients(T, k, G, H, dt, kind)


@pytest.mark.parametrize("H", [40, 520])
def test_gradients_of_many_slots_pass_over_bad_positions(H):
    T, k = 300, 4
    pos = torch.arange(T * k, dtype=torch.int32, device=DEV).view(T, k)
    bad = pos.clone()
    bad[1, 0], bad[2, 1], bad[299, 3], bad[4, 1] = T * k, 2**31 - 1, -2**31, ~(T * k)
    ok = (bad == pos).view(-1)
    X, Y = torch.randn((T, H), device=DEV), torch.randn((T * k, H), device=DEV)
    dY, dw = kg.kg_combine_bwd(X, Y, bad, None, torch.full((T * k, H), 9.0, device=DEV))
    assert (dY[~ok] == 9).all() and (dw.view(-1)[~ok] == 0).all()
    assert torch.equal(dY[ok], X.repeat_interleave(k, 0)[ok])
    assert (dw.view(-1)[ok] != 0).all()


@pytest.mark.parametrize("T,k,G,H", [(64, 8, 16, 7000), (65, 8, 16, 7000), (2100, 2, 8, 1100), (4200, 2, 8, 1100),
                                     (3000, 11, 40, 30), (1, 4096, 9, 66), (5000, 9, 3, 20)])
@pytest.mark.parametrize("dt", [BF16, F32])
def test_gradients_of_many_slots(T, k, G, H, dt):
    test_dispatch_combine_and_gradients(T, k, G, H, dt, "wild")
