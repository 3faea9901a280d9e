"""kg_gate and kg_gate_bwd against the definition in 64 bits.

Tolerances. A score is an exponential (or a sigmoid) of a logit's difference and a quotient: the
difference is rounded by 2^-24 of its size, which the exponential turns into a relative error of
|x - max| 2^-24, at most 2^-24 / e of the largest score; the exponential and the reciprocal are off
by about 2^-23 each, sums of up to 1024 terms by at most 22 roundings. So scores and weights are
within 40 * 2^-24 = TOL of the larger of themselves and the row's largest. psum adds T such terms in
runs of at most T / 64 + 20 roundings. Gradients add five products of those: 8 TOL of the sum of
magnitudes. bf16 outputs add half a step, 2^-8
relative."""
import math

import pytest
import torch

import fp8_grouped_gemm_tn_amd as kg

pytestmark = pytest.mark.gpu
TOL = 40 * 2.0 ** -24
INF, LOWEST = math.inf, torch.finfo(torch.float32).min
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


def logits(T, G, seed, dtype="f32", mask=None):
    gen = torch.Generator("cuda").manual_seed(seed)
    x = 2 * torch.randn((T, G), generator=gen, device="cuda")
    if mask is not None:
        x[torch.rand((T, G), generator=gen, device="cuda") < 0.3] = mask
        x[::5] = mask  # whole rows
        if T > 1:
            x[1, : G // 2] = mask
    return x.to(TYPES[dtype])


def scores64(x, sigmoid):
    """Scores and balance probabilities of the definition, in 64 bits on the CPU."""
    x = x.detach().cpu().double()
    dead = torch.isneginf(x).all(1, keepdim=True)
    if sigmoid:
        s = torch.special.expit(x)
        total = s.sum(1, keepdim=True)
        return s, torch.where(total == 0, 0.0, s / torch.where(total == 0, 1.0, total))
    p = torch.where(dead, 0.0, torch.softmax(torch.where(dead, 0.0, x), 1))
    return p, p


def choice64(x, k, sigmoid=False, bias=None):
    x64 = x.detach().cpu().double()
    key = x64 if bias is None else scores64(x, sigmoid)[0] + bias.cpu().double()
    key = torch.where((x64 == -INF) | x64.isnan() | key.isnan(), -INF, key)
    top, idx = torch.sort(key, dim=1, descending=True, stable=True)
    return torch.where(top[:, :k] == -INF, -1, idx[:, :k])


def weights64(x, idx, sigmoid, norm, scale):
    s = scores64(x, sigmoid)[0]
    w = torch.where(idx < 0, 0.0, s.gather(1, idx.clamp(min=0)))
    if norm:
        w = w / (w.sum(1, keepdim=True) + 1e-20)
    return scale * w


def near(got, want, tol, size=None):
    got, size = got.detach().cpu().double(), want.abs() if size is None else size
    off = (got - want).abs() - tol * size
    assert got.isfinite().all() and float(off.max() if off.numel() else 0) <= 0, float(off.max())


def flags_of(sigmoid, norm):
    return (kg.KG_GATE_SIGMOID if sigmoid else 0) | (kg.KG_GATE_NORM if norm else 0)


def check(x, k, sigmoid=False, norm=False, scale=1.0, bias=None, coef=0.5):
    T, G = x.shape
    counts = torch.full((G,), -7, dtype=torch.int32, device="cuda")
    psum, loss = torch.full((G,), math.nan, device="cuda"), torch.full((1,), math.nan, device="cuda")
    idx, w = kg.kg_gate(x, k, bias, flags_of(sigmoid, norm), scale, coef, counts=counts, psum=psum,
                        loss=loss)
    only, w2 = kg.kg_gate(x, k, bias, flags_of(sigmoid, norm), scale)
    want = choice64(x, k, sigmoid, bias)
    assert torch.equal(idx.cpu().long(), want)
    assert torch.equal(only, idx) and torch.equal(w2, w)
    ww = weights64(x, want, sigmoid, norm, scale)
    top = ww.amax(1, keepdim=True) if not norm else torch.full((T, 1), scale, dtype=torch.float64)
    near(w, ww, TOL, torch.maximum(ww.abs(), top.expand_as(ww)) if not sigmoid else ww.abs() + 1e-30)
    n = torch.stack([(want == g).sum() for g in range(G)])
    assert torch.equal(counts.cpu().long(), n)
    p = scores64(x, sigmoid)[1].sum(0)
    tol = TOL + (T / 64 + 20) * 2.0 ** -24
    near(psum, p, tol, p + 1e-6 * T)
    near(loss, coef * (n * p).sum().view(1), 2 * tol)
    return idx, w, counts


@pytest.mark.parametrize("G", [1, 2, 15, 37, 64, 65, 128, 200, 256, 257, 512, 513, 1000, 1024])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_sizes(G, dtype):
    for T, k in ((1, 1), (3, min(G, 8)), (129, min(G, 3)), (700, min(G, 16))):
        check(logits(T, G, T + G, dtype), k, norm=T % 2 == 1)


@pytest.mark.parametrize("G,k", [(8, 2), (256, 8), (200, 14), (256, 15), (250, 16), (700, 16), (33, 1)])
@pytest.mark.parametrize("sigmoid", [True, False])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_biased(G, k, sigmoid, dtype):
    gen = torch.Generator("cuda").manual_seed(G + k)
    bias = 0.05 * torch.randn(G, generator=gen, device="cuda")
    check(logits(901, G, G, dtype), k, sigmoid, norm=True, scale=2.5, bias=bias)


@pytest.mark.parametrize("mask", [-INF, LOWEST])
@pytest.mark.parametrize("sigmoid", [True, False])
@pytest.mark.parametrize("biased", [True, False])
@pytest.mark.parametrize("G", [8, 100, 300])
def test_masked(mask, sigmoid, biased, G):
    bias = torch.linspace(-0.1, 0.1, G, device="cuda") if biased else None
    idx, w, _ = check(logits(333, G, G, mask=mask), 7, sigmoid, norm=not sigmoid, bias=bias)
    if mask == -INF:
        assert (idx[::5] == -1).all() and (w[::5] == 0).all()


@pytest.mark.parametrize("G", [8, 129, 256, 1024])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("biased", [True, False])
def test_equal_logits(G, dtype, biased):
    """Ties go to the lower index: equal rows, rows of few values, both zeros."""
    gen = torch.Generator("cuda").manual_seed(G)
    x = torch.zeros((64, G), device="cuda")
    x[16:32] = torch.randint(-2, 3, (16, G), generator=gen, device="cuda").float()
    x[32:48] = torch.where(torch.rand((16, G), generator=gen, device="cuda") < 0.5, 0.0, -0.0)
    x[48:] = 1.0 + torch.randint(0, 3, (16, G), generator=gen, device="cuda") * 2.0 ** -23
    bias = torch.full((G,), 0.25, device="cuda") if biased else None
    check(x.to(TYPES[dtype]), min(G, 8), sigmoid=biased, bias=bias)


@pytest.mark.parametrize("sigmoid", [True, False])
@pytest.mark.parametrize("step", [2.0 ** -21, 2.0 ** -24, 2.0 ** -30])
@pytest.mark.parametrize("G,k", [(64, 6), (256, 8), (512, 8)])
def test_keys_a_few_last_bits_apart(sigmoid, step, G, k):
    """Biases that bring many keys together closer than 32 bits tell apart."""
    gen = torch.Generator("cuda").manual_seed(G)
    x = torch.randn((500, G), generator=gen, device="cuda")
    s = scores64(x[:1], sigmoid)[0][0]
    bias = (0.75 - s + step * torch.randint(-3, 4, (G,), generator=gen, device="cuda").cpu()).float()
    x[::2] = x[0]
    check(x, k, sigmoid, bias=bias.cuda())


def test_nan_and_infinite_logits():
    x = logits(64, 100, 3)
    x[3, 5] = math.nan
    x[4, 7] = INF
    x[6] = math.nan
    for sigmoid in (False, True):
        for bias in (None, torch.zeros(100, device="cuda")):
            idx, w = kg.kg_gate(x, 4, bias, kg.KG_GATE_SIGMOID if sigmoid else 0)
            rest = [t for t in range(64) if t not in (3, 4, 6)]
            want = choice64(x, 4, sigmoid, bias)
            assert torch.equal(idx.cpu().long()[rest], want[rest])
            assert (idx[3] != 5).all() and (idx[6] == -1).all() and (w[6] == 0).all()
            if bias is None:
                assert torch.equal(idx.cpu().long(), want)
            if not sigmoid and bias is None:
                assert w[3].isnan().all() and w[4, 0].isnan()


def test_very_negative_sigmoids():
    """Scores down to nothing: weights and probabilities stay finite."""
    x = torch.full((8, 40), -95.0, device="cuda") - torch.arange(40, device="cuda") * 0.5
    psum = torch.empty(40, device="cuda")
    idx, w = kg.kg_gate(x, 4, None, kg.KG_GATE_SIGMOID | kg.KG_GATE_NORM, psum=psum)
    assert w.isfinite().all() and psum.isfinite().all() and (psum <= 8).all()
    dx = kg.kg_gate_bwd(x, idx, torch.ones_like(w), torch.ones(40, dtype=torch.int32, device="cuda"),
                        None, kg.KG_GATE_SIGMOID | kg.KG_GATE_NORM, 1.0, 1.0)
    assert dx.isfinite().all()


def test_rows_of_a_wider_matrix_and_no_tokens():
    wide = logits(100, 300, 1)
    x = wide[:, 7:207]
    check(x, 5)
    check(logits(100, 301, 1, "bf16")[:, 1:201], 5, sigmoid=True, bias=torch.zeros(200, device="cuda"))
    check(x[:0], 5)
    dx = torch.full((100, 300), 5.0, device="cuda")
    idx, w = kg.kg_gate(x, 5)
    kg.kg_gate_bwd(x, idx, torch.ones_like(w), dX=dx[:, 50:250])
    assert (dx[:, :50] == 5).all() and (dx[:, 250:] == 5).all() and (dx[:, 50:250] != 5).all()


def test_long():
    check(logits(70001, 256, 1), 8, norm=True)


def test_the_same_in_every_run():
    x = logits(30000, 64, 2)
    outs = []
    for _ in range(3):
        o = [torch.empty(64, device="cuda"), torch.empty(1, device="cuda")]
        kg.kg_gate(x, 4, psum=o[0], loss=o[1], coef=1.0)
        outs.append(o)
    assert all(torch.equal(a, b) for o in outs[1:] for a, b in zip(o, outs[0]))


# ------------------------------------------------------------------------------- gradient

def grad64(x, idx, dw, counts, dloss, sigmoid, norm, scale, coef):
    """The derivative of sum(w dw) + dloss coef counts . psum, and the sum of magnitudes."""
    x64 = x.detach().cpu().double()
    dead = torch.isneginf(x64)
    leaf = torch.where(dead, -800.0 if not sigmoid else -700.0, x64).requires_grad_()
    some = (~dead).any(1, keepdim=True)
    if sigmoid:
        s = torch.sigmoid(leaf) * ~dead
        p = s / s.sum(1, keepdim=True).clamp(min=1e-300)
    else:
        s = p = torch.softmax(leaf, 1) * some * ~dead
    ok = (idx >= 0) & (idx < x.shape[1])
    w = torch.where(ok, s.gather(1, torch.where(ok, idx, 0)), 0.0)
    if norm:
        w = w / (w.sum(1, keepdim=True) + 1e-20)
    total = 0 * leaf.sum()
    if dw is not None:
        total = total + (scale * w * dw.cpu().double()).sum()
    if counts is not None:
        total = total + dloss * coef * (p * counts.cpu().double()).sum()
    total.backward()
    return torch.where(dead, 0.0, leaf.grad)


def check_back(x, k, sigmoid, norm, scale, with_dw=True, with_loss=True, idx=None):
    T, G = x.shape
    gen = torch.Generator("cuda").manual_seed(T)
    if idx is None:
        idx = kg.kg_gate(x, k, None, flags_of(sigmoid, norm))[0]
    dw = torch.randn((T, k), generator=gen, device="cuda") if with_dw else None
    counts = torch.randint(0, T + 1, (G,), generator=gen, device="cuda", dtype=torch.int32) if with_loss else None
    dloss, coef = torch.full((1,), 0.7, device="cuda"), 1.0 / max(T, 1)
    dx = kg.kg_gate_bwd(x, idx, dw, counts, dloss, flags_of(sigmoid, norm), scale, coef)
    want = grad64(x, idx.cpu().long(), dw, counts, float(dloss), sigmoid, norm, scale, coef)
    size = scale * (4 if with_dw else 0) + (1.5 if with_loss else 0)
    if norm and with_dw:  # the quotient by a small sum
        s = scores64(x, sigmoid)[0]
        own = torch.where(idx.cpu() < 0, 0.0, s.gather(1, idx.cpu().long().clamp(0, G - 1)))
        size = size + 8 * scale / (own.sum(1, keepdim=True) + 1e-20)
    s, p = scores64(x, sigmoid)
    bound = 8 * TOL * size * (s + p + 1e-9)  # (the loss's part is a multiple of p)
    if dx.dtype == torch.bfloat16:
        bound = bound + 2.0 ** -8 * want.abs()
    off = (dx.cpu().double() - want).abs() - bound
    assert dx.isfinite().all() and float(off.max()) <= 0, float(off.max())
    return dx


@pytest.mark.parametrize("G,k", [(1, 1), (2, 2), (37, 3), (64, 8), (129, 16), (256, 8), (300, 6), (1024, 16)])
@pytest.mark.parametrize("sigmoid", [True, False])
@pytest.mark.parametrize("norm", [True, False])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_gradient(G, k, sigmoid, norm, dtype):
    for T in (1, 5, 333):
        check_back(logits(T, G, T + G, dtype), k, sigmoid, norm, 2.5)
    check_back(logits(50, G, 7, dtype), k, sigmoid, norm, 1.0, with_dw=False)
    check_back(logits(50, G, 7, dtype), k, sigmoid, norm, 1.0, with_loss=False)


@pytest.mark.parametrize("sigmoid", [True, False])
@pytest.mark.parametrize("norm", [True, False])
def test_gradient_of_masked_logits(sigmoid, norm):
    x = logits(333, 100, 1, mask=-INF)
    dx = check_back(x, 5, sigmoid, norm, 1.0)
    assert (dx[x == -INF] == 0).all()


def test_gradient_of_slots_named_by_hand():
    """Experts named twice, entries outside [0, G)."""
    x = logits(200, 30, 1)
    gen = torch.Generator("cuda").manual_seed(1)
    idx = torch.randint(-2, 33, (200, 6), generator=gen, device="cuda", dtype=torch.int32)
    idx[:, 3] = idx[:, 1]
    idx[0] = 4
    check_back(x, 6, False, False, 1.0, idx=idx)
    check_back(x, 6, True, False, 1.0, idx=idx)


@pytest.mark.parametrize("sigmoid", [True, False])
@pytest.mark.parametrize("norm", [True, False])
def test_gradient_against_differences(sigmoid, norm):
    """Central differences of the call's own weights and loss; the choice does not change."""
    x = logits(1, 12, 9) + torch.arange(12, device="cuda") * 0.5
    dw = torch.tensor([[0.3, -0.9, 0.5]], device="cuda")
    f, h = flags_of(sigmoid, norm), 2.0 ** -6

    def value(x):
        loss, counts = torch.empty(1, device="cuda"), torch.empty(12, dtype=torch.int32, device="cuda")
        idx, w = kg.kg_gate(x, 3, None, f, 1.5, 0.25, counts=counts, loss=loss)
        return float((w.double() * dw).sum() + loss.double()), idx, counts

    _, idx, counts = value(x)
    dx = kg.kg_gate_bwd(x, idx, dw, counts, None, f, 1.5, 0.25)
    for i in range(12):
        e = torch.zeros_like(x)
        e[0, i] = h
        (a, ia, _), (b, ib, _) = value(x + e), value(x - e)
        assert torch.equal(ia, ib)
        # rounding of values of about 2 by 2^-21, over 2 h; the third derivative, below 2, h^2 / 6
        assert abs((a - b) / (2 * h) - float(dx[0, i])) <= 2.0 ** -20 / h + 2 * h * h / 6


# ------------------------------------------------------------------ streams, graphs, together

def test_on_another_stream():
    x = logits(5000, 64, 4)
    want = kg.kg_gate(x, 4)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    counts = torch.empty(64, dtype=torch.int32, device="cuda")
    idx, w = kg.kg_gate(x, 4, counts=counts, stream=s)
    dx = kg.kg_gate_bwd(x, idx, w, counts, stream=s, coef=1.0)
    torch.cuda.current_stream().wait_stream(s)
    assert torch.equal(idx, want[0]) and torch.equal(w, want[1])
    assert torch.equal(dx, kg.kg_gate_bwd(x, idx, w, counts, coef=1.0))


def test_in_a_graph():
    """Captured and replayed with other logits, eager work between the replays."""
    x = logits(4000, 96, 5)
    ws = kg.new_gate_workspace(4000, 96, "cuda")
    new = lambda *s, dtype=torch.float32: torch.empty(s, dtype=dtype, device="cuda")
    idx, w, counts = new(4000, 4, dtype=torch.int32), new(4000, 4), new(96, dtype=torch.int32)
    psum, loss, dx = new(96), new(1), new(4000, 96)

    def step():
        kg.kg_gate(x, 4, None, 2, 1.0, 0.1, idx, w, counts, psum, loss, ws)
        kg.kg_gate_bwd(x, idx, w, counts, loss, 2, 1.0, 0.1, dx)

    step()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    for seed in range(3):
        x.copy_(logits(4000, 96, 50 + seed))
        g.replay()
        got = [t.clone() for t in (idx, w, counts, psum, loss, dx)]
        torch.cuda.synchronize()
        step()
        assert all(torch.equal(a, b) for a, b in zip(got, (idx, w, counts, psum, loss, dx)))


def test_choice_to_rows_and_back():
    """kg_gate's choice through kg_route, kg_dispatch and kg_combine; its counts are kg_route's."""
    T, G, k, H = 500, 24, 4, 64
    x = logits(T, G, 6, mask=-INF)
    counts, ks = (torch.empty(G, dtype=torch.int32, device="cuda") for _ in range(2))
    idx, w = kg.kg_gate(x, k, None, kg.KG_GATE_NORM, counts=counts)
    pos, _ = kg.kg_route(idx, ks)
    assert torch.equal(counts, ks)
    rows = torch.randn((T, H), device="cuda")
    out = kg.kg_combine(kg.kg_dispatch(rows, pos), pos, w)
    full = (w.double().sum(1, keepdim=True) * rows.double()).cpu()
    assert float((out.cpu().double() - full).abs().max()) <= 16 * 2.0 ** -24 * float(rows.abs().max())
