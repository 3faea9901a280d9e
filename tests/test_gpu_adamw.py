"""kg_adamw against its formula in 64 bits.

Tolerances. u = 2^-24. m and v are two products and a sum, their coefficients rounded once, v with
a square, and the gradient with its factor: off by at most 8 u of the sum of the terms' absolute
values. The step m / (sqrt(v) c + eps) adds six operations: 24 u of itself plus what m's
cancellation leaves, 8 u of its terms over the denominator; p adds 4 u |p| and, rounded to bf16,
2^-8 |p|. 8-bit states are within half a step of the value: 2^-4 of it, or half of the
smallest step, 2^-10 of the scale (for a nonzero square root up to 2^-9, as it may not become
zero), and their scales within 16 u of the block's largest."""
import math

import numpy as np
import pytest
import torch

import fp8_grouped_gemm_tn_amd as kg

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
BF16, F32, E4M3 = torch.bfloat16, torch.float32, torch.float8_e4m3fn
U = 2.0 ** -24
HYPER = dict(lr=3e-3, beta1=0.9, beta2=0.95, eps=1e-8, weight_decay=0.1)
SIZES = [1, 7, 8, 127, 128, 129, 1000, 2047, 2048, 2049, 5000, 0, 70001]


def unpack(q, s):
    n = q.numel()
    return q.view(E4M3).double() * s.double().repeat_interleave(128)[:n]


def make(sizes, pt, gt, packed, seed=0, offset=0):
    """Lists of tensors; `offset` elements of slack in front of each, which unaligns it."""
    g = torch.Generator(DEV).manual_seed(seed)
    cut = lambda n, dt, x: torch.cat([torch.zeros(offset, device=DEV), x]).to(dt)[offset:]
    rnd = lambda n: torch.randn(n, generator=g, device=DEV)
    t = dict(p=[cut(n, pt, rnd(n) * 0.1) for n in sizes], g=[cut(n, gt, rnd(n) * 1e-3) for n in sizes])
    if packed:
        byte = lambda n, lo: torch.randint(lo, 0x7F, (n + offset,), generator=g, device=DEV).to(torch.uint8)[offset:]
        t["m"] = [byte(n, 0) | (byte(n, 0) & 1) << 7 for n in sizes]
        t["v"] = [byte(n, 1) for n in sizes]
        t["ms"] = [torch.rand(-(-n // 128), generator=g, device=DEV) * 1e-5 for n in sizes]
        t["vs"] = [torch.rand(-(-n // 128), generator=g, device=DEV) * 1e-5 for n in sizes]
    else:
        t["m"] = [cut(n, F32, rnd(n) * 1e-3) for n in sizes]
        t["v"] = [cut(n, F32, (rnd(n) * 1e-3).square()) for n in sizes]
    t["copy"] = [cut(n, BF16, rnd(n)) for n in sizes]
    return t


def table(t, copies=True):
    return kg.AdamWTable(t["p"], t["g"], t["m"], t["v"], t.get("ms"), t.get("vs"),
                         t["copy"] if copies else None)


def clone(t):
    return {k: [x.clone() for x in v] for k, v in t.items()}


def check(before, after, step, gscale=1.0, copies=True, lr=HYPER["lr"]):
    b1, b2, eps, wd = HYPER["beta1"], HYPER["beta2"], HYPER["eps"], HYPER["weight_decay"]
    packed = "ms" in before
    for i in range(len(before["p"])):
        n = before["p"][i].numel()
        if n == 0:
            continue
        p, g = before["p"][i].double(), before["g"][i].double() * gscale
        if packed:
            m0 = unpack(before["m"][i], before["ms"][i])
            v0 = unpack(before["v"][i], before["vs"][i]).square()
        else:
            m0, v0 = before["m"][i].double(), before["v"][i].double()
        m, v = b1 * m0 + (1 - b1) * g, b2 * v0 + (1 - b2) * g * g
        tm, tv = 8 * U * ((b1 * m0).abs() + ((1 - b1) * g).abs()), 8 * U * v
        den = (v / (1 - b2 ** step)).sqrt() + eps
        rate = lr / (1 - b1 ** step)
        want = p * (1 - lr * wd) - rate * m / den
        tol = 4 * U * (p.abs() + want.abs()) + rate * (24 * U * m.abs() + tm) / den
        half = 2.0 ** -8 if before["p"][i].dtype == BF16 else 0.0
        got = after["p"][i].double()
        assert ((got - want).abs() <= tol * (1 + half) + half * want.abs()).all(), i
        if copies:
            assert torch.equal(after["copy"][i], after["p"][i].to(BF16)), i
        else:
            assert torch.equal(after["copy"][i], before["copy"][i]), i
        if not packed:
            assert ((after["m"][i].double() - m).abs() <= tm).all(), i
            assert ((after["v"][i].double() - v).abs() <= tv).all(), i
            continue
        for x, q, s, up in ((m, after["m"][i], after["ms"][i], False),
                            (v.sqrt(), after["v"][i], after["vs"][i], True)):
            pad = torch.zeros(-(-n // 128) * 128, dtype=torch.float64, device=DEV)
            pad[:n] = x.abs()
            amax = pad.view(-1, 128).amax(1)
            assert ((s.double() * 448 - amax).abs() <= 16 * U * amax + 448 * 8 * U * 1e-3 * (not up)).all(), i
            sc = s.double().repeat_interleave(128)[:n]
            small = sc * (2.0 ** -9 if up else 2.0 ** -10)
            err = (unpack(q, s) - x).abs()
            assert (err <= torch.maximum(2.0 ** -4 * x.abs(), small) * (1 + 2.0 ** -15) + tm * (not up)).all(), i
            if up:
                assert ((q.view(E4M3).float() > 0) | (x == 0)).all(), i


@pytest.mark.parametrize("pt", [F32, BF16])
@pytest.mark.parametrize("gt", [F32, BF16])
@pytest.mark.parametrize("packed", [False, True])
@pytest.mark.parametrize("offset", [0, 1, 3])
def test_step(pt, gt, packed, offset):
    t = make(SIZES, pt, gt, packed, seed=offset, offset=offset)
    before = clone(t)
    kg.kg_adamw(table(t), step=7, **HYPER)
    check(before, t, 7)


@pytest.mark.parametrize("packed", [False, True])
def test_first_step_from_zeros_and_factor(packed):
    """States of zeros are the start; gscale multiplies the gradients; no copies."""
    t = make(SIZES, F32, F32, packed)
    for k in ("m", "v", "ms", "vs"):
        for x in t.get(k, []):
            x.zero_()
    before = clone(t)
    kg.kg_adamw(table(t, copies=False), step=1, gscale=torch.tensor([0.25], device=DEV), **HYPER)
    check(before, t, 1, gscale=0.25, copies=False)


@pytest.mark.parametrize("packed", [False, True])
def test_many_tensors_equal_one_by_one(packed):
    """One table of 400 tensors gives the bits of 400 tables."""
    sizes = [int(x) for x in np.exp(np.random.default_rng(0).uniform(0, np.log(9000), 400))]
    a = make(sizes, F32, BF16, packed, 3)
    b = clone(a)
    kg.kg_adamw(table(a), step=3, **HYPER)
    for i in range(len(sizes)):
        kg.kg_adamw(table({k: [v[i]] for k, v in b.items()}), step=3, **HYPER)
    for k in a:
        for x, y in zip(a[k], b[k]):
            assert torch.equal(x.view(torch.uint8), y.view(torch.uint8))


@pytest.mark.parametrize("packed", [False, True])
def test_zero_gradients_and_tiny_states(packed):
    """A block of zeros stays zero (p only decays); values whose scale would underflow are
    held as zeros, and nothing becomes infinite or NaN."""
    t = make([256, 300], F32, F32, packed, 5)
    for k in ("m", "v", "ms", "vs"):
        for x in t.get(k, []):
            x.zero_()
    t["g"][0].zero_()
    t["g"][1].fill_(1e-37)
    p = [x.clone() for x in t["p"]]
    kg.kg_adamw(table(t), step=1, **HYPER)
    assert all(torch.isfinite(x.float()).all() for x in t["p"])
    assert torch.allclose(t["p"][0], p[0] * (1 - 3e-4), rtol=4 * U, atol=0)
    assert torch.allclose(t["p"][1], p[1] * (1 - 3e-4), rtol=4 * U, atol=0)  # 1e-37 / eps is nothing
    for k in ("m", "v"):
        assert (t[k][0].view(torch.uint8) & 0x7F == 0).all()


@pytest.mark.parametrize("packed", [False, True])
@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_gradients_that_are_not_finite(packed, bad):
    """Such a gradient shows in its element, and with 8-bit states in its block of 128; the
    neighbouring blocks and tensors are as without it."""
    a = make([384, 200], F32, F32, packed, 6)
    b = clone(a)
    a["g"][0][130] = bad
    kg.kg_adamw(table(a), step=2, **HYPER)
    kg.kg_adamw(table(b), step=2, **HYPER)
    assert not torch.isfinite(a["p"][0][130]) or not torch.isfinite(a["m"][0].view(E4M3).float()[130] if packed else a["m"][0][130])
    keep = torch.ones(384, dtype=torch.bool, device=DEV)
    keep[130] = False
    assert torch.equal(a["p"][0][keep], b["p"][0][keep])
    keep[128:256] = False
    for k in ("m", "v"):
        assert torch.equal(a[k][0][keep], b[k][0][keep]) and torch.equal(a[k][1], b[k][1])
    assert torch.equal(a["p"][1], b["p"][1])
    if packed:
        assert not torch.isfinite(unpack(a["m"][0], a["ms"][0])[128:256]).any()
        assert not torch.isfinite(unpack(a["v"][0], a["vs"][0])[128:256]).any()


def test_device_hyperparameters_and_graph():
    """A captured step follows lr and the bias corrections that it finds in device memory."""
    t = make([3000, 77], F32, BF16, True, 8)
    tab = table(t)
    dyn = torch.zeros(3, device=DEV)

    def put(step, lr):
        dyn.copy_(torch.tensor([lr, 1 - HYPER["beta1"] ** step, 1 - HYPER["beta2"] ** step]))

    put(1, 1e-3)
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):
        kg.kg_adamw(tab, dyn=dyn, **HYPER)
    stream.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        kg.kg_adamw(tab, dyn=dyn, **HYPER)
    for step in range(2, 6):
        for x in t["g"]:
            x.copy_(torch.randn(x.numel(), device=DEV) * 1e-3)
        put(step, 1e-3 * step)
        before = clone(t)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        check(before, t, step, lr=1e-3 * step)


def test_more_than_32_bits_of_bytes():
    """A parameter of 2^30 + 300 elements: its bytes pass 2^32."""
    n = 2 ** 30 + 300
    t = dict(p=[torch.full((n,), 0.5, device=DEV)], g=[torch.full((n,), 1e-3, dtype=BF16, device=DEV)],
             m=[torch.zeros(n, dtype=torch.uint8, device=DEV)], v=[torch.zeros(n, dtype=torch.uint8, device=DEV)],
             ms=[torch.zeros(-(-n // 128), device=DEV)], vs=[torch.zeros(-(-n // 128), device=DEV)])
    kg.kg_adamw(kg.AdamWTable(t["p"], t["g"], t["m"], t["v"], t["ms"], t["vs"]), step=1, **HYPER)
    p = t["p"][0]
    assert (p == p[0]).all() and abs(float(p[0]) - (0.5 * (1 - 3e-4) - 3e-3)) < 1e-6
    for k in ("m", "v"):
        assert (t[k][0] == 0x7E).all()  # every element is its block's largest: 448


@pytest.mark.parametrize("packed", [False, True])
def test_training_reaches_the_64_bit_loss(packed):
    """Least squares with noisy gradients: the loss after 300 steps is near what the same
    gradients give in 64 bits (8-bit states within 15 %, fp32 ones within 0.1 %)."""
    g = torch.Generator(DEV).manual_seed(12)
    d, n = 1536, 4096
    X = torch.randn((n, d), generator=g, device=DEV) * torch.exp(torch.randn(d, generator=g, device=DEV) * 0.7)
    goal = torch.randn(d, generator=g, device=DEV)
    y = X @ goal + torch.randn(n, generator=g, device=DEV)
    hyper = dict(lr=2e-2, beta1=0.9, beta2=0.99, eps=1e-8, weight_decay=0.0)
    p = torch.zeros(d, device=DEV)
    grad = torch.zeros(d, device=DEV)
    nb = d // 128
    if packed:
        st = [torch.zeros(d, dtype=torch.uint8, device=DEV) for _ in "mv"]
        tab = kg.AdamWTable([p], [grad], [st[0]], [st[1]], [torch.zeros(nb, device=DEV)], [torch.zeros(nb, device=DEV)])
    else:
        st = [torch.zeros(d, device=DEV) for _ in "mv"]
        tab = kg.AdamWTable([p], [grad], [st[0]], [st[1]])
    q, m, v = (torch.zeros(d, dtype=torch.float64, device=DEV) for _ in range(3))
    for step in range(1, 301):
        rows = torch.randint(0, n, (256,), generator=g, device=DEV)
        x, t = X[rows], y[rows]
        grad.copy_(x.t() @ (x @ p - t) / 256)
        kg.kg_adamw(tab, step=step, **hyper)
        gq = (x.double().t() @ (x.double() @ q - t.double())) / 256
        m, v = 0.9 * m + 0.1 * gq, 0.99 * v + 0.01 * gq * gq
        q = q - 2e-2 * (m / (1 - 0.9 ** step)) / ((v / (1 - 0.99 ** step)).sqrt() + 1e-8)
    loss = lambda w: float((X.double() @ w.double() - y.double()).square().mean())
    start, ref, got = loss(torch.zeros(d, device=DEV)), loss(q), loss(p)
    print(f"[loss] start {start:.4f} 64-bit {ref:.4f} here {got:.4f}", flush=True)
    assert ref < 0.5 * start
    assert got <= ref * (1.15 if packed else 1.001)
