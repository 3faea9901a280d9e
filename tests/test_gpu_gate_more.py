"""kg_gate and kg_gate_bwd: calls between those of test_gpu_gate, with its definition in 64 bits."""
import pytest
import torch

import fp8_grouped_gemm_tn_amd as kg
import test_gpu_gate as base

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("G", [100, 256])
def test_smaller_batches_in_a_workspace_of_the_largest(G):
    """A workspace for 2000 tokens serves every batch up to that, the most workgroups (1024 tokens) too, and
    nothing behind it is written."""
    n = kg.new_gate_workspace(2000, G, "cuda").numel()
    store = torch.full((n + 256,), 77, dtype=torch.uint8, device="cuda")
    ws = store[:n]
    for T in (2000, 1, 512, 1024, 1025, 0):
        x = base.logits(T, G, T)
        counts = torch.empty(G, dtype=torch.int32, device="cuda")
        psum, loss = torch.empty(G, device="cuda"), torch.empty(1, device="cuda")
        other = torch.empty_like(psum), torch.empty_like(loss), torch.empty_like(counts)
        kg.kg_gate(x, 4, coef=0.5, counts=counts, psum=psum, loss=loss, ws=ws)
        kg.kg_gate(x, 4, coef=0.5, counts=other[2], psum=other[0], loss=other[1])
        assert torch.equal(psum, other[0]) and torch.equal(loss, other[1]) and torch.equal(counts, other[2])
        assert int(counts.sum()) == 4 * T
    assert (store[n:] == 77).all()


@pytest.mark.parametrize("T,G", [(70, 17), (333, 40), (3000, 64), (1500, 100), (2000, 256), (500, 300)])
@pytest.mark.parametrize("k", [15, 16])
def test_last_choices_that_differ_in_the_last_bits(T, G, k):
    """The k-th and the next logit a few last bits apart, which cut keys do not tell apart, or equal, or far
    apart, and with fewer experts left than k: with 16 choices of 16 lanes the 17th key has no lane."""
    x = base.logits(T, G, T + k)
    order = x.argsort(1, descending=True)
    last = x.gather(1, order[:, k - 1:k])
    step = torch.tensor([0, 1, 2, 7, 100, 200, 1 << 12], device="cuda")[torch.arange(T, device="cuda") % 7][:, None]
    bits = last.view(torch.int32)
    near = torch.where(bits >= 0, bits - step, bits + step).int()  # below by `step` places
    x.scatter_(1, order[:, k:k + 1], near.view(torch.float32))
    x[3::11, G // 2:] = -float("inf")
    x[5::11] = -float("inf")
    base.check(x, k, norm=True)
    base.check(-x.masked_fill(x.isinf(), 0), k)


# The gradient's roundings, one by one. With u = 2^-24: a score's relative error e is 3 u |x - max| from its
# exponent (difference, factor, product) plus 2 u of v_exp_f32, and 24 u + u from the sum of up to 16 terms a
# lane and six steps across lanes and the quotient; a sigmoid's is 3 u |x| + 2 u for the exponential, u for the
# sum and 2 u for v_rcp_f32. The formulas then round each operation by u.
U = 2.0 ** -24


def gradient_bound(x, idx, dw, counts, dloss, sigmoid, norm, scale, coef):
    """|dx - the definition's|, by element."""
    x64 = x.detach().cpu().double()
    live = ~torch.isneginf(x64)
    far = torch.where(live, x64, 0.0).abs() if sigmoid else \
        torch.where(live, x64.amax(1, keepdim=True) - x64, 0.0)
    s, p = base.scores64(x, sigmoid)
    e = (3 * far + (5 if sigmoid else 27)) * U
    ok = (idx >= 0) & (idx < x.shape[1])
    at = torch.where(ok, idx, 0)
    dw64 = torch.where(ok, dw.cpu().double(), 0.0) if dw is not None else torch.zeros(idx.shape, dtype=torch.float64)
    sj, ej = torch.where(ok, s.gather(1, at), 0.0), torch.where(ok, e.gather(1, at), 0.0)
    if norm:
        total, et = sj.sum(1, keepdim=True) + 1e-20, ej.amax(1, keepdim=True) + 7 * U
        mean = (dw64 * sj).sum(1, keepdim=True) / total
        off_mean = ((dw64 * sj).abs() * (ej + et + 9 * U)).sum(1, keepdim=True) / total
        d = (dw64 - mean) / total
        off = (off_mean + U * (dw64.abs() + mean.abs())) / total + d.abs() * (et + 3 * U)
    else:
        d, off = dw64, torch.zeros_like(dw64)
    d, off = scale * d, scale * (off + U * d.abs())
    zero = torch.zeros_like(x64)
    d, off = zero.scatter_add(1, at, torch.where(ok, d, 0.0)), zero.scatter_add(1, at, torch.where(ok, off, 0.0))
    size = zero.scatter_add(1, at, torch.where(ok, d.gather(1, at).abs(), 0.0))  # (sums of a few named twice)
    off = off + 16 * U * size
    c = dloss * coef * counts.cpu().double()[None] if counts is not None else zero
    off_c = 4 * U * c.abs()
    if sigmoid:
        whole = s.sum(1, keepdim=True)
        mean = (p * c).sum(1, keepdim=True)
        et = e.amax(1, keepdim=True) + 26 * U
        off_mean = (p * (c.abs() * (e + et + 26 * U) + off_c)).sum(1, keepdim=True)
        even, off_even = (c - mean) / whole, (off_c + off_mean + U * (c - mean).abs()) / whole
        off_even = off_even + even.abs() * (et + 3 * U)
        t = d + even
        return s * (1 - s) * ((2 * e + 6 * U) * t.abs() + off + off_even + U * (d.abs() + even.abs()))
    v, off_v = d + c, off + off_c + U * (d.abs() + c.abs())
    mean = (p * v).sum(1, keepdim=True)
    off_mean = (p * (v.abs() * (e + 26 * U) + off_v)).sum(1, keepdim=True)
    return p * ((e + 3 * U) * (v - mean).abs() + off_v + off_mean + U * (v.abs() + mean.abs()))


@pytest.mark.parametrize("G,k", [(2, 1), (8, 2), (37, 3), (64, 8), (200, 16), (256, 8), (300, 6), (1024, 8)])
@pytest.mark.parametrize("sigmoid", [True, False])
@pytest.mark.parametrize("norm", [True, False])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_gradient_to_its_last_roundings(G, k, sigmoid, norm, dtype):
    for T, with_dw, with_loss in ((1100, True, True), (70, True, False), (70, False, True)):
        x = base.logits(T, G, T + G, dtype)
        flags, scale, coef = base.flags_of(sigmoid, norm), 2.5, 1.0 / T
        idx = kg.kg_gate(x, k, None, flags)[0]
        gen = torch.Generator("cuda").manual_seed(T + G)
        dw = torch.randn((T, k), generator=gen, device="cuda") if with_dw else None
        counts = torch.randint(0, T, (G,), generator=gen, device="cuda", dtype=torch.int32) if with_loss else None
        dloss = torch.full((1,), 0.625, device="cuda")
        dx = kg.kg_gate_bwd(x, idx, dw, counts, dloss, flags, scale, coef)
        args = (x, idx.cpu().long(), dw, counts, 0.625, sigmoid, norm, scale, coef)
        want, bound = base.grad64(*args), gradient_bound(*args)
        if dtype == "bf16":
            bound = bound * (1 + 2.0 ** -8) + 2.0 ** -8 * want.abs()
        off = (dx.cpu().double() - want).abs()
        # (2^-120: exponentials below fp32's range are zeros, bf16's last steps of what is next to zero)
        assert bool((off <= bound + 2.0 ** -120).all()), float((off / (bound + 2.0 ** -120)).max())


@pytest.mark.parametrize("sigmoid", [True, False])
@pytest.mark.parametrize("norm", [True, False])
@pytest.mark.parametrize("biased", [True, False])
@pytest.mark.parametrize("G", [6, 100, 300])
def test_empty_slots_of_rows_with_nan(G, norm, sigmoid, biased):
    """A slot without an expert has weight 0 whatever else its row holds."""
    x = base.logits(40, G, G)
    x[::2, 3:] = -float("inf")
    x[::4, 1] = float("nan")
    x[1] = float("nan")
    x[2, 0] = float("inf")
    idx, w = kg.kg_gate(x, 5, torch.zeros(G, device="cuda") if biased else None, base.flags_of(sigmoid, norm), 2.0)
    assert (idx[::2, 3:] == -1).all() and (idx[1] == -1).all()
    assert (w[idx == -1] == 0).all()
    good = torch.tensor([t for t in range(40) if t % 4 and t > 2])
    assert (idx[good, :2] >= 0).all() and w[good].isfinite().all()


@pytest.mark.parametrize("sigmoid", [True, False])
def test_logits_past_32_bit_offsets(sigmoid):
    """More than 2^31 logits: rows behind that are what they are alone, in choice and gradient, and the sums
    are those of all rows."""
    T, G, k = 2_200_000, 1024, 4
    gen = torch.Generator("cuda").manual_seed(1)
    x = torch.empty((T, G), dtype=torch.bfloat16, device="cuda")
    for at in range(0, T, 200_000):
        x[at:at + 200_000] = torch.randn((200_000, G), generator=gen, device="cuda")
    flags = base.flags_of(sigmoid, True)
    counts, psum = torch.empty(G, dtype=torch.int32, device="cuda"), torch.empty(G, device="cuda")
    idx, w = kg.kg_gate(x, k, None, flags, counts=counts, psum=psum)
    dx = kg.kg_gate_bwd(x, idx, w, counts, None, flags, 1.0, 1.0 / T)
    for rows in (slice(0, 500), slice(2 ** 21 - 300, 2 ** 21 + 300), slice(T - 700, T)):
        i, v = kg.kg_gate(x[rows], k, None, flags)
        assert torch.equal(i, idx[rows]) and torch.equal(v, w[rows])
        assert torch.equal(kg.kg_gate_bwd(x[rows], i, v, counts, None, flags, 1.0, 1.0 / T), dx[rows])
    base.check(x[T - 300:], k, sigmoid, True)
    want, n = torch.zeros(G, dtype=torch.float64, device="cuda"), torch.zeros(G, dtype=torch.int64, device="cuda")
    for at in range(0, T, 100_000):
        y = x[at:at + 100_000].double()
        s = torch.sigmoid(y) if sigmoid else torch.softmax(y, 1)
        want += (s / s.sum(1, keepdim=True)).sum(0)
        n += torch.bincount(idx[at:at + 100_000].flatten(), minlength=G)
    assert torch.equal(counts.long(), n)
    # a lane adds T / 4096 rows, then 8 waves and, in 64 bits, the workgroups
    assert bool(((psum.double() - want).abs() <= want * (base.TOL + (T / 4096 + 8) * 2.0 ** -24)).all())
