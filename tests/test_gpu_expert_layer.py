"""The operators together, as examples/expert_layer.py uses them: its gradients against the
64-bit derivative of the same layer, and its training with 8-bit and 32-bit optimizer states.

Tolerances. The example's fp8 operands are rounded by at most 2^-4 of a value (half a step of
3 mantissa bits), in products with rounding errors of both operands that are independent of
each other: results are within 2 * 2^-4 of their norm."""
import importlib.util
import os

import pytest
import torch

import fp8_grouped_gemm_tn_amd as kg

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def example():
    spec = importlib.util.spec_from_file_location("expert_layer",
                                                  os.path.join(ROOT, "examples", "expert_layer.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


@pytest.mark.parametrize("T,G,K,N,k", [(300, 5, 128, 256, 2), (1, 8, 256, 128, 3), (1000, 3, 384, 128, 1)])
def test_gradients(T, G, K, N, k):
    layer = example().ExpertLayer(G, K, N, k, seed=4)
    gen = torch.Generator("cuda").manual_seed(5)
    x = torch.randn((T, K), generator=gen, device="cuda").to(torch.bfloat16)
    dout = torch.randn((T, N), generator=gen, device="cuda").to(torch.bfloat16)
    out = layer.forward(x)
    dx = layer.backward(dout)
    assert kg.kg_status() == kg.KG_OK
    leaf = lambda t: t.detach().cpu().double().requires_grad_()
    x64, w64, r64 = leaf(x), leaf(layer.w), leaf(layer.router)
    idx = layer.idx.cpu().long()
    p = torch.softmax((x64 @ r64.t()).gather(1, idx), 1)
    want = sum(p[:, j, None] * torch.bmm(w64[idx[:, j]], x64[:, :, None])[:, :, 0] for j in range(k))
    want.backward(dout.cpu().double())
    near = lambda a, b: float((a.detach().cpu().double() - b).norm()) <= 2 * 2.0 ** -4 * float(b.norm())
    assert near(out, want.detach())
    assert near(dx, x64.grad)
    assert near(layer.grads[0], w64.grad)
    if k > 1:  # (a softmax over one score has no gradient)
        assert near(layer.grads[1], r64.grad)


@pytest.mark.parametrize("bits", [8, 32])
def test_training(bits):
    losses = example().train(steps=80, bits=bits)
    print(f"[loss] {bits}-bit states: {losses[0]:.4f} -> {losses[-1]:.4f}", flush=True)
    assert losses[-1] < 0.2 * losses[0]


@pytest.mark.parametrize("T,G,K,N,k", [(200, 6, 256, 256, 3), (4, 3, 128, 128, 2)])
def test_dropped_slots_through_the_products(T, G, K, N, k):
    """Experts held elsewhere: the products take the kept rows, the sums leave the others out."""
    gen = torch.Generator("cuda").manual_seed(T)
    rand = lambda *s: torch.randn(s, generator=gen, device="cuda")
    idx = torch.randint(-2, G + 2, (T, k), generator=gen, device="cuda", dtype=torch.int32)
    idx[0, 0], idx[1, 0] = 0, G  # one slot of either kind at least
    x, w, p = rand(T, K).to(torch.bfloat16), rand(G, N, K), rand(T, k)
    ks = torch.empty(G, dtype=torch.int32, device="cuda")
    pos, _ = kg.kg_route(idx, ks)
    rows, sa = kg.kg_dispatch_fp8(x, pos)
    n = int(ks.sum())
    wq, sw = example().inputs.quantize_blocks_128x128(w)
    y = torch.full((T * k, N), float("nan"), dtype=torch.bfloat16, device="cuda")
    kg.kg_fprop(rows[:n], sa[:, :n].contiguous(), wq, sw, y[:n], ks, kg.KG_FLAG_FP8_MFMA)
    assert kg.kg_status() == kg.KG_OK
    assert y[n:].isnan().all()
    out = kg.kg_combine(y, pos, p)
    on = (idx >= 0) & (idx < G)
    at = idx.clamp(0, G - 1).long().cpu()
    one = torch.einsum("tk,tjnk->tjn", x.cpu().double(), w.cpu().double()[at])
    want = (one * (p * on).cpu().double()[..., None]).sum(1)
    assert float((out.cpu().double() - want).norm()) <= 2 * 2.0 ** -4 * float(want.norm())
