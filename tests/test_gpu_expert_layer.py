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
