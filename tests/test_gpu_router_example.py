"""examples/expert_layer.py with kg_gate as its router and kg_orthogonalize as its experts' step: it runs,
and its router's gradients are those of the plain router.

Tolerances, u = 2^-24 being a rounding to fp32. A weight p goes through some ten roundings on either
side (the exponential's argument, itself, the sums over 8 experts, a quotient), and 1.5 u of the
exponential unit on one: 16 u of itself. A score's gradient is p (dp - sum p dp): 64 u of
p (|dp| + sum p |dp|). The router's gradient sums T of them: (T + 64) u of the sum of magnitudes on
either side."""
import importlib.util
import os

import pytest
import torch

import fp8_grouped_gemm_tn_amd as kg

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
U = 2.0 ** -24


def example():
    spec = importlib.util.spec_from_file_location("expert_layer",
                                                  os.path.join(ROOT, "examples", "expert_layer.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


@pytest.mark.parametrize("k", [1, 2, 5])
def test_router_gradients(k):
    G, K, N, T = 8, 256, 128, 300
    layers = [example().ExpertLayer(G, K, N, k, seed=4, balance=b) for b in (None, 0.0)]
    gen = torch.Generator("cuda").manual_seed(5)
    x, dout = (torch.randn((T, n), generator=gen, device="cuda").to(torch.bfloat16) for n in (K, N))
    for layer in layers:
        layer.forward(x)
    plain, own = layers
    assert torch.equal(plain.idx, own.idx) and torch.equal(plain.ks, own.ks)
    assert torch.equal(own.counts, own.ks)
    assert ((plain.p - own.p).abs() <= 32 * U * plain.p).all()
    for layer in layers:
        layer.backward(dout)
    # |dp| from the plain layer's rows (its own y: the same rows and weights in both)
    _, dp = kg.kg_combine_bwd(dout, plain.y, plain.pos, plain.p)
    p, dp = plain.p.double(), dp.double().abs()
    size = p * (dp + (p * dp).sum(1, keepdim=True))
    full = torch.zeros((T, G), device="cuda", dtype=torch.float64).scatter_(1, plain.idx.long(), size)
    bound = 2 * (T + 64) * U * (full.t() @ x.double().abs())
    assert ((plain.grads[1] - own.grads[1]).double().abs() <= bound).all()


@pytest.mark.parametrize("bits", [8, 32])
def test_runs(bits):
    losses = example().train(steps=4, bits=bits, T=512, balance=0.01, orthogonal=True)
    assert len(losses) == 4 and torch.tensor(losses).isfinite().all()
