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
