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
