"""kg_route: a workspace made for the largest call serves the smaller ones."""
import pytest
import torch

import fp8_grouped_gemm_tn_amd as kg

pytestmark = pytest.mark.gpu


def test_fewer_slots_in_a_workspace_of_the_most():
    """200000 tokens of 8 slots take 241 blocks, 65536 tokens 256: the plan is a stable sort by expert
    each time, and nothing behind the workspace is written."""
    G, k = 16, 8
    n = kg.new_route_workspace(200000, k, G, "cuda").numel()
    store = torch.full((n + 256,), 77, dtype=torch.uint8, device="cuda")
    gen = torch.Generator("cuda").manual_seed(1)
    ks = torch.empty(G, dtype=torch.int32, device="cuda")
    for T in (200000, 65536, 65537, 5000, 600, 100):
        idx = torch.randint(0, G, (T, k), generator=gen, device="cuda", dtype=torch.int32)
        pos, src = kg.kg_route(idx, ks, ws=store[:n])
        order = torch.sort(idx.flatten(), stable=True)[1]
        assert torch.equal(src.long(), order)
        assert torch.equal(pos.flatten().long()[order], torch.arange(T * k, device="cuda"))
        assert torch.equal(ks.long(), torch.bincount(idx.flatten(), minlength=G))
    assert (store[n:] == 77).all()
