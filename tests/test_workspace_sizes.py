"""A workspace made for the largest call is enough for the smaller ones."""
import pytest

from fp8_grouped_gemm_tn_amd import _binding as B


def test_gate_workspaces_grow_with_tokens_and_experts():
    L = B.lib()
    tokens = [0, 1, 7, 8, 9, 31, 32, 33, 500, 512, 1000, 1023, 1024, 1025, 1026, 2000, 4095, 4096, 4097, 16384,
              16385, 20000, 100000, 1 << 24]
    experts = [1, 2, 8, 63, 64, 65, 128, 255, 256, 257, 300, 512, 513, 1024]
    size = {(T, G): L.kg_gate_workspace_bytes(T, G) for T in tokens for G in experts}
    for i, T in enumerate(tokens):
        for j, G in enumerate(experts):
            assert size[T, G] > 0
            assert i == 0 or size[tokens[i - 1], G] <= size[T, G], (T, G)
            assert j == 0 or size[T, experts[j - 1]] <= size[T, G], (T, G)
    for G in (65, 200, 256, 257):
        assert all(L.kg_gate_workspace_bytes(T, G) <= L.kg_gate_workspace_bytes(T + 1, G)
                   for T in range(0, 6000))


@pytest.mark.parametrize("sizes", [[0, 1, 63, 64, 65, 2047, 2048, 2049, 2112, 4096, 4100, 16384, 65536]])
def test_orthogonalize_workspaces_grow(sizes):
    L = B.lib()
    for G in (1, 2, 40):
        for R in sizes:
            row = [L.kg_orthogonalize_workspace_bytes(G, R, C) for C in sizes]
            assert row == sorted(row) and row[0] == 0
            assert all(a <= L.kg_orthogonalize_workspace_bytes(G + 1, R, C) for a, C in zip(row, sizes))
            assert row == [L.kg_orthogonalize_workspace_bytes(G, C, R) for C in sizes]


def test_route_workspaces_grow():
    L = B.lib()
    for G in (1, 8, 256, 1024):
        for k in (1, 8):
            row = [L.kg_route_workspace_bytes(T, k, G) for T in (0, 1, 100, 2000, 4096, 5000, 65536, 200000)]
            assert row == sorted(row)
    row = [L.kg_route_workspace_bytes(n, 1, 16) for n in range(4000, 1100000, 97)]
    assert row == sorted(row)
