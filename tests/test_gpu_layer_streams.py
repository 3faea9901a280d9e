"""Calls on a stream of their own while other streams are busy, against the same calls made with
the whole GPU idle: the bits are the same."""
import numpy as np
import pytest
import torch

import fp8_grouped_gemm_tn_amd as kg

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
BF16 = torch.bfloat16


def busy(x, n=6):
    """Work of some milliseconds for the current stream."""
    for _ in range(n):
        x @ x


def test_memory_freed_on_a_busy_current_stream():
    """The current stream still writes to blocks that it has freed when the calls on another
    stream make their outputs and workspaces (sizes of those blocks among them)."""
    T, k, G, H = 3000, 8, 64, 256
    R = T * k
    rng = np.random.default_rng(4)
    idx = torch.from_numpy(rng.integers(0, G, (T, k)).astype(np.int32)).to(DEV)
    X = torch.randn((T, H), device=DEV).to(BF16)
    w = torch.rand((T, k), device=DEV)
    ks = torch.empty(G, dtype=torch.int32, device=DEV)

    def all_calls(stream):
        pos, src = kg.kg_route(idx, ks, stream=stream)
        Xp = kg.kg_dispatch(X, pos, stream=stream)
        Q, sa = kg.kg_dispatch_fp8(X, pos, stream=stream)
        out = kg.kg_combine(Xp, pos, w, stream=stream)
        dY, dw = kg.kg_combine_bwd(X, Xp, pos, w, stream=stream)
        return pos, src, Xp, Q, sa, out, dY, dw

    want = all_calls(None)
    sizes = [t.numel() * t.element_size() for t in want]
    sizes.append(kg.layer.lib().kg_route_workspace_bytes(T, k, G))
    x = torch.randn((4096, 4096), device=DEV)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(3):
        busy(x)
        for n in sizes:  # freed at once, written when the work before it is done
            torch.full((n,), 0x5A, dtype=torch.uint8, device=DEV)
        got = all_calls(side)
        torch.cuda.synchronize()
        for a, b in zip(got, want):
            assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))
        del got


def test_what_is_handed_back_outlives_the_current_streams_use():
    """A tensor made for another stream and freed while the current stream has yet to read it:
    that stream's next tensors do not take its memory."""
    T, k, G, H = 2000, 4, 16, 512
    rng = np.random.default_rng(5)
    idx = torch.from_numpy(rng.integers(0, G, (T, k)).astype(np.int32)).to(DEV)
    X = torch.randn((T, H), device=DEV).to(BF16)
    pos, src = kg.kg_route(idx, torch.empty(G, dtype=torch.int32, device=DEV))
    want = kg.kg_dispatch(X, pos)
    x = torch.randn((4096, 4096), device=DEV)
    side, here = torch.cuda.Stream(), torch.cuda.current_stream()
    torch.cuda.synchronize()
    for _ in range(3):
        Xp = kg.kg_dispatch(X, pos, stream=side)
        here.wait_stream(side)
        busy(x)
        kept = Xp.clone()
        del Xp
        with torch.cuda.stream(side):
            for _ in range(20):
                torch.zeros((T * k, H), dtype=BF16, device=DEV)
        torch.cuda.synchronize()
        assert torch.equal(kept, want)


@pytest.mark.parametrize("packed", [False, True])
def test_a_table_dropped_behind_a_step_on_another_stream(packed):
    """The step waits behind other work when its table goes, with the gradients that only the
    table kept; the current stream then fills the memory that is free."""
    g = torch.Generator(DEV).manual_seed(7)
    sizes = [5000, 130, 70000]
    rnd = lambda n: torch.randn(n, generator=g, device=DEV)
    x = torch.randn((4096, 4096), device=DEV)
    side = torch.cuda.Stream()
    for _ in range(3):
        p, g0 = [rnd(n) for n in sizes], [rnd(n) * 1e-3 for n in sizes]
        state = (lambda: [torch.zeros(n, dtype=torch.uint8, device=DEV) for n in sizes]) if packed else \
            (lambda: [torch.zeros(n, device=DEV) for n in sizes])
        scales = lambda: [torch.zeros(-(-n // 128), device=DEV) for n in sizes]
        more = lambda: [scales(), scales()] if packed else []
        want = [t.clone() for t in p]
        kg.kg_adamw(kg.AdamWTable(want, g0, state(), state(), *more()), 1e-3)
        torch.cuda.synchronize()
        table = kg.AdamWTable(p, [t.clone() for t in g0], state(), state(), *more())
        torch.cuda.synchronize()
        with torch.cuda.stream(side):
            busy(x)
        kg.kg_adamw(table, 1e-3, stream=side)
        del table
        for n in [256, 1024, 2048] + [4 * n for n in sizes] + sizes:
            for _ in range(8):  # (were it reused: pointers and lengths of zeros)
                torch.zeros(n, dtype=torch.uint8, device=DEV)
        torch.cuda.synchronize()
        for a, b in zip(p, want):
            assert torch.equal(a, b)
