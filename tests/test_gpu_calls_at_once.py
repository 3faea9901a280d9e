"""The router, the 4-bit products and the orthogonal updates on two streams at once, each with what it
makes for itself."""
import pytest
import torch

import fp8_grouped_gemm_tn_amd as kg
import test_gpu_fprop_w4 as w4
import test_gpu_gate as gate
import test_gpu_ortho as ortho

pytestmark = pytest.mark.gpu


def at_once(calls, times=8):
    """What `calls` give one by one, and `times` times on a stream each, interleaved."""
    alone = [call(None) for call in calls]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in calls]
    outs = [[call(s) for call, s in zip(calls, streams)] for _ in range(times)]
    torch.cuda.synchronize()
    for turn in outs:
        for got, want in zip(turn, alone):
            assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_two_routers():
    def call(T, G, k, seed):
        x = gate.logits(T, G, seed)

        def run(s):
            idx, w = kg.kg_gate(x, k, None, kg.KG_GATE_NORM, stream=s)
            with torch.cuda.stream(s):
                counts = torch.empty(G, dtype=torch.int32, device="cuda")
                psum, loss = torch.empty(G, device="cuda"), torch.empty(1, device="cuda")
            kg.kg_gate(x, k, None, kg.KG_GATE_NORM, 1.0, 0.5, idx, w, counts, psum, loss, stream=s)
            dx = kg.kg_gate_bwd(x, idx, w, counts, loss, kg.KG_GATE_NORM, 1.0, 0.5, stream=s)
            return idx, w, counts, psum, loss, dx
        return run

    at_once([call(5000, 64, 4, 1), call(700, 256, 8, 2)])


@pytest.mark.parametrize("ms", [[3, 0, 9], [50, 200, 70]], ids=str)
def test_two_products(ms):
    def call(kind, group, seed):
        A, W, sw, zp, m = w4.make(ms, 700, 1024, group, kind, seed)

        def run(s):
            with torch.cuda.stream(s):
                D = torch.empty((sum(ms), 700), device="cuda")
            return kg.kg_fprop_w4(A, W, sw, D, m, zp, stream=s),
        return run

    at_once([call("bf16", 128, 1), call("e2m1", 32, 2)])
    assert kg.kg_status() == kg.KG_OK


def test_two_updates():
    us = [torch.stack([ortho.update(R, C, i) for i in range(G)]) for G, R, C in ((3, 300, 400), (2, 64, 256))]
    at_once([lambda s, u=u: (kg.kg_orthogonalize(u, stream=s),) for u in us])
