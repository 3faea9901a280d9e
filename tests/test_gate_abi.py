"""Host-side checks of kg_gate and kg_gate_bwd: bad arguments are refused before anything is
enqueued (no HIP call is made here)."""
import pytest
import torch

import fp8_grouped_gemm_tn_amd as kg
from fp8_grouped_gemm_tn_amd import _binding as B

GB = 1 << 30
FAKE = [(i + 1) * 64 * GB for i in range(12)]  # aligned, far apart, never dereferenced


def gate(X=FAKE[0], ldx=64, bias=FAKE[1], T=100, G=64, k=4, type=B.KG_ROWS_F32, flags=3, scale=1.0,
         coef=1.0, idx=FAKE[2], w=FAKE[3], counts=FAKE[4], psum=FAKE[5], loss=FAKE[6], ws=FAKE[7],
         wb=1 << 20):
    return B.lib().kg_gate(X, ldx, bias, T, G, k, type, flags, scale, coef, idx, w, counts, psum,
                           loss, ws, wb, None)


@pytest.mark.parametrize("kw,code", [
    (dict(type=2), B.KG_ERR_DTYPE),
    (dict(flags=4), B.KG_ERR_DTYPE),
    (dict(T=-1), B.KG_ERR_SHAPE),
    (dict(G=0, ldx=0, k=0), B.KG_ERR_SHAPE),
    (dict(k=0), B.KG_ERR_SHAPE),
    (dict(G=8, k=9), B.KG_ERR_SHAPE),
    (dict(ldx=63), B.KG_ERR_SHAPE),
    (dict(wb=-1), B.KG_ERR_SHAPE),
    (dict(wb=64), B.KG_ERR_SHAPE),
    (dict(G=1025, ldx=1025), B.KG_ERR_UNSUPPORTED),
    (dict(k=17), B.KG_ERR_UNSUPPORTED),
    (dict(T=1 << 30), B.KG_ERR_UNSUPPORTED),
    (dict(ldx=(1 << 30) + 1), B.KG_ERR_UNSUPPORTED),
    (dict(X=None), B.KG_ERR_NULL),
    (dict(idx=None), B.KG_ERR_NULL),
    (dict(w=None), B.KG_ERR_NULL),
    (dict(ws=None), B.KG_ERR_NULL),
    (dict(X=FAKE[0] + 2), B.KG_ERR_ALIGN),
    (dict(X=FAKE[0] + 1, type=B.KG_ROWS_BF16), B.KG_ERR_ALIGN),
    (dict(bias=FAKE[1] + 2), B.KG_ERR_ALIGN),
    (dict(idx=FAKE[2] + 1), B.KG_ERR_ALIGN),
    (dict(w=FAKE[3] + 2), B.KG_ERR_ALIGN),
    (dict(counts=FAKE[4] + 2), B.KG_ERR_ALIGN),
    (dict(psum=FAKE[5] + 2), B.KG_ERR_ALIGN),
    (dict(loss=FAKE[6] + 2), B.KG_ERR_ALIGN),
    (dict(ws=FAKE[7] + 8), B.KG_ERR_ALIGN),
    (dict(w=FAKE[2] + 4 * 399), B.KG_ERR_ALIAS),
    (dict(idx=FAKE[0] + 4 * 6396), B.KG_ERR_ALIAS),
    (dict(counts=FAKE[1]), B.KG_ERR_ALIAS),
    (dict(psum=FAKE[4] + 4 * 63), B.KG_ERR_ALIAS),
    (dict(loss=FAKE[7] + 16), B.KG_ERR_ALIAS),
    (dict(T=0, counts=None, psum=None, loss=None), B.KG_OK),
])
def test_gate_refusals(kw, code):
    assert gate(**kw) == code


def back(X=FAKE[0], ldx=64, idx=FAKE[1], dw=FAKE[2], counts=FAKE[3], dloss=FAKE[4], T=100, G=64,
         k=4, type=B.KG_ROWS_F32, flags=3, scale=1.0, coef=1.0, dX=FAKE[5], ldd=64):
    return B.lib().kg_gate_bwd(X, ldx, idx, dw, counts, dloss, T, G, k, type, flags, scale, coef,
                               dX, ldd, None)


@pytest.mark.parametrize("kw,code", [
    (dict(type=2), B.KG_ERR_DTYPE),
    (dict(flags=8), B.KG_ERR_DTYPE),
    (dict(T=-1), B.KG_ERR_SHAPE),
    (dict(k=65), B.KG_ERR_SHAPE),
    (dict(ldx=63), B.KG_ERR_SHAPE),
    (dict(ldd=63), B.KG_ERR_SHAPE),
    (dict(k=17), B.KG_ERR_UNSUPPORTED),
    (dict(G=2000, ldx=2000, ldd=2000), B.KG_ERR_UNSUPPORTED),
    (dict(X=None), B.KG_ERR_NULL),
    (dict(dX=None), B.KG_ERR_NULL),
    (dict(idx=None), B.KG_ERR_NULL),
    (dict(X=FAKE[0] + 2), B.KG_ERR_ALIGN),
    (dict(dX=FAKE[5] + 2), B.KG_ERR_ALIGN),
    (dict(idx=FAKE[1] + 2), B.KG_ERR_ALIGN),
    (dict(dw=FAKE[2] + 2), B.KG_ERR_ALIGN),
    (dict(counts=FAKE[3] + 2), B.KG_ERR_ALIGN),
    (dict(dloss=FAKE[4] + 2), B.KG_ERR_ALIGN),
    (dict(dX=FAKE[0]), B.KG_ERR_ALIAS),
    (dict(dX=FAKE[2] - 4), B.KG_ERR_ALIAS),
    (dict(counts=FAKE[5] + 4 * 6396), B.KG_ERR_ALIAS),
    (dict(T=0), B.KG_OK),
])
def test_gate_bwd_refusals(kw, code):
    assert back(**kw) == code


def test_workspace_sizes():
    L = B.lib()
    assert L.kg_gate_workspace_bytes(-1, 8) == -1
    assert L.kg_gate_workspace_bytes(8, 0) == -1
    assert L.kg_gate_workspace_bytes(8, 1025) == -1
    assert L.kg_gate_workspace_bytes(1 << 31, 8) == -1
    assert 0 < L.kg_gate_workspace_bytes(0, 1) <= L.kg_gate_workspace_bytes(1 << 20, 1024)


@pytest.mark.parametrize("kw", [
    dict(X=torch.zeros(4, 8, dtype=torch.float16)),
    dict(X=torch.zeros(4, 8, 2)),
    dict(X=torch.zeros(8, 4).t()),
    dict(idx=torch.zeros(4, 2, dtype=torch.int64)),
    dict(idx=torch.zeros(4, 3, dtype=torch.int32)),
    dict(w=torch.zeros(4, 2, dtype=torch.float64)),
    dict(bias=torch.zeros(7)),
    dict(counts=torch.zeros(8)),
    dict(psum=torch.zeros(9)),
    dict(loss=torch.zeros(2)),
    dict(),  # not on a GPU
])
def test_gate_binding_refuses(kw):
    with pytest.raises(ValueError):
        kg.kg_gate(**{"X": torch.zeros(4, 8), "k": 2, **kw})


@pytest.mark.parametrize("kw", [
    dict(X=torch.zeros(5, 8)),
    dict(idx=torch.zeros(4, 2)),
    dict(dw=torch.zeros(4, 3)),
    dict(counts=torch.zeros(8)),
    dict(dloss=torch.zeros(1, dtype=torch.float64)),
    dict(dX=torch.zeros(4, 8, dtype=torch.bfloat16)),
    dict(dX=torch.zeros(4, 9)),
    dict(),
])
def test_gate_bwd_binding_refuses(kw):
    with pytest.raises(ValueError):
        kg.kg_gate_bwd(**{"X": torch.zeros(4, 8), "idx": torch.zeros(4, 2, dtype=torch.int32), **kw})
