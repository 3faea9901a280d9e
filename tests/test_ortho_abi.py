"""Host-side checks of kg_orthogonalize: bad arguments are refused before anything is enqueued (no
HIP call is made here)."""
import pytest
import torch

import fp8_grouped_gemm_tn_amd as kg
from fp8_grouped_gemm_tn_amd import _binding as B

GB = 1 << 30
FAKE = [(i + 1) * 64 * GB for i in range(4)]  # aligned, far apart, never dereferenced


def ortho(U=FAKE[0], O=FAKE[1], G=2, R=100, C=60, type=B.KG_ROWS_F32, steps=5, ws=FAKE[2], wb=1 << 30):
    return B.lib().kg_orthogonalize(U, O, G, R, C, type, steps, ws, wb, None)


def need(G=2, R=100, C=60):
    return B.lib().kg_orthogonalize_workspace_bytes(G, R, C)


@pytest.mark.parametrize("kw,code", [
    (dict(type=2), B.KG_ERR_DTYPE),
    (dict(G=-1), B.KG_ERR_SHAPE),
    (dict(R=-1), B.KG_ERR_SHAPE),
    (dict(C=-1), B.KG_ERR_SHAPE),
    (dict(steps=0), B.KG_ERR_SHAPE),
    (dict(wb=-1), B.KG_ERR_SHAPE),
    (dict(wb=need() - 1), B.KG_ERR_SHAPE),
    (dict(G=65536), B.KG_ERR_UNSUPPORTED),
    (dict(R=65537), B.KG_ERR_UNSUPPORTED),
    (dict(C=65537), B.KG_ERR_UNSUPPORTED),
    (dict(steps=65), B.KG_ERR_UNSUPPORTED),
    (dict(U=None), B.KG_ERR_NULL),
    (dict(O=None), B.KG_ERR_NULL),
    (dict(ws=None), B.KG_ERR_NULL),
    (dict(U=FAKE[0] + 2), B.KG_ERR_ALIGN),
    (dict(U=FAKE[0] + 1, type=B.KG_ROWS_BF16), B.KG_ERR_ALIGN),
    (dict(O=FAKE[1] + 1), B.KG_ERR_ALIGN),
    (dict(ws=FAKE[2] + 128), B.KG_ERR_ALIGN),
    (dict(U=FAKE[2] + need() - 4), B.KG_ERR_ALIAS),
    (dict(O=FAKE[2] - 2), B.KG_ERR_ALIAS),
    (dict(G=0), B.KG_OK),
    (dict(R=0), B.KG_OK),
    (dict(C=0), B.KG_OK),
])
def test_refusals(kw, code):
    assert ortho(**kw) == code


def test_workspace_sizes():
    assert need(-1) == need(1, -1) == need(1, 1, -1) == need(65536) == need(1, 65537) == -1
    assert need(0) == need(1, 0) == need(1, 1, 0) == 0
    assert need(2, 100, 60) == need(2, 60, 100) > 2 * 100 * 60 * 8


@pytest.mark.parametrize("kw", [
    dict(U=torch.zeros(4, 8, dtype=torch.float16)),
    dict(U=torch.zeros(8)),
    dict(U=torch.zeros(2, 2, 2, 2)),
    dict(U=torch.zeros(8, 4).t()),
    dict(O=torch.zeros(4, 8)),
    dict(O=torch.zeros(8, 4, dtype=torch.bfloat16)),
    dict(ws=torch.zeros(8)),
    dict(),  # not on a GPU
])
def test_binding_refuses(kw):
    with pytest.raises(ValueError):
        kg.kg_orthogonalize(**{"U": torch.zeros(4, 8), **kw})
