"""Host-side checks of the expert layer's operators (kg_route, kg_dispatch, kg_dispatch_fp8,
kg_combine, kg_combine_bwd, kg_fprop, kg_adamw): bad arguments are refused before anything is
enqueued (no HIP call is made here), and the host-built AdamW table."""
import ctypes

import numpy as np
import pytest
import torch

import fp8_grouped_gemm_tn_amd as kg
from fp8_grouped_gemm_tn_amd import _binding as B
from fp8_grouped_gemm_tn_amd.layer import AdamWTensor

GB = 1 << 30
FAKE = [(i + 1) * 64 * GB for i in range(12)]  # aligned, far apart, never dereferenced


def fprop(A=FAKE[0], lda=256, sa=FAKE[1], W=FAKE[2], sw=FAKE[3], D=FAKE[4], ldd=64, ms=FAKE[5],
          G=3, N=64, K=256, M=100, flags=0):
    return B.lib().kg_fprop(A, lda, sa, W, sw, D, ldd, ms, G, N, K, M, flags, None)


@pytest.mark.parametrize("kw,code", [
    (dict(flags=0x400), B.KG_ERR_DTYPE),
    (dict(G=-1), B.KG_ERR_SHAPE),
    (dict(M=-1), B.KG_ERR_SHAPE),
    (dict(lda=240), B.KG_ERR_SHAPE),
    (dict(ldd=63), B.KG_ERR_SHAPE),
    (dict(G=1025), B.KG_ERR_UNSUPPORTED),
    (dict(K=1 << 24, lda=1 << 24), B.KG_ERR_UNSUPPORTED),
    (dict(lda=(1 << 23) + 16), B.KG_ERR_UNSUPPORTED),
    (dict(K=250), B.KG_ERR_ALIGN),
    (dict(lda=264), B.KG_ERR_ALIGN),
    (dict(A=None), B.KG_ERR_NULL),
    (dict(sa=None), B.KG_ERR_NULL),
    (dict(W=None), B.KG_ERR_NULL),
    (dict(sw=None), B.KG_ERR_NULL),
    (dict(D=None), B.KG_ERR_NULL),
    (dict(ms=None), B.KG_ERR_NULL),
    (dict(A=FAKE[0] + 8), B.KG_ERR_ALIGN),
    (dict(W=FAKE[2] + 4), B.KG_ERR_ALIGN),
    (dict(sa=FAKE[1] + 2), B.KG_ERR_ALIGN),
    (dict(D=FAKE[4] + 2), B.KG_ERR_ALIGN),
    (dict(D=FAKE[4] + 1, flags=kg.KG_FLAG_D_BF16), B.KG_ERR_ALIGN),
    (dict(D=FAKE[0] + 16), B.KG_ERR_ALIAS),
    (dict(D=FAKE[2] + 3 * 64 * 256 - 16), B.KG_ERR_ALIAS),
    (dict(D=FAKE[1]), B.KG_ERR_ALIAS),
    (dict(D=FAKE[3]), B.KG_ERR_ALIAS),
    (dict(ms=FAKE[4] + 4 * 64 * 99), B.KG_ERR_ALIAS),
    (dict(G=0), B.KG_OK),
    (dict(N=0), B.KG_OK),
    (dict(M=0), B.KG_OK),
])
def test_fprop_refusals(kw, code):
    assert fprop(**kw) == code


def route(idx=FAKE[0], T=10, k=4, G=8, ks=FAKE[1], pos=FAKE[2], src=FAKE[3], ws=None, wb=0):
    return B.lib().kg_route(idx, T, k, G, ks, pos, src, ws, wb, None)


@pytest.mark.parametrize("kw,code", [
    (dict(T=-1), B.KG_ERR_SHAPE),
    (dict(k=-1), B.KG_ERR_SHAPE),
    (dict(G=-1), B.KG_ERR_SHAPE),
    (dict(wb=-1), B.KG_ERR_SHAPE),
    (dict(G=1025), B.KG_ERR_UNSUPPORTED),
    (dict(k=4097), B.KG_ERR_UNSUPPORTED),
    (dict(T=1 << 30, k=2), B.KG_ERR_UNSUPPORTED),
    (dict(idx=None), B.KG_ERR_NULL),
    (dict(ks=None), B.KG_ERR_NULL),
    (dict(pos=None), B.KG_ERR_NULL),
    (dict(T=100000), B.KG_ERR_NULL),                       # needs a workspace
    (dict(T=100000, ws=FAKE[4], wb=64), B.KG_ERR_SHAPE),   # ... a larger one
    (dict(idx=FAKE[0] + 2), B.KG_ERR_ALIGN),
    (dict(pos=FAKE[0] + 4 * 39), B.KG_ERR_ALIAS),
    (dict(src=FAKE[2] + 4), B.KG_ERR_ALIAS),
    (dict(ks=FAKE[2]), B.KG_ERR_ALIAS),
    (dict(T=0, G=0), B.KG_OK),
])
def test_route_refusals(kw, code):
    assert route(**kw) == code


def test_route_workspace_sizes():
    need = B.lib().kg_route_workspace_bytes
    assert need(8, 8, 256) == 0
    assert need(-1, 8, 256) == need(8, 8, 1025) == need(1 << 30, 2, 8) == -1
    assert 0 < need(16384, 8, 256) < need(1 << 20, 8, 256)


def test_fp8_workspace_sizes():
    need = B.lib().kg_dispatch_fp8_workspace_bytes
    assert need(8, 8, 7168) == 0
    assert need(-1, 8, 128) == need(8, 5000, 128) == -1
    assert need(8192, 8, 7168) == 8192 * 56 * 4 + 65536 * 4
    assert need(1024, 8, 7168) == 0
    assert need(131072, 8, 144) == 131072 * 4 * 4 + 1048576 * 4


def rows(fn, X=FAKE[0], ld=32, pos=FAKE[1], T=10, k=4, H=32, ty=0, out=FAKE[2], w=FAKE[3],
         sa=FAKE[4], dw=FAKE[5], Y=FAKE[6], ws=None, wb=0):
    L = B.lib()
    if fn == "dispatch":
        return L.kg_dispatch(X, ld, pos, T, k, H, ty, out, None)
    if fn == "dispatch_fp8":
        return L.kg_dispatch_fp8(X, ld, pos, T, k, H, out, sa, ws, wb, None)
    if fn == "combine":
        return L.kg_combine(X, pos, w, out, ld, T, k, H, ty, None)
    return L.kg_combine_bwd(X, ld, Y, pos, w, out, dw, T, k, H, ty, None)


ALL = ("dispatch", "dispatch_fp8", "combine", "combine_bwd")


@pytest.mark.parametrize("fn", ALL)
@pytest.mark.parametrize("kw,code", [
    (dict(T=-1), B.KG_ERR_SHAPE),
    (dict(k=-1), B.KG_ERR_SHAPE),
    (dict(H=-16), B.KG_ERR_SHAPE),
    (dict(ld=31), B.KG_ERR_SHAPE),
    (dict(H=1 << 25, ld=1 << 25), B.KG_ERR_UNSUPPORTED),
    (dict(T=1 << 30, k=2), B.KG_ERR_UNSUPPORTED),
    (dict(k=5000), B.KG_ERR_UNSUPPORTED),
    (dict(X=None), B.KG_ERR_NULL),
    (dict(pos=None), B.KG_ERR_NULL),
    (dict(out=None), B.KG_ERR_NULL),
    (dict(X=FAKE[0] + 1), B.KG_ERR_ALIGN),
    (dict(pos=FAKE[1] + 2), B.KG_ERR_ALIGN),
    (dict(out=FAKE[0] + 32), B.KG_ERR_ALIAS),
    (dict(out=FAKE[1] + 32), B.KG_ERR_ALIAS),
    (dict(T=0), B.KG_OK),
    (dict(H=0), B.KG_OK),
])
def test_row_refusals(fn, kw, code):
    if fn == "combine_bwd" and kw == dict(H=0):
        kw = dict(H=0, T=0)  # (with tokens it writes zeros to dw)
    assert rows(fn, **kw) == code


@pytest.mark.parametrize("fn,kw,code", [
    ("dispatch", dict(ty=2), B.KG_ERR_DTYPE),
    ("combine", dict(ty=-1), B.KG_ERR_DTYPE),
    ("combine_bwd", dict(ty=7), B.KG_ERR_DTYPE),
    ("dispatch", dict(ty=1, X=FAKE[0] + 2), B.KG_ERR_ALIGN),
    ("dispatch_fp8", dict(H=24), B.KG_ERR_ALIGN),
    ("dispatch_fp8", dict(sa=None), B.KG_ERR_NULL),
    ("dispatch_fp8", dict(sa=FAKE[2] + 4), B.KG_ERR_ALIAS),
    ("dispatch_fp8", dict(sa=FAKE[1]), B.KG_ERR_ALIAS),
    ("dispatch_fp8", dict(wb=-1), B.KG_ERR_SHAPE),
    ("dispatch_fp8", dict(T=1000000, ws=FAKE[7] + 8, wb=1 << 26), B.KG_ERR_ALIGN),
    ("dispatch_fp8", dict(T=1000000, ws=FAKE[2] + 64, wb=1 << 26), B.KG_ERR_ALIAS),
    ("dispatch_fp8", dict(T=1000000, ws=FAKE[0], wb=1 << 26), B.KG_ERR_ALIAS),
    ("combine", dict(w=FAKE[3] + 2), B.KG_ERR_ALIGN),
    ("combine", dict(w=FAKE[2]), B.KG_ERR_ALIAS),
    ("combine_bwd", dict(Y=None), B.KG_ERR_NULL),
    ("combine_bwd", dict(dw=FAKE[3]), B.KG_ERR_ALIAS),
    ("combine_bwd", dict(dw=FAKE[2]), B.KG_ERR_ALIAS),
    ("combine_bwd", dict(out=FAKE[6]), B.KG_ERR_ALIAS),
])
def test_row_refusals_of_one(fn, kw, code):
    assert rows(fn, **kw) == code


def table(ts, kinds=0, room=None):
    """Packs tensors given as dicts; returns (code, image, items)."""
    arr = (AdamWTensor * max(1, len(ts)))(*[AdamWTensor(**t) for t in ts])
    L = B.lib()
    size = L.kg_adamw_table_bytes(arr, len(ts))
    img = np.zeros(max(size, 8) if room is None else max(room, 1), np.uint8)
    rc = L.kg_adamw_pack(arr, len(ts), kinds, img.ctypes.data, size if room is None else room)
    return rc, img, L.kg_adamw_items(arr, len(ts))


def one(n=1000, at=0, **kw):
    t = dict(p=FAKE[0] + at, g=FAKE[1] + at, m=FAKE[2] + at, v=FAKE[3] + at, m_scale=FAKE[4] + at,
             v_scale=FAKE[5] + at, copy=FAKE[6] + at, n=n)
    t.update(kw)
    return t


def test_adamw_table_layout():
    sizes = [1, 2048, 0, 2049, 10000]
    at, ts = 0, []
    for n in sizes:
        ts.append(one(n, at))
        at += 4 * n
    rc, img, items = table(ts)
    assert rc == B.KG_OK
    per = [-(-n // 2048) for n in sizes]
    assert items == sum(per)
    desc = np.frombuffer(img[:72 * 5].tobytes(), np.int64).reshape(5, 9)
    assert desc[:, 7].tolist() == sizes
    assert desc[:, 8].tolist() == [0] + np.cumsum(per)[:-1].tolist()
    owner = np.frombuffer(img[72 * 5:].tobytes(), np.int32)
    assert owner.tolist() == [i for i, c in enumerate(per) for _ in range(c)]


@pytest.mark.parametrize("ts,kinds,code", [
    ([one()], 8, B.KG_ERR_DTYPE),
    ([one(p=None)], 0, B.KG_ERR_NULL),
    ([one(g=None)], 0, B.KG_ERR_NULL),
    ([one(m=None)], 0, B.KG_ERR_NULL),
    ([one(v=None)], 4, B.KG_ERR_NULL),
    ([one(m_scale=None)], 4, B.KG_ERR_NULL),
    ([one(m_scale=None, v_scale=None, copy=None)], 0, B.KG_OK),
    ([one(p=FAKE[0] + 2)], 0, B.KG_ERR_ALIGN),
    ([one(p=FAKE[0] + 2)], 1, B.KG_OK),
    ([one(g=FAKE[1] + 1)], 2, B.KG_ERR_ALIGN),
    ([one(m=FAKE[2] + 1)], 0, B.KG_ERR_ALIGN),
    ([one(m=FAKE[2] + 1)], 4, B.KG_OK),
    ([one(v_scale=FAKE[5] + 2)], 4, B.KG_ERR_ALIGN),
    ([one(copy=FAKE[6] + 1)], 0, B.KG_ERR_ALIGN),
    ([one(n=-1)], 0, B.KG_ERR_SHAPE),
    ([one(m=FAKE[0] + 3996)], 0, B.KG_ERR_ALIAS),            # m starts in p's last element
    ([one(m=FAKE[0] + 4000)], 0, B.KG_OK),
    ([one(g=FAKE[0])], 0, B.KG_ERR_ALIAS),                   # a gradient in the parameter
    ([one(), one(at=4000, g=FAKE[1])], 0, B.KG_OK),          # two tensors, one gradient
    ([one(), one(at=3996)], 0, B.KG_ERR_ALIAS),              # neighbours that overlap
    ([one(copy=FAKE[1])], 0, B.KG_ERR_ALIAS),
])
def test_adamw_table_refusals(ts, kinds, code):
    assert table(ts, kinds)[0] == code


def test_adamw_table_too_small_and_too_large():
    assert table([one()], room=8)[0] == B.KG_ERR_SHAPE
    assert table([one(n=1 << 45)], room=8)[0] == B.KG_ERR_UNSUPPORTED
    assert table([])[0] == B.KG_OK


def adamw(tab=FAKE[0], count=1, items=1, kinds=0, lr=1e-3, b1=0.9, b2=0.99, eps=1e-8, wd=0.1,
          step=1, gscale=None, dyn=None):
    return B.lib().kg_adamw(tab, count, items, kinds, lr, b1, b2, eps, wd, step, gscale, dyn, None)


@pytest.mark.parametrize("kw,code", [
    (dict(kinds=16), B.KG_ERR_DTYPE),
    (dict(count=-1), B.KG_ERR_SHAPE),
    (dict(items=-1), B.KG_ERR_SHAPE),
    (dict(step=0), B.KG_ERR_SHAPE),
    (dict(b1=1.0), B.KG_ERR_SHAPE),
    (dict(b2=-0.1), B.KG_ERR_SHAPE),
    (dict(b2=float("nan")), B.KG_ERR_SHAPE),
    (dict(lr=-1.0), B.KG_ERR_SHAPE),
    (dict(lr=float("nan")), B.KG_ERR_SHAPE),
    (dict(eps=-1.0), B.KG_ERR_SHAPE),
    (dict(wd=-1.0), B.KG_ERR_SHAPE),
    (dict(tab=None), B.KG_ERR_NULL),
    (dict(tab=FAKE[0] + 4), B.KG_ERR_ALIGN),
    (dict(gscale=FAKE[1] + 2), B.KG_ERR_ALIGN),
    (dict(dyn=FAKE[1] + 1), B.KG_ERR_ALIGN),
    (dict(items=1 << 31), B.KG_ERR_UNSUPPORTED),
    (dict(items=1 << 24), B.KG_ERR_UNSUPPORTED),
    (dict(count=0, items=0, tab=None), B.KG_OK),
    (dict(items=0), B.KG_OK),
])
def test_adamw_refusals(kw, code):
    assert adamw(**kw) == code


def test_python_shape_checks():
    z = torch.zeros
    i32 = torch.int32
    f8 = torch.uint8
    bad = [
        lambda: kg.kg_route(z(4, 2), z(3, dtype=i32)),
        lambda: kg.kg_route(z(8, dtype=i32), z(3, dtype=i32)),
        lambda: kg.kg_route(z(4, 2, dtype=i32), z(3, dtype=torch.int64)),
        lambda: kg.kg_route(z(4, 2, dtype=i32), z(3, dtype=i32), src=z(7, dtype=i32)),
        lambda: kg.kg_dispatch(z(4, 8, dtype=torch.float16), z(4, 2, dtype=i32)),
        lambda: kg.kg_dispatch(z(4, 8), z(5, 2, dtype=i32)),
        lambda: kg.kg_dispatch(z(8, 4).t(), z(4, 2, dtype=i32)),
        lambda: kg.kg_dispatch(z(4, 8), z(4, 2, dtype=i32), z(8, 9)),
        lambda: kg.kg_dispatch_fp8(z(4, 16), z(4, 2, dtype=i32)),
        lambda: kg.kg_combine(z(7, 8), z(4, 2, dtype=i32)),
        lambda: kg.kg_combine(z(8, 8), z(4, 2, dtype=i32), z(4, 3)),
        lambda: kg.kg_combine(z(8, 8), z(4, 2, dtype=i32), out=z(4, 8, dtype=torch.bfloat16)),
        lambda: kg.kg_combine_bwd(z(4, 8), None, z(4, 2, dtype=i32)),
        lambda: kg.kg_combine_bwd(z(4, 8), z(8, 9), z(4, 2, dtype=i32)),
        lambda: kg.kg_fprop(z(4, 32, dtype=f8), z(1, 4), z(2, 8, 16, dtype=f8), z(2, 1, 1), z(4, 8),
                            z(2, dtype=i32)),
        lambda: kg.kg_fprop(z(4, 32, dtype=f8), z(4, 1), z(2, 8, 32, dtype=f8), z(2, 1, 1), z(4, 8),
                            z(2, dtype=i32)),
        lambda: kg.kg_fprop(z(4, 32, dtype=f8), z(1, 4), z(2, 8, 32, dtype=f8), z(2, 1, 1), z(4, 9),
                            z(2, dtype=i32)),
        lambda: kg.AdamWTable([z(4)], [z(4)], [z(4)], [z(4)], [z(1)], None),
        lambda: kg.AdamWTable([z(4)], [], [z(4)], [z(4)]),
    ]
    for i, call in enumerate(bad):
        with pytest.raises(ValueError):
            call()
            pytest.fail(f"call {i} was accepted")
    # shapes right, but not on a GPU
    for call in (lambda: kg.kg_route(z(4, 2, dtype=i32), z(3, dtype=i32)),
                 lambda: kg.kg_dispatch(z(4, 8), z(4, 2, dtype=i32)),
                 lambda: kg.AdamWTable([z(4)], [z(4)], [z(4)], [z(4)])):
        with pytest.raises(ValueError, match="GPU"):
            call()
