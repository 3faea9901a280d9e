"""Bindings of the operators around an expert layer's products (the C ABI in
include/kgwgrad.h): the sort of tokens by expert and the row copies (kg_route, kg_dispatch,
kg_dispatch_fp8, kg_combine, kg_combine_bwd), the forward product (kg_fprop) and the AdamW
step (AdamWTable, kg_adamw).

Argument marshalling only, as in _binding. A small call costs about as much here as on the
GPU, so the checks read each property of a tensor once.
"""
import ctypes

from ._binding import (KG_ADAMW_8BIT, KG_ADAMW_G_BF16, KG_ADAMW_P_BF16, KG_ERR_SHAPE,
                       KG_FLAG_D_BF16, KG_OK, KG_ROWS_BF16, KG_ROWS_F32, KgError, _need, lib)


def _on(stream):
    import torch
    return (torch.cuda.current_stream() if stream is None else stream).cuda_stream


def _check(rc, what):
    if rc != KG_OK:
        raise KgError(rc, what)


def _at(t):
    return None if t is None else t.data_ptr()


def _gpu(ref, **named):
    """Every given tensor is on `ref`'s GPU."""
    _need(ref.is_cuda, "the tensors must be on a GPU")
    for name, t in named.items():
        if t is not None and t.device != ref.device:
            raise ValueError(f"{name} is on {t.device}, not on {ref.device}")


def _i32(t, shape, name):
    import torch
    _need(t.dtype == torch.int32 and t.shape == shape and t.is_contiguous(),
          f"{name} must be a contiguous int32 {list(shape)} tensor")


def _row_type(t, name):
    import torch
    if t.dtype == torch.bfloat16:
        return KG_ROWS_BF16
    _need(t.dtype == torch.float32, f"{name} must be bfloat16 or float32")
    return KG_ROWS_F32


def _row_stride(t, name):
    """Row stride in elements of a 2-D tensor whose rows are contiguous (its width where it
    has at most one row, or no columns: torch gives those any stride)."""
    _need(t.dim() == 2 and (t.stride(1) == 1 or t.shape[1] <= 1),
          f"{name} must be 2-D with contiguous rows")
    return t.stride(0) if t.shape[0] > 1 and t.shape[1] > 0 else t.shape[1]


def new_route_workspace(T, k, G, device):
    """The workspace of kg_route for T tokens of k slots and G experts (None where it needs
    none); keep it for later calls of at most these sizes."""
    import torch
    n = lib().kg_route_workspace_bytes(T, k, G)
    if n < 0:
        raise KgError(KG_ERR_SHAPE, "kg_route_workspace_bytes")
    return torch.empty(n, dtype=torch.uint8, device=device) if n else None


def kg_route(idx, ks, pos=None, src=None, ws=None, stream=None):
    """Plan that puts tokens into expert order: idx int32 [T, k] (an entry outside [0, G) is
    dropped), ks int32 [G] (out). pos int32 [T, k] and src int32 [T * k] are written (made if
    not given); ws: new_route_workspace (made if not given and needed). Returns (pos, src)."""
    import torch
    _need(idx.dim() == 2, "idx must be [T, k]")
    T, k = idx.shape
    _i32(idx, idx.shape, "idx")
    _need(ks.dim() == 1, "ks must be [G]")
    _i32(ks, ks.shape, "ks")
    G = ks.shape[0]
    if pos is None:
        pos = torch.empty_like(idx)
    if src is None:
        src = torch.empty(T * k, dtype=torch.int32, device=idx.device)
    _i32(pos, idx.shape, "pos")
    _i32(src, (T * k,), "src")
    L = lib()
    if ws is None and L.kg_route_workspace_bytes(T, k, G) > 0:
        ws = new_route_workspace(T, k, G, idx.device)
    if ws is not None:
        _need(ws.dtype == torch.uint8 and ws.is_contiguous(), "ws must be contiguous uint8")
    _gpu(idx, ks=ks, pos=pos, src=src, ws=ws)
    _check(L.kg_route(idx.data_ptr(), T, k, G, ks.data_ptr(), pos.data_ptr(), src.data_ptr(),
                      _at(ws), 0 if ws is None else ws.numel(), _on(stream)), "kg_route")
    return pos, src


def kg_dispatch(X, pos, Xp=None, stream=None):
    """X [T, H] (bfloat16 or float32, rows contiguous) copied to Xp [T * k, H] (made if not
    given): every token's row to the rows that pos (kg_route) names, zeros for dropped slots."""
    import torch
    ty, ldx = _row_type(X, "X"), _row_stride(X, "X")
    T, H = X.shape
    _need(pos.dim() == 2 and pos.shape[0] == T, "pos must be [T, k]")
    k = pos.shape[1]
    _i32(pos, pos.shape, "pos")
    if Xp is None:
        Xp = torch.empty((T * k, H), dtype=X.dtype, device=X.device)
    _need(Xp.dtype == X.dtype and Xp.shape == (T * k, H) and Xp.is_contiguous(),
          "Xp must be a contiguous [T * k, H] tensor of X's dtype")
    _gpu(X, pos=pos, Xp=Xp)
    _check(lib().kg_dispatch(X.data_ptr(), ldx, pos.data_ptr(), T, k, H, ty, Xp.data_ptr(),
                             _on(stream)), "kg_dispatch")
    return Xp


def kg_dispatch_fp8(X, pos, Q=None, sa=None, stream=None):
    """kg_dispatch as e4m3 codes: X bfloat16 [T, H], H a multiple of 16; Q 1-byte [T * k, H] and
    sa float32 [ceil(H / 128), T * k] as kg_fprop and kg_dgrad read them (made if not given).
    Returns (Q, sa)."""
    import torch
    _need(X.dtype == torch.bfloat16, "X must be bfloat16")
    ldx = _row_stride(X, "X")
    T, H = X.shape
    _need(pos.dim() == 2 and pos.shape[0] == T, "pos must be [T, k]")
    k = pos.shape[1]
    _i32(pos, pos.shape, "pos")
    if Q is None:
        Q = torch.empty((T * k, H), dtype=torch.uint8, device=X.device)
    if sa is None:
        sa = torch.empty((-(-H // 128), T * k), device=X.device)
    _need(Q.element_size() == 1 and Q.shape == (T * k, H) and Q.is_contiguous(),
          "Q must be a contiguous 1-byte [T * k, H] tensor")
    _need(sa.dtype == torch.float32 and sa.shape == (-(-H // 128), T * k) and sa.is_contiguous(),
          "sa must be a contiguous float32 [ceil(H / 128), T * k] tensor")
    _gpu(X, pos=pos, Q=Q, sa=sa)
    _check(lib().kg_dispatch_fp8(X.data_ptr(), ldx, pos.data_ptr(), T, k, H, Q.data_ptr(),
                                 sa.data_ptr(), _on(stream)), "kg_dispatch_fp8")
    return Q, sa


def _rows_of(Y, pos, name):
    T, k = pos.shape
    _need(Y.dim() == 2 and Y.shape[0] == T * k and Y.is_contiguous(),
          f"{name} must be a contiguous [T * k, H] tensor")
    return Y.shape[1]


def _weights(w, pos, name):
    import torch
    _need(w.dtype == torch.float32 and w.shape == pos.shape and w.is_contiguous(),
          f"{name} must be a contiguous float32 [T, k] tensor")


def kg_combine(Y, pos, w=None, out=None, stream=None):
    """out[t] = sum_j w[t][j] Y[pos[t][j]] over the kept slots: Y [T * k, H] (bfloat16 or
    float32), pos int32 [T, k] from kg_route, w float32 [T, k] (None: ones), out [T, H] (rows
    contiguous; made if not given). With w None this is kg_dispatch's gradient."""
    import torch
    ty = _row_type(Y, "Y")
    _need(pos.dim() == 2, "pos must be [T, k]")
    _i32(pos, pos.shape, "pos")
    T, k = pos.shape
    H = _rows_of(Y, pos, "Y")
    if w is not None:
        _weights(w, pos, "w")
    if out is None:
        out = torch.empty((T, H), dtype=Y.dtype, device=Y.device)
    _need(out.dtype == Y.dtype and out.shape == (T, H), "out must be [T, H] of Y's dtype")
    ldo = _row_stride(out, "out")
    _gpu(Y, pos=pos, w=w, out=out)
    _check(lib().kg_combine(Y.data_ptr(), pos.data_ptr(), _at(w), out.data_ptr(), ldo, T, k, H, ty,
                            _on(stream)), "kg_combine")
    return out


def kg_combine_bwd(dOut, Y, pos, w=None, dY=None, dw=None, need_dw=True, stream=None):
    """Gradients of kg_combine: dOut [T, H] (rows contiguous), Y [T * k, H], pos, w as given to
    it. Returns (dY [T * k, H], dw float32 [T, k]); with need_dw False dw is not computed (None)
    and Y is not read (it may be None)."""
    import torch
    ty, ldo = _row_type(dOut, "dOut"), _row_stride(dOut, "dOut")
    _need(pos.dim() == 2 and pos.shape[0] == dOut.shape[0], "pos must be [T, k]")
    _i32(pos, pos.shape, "pos")
    T, k = pos.shape
    H = dOut.shape[1]
    if w is not None:
        _weights(w, pos, "w")
    if dY is None:
        dY = torch.empty((T * k, H), dtype=dOut.dtype, device=dOut.device)
    _need(dY.dtype == dOut.dtype and dY.shape == (T * k, H) and dY.is_contiguous(),
          "dY must be a contiguous [T * k, H] tensor of dOut's dtype")
    if need_dw:
        _need(Y is not None and Y.dtype == dOut.dtype and _rows_of(Y, pos, "Y") == H,
              "Y must be a contiguous [T * k, H] tensor of dOut's dtype")
        if dw is None:
            dw = torch.empty((T, k), device=dOut.device)
        _weights(dw, pos, "dw")
    else:
        Y = dw = None
    _gpu(dOut, Y=Y, pos=pos, w=w, dY=dY, dw=dw)
    _check(lib().kg_combine_bwd(dOut.data_ptr(), ldo, _at(Y), pos.data_ptr(), _at(w),
                                dY.data_ptr(), _at(dw), T, k, H, ty, _on(stream)),
           "kg_combine_bwd")
    return dY, dw


def kg_fprop(A, sa, W, sw, D, ms, flags=0, stream=None):
    """D = rows . W^T per expert: A fp8 codes [M_total, K] (rows contiguous), sa float32
    [ceil(K / 128), M_total], W fp8 codes [G, N, K], sw float32 [G, ceil(N / 128),
    ceil(K / 128)], ms int32 [G], D [M_total, N] (float32 or bfloat16, rows contiguous)."""
    import torch
    _need(W.dim() == 3 and W.element_size() == 1 and W.is_contiguous(),
          "W must be contiguous fp8 codes [G, N, K]")
    G, N, K = W.shape
    lda = _row_stride(A, "A")
    M, nk = A.shape[0], -(-K // 128)
    _need(A.shape[1] == K and A.element_size() == 1, "A must be fp8 codes [M_total, K]")
    _need(sa.dtype == torch.float32 and sa.shape == (nk, M) and sa.is_contiguous(),
          "sa must be contiguous float32 [ceil(K / 128), M_total]")
    _need(sw.dtype == torch.float32 and sw.shape == (G, -(-N // 128), nk) and sw.is_contiguous(),
          "sw must be contiguous float32 [G, ceil(N / 128), ceil(K / 128)]")
    _i32(ms, (G,), "ms")
    ldd = _row_stride(D, "D")
    _need(D.shape == (M, N) and D.dtype in (torch.float32, torch.bfloat16),
          "D must be a float32 or bfloat16 [M_total, N] tensor")
    _gpu(D, A=A, sa=sa, W=W, sw=sw, ms=ms)
    if D.dtype == torch.bfloat16:
        flags |= KG_FLAG_D_BF16
    _check(lib().kg_fprop(A.data_ptr(), lda, sa.data_ptr(), W.data_ptr(), sw.data_ptr(),
                          D.data_ptr(), ldd, ms.data_ptr(), G, N, K, M, flags, _on(stream)),
           "kg_fprop")
    return D


class AdamWTensor(ctypes.Structure):
    """kg_adamw_tensor."""
    _fields_ = [("p", ctypes.c_void_p), ("g", ctypes.c_void_p), ("m", ctypes.c_void_p),
                ("v", ctypes.c_void_p), ("m_scale", ctypes.c_void_p),
                ("v_scale", ctypes.c_void_p), ("copy", ctypes.c_void_p), ("n", ctypes.c_int64)]


class AdamWTable:
    """The tensors of kg_adamw, laid out once: lists of params (float32 or bfloat16), grads
    (float32 or bfloat16) and states exp_avgs, exp_avg_sqs: float32, or with m_scales and
    v_scales 1-byte e4m3 codes of the first moment and of the second one's square root (each
    scale tensor float32 [ceil(n / 128)]); copies: bfloat16 tensors that receive the new
    parameters (None: none). All contiguous, on one GPU; all of a list have one dtype. The
    table keeps the tensors; it is made anew when one of them moves (a gradient that autograd
    allocated anew)."""

    def __init__(self, params, grads, exp_avgs, exp_avg_sqs, m_scales=None, v_scales=None,
                 copies=None):
        import torch
        n = len(params)
        self.count, self.kinds, self.items, self.table = n, 0, 0, None
        none = [None] * n
        _need((m_scales is None) == (v_scales is None), "m_scales and v_scales go together")
        packed = m_scales is not None
        lists = [list(params), list(grads), list(exp_avgs), list(exp_avg_sqs),
                 list(m_scales) if packed else none, list(v_scales) if packed else none,
                 list(copies) if copies is not None else none]
        _need(all(len(x) == n for x in lists), "the lists must have one length")
        self.tensors = lists
        if n == 0:
            return
        ref = lists[0][0]
        _need(ref.is_cuda, "the tensors must be on a GPU")
        f32, bf16 = torch.float32, torch.bfloat16
        p16, g16 = ref.dtype == bf16, lists[1][0].dtype == bf16
        names = ("params", "grads", "exp_avgs", "exp_avg_sqs", "m_scales", "v_scales", "copies")
        kinds = (bf16 if p16 else f32, bf16 if g16 else f32, None if packed else f32,
                 None if packed else f32, f32, f32, bf16)
        rows = (AdamWTensor * n)()
        for i in range(n):
            size = lists[0][i].numel()
            for name, kind, x in zip(names, kinds, (col[i] for col in lists)):
                if x is None:
                    continue
                _need(x.device == ref.device and x.is_contiguous(),
                      f"{name}[{i}] must be contiguous and on {ref.device}")
                _need(x.dtype == kind if kind is not None else
                      x.element_size() == 1 and x.dtype != torch.bool,
                      f"{name}[{i}] must be {kind if kind is not None else 'e4m3 codes'}")
                _need(x.numel() == (-(-size // 128) if name in ("m_scales", "v_scales") else size),
                      f"{name}[{i}] has {x.numel()} elements for a parameter of {size}")
            rows[i] = AdamWTensor(*(_at(col[i]) for col in lists), size)
        self.kinds = (KG_ADAMW_P_BF16 if p16 else 0) | (KG_ADAMW_G_BF16 if g16 else 0) | \
            (KG_ADAMW_8BIT if packed else 0)
        L = lib()
        self.items, size = L.kg_adamw_items(rows, n), L.kg_adamw_table_bytes(rows, n)
        if size < 0:
            raise KgError(KG_ERR_SHAPE, "kg_adamw_table_bytes")
        image = torch.empty(size, dtype=torch.uint8)
        _check(L.kg_adamw_pack(rows, n, self.kinds, image.data_ptr(), size), "kg_adamw_pack")
        self.table = image.to(ref.device)


def kg_adamw(table, lr, beta1=0.9, beta2=0.999, eps=1e-8, weight_decay=0.0, step=1, gscale=None,
             dyn=None, stream=None):
    """One AdamW step over an AdamWTable's tensors, in place. step: 1 for the first. gscale:
    a one-element float32 GPU tensor that multiplies every gradient. dyn: float32 GPU tensor
    {lr, 1 - beta1^step, 1 - beta2^step}, read in the place of lr and step."""
    import torch
    if gscale is not None:
        _need(gscale.dtype == torch.float32 and gscale.numel() == 1, "gscale must be one float32")
    if dyn is not None:
        _need(dyn.dtype == torch.float32 and dyn.numel() == 3 and dyn.is_contiguous(),
              "dyn must be three contiguous float32")
    if table.count and (gscale is not None or dyn is not None):
        _gpu(table.table, gscale=gscale, dyn=dyn)
    _check(lib().kg_adamw(_at(table.table), table.count, table.items, table.kinds, lr, beta1, beta2,
                          eps, weight_decay, step, _at(gscale), _at(dyn), _on(stream)), "kg_adamw")
