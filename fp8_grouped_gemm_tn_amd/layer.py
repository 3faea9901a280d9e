"""Bindings of the operators around an expert layer's products (the C ABI in
include/kgwgrad.h): the sort of tokens by expert and the row copies (kg_route, kg_dispatch,
kg_dispatch_fp8, kg_combine, kg_combine_bwd), the router's choice in front of it (kg_gate,
kg_gate_bwd), the forward products (kg_fprop, kg_fprop_w4) and the steps
of the optimizers (AdamWTable, kg_adamw; kg_orthogonalize).

Argument marshalling only, as in _binding. With `stream` given, what a call makes is of that
stream's memory, and the current stream may use it once it waits for `stream`; the order of the
given tensors' uses is the caller's. A small call costs about as much here as on the
GPU, so the checks read each property of a tensor once.
"""
import ctypes

import numpy as np

from ._binding import (KG_ADAMW_8BIT, KG_ADAMW_G_BF16, KG_ADAMW_P_BF16, KG_ERR_SHAPE,
                       KG_FLAG_D_BF16, KG_OK, KG_ROWS_BF16, KG_ROWS_F32, KG_W4_E2M1,
                       KG_W4_INT_BF16, KG_W4_INT_F32, KgError, _need, lib, made)

torch = None  # imported with the first call, as the library itself is loaded
_lib = None
_f32 = _bf16 = _int32 = None
_row_types, _w4_kinds = {}, {}
_current_gpu = _current_stream = None


def _load():
    """The loaded library; sets what the calls read of torch."""
    global torch, _lib, _f32, _bf16, _int32, _row_types, _w4_kinds, _current_gpu, _current_stream
    if _lib is None:
        import torch as t
        L = lib()
        _f32, _bf16, _int32 = t.float32, t.bfloat16, t.int32
        _row_types = {t.bfloat16: KG_ROWS_BF16, t.float32: KG_ROWS_F32}
        _w4_kinds = {t.bfloat16: KG_W4_INT_BF16, t.float32: KG_W4_INT_F32, t.uint8: KG_W4_E2M1}
        _current_gpu, _current_stream = t._C._cuda_getDevice, t._C._cuda_getCurrentRawStream
        torch, _lib = t, L
    return _lib


def _on(gpu, stream):
    """hipStream_t: `stream`'s, or the current one. The call goes to the current GPU, so that
    has to be `gpu`."""
    if gpu != _current_gpu():
        raise ValueError(f"the tensors are on GPU {gpu}, which is not the current one")
    return _current_stream(gpu) if stream is None else stream.cuda_stream


def _made(shape, dtype, ref, stream, back=True):
    return made(torch, shape, dtype, ref.device, stream, back)


def _fail(rc, what):
    raise KgError(rc, what)


def _at(t):
    return None if t is None else t.data_ptr()


def _gpu(ref, *others):
    """The GPU that `ref` and every given tensor are on."""
    gpu = ref.get_device()
    if gpu < 0:
        raise ValueError("the tensors must be on a GPU")
    for t in others:
        if t is not None and t.get_device() != gpu:
            raise ValueError(f"a tensor is on {t.device}, another on {ref.device}")
    return gpu


def _i32(t, shape, name):
    if t.dtype is not _int32 or t.shape != shape or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous int32 {list(shape)} tensor")


def _row_type(dtype, name):
    ty = _row_types.get(dtype)
    if ty is None:
        raise ValueError(f"{name} must be bfloat16 or float32")
    return ty


def _rows(t, name):
    """(rows, columns, row stride in elements) of a 2-D tensor whose rows are contiguous (its
    width where it has at most one row, or no columns: torch gives those any stride)."""
    shape = t.shape
    if len(shape) != 2:
        raise ValueError(f"{name} must be 2-D")
    rows, cols = shape
    ld, one = t.stride()
    if one != 1 and cols > 1:
        raise ValueError(f"{name} must have contiguous rows")
    return rows, cols, ld if rows > 1 and cols > 0 else cols


def new_route_workspace(T, k, G, device):
    """The workspace of kg_route for T tokens of k slots and G experts (None where it needs
    none); keep it for later calls of at most these sizes."""
    n = _load().kg_route_workspace_bytes(T, k, G)
    if n < 0:
        _fail(KG_ERR_SHAPE, "kg_route_workspace_bytes")
    return torch.empty(n, dtype=torch.uint8, device=device) if n else None


def _workspace(ws):
    """(address, bytes) of a workspace tensor or None."""
    if ws is None:
        return None, 0
    if ws.dtype is not torch.uint8 or not ws.is_contiguous():
        raise ValueError("ws must be contiguous uint8")
    return ws.data_ptr(), ws.numel()


def kg_route(idx, ks, pos=None, src=None, ws=None, stream=None):
    """Plan that puts tokens into expert order: idx int32 [T, k] (an entry outside [0, G) is
    dropped), ks int32 [G] (out). pos int32 [T, k] and src int32 [T * k] are written (made if
    not given); ws: new_route_workspace (made if not given and needed). Returns (pos, src)."""
    L = _lib or _load()
    shape, experts = idx.shape, ks.shape
    if len(shape) != 2 or len(experts) != 1:
        raise ValueError("idx must be [T, k] and ks [G]")
    T, k = shape
    G = experts[0]
    _i32(idx, shape, "idx")
    _i32(ks, experts, "ks")
    if pos is None:
        pos = _made(shape, _int32, idx, stream)
    if src is None:
        src = _made((T * k,), _int32, idx, stream)
    _i32(pos, shape, "pos")
    _i32(src, (T * k,), "src")
    if ws is None:
        n = L.kg_route_workspace_bytes(T, k, G)
        if n > 0:
            ws = _made((n,), torch.uint8, idx, stream, back=False)
    at, size = _workspace(ws)
    gpu = _gpu(idx, ks, pos, src, ws)
    rc = L.kg_route(idx.data_ptr(), T, k, G, ks.data_ptr(), pos.data_ptr(), src.data_ptr(), at,
                    size, _on(gpu, stream))
    if rc:
        _fail(rc, "kg_route")
    return pos, src


def new_gate_workspace(T, G, device):
    """The workspace of kg_gate with statistics, for T tokens and G experts; keep it for later
    calls of at most these sizes."""
    n = _load().kg_gate_workspace_bytes(T, G)
    if n < 0:
        _fail(KG_ERR_SHAPE, "kg_gate_workspace_bytes")
    return torch.empty(n, dtype=torch.uint8, device=device)


def _one(t, name):
    if t is not None and (t.dtype is not _f32 or t.numel() != 1):
        raise ValueError(f"{name} must be one float32")


def kg_gate(X, k, bias=None, flags=0, scale=1.0, coef=0.0, idx=None, w=None, counts=None,
            psum=None, loss=None, ws=None, stream=None):
    """The router's choice: X [T, G] logits (bfloat16 or float32, rows contiguous), bias float32
    [G] or None, flags KG_GATE_SIGMOID and KG_GATE_NORM. Writes idx int32 [T, k] and w float32
    [T, k] (made if not given), and what is given of counts int32 [G], psum float32 [G] and loss,
    one float32; ws: new_gate_workspace (made if not given and needed). Returns (idx, w)."""
    L = _lib or _load()
    ty, (T, G, ldx) = _row_type(X.dtype, "X"), _rows(X, "X")
    if idx is None:
        idx = _made((T, k), _int32, X, stream)
    if w is None:
        w = _made((T, k), _f32, X, stream)
    _i32(idx, (T, k), "idx")
    _expert_rows(w, (T, k), _f32, "w")
    if bias is not None:
        _expert_rows(bias, (G,), _f32, "bias")
    at = size = None
    if counts is not None or psum is not None or loss is not None:
        if counts is not None:
            _i32(counts, (G,), "counts")
        if psum is not None:
            _expert_rows(psum, (G,), _f32, "psum")
        _one(loss, "loss")
        if ws is None:
            n = L.kg_gate_workspace_bytes(T, G)
            if n > 0:
                ws = _made((n,), torch.uint8, X, stream, back=False)
        at, size = _workspace(ws)
    gpu = _gpu(X, bias, idx, w, counts, psum, loss, ws)
    rc = L.kg_gate(X.data_ptr(), ldx, _at(bias), T, G, k, ty, flags, scale, coef, idx.data_ptr(),
                   w.data_ptr(), _at(counts), _at(psum), _at(loss), at, size or 0,
                   _on(gpu, stream))
    if rc:
        _fail(rc, "kg_gate")
    return idx, w


def kg_gate_bwd(X, idx, dw=None, counts=None, dloss=None, flags=0, scale=1.0, coef=0.0, dX=None,
                stream=None):
    """The logits' gradient of kg_gate: X, idx, flags, scale and coef as given to and made by it,
    dw float32 [T, k] (None: zeros), counts int32 [G] (None: no gradient of the loss), dloss one
    float32 on the GPU (None: 1). Returns dX [T, G] of X's dtype (rows contiguous; made if not
    given)."""
    L = _lib or _load()
    dtype = X.dtype
    ty, (T, G, ldx) = _row_type(dtype, "X"), _rows(X, "X")
    shape = idx.shape
    if len(shape) != 2 or shape[0] != T:
        raise ValueError(f"idx must be [{T}, k]")
    _i32(idx, shape, "idx")
    if dw is not None:
        _expert_rows(dw, shape, _f32, "dw")
    if counts is not None:
        _i32(counts, (G,), "counts")
    _one(dloss, "dloss")
    if dX is None:
        dX = _made((T, G), dtype, X, stream)
    rows, cols, ldd = _rows(dX, "dX")
    if dX.dtype is not dtype or rows != T or cols != G:
        raise ValueError("dX must be [T, G] of X's dtype")
    gpu = _gpu(X, idx, dw, counts, dloss, dX)
    rc = L.kg_gate_bwd(X.data_ptr(), ldx, idx.data_ptr(), _at(dw), _at(counts), _at(dloss), T, G,
                       shape[1], ty, flags, scale, coef, dX.data_ptr(), ldd, _on(gpu, stream))
    if rc:
        _fail(rc, "kg_gate_bwd")
    return dX


def _positions(pos, T):
    """k of the int32 [T, k] tensor pos."""
    shape = pos.shape
    if (len(shape) != 2 or shape[0] != T or pos.dtype is not _int32 or
            not pos.is_contiguous()):
        raise ValueError(f"pos must be a contiguous int32 [{T}, k] tensor")
    return shape[1]


def _expert_rows(t, shape, dtype, name):
    if t.dtype is not dtype or t.shape != shape or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous {dtype} {list(shape)} tensor")


def kg_dispatch(X, pos, Xp=None, stream=None):
    """X [T, H] (bfloat16 or float32, rows contiguous) copied to Xp [T * k, H] (made if not
    given): every token's row to the rows that pos (kg_route) names, zeros for dropped slots."""
    L = _lib or _load()
    dtype = X.dtype
    ty, (T, H, ldx) = _row_type(dtype, "X"), _rows(X, "X")
    k = _positions(pos, T)
    if Xp is None:
        Xp = _made((T * k, H), dtype, X, stream)
    _expert_rows(Xp, (T * k, H), dtype, "Xp")
    gpu = _gpu(X, pos, Xp)
    rc = L.kg_dispatch(X.data_ptr(), ldx, pos.data_ptr(), T, k, H, ty, Xp.data_ptr(),
                       _on(gpu, stream))
    if rc:
        _fail(rc, "kg_dispatch")
    return Xp


def kg_dispatch_fp8(X, pos, Q=None, sa=None, ws=None, stream=None):
    """kg_dispatch as e4m3 codes: X bfloat16 [T, H], H a multiple of 16; Q 1-byte [T * k, H] and
    sa float32 [ceil(H / 128), T * k] as kg_fprop and kg_dgrad read them (made if not given);
    ws: a uint8 workspace of kg_dispatch_fp8_workspace_bytes (made if not given and of use).
    Returns (Q, sa)."""
    L = _lib or _load()
    if X.dtype is not _bf16:
        raise ValueError("X must be bfloat16")
    T, H, ldx = _rows(X, "X")
    k = _positions(pos, T)
    if Q is None:
        Q = _made((T * k, H), torch.uint8, X, stream)
    if sa is None:
        sa = _made((-(-H // 128), T * k), _f32, X, stream)
    if Q.element_size() != 1 or Q.shape != (T * k, H) or not Q.is_contiguous():
        raise ValueError("Q must be a contiguous 1-byte [T * k, H] tensor")
    _expert_rows(sa, (-(-H // 128), T * k), _f32, "sa")
    if ws is None:
        n = L.kg_dispatch_fp8_workspace_bytes(T, k, H)
        if n > 0:
            ws = _made((n,), torch.uint8, X, stream, back=False)
    at, size = _workspace(ws)
    gpu = _gpu(X, pos, Q, sa, ws)
    rc = L.kg_dispatch_fp8(X.data_ptr(), ldx, pos.data_ptr(), T, k, H, Q.data_ptr(),
                           sa.data_ptr(), at, size, _on(gpu, stream))
    if rc:
        _fail(rc, "kg_dispatch_fp8")
    return Q, sa


def kg_combine(Y, pos, w=None, out=None, stream=None):
    """out[t] = sum_j w[t][j] Y[pos[t][j]] over the kept slots: Y [T * k, H] (bfloat16 or
    float32), pos int32 [T, k] from kg_route, w float32 [T, k] (None: ones), out [T, H] (rows
    contiguous; made if not given). With w None this is kg_dispatch's gradient."""
    L = _lib or _load()
    dtype, shape = Y.dtype, Y.shape
    ty = _row_type(dtype, "Y")
    T = pos.shape[0] if pos.dim() else -1
    k = _positions(pos, T)
    if len(shape) != 2 or shape[0] != T * k or not Y.is_contiguous():
        raise ValueError(f"Y must be a contiguous [{T * k}, H] tensor")
    H = shape[1]
    if w is not None:
        _expert_rows(w, (T, k), _f32, "w")
    if out is None:
        out = _made((T, H), dtype, Y, stream)
    rows, cols, ldo = _rows(out, "out")
    if out.dtype is not dtype or rows != T or cols != H:
        raise ValueError("out must be [T, H] of Y's dtype")
    gpu = _gpu(Y, pos, w, out)
    rc = L.kg_combine(Y.data_ptr(), pos.data_ptr(), _at(w), out.data_ptr(), ldo, T, k, H, ty,
                      _on(gpu, stream))
    if rc:
        _fail(rc, "kg_combine")
    return out


def kg_combine_bwd(dOut, Y, pos, w=None, dY=None, dw=None, need_dw=True, stream=None):
    """Gradients of kg_combine: dOut [T, H] (rows contiguous), Y [T * k, H], pos, w as given to
    it. Returns (dY [T * k, H], dw float32 [T, k]); with need_dw False dw is not computed (None)
    and Y is not read (it may be None)."""
    L = _lib or _load()
    dtype = dOut.dtype
    ty, (T, H, ldo) = _row_type(dtype, "dOut"), _rows(dOut, "dOut")
    k = _positions(pos, T)
    if w is not None:
        _expert_rows(w, (T, k), _f32, "w")
    if dY is None:
        dY = _made((T * k, H), dtype, dOut, stream)
    _expert_rows(dY, (T * k, H), dtype, "dY")
    if need_dw:
        if Y is None:
            raise ValueError("dw needs Y")
        _expert_rows(Y, (T * k, H), dtype, "Y")
        if dw is None:
            dw = _made((T, k), _f32, dOut, stream)
        _expert_rows(dw, (T, k), _f32, "dw")
    else:
        Y = dw = None
    gpu = _gpu(dOut, Y, pos, w, dY, dw)
    rc = L.kg_combine_bwd(dOut.data_ptr(), ldo, _at(Y), pos.data_ptr(), _at(w), dY.data_ptr(),
                          _at(dw), T, k, H, ty, _on(gpu, stream))
    if rc:
        _fail(rc, "kg_combine_bwd")
    return dY, dw


def kg_fprop(A, sa, W, sw, D, ms, flags=0, stream=None):
    """D = rows . W^T per expert: A fp8 codes [M_total, K] (rows contiguous), sa float32
    [ceil(K / 128), M_total], W fp8 codes [G, N, K], sw float32 [G, ceil(N / 128),
    ceil(K / 128)], ms int32 [G], D [M_total, N] (float32 or bfloat16, rows contiguous)."""
    L = _lib or _load()
    if W.dim() != 3 or W.element_size() != 1 or not W.is_contiguous():
        raise ValueError("W must be contiguous fp8 codes [G, N, K]")
    G, N, K = W.shape
    (M, cols, lda), (rows, outs, ldd) = _rows(A, "A"), _rows(D, "D")
    nk = -(-K // 128)
    if cols != K or A.element_size() != 1:
        raise ValueError("A must be fp8 codes [M_total, K]")
    _expert_rows(sa, (nk, M), _f32, "sa")
    _expert_rows(sw, (G, -(-N // 128), nk), _f32, "sw")
    _i32(ms, (G,), "ms")
    if D.dtype is _bf16:
        flags |= KG_FLAG_D_BF16
    elif D.dtype is not _f32:
        raise ValueError("D must be float32 or bfloat16")
    if rows != M or outs != N:
        raise ValueError("D must be [M_total, N]")
    gpu = _gpu(D, A, sa, W, sw, ms)
    rc = L.kg_fprop(A.data_ptr(), lda, sa.data_ptr(), W.data_ptr(), sw.data_ptr(), D.data_ptr(),
                    ldd, ms.data_ptr(), G, N, K, M, flags, _on(gpu, stream))
    if rc:
        _fail(rc, "kg_fprop")
    return D


def kg_fprop_w4(A, W, sw, D, ms, zp=None, stream=None):
    """kg_fprop's product with 4-bit weights: A bfloat16 [M_total, K] (rows contiguous), W bytes
    [G, N, K / 2] of two codes each (the even channel's in the low half), ms int32 [G], D
    [M_total, N] (float32 or bfloat16, rows contiguous). sw [G, N, K / group] says what the codes
    are: bfloat16 or float32, whole numbers w = (q - z) s with group 32, 64 or 128 and zp uint8 of
    the same shape (None: 8); uint8, e2m1 codes times 2^(sw - 127) with group 32."""
    L = _lib or _load()
    if W.dim() != 3 or W.element_size() != 1 or not W.is_contiguous():
        raise ValueError("W must be contiguous bytes [G, N, K / 2]")
    G, N, K = W.shape
    K *= 2
    (M, cols, lda), (rows, outs, ldd) = _rows(A, "A"), _rows(D, "D")
    if cols != K or A.dtype is not _bf16:
        raise ValueError("A must be bfloat16 [M_total, K]")
    shape, kind = sw.shape, _w4_kinds.get(sw.dtype)
    if kind is None or len(shape) != 3 or shape[0] != G or shape[1] != N or not sw.is_contiguous():
        raise ValueError("sw must be contiguous [G, N, K / group]: bfloat16, float32 or uint8")
    group = K // shape[2] if shape[2] else 32
    if group * shape[2] != K:
        raise ValueError("sw must hold one scale per group of channels")
    if zp is not None and (zp.dtype is not torch.uint8 or zp.shape != shape or
                           not zp.is_contiguous()):
        raise ValueError("zp must be contiguous uint8 of sw's shape")
    _i32(ms, (G,), "ms")
    flags = 0
    if D.dtype is _bf16:
        flags = KG_FLAG_D_BF16
    elif D.dtype is not _f32:
        raise ValueError("D must be float32 or bfloat16")
    if rows != M or outs != N:
        raise ValueError("D must be [M_total, N]")
    gpu = _gpu(D, A, W, sw, ms, zp)
    rc = L.kg_fprop_w4(A.data_ptr(), lda, W.data_ptr(), sw.data_ptr(), _at(zp), D.data_ptr(), ldd,
                       ms.data_ptr(), G, N, K, M, group, kind, flags, _on(gpu, stream))
    if rc:
        _fail(rc, "kg_fprop_w4")
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
    allocated anew). It is made on the stream that its tensors' memory belongs to; a step may
    run on any stream, and the table be dropped as soon as the call returns. A graph that
    captured a step needs the table as long as it is replayed."""

    def __init__(self, params, grads, exp_avgs, exp_avg_sqs, m_scales=None, v_scales=None,
                 copies=None):
        L = _lib or _load()
        n = len(params)
        self.count, self.kinds, self.items, self.table = n, 0, 0, None
        self.streams = set()  # those whose steps the allocator knows of
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
        _gpu(ref)
        device = ref.device
        p16, g16 = ref.dtype is _bf16, lists[1][0].dtype is _bf16
        names = ("params", "grads", "exp_avgs", "exp_avg_sqs", "m_scales", "v_scales", "copies")
        kinds = (_bf16 if p16 else _f32, _bf16 if g16 else _f32, None if packed else _f32,
                 None if packed else _f32, _f32, _f32, _bf16)
        sizes = [x.numel() for x in lists[0]]
        blocks = [-(-s // 128) for s in sizes]
        rows = np.zeros((n, 8), np.int64)  # kg_adamw_tensor: seven pointers, n
        rows[:, 7] = sizes
        for col, (name, kind, xs) in enumerate(zip(names, kinds, lists)):
            if xs is none:
                continue
            if kind is None:  # e4m3 codes
                ok = all(x.element_size() == 1 and x.dtype is not torch.bool for x in xs)
            else:
                ok = all(x.dtype is kind for x in xs)
            _need(ok, f"{name} must all be {'1-byte e4m3 codes' if kind is None else kind}")
            _need(all(x.device == device and x.is_contiguous() for x in xs),
                  f"{name} must be contiguous and on {device}")
            _need([x.numel() for x in xs] == (blocks if name.endswith("scales") else sizes),
                  f"{name} must have {'ceil(n / 128)' if name.endswith('scales') else 'n'} "
                  "elements for a parameter of n")
            rows[:, col] = [x.data_ptr() for x in xs]
        at = rows.ctypes.data
        self.kinds = (KG_ADAMW_P_BF16 if p16 else 0) | (KG_ADAMW_G_BF16 if g16 else 0) | \
            (KG_ADAMW_8BIT if packed else 0)
        self.items, size = L.kg_adamw_items(at, n), L.kg_adamw_table_bytes(at, n)
        if size < 0:
            _fail(KG_ERR_SHAPE, "kg_adamw_table_bytes")
        image = torch.empty(size, dtype=torch.uint8)
        rc = L.kg_adamw_pack(at, n, self.kinds, image.data_ptr(), size)
        if rc:
            _fail(rc, "kg_adamw_pack")
        self.table = image.to(device)
        self.streams.add(_current_stream(device.index))

    def used_on(self, handle, stream):
        """A step goes to `stream` (None: the current one): from the first one on, the memory of
        the table and of the tensors that it may be the last to keep is not handed on before
        that stream is done with it."""
        if stream is None:
            stream = torch.cuda.current_stream(self.table.device)
        with torch.cuda.stream(stream):
            if torch.cuda.is_current_stream_capturing():
                return  # nothing runs now
        for xs in self.tensors:
            for x in xs:
                if x is not None:
                    x.record_stream(stream)
        self.table.record_stream(stream)
        self.streams.add(handle)


def kg_adamw(table, lr, beta1=0.9, beta2=0.999, eps=1e-8, weight_decay=0.0, step=1, gscale=None,
             dyn=None, stream=None):
    """One AdamW step over an AdamWTable's tensors, in place. step: 1 for the first. gscale:
    a one-element float32 GPU tensor that multiplies every gradient. dyn: float32 GPU tensor
    {lr, 1 - beta1^step, 1 - beta2^step}, read in the place of lr and step."""
    L = _lib or _load()
    if gscale is not None and (gscale.dtype is not _f32 or gscale.numel() != 1):
        raise ValueError("gscale must be one float32")
    if dyn is not None and (dyn.dtype is not _f32 or dyn.shape != (3,) or not dyn.is_contiguous()):
        raise ValueError("dyn must be three contiguous float32")
    if table.table is None:  # no tensors
        return
    on = _on(_gpu(table.table, gscale, dyn), stream)
    rc = L.kg_adamw(table.table.data_ptr(), table.count, table.items, table.kinds, lr, beta1,
                    beta2, eps, weight_decay, step, _at(gscale), _at(dyn), on)
    if on not in table.streams:
        table.used_on(on, stream)
    if rc:
        _fail(rc, "kg_adamw")


def new_orthogonalize_workspace(G, R, C, device):
    """The workspace of kg_orthogonalize for G matrices [R, C]; keep it for later calls of at most
    these sizes."""
    n = _load().kg_orthogonalize_workspace_bytes(G, R, C)
    if n < 0:
        _fail(KG_ERR_SHAPE, "kg_orthogonalize_workspace_bytes")
    return torch.empty(n, dtype=torch.uint8, device=device)


def kg_orthogonalize(U, O=None, steps=5, ws=None, stream=None):
    """The nearly orthogonal form of weight updates by Newton-Schulz steps: U [R, C] or [G, R, C]
    (bfloat16 or float32, contiguous), O bfloat16 of U's shape (made if not given; may be U); ws:
    new_orthogonalize_workspace (made if not given). Returns O."""
    L = _lib or _load()
    ty, shape = _row_type(U.dtype, "U"), U.shape
    if len(shape) not in (2, 3) or not U.is_contiguous():
        raise ValueError("U must be contiguous [R, C] or [G, R, C]")
    G, R, C = shape if len(shape) == 3 else (1, *shape)
    if O is None:
        O = _made(shape, _bf16, U, stream)
    _expert_rows(O, shape, _bf16, "O")
    if ws is None:
        n = L.kg_orthogonalize_workspace_bytes(G, R, C)
        if n > 0:
            ws = _made((n,), torch.uint8, U, stream, back=False)
    at, size = _workspace(ws)
    gpu = _gpu(U, O, ws)
    rc = L.kg_orthogonalize(U.data_ptr(), O.data_ptr(), G, R, C, ty, steps, at, size,
                            _on(gpu, stream))
    if rc:
        _fail(rc, "kg_orthogonalize")
    return O
