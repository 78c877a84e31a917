"""Python binding of the batch operators in include/moe.h: the router's selection with rows grouped by
expert, the 16-bit grouped products and their gradients, the verification of drafted tokens.

Argument marshalling only: shapes, types and devices of the tensors are checked here (ValueError),
everything else by the library (MoeError).  Outputs are allocated where ``out`` is not given; with
``stream`` they then belong to that stream.  The launch goes to the tensors' device, whichever is
current.
"""
from __future__ import annotations

import contextlib
import ctypes

from .moe import OK, ROUTER_SOFTMAX, MoeError, _stream, lib

T_BF16, T_FP16, T_FP32 = 0, 1, 2
GROUP_NK, GROUP_KN = 0, 1
ACT_NONE, ACT_SWIGLU = 0, 1

_vp, _i, _ll = ctypes.c_void_p, ctypes.c_int, ctypes.c_longlong


class GroupedArgs(ctypes.Structure):
    _fields_ = [(n, _vp) for n in ("x", "w", "offsets", "rows", "out_rows", "out")] + \
        [(n, _ll) for n in ("x_rows", "ldx", "ldw", "w_stride", "out_rows_n", "ldo", "m")] + \
        [(n, _i) for n in ("groups", "n", "k", "dtype", "out_dtype", "layout", "act")] + \
        [("workspace", _vp), ("workspace_bytes", ctypes.c_size_t)]


class GroupedWgradArgs(ctypes.Structure):
    _fields_ = [(n, _vp) for n in ("dy", "x", "offsets", "dy_rows", "x_rows", "dw")] + \
        [(n, _ll) for n in ("dy_rows_n", "lddy", "x_rows_n", "ldx", "lddw", "dw_stride", "m")] + \
        [(n, _i) for n in ("groups", "n", "k", "dtype", "out_dtype")] + \
        [("workspace", _vp), ("workspace_bytes", ctypes.c_size_t)]


class VerifyArgs(ctypes.Structure):
    _fields_ = [(n, _vp) for n in ("p", "q", "draft", "lengths", "u", "accepted", "tokens")] + \
        [(n, _ll) for n in ("p_seq", "p_row", "q_seq", "q_row")] + [(n, _i) for n in ("B", "D", "V", "dtype")]


_calls = None


def _lib():
    global _calls
    if _calls is None:
        L = lib()
        L.moe_group_route.argtypes = [_vp, _ll, _i, _i, _i, _i, _i, _vp, _vp, _vp, _vp, _vp, _vp, ctypes.c_size_t, _vp]
        L.moe_group_route_workspace.argtypes = [_i, _i, _i]
        L.moe_group_route_workspace.restype = ctypes.c_size_t
        L.moe_grouped_workspace.argtypes = [_ll, _i]
        L.moe_grouped_workspace.restype = ctypes.c_size_t
        L.moe_grouped_matmul.argtypes = [ctypes.POINTER(GroupedArgs), _vp]
        L.moe_grouped_wgrad.argtypes = [ctypes.POINTER(GroupedWgradArgs), _vp]
        L.moe_verify_draft.argtypes = [ctypes.POINTER(VerifyArgs), _vp]
        for n in ("moe_group_route", "moe_grouped_matmul", "moe_grouped_wgrad", "moe_verify_draft"):
            getattr(L, n).restype = _i
        _calls = L
    return _calls


_torch = None
_types = {}


def _dtypes():
    global _torch
    if _torch is None:
        import torch
        _types.update({torch.bfloat16: T_BF16, torch.float16: T_FP16, torch.float32: T_FP32})
        _torch = torch
    return _torch


def _type(t, what, fp32=True):
    c = _types.get(t.dtype)
    if c is None or (c == T_FP32 and not fp32):
        raise ValueError("%s: dtype %s is not supported" % (what, t.dtype))
    return c


def _dense(t, what, dims, device):
    """A tensor of `dims` dimensions on `device`, its last dimension contiguous."""
    if t.dim() != dims or t.device != device or (t.shape[-1] > 1 and t.stride(-1) != 1):
        raise ValueError("%s: a %d-dimensional tensor on %s with a contiguous last dimension is wanted, got %s on %s" %
                         (what, dims, device, tuple(t.shape), t.device))
    return t


def _ints(t, what, shape, device):
    """A contiguous int32 tensor of the shape on the device."""
    if t.dtype != _torch.int32 or tuple(t.shape) != shape or t.device != device or not t.is_contiguous():
        raise ValueError("%s: a contiguous int32 tensor of shape %s on %s is wanted, got %s %s on %s" %
                         (what, shape, device, t.dtype, tuple(t.shape), t.device))
    return t.data_ptr()


def _pitch(t, dim, least):
    """Elements between neighbours along `dim`; at least `least` where there is only one."""
    return t.stride(dim) if t.shape[dim] > 1 else max(t.stride(dim), least)


def _device(t):
    if t.device.type != "cuda":
        raise ValueError("the tensors must be on a CUDA device, got %s" % t.device)
    return t.device


def _on(device, stream, allocates):
    """The context a call runs in: its device current, and its stream too where it allocates."""
    torch = _torch
    if allocates and stream is not None:
        s = torch.cuda.ExternalStream(stream, device=device) if isinstance(stream, int) else stream
        return torch.cuda.stream(s)
    if device.index != torch.cuda.current_device():
        return torch.cuda.device(device)
    return None


def _check(st, what):
    if st != OK:
        raise MoeError(st, what)


def group_route(logits, k, router=ROUTER_SOFTMAX, out=None, workspace=None, stream=None):
    """Router selection of a batch with its pairs grouped by expert (moe_group_route).

    logits [T, E] bf16, fp16 or fp32.  Returns (idx [T, k] int32, weights [T, k] fp32, offsets [E + 1]
    int32, rows [T k] int32, pairs [T k] int32): rows is what ``grouped_matmul`` gathers its input by, pairs
    the (token, rank) slots t k + j that its output is scattered to.  A logit of -inf is never selected: idx -1,
    weight 0, in no group.  out: the five tensors to write instead of new ones.  workspace: uint8 device
    memory of group_route_workspace(T, E, k) bytes; calls that may overlap on the GPU need one each."""
    torch = _dtypes()
    dev = _device(logits)
    _dense(logits, "logits", 2, dev)
    dt = _type(logits, "logits")
    T, E = logits.shape
    L = _lib()
    ctx = _on(dev, stream, out is None or workspace is None)
    with ctx if ctx is not None else contextlib.nullcontext():
        if out is None:
            i32 = torch.empty(2 * T * k + T * k + E + 1, dtype=torch.int32, device=dev)
            idx, rows, pairs, offsets = i32[:T * k].view(T, k), i32[T * k:2 * T * k], i32[2 * T * k:3 * T * k], i32[3 * T * k:]
            out = (idx, torch.empty(T, k, dtype=torch.float32, device=dev), offsets, rows, pairs)
        idx, weights, offsets, rows, pairs = out
        if weights.dtype != torch.float32 or tuple(weights.shape) != (T, k) or weights.device != dev or \
                not weights.is_contiguous():
            raise ValueError("out: weights must be a contiguous float32 tensor of shape %s" % ((T, k),))
        need = L.moe_group_route_workspace(T, E, k)
        if workspace is None and need:
            workspace = torch.empty(need, dtype=torch.uint8, device=dev)
        if workspace is not None and workspace.device != dev:
            raise ValueError("workspace: on %s, wanted on %s" % (workspace.device, dev))
        _check(L.moe_group_route(
            logits.data_ptr(), _pitch(logits, 0, E), dt, T, E, k, router, _ints(idx, "out: idx", (T, k), dev),
            weights.data_ptr(), _ints(offsets, "out: offsets", (E + 1,), dev), _ints(rows, "out: rows", (T * k,), dev),
            _ints(pairs, "out: pairs", (T * k,), dev), workspace.data_ptr() if workspace is not None else None,
            workspace.numel() * workspace.element_size() if workspace is not None else 0, _stream(stream)),
            "moe_group_route")
    return out


def group_route_workspace(T, E, k):
    """Bytes of workspace that group_route needs at these sizes (0 for sizes it refuses)."""
    return int(_lib().moe_group_route_workspace(T, E, k))


def _row_space(workspace, need, dev):
    """The workspace of a call that names rows by number: what is given, or new memory of `need` bytes."""
    if workspace is None and need:
        workspace = _torch.empty(need, dtype=_torch.uint8, device=dev)
    if workspace is None:
        return None, 0
    if workspace.device != dev:
        raise ValueError("workspace: on %s, wanted on %s" % (workspace.device, dev))
    return workspace.data_ptr(), workspace.numel() * workspace.element_size()


def grouped_workspace(m, k):
    """Bytes of workspace for m rows of length k that a grouped product names by number."""
    return int(_lib().moe_grouped_workspace(m, k))


def grouped_matmul(x, w, offsets, rows=None, out_rows=None, w_layout="nk", act=None, out=None, out_dtype=None, stream=None,
                   workspace=None):
    """The products of ragged groups of rows with their experts' weights (moe_grouped_matmul).

    x [R, k] bf16 or fp16; w [E, n, k] ("nk") or [E, k, n] ("kn") of the same type; offsets [E + 1] int32: sorted
    row i of [offsets[e], offsets[e + 1]) gives out = W_e x[rows[i]] (x[i] without rows), written to
    out[out_rows[i]] (out[i] without out_rows).  act="swiglu" ("nk" only): the first n / 2 rows of W_e are gate, the others
    up, and out = silu(gate x) * (up x) has n / 2 columns.  Rows of out that no sorted row names are left as they
    were (undefined in a new tensor).  The gradient of x is the same call on dy with the other w_layout.
    workspace (with rows): uint8 device memory of grouped_workspace(m, k) bytes; new memory without it."""
    torch = _dtypes()
    dev = _device(x)
    dt = _type(_dense(x, "x", 2, dev), "x", fp32=False)
    _dense(w, "w", 3, dev)
    if w.dtype != x.dtype:
        raise ValueError("w: dtype %s, x has %s" % (w.dtype, x.dtype))
    E = w.shape[0]
    R, k = x.shape
    if w_layout == "nk":
        layout, n, kw = GROUP_NK, w.shape[1], w.shape[2]
    elif w_layout == "kn":
        layout, n, kw = GROUP_KN, w.shape[2], w.shape[1]
    else:
        raise ValueError("w_layout: 'nk' or 'kn', got %r" % (w_layout,))
    if kw != k:
        raise ValueError("x has %d columns, w takes %d" % (k, kw))
    if act not in (None, "swiglu"):
        raise ValueError("act: None or 'swiglu', got %r" % (act,))
    n_out = n // 2 if act else n
    m = rows.shape[0] if rows is not None else out_rows.shape[0] if out_rows is not None else R
    ctx = _on(dev, stream, out is None or (rows is not None and workspace is None))
    with ctx if ctx is not None else contextlib.nullcontext():
        space = (None, 0) if rows is None else _row_space(workspace, _lib().moe_grouped_workspace(m, k), dev)
        if out is None:
            out = torch.empty(m, n_out, dtype=out_dtype or x.dtype, device=dev)
        _dense(out, "out", 2, dev)
        if out.shape[1] != n_out or (out_dtype is not None and out.dtype != out_dtype):
            raise ValueError("out: %s %s, wanted %d columns" % (tuple(out.shape), out.dtype, n_out))
        a = GroupedArgs(
            x.data_ptr(), w.data_ptr(), _ints(offsets, "offsets", (E + 1,), dev),
            None if rows is None else _ints(rows, "rows", (m,), dev),
            None if out_rows is None else _ints(out_rows, "out_rows", (m,), dev), out.data_ptr(),
            R, _pitch(x, 0, k), _pitch(w, 1, w.shape[2]), w.stride(0) if E > 1 else 0, out.shape[0], _pitch(out, 0, n_out), m,
            E, n, k, dt, _type(out, "out"), layout, ACT_SWIGLU if act else ACT_NONE, *space)
        if m:
            _check(_lib().moe_grouped_matmul(ctypes.byref(a), _stream(stream)), "moe_grouped_matmul")
    return out


def grouped_wgrad(dy, x, offsets, dy_rows=None, x_rows=None, out=None, out_dtype=None, stream=None, workspace=None):
    """The weights' gradient of grouped_matmul (moe_grouped_wgrad): out[e] = sum over the sorted rows i of
    expert e of dy[dy_rows[i]]^T x[x_rows[i]], [E, n, k] (zeros where a group is empty).

    dy [R, n] and x [S, k] bf16 or fp16 of one type; offsets [E + 1] int32.  For "kn" weights exchange dy and x.
    workspace (with row numbers): uint8 device memory of grouped_workspace(m, n) bytes for dy_rows and
    grouped_workspace(m, k) for x_rows; new memory without it."""
    torch = _dtypes()
    dev = _device(dy)
    dt = _type(_dense(dy, "dy", 2, dev), "dy", fp32=False)
    _dense(x, "x", 2, dev)
    if x.dtype != dy.dtype:
        raise ValueError("x: dtype %s, dy has %s" % (x.dtype, dy.dtype))
    n, k, E = dy.shape[1], x.shape[1], offsets.shape[0] - 1
    if dy_rows is not None:
        m = dy_rows.shape[0]
    elif x_rows is not None:
        m = x_rows.shape[0]
    else:
        m = min(dy.shape[0], x.shape[0])
    L = _lib()
    need = (L.moe_grouped_workspace(m, n) if dy_rows is not None else 0) + \
        (L.moe_grouped_workspace(m, k) if x_rows is not None else 0)
    ctx = _on(dev, stream, out is None or (need and workspace is None))
    with ctx if ctx is not None else contextlib.nullcontext():
        space = _row_space(workspace, need, dev)
        if out is None:
            out = torch.empty(E, n, k, dtype=out_dtype or dy.dtype, device=dev)
        _dense(out, "out", 3, dev)
        if tuple(out.shape) != (E, n, k) or (out_dtype is not None and out.dtype != out_dtype):
            raise ValueError("out: %s %s, wanted %s" % (tuple(out.shape), out.dtype, (E, n, k)))
        ldw = _pitch(out, 1, k)
        a = GroupedWgradArgs(
            dy.data_ptr() if dy.shape[0] else None, x.data_ptr() if x.shape[0] else None,
            _ints(offsets, "offsets", (E + 1,), dev),
            None if dy_rows is None else _ints(dy_rows, "dy_rows", (m,), dev),
            None if x_rows is None else _ints(x_rows, "x_rows", (m,), dev), out.data_ptr(),
            dy.shape[0], _pitch(dy, 0, n), x.shape[0], _pitch(x, 0, k), ldw,
            out.stride(0) if E > 1 else max(out.stride(0), (n - 1) * ldw + k), m, E, n, k, dt, _type(out, "out"), *space)
        _check(L.moe_grouped_wgrad(ctypes.byref(a), _stream(stream)), "moe_grouped_wgrad")
    return out


def verify_draft(p, draft, u, q=None, lengths=None, out=None, stream=None):
    """Which drafted tokens stand, and the token drawn after them (moe_verify_draft).

    p [B, D + 1, V]: the target's probabilities (bf16, fp16 or fp32); draft [B, D] int32; u [B, D + 1] fp32 in [0, 1);
    q [B, D, V]: the draft's probabilities, of p's type, or None for drafts given without; lengths [B] int32:
    drafts per sequence (D without it).  Returns (accepted [B] int32, tokens [B, D + 1] int32): the accepted drafts,
    the drawn token, then -1."""
    torch = _dtypes()
    dev = _device(p)
    dt = _type(_dense(p, "p", 3, dev), "p")
    B, D1, V = p.shape
    D = D1 - 1
    if q is not None:
        _dense(q, "q", 3, dev)
        if q.dtype != p.dtype or tuple(q.shape) != (B, D, V):
            raise ValueError("q: %s %s, wanted %s %s" % (tuple(q.shape), q.dtype, (B, D, V), p.dtype))
    if u.dtype != torch.float32 or tuple(u.shape) != (B, D1) or u.device != dev or not u.is_contiguous():
        raise ValueError("u: a contiguous float32 tensor of shape %s on %s is wanted" % ((B, D1), dev))
    ctx = _on(dev, stream, out is None)
    with ctx if ctx is not None else contextlib.nullcontext():
        if out is None:
            out = (torch.empty(B, dtype=torch.int32, device=dev), torch.empty(B, D1, dtype=torch.int32, device=dev))
        has_q = q is not None and D > 0
        a = VerifyArgs(
            p.data_ptr(), q.data_ptr() if has_q else None, _ints(draft, "draft", (B, D), dev) if D else None,
            None if lengths is None else _ints(lengths, "lengths", (B,), dev), u.data_ptr(),
            _ints(out[0], "out: accepted", (B,), dev), _ints(out[1], "out: tokens", (B, D1), dev),
            _pitch(p, 0, D1 * V), _pitch(p, 1, V), _pitch(q, 0, D * V) if has_q else 0, _pitch(q, 1, V) if has_q else 0,
            B, D, V, dt)
        _check(_lib().moe_verify_draft(ctypes.byref(a), _stream(stream)), "moe_verify_draft")
    return out
