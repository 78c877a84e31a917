"""Python binding of the batch operators in include/moe.h: the router's selection with rows grouped by
expert, the 16-bit grouped products and their gradients, the verification of drafted tokens.

Argument marshalling only: shapes, types and devices of the tensors are checked here (ValueError),
everything else by the library (MoeError).  Outputs and workspaces are allocated where they are not
given; with ``stream`` they then belong to that stream.  The launch goes to the tensors' device,
whichever is current.  The calls take a few microseconds of host time, which decides what the smallest
products take, so the checks are kept lean.
"""
from __future__ import annotations

import ctypes
import functools
import struct

from .moe import OK, ROUTER_SOFTMAX, MoeError, lib

T_BF16, T_FP16, T_FP32 = 0, 1, 2
GROUP_NK, GROUP_KN = 0, 1
ACT_NONE, ACT_SWIGLU = 0, 1
GROUPED_NONE, GROUPED_FEW, GROUPED_PAIR, GROUPED_ANY = range(4)

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


def _packer(cls):
    """The structure's packed form: the same bytes as the ctypes structure, made in one call (pointers and sizes as
    unsigned numbers)."""
    code = {_vp: "Q", _ll: "q", _i: "i", ctypes.c_size_t: "Q"}
    return struct.Struct("@" + "".join(code[t] for _, t in cls._fields_)).pack


_pack_matmul, _pack_wgrad, _pack_verify = _packer(GroupedArgs), _packer(GroupedWgradArgs), _packer(VerifyArgs)
_calls = None


def _lib():
    global _calls
    if _calls is None:
        L = lib()
        L.moe_group_route.argtypes = [_vp, _ll, _i, _i, _i, _i, _i, _vp, _vp, _vp, _vp, _vp, _vp, ctypes.c_size_t, _vp]
        L.moe_group_route_workspace.argtypes = [_i, _i, _i]
        L.moe_grouped_workspace.argtypes = [_ll, _i, _i]
        L.moe_grouped_wgrad_workspace.argtypes = [_ll, _i]
        for n in ("moe_group_route_workspace", "moe_grouped_workspace", "moe_grouped_wgrad_workspace"):
            getattr(L, n).restype = ctypes.c_size_t
        for n in ("moe_grouped_matmul", "moe_grouped_wgrad", "moe_verify_draft"):
            getattr(L, n).argtypes = [_vp, _vp]
        L.moe_debug_batch_wait.argtypes = [_ll]
        L.moe_debug_batch_wait.restype = _i
        for n in ("moe_grouped_kernel", "moe_grouped_wgrad_kernel"):
            getattr(L, n).argtypes = [_vp, _i]
            getattr(L, n).restype = _i
        for n in ("moe_group_route", "moe_grouped_matmul", "moe_grouped_wgrad", "moe_verify_draft"):
            getattr(L, n).restype = _i
        _calls = L
    return _calls


_torch = None
_types = {}
_raw_stream = None    # torch's current stream of a device as an address, without a Stream object (2 us less)
_current = None       # the current device's index


def _start():
    """(torch, the library)"""
    global _torch, _raw_stream, _current
    if _torch is None:
        import torch
        _raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or \
            (lambda index: torch.cuda.current_stream(index).cuda_stream)
        _current = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device
        _types.update({torch.bfloat16: T_BF16, torch.float16: T_FP16, torch.float32: T_FP32})
        _torch = torch
    return _torch, _calls or _lib()


# The workspaces' sizes depend on the numbers alone; remembered, as a call through ctypes takes 0.5 us.
@functools.lru_cache(4096)
def _route_space(T, E, k):
    return _lib().moe_group_route_workspace(T, E, k)


@functools.lru_cache(4096)
def _matmul_space(m, k, groups):
    return _lib().moe_grouped_workspace(m, k, groups)


@functools.lru_cache(4096)
def _wgrad_space(m, length):
    return _lib().moe_grouped_wgrad_workspace(m, length)


def _type(t, what, fp32=True):
    c = _types.get(t.dtype)
    if c is None or (c == T_FP32 and not fp32):
        raise ValueError("%s: dtype %s is not supported" % (what, t.dtype))
    return c


def _cuda(t, what):
    """The index of the tensor's CUDA device."""
    index = t.get_device()
    if index < 0 or not t.is_cuda:
        raise ValueError("%s: the tensors must be on a CUDA device, got %s" % (what, t.device))
    return index


def _dense(t, what, dims, index):
    """(shape, strides) of a tensor of `dims` dimensions on the device, its last dimension contiguous."""
    shape, stride = t.shape, t.stride()
    if len(shape) != dims or t.get_device() != index or (stride[-1] != 1 and shape[-1] > 1):
        raise ValueError("%s: a %d-dimensional tensor on cuda:%d with a contiguous last dimension is wanted, got %s on %s" %
                         (what, dims, index, tuple(shape), t.device))
    return shape, stride


def _flat(t, what, dtype, shape, index):
    """The address of a contiguous tensor of that type and shape on the device."""
    if t.dtype is not dtype or t.shape != shape or t.get_device() != index or not t.is_contiguous():
        raise ValueError("%s: a contiguous %s tensor of shape %s on cuda:%d is wanted, got %s %s on %s" %
                         (what, dtype, tuple(shape), index, t.dtype, tuple(t.shape), t.device))
    return t.data_ptr()


def _pitch(stride, size, least):
    """Elements between neighbours along a dimension; at least `least` where there is only one."""
    return stride if size > 1 or stride > least else least


def _new(stream, index, *wanted):
    """New tensors of the given (shape, dtype), belonging to the stream that will use them."""
    torch = _torch
    dev = torch.device("cuda", index)
    if stream is None:
        return [torch.empty(s, dtype=t, device=dev) for s, t in wanted]
    s = torch.cuda.ExternalStream(stream, device=dev) if isinstance(stream, int) else stream
    with torch.cuda.stream(s):
        return [torch.empty(s, dtype=t, device=dev) for s, t in wanted]


def _space(workspace, need, stream, index):
    """(address, bytes) of a call's workspace: what is given, or new memory; and the tensor, to be held until the
    launch."""
    if workspace is None:
        if not need:
            return 0, 0, None
        workspace, = _new(stream, index, ((need,), _torch.uint8))
    elif workspace.get_device() != index or not workspace.is_contiguous():
        raise ValueError("workspace: a contiguous tensor on cuda:%d is wanted, got one on %s" % (index, workspace.device))
    return workspace.data_ptr(), workspace.numel() * workspace.element_size(), workspace


def _run(what, call, index, stream, *args):
    """The call on the tensors' device, on `stream` or that device's current one."""
    if stream is None:
        stream = _raw_stream(index)
    elif not isinstance(stream, int):
        stream = stream.cuda_stream
    if index == _current():
        st = call(*args, stream)
    else:
        with _torch.cuda.device(index):
            st = call(*args, stream)
    if st != OK:
        raise MoeError(st, what)


def group_route(logits, k, router=ROUTER_SOFTMAX, out=None, workspace=None, stream=None):
    """Router selection of a batch with its pairs grouped by expert (moe_group_route).

    logits [T, E] bf16, fp16 or fp32.  Returns (idx [T, k] int32, weights [T, k] fp32, offsets [E + 1]
    int32, rows [T k] int32, pairs [T k] int32): rows is what ``grouped_matmul`` gathers its input by, pairs
    the (token, rank) slots t k + j that its output is scattered to.  A logit of -inf is never selected: idx -1,
    weight 0, in no group.  out: the five tensors to write instead of new ones.  workspace: uint8 device
    memory of group_route_workspace(T, E, k) bytes; calls that may overlap on the GPU need one each."""
    torch, L = _start()
    dev = _cuda(logits, "logits")
    (T, E), stride = _dense(logits, "logits", 2, dev)
    dt = _type(logits, "logits")
    i32, P, TK = torch.int32, (T * k,), (T, k)
    if out is None:
        if k < 1:
            raise ValueError("k: at least 1, got %d" % k)
        out = tuple(_new(stream, dev, (TK, i32), (TK, torch.float32), ((E + 1,), i32), (P, i32), (P, i32)))
    idx, weights, offsets, rows, pairs = out
    ws, ws_bytes, _held = _space(workspace, _route_space(T, E, k), stream, dev)
    _run("moe_group_route", L.moe_group_route, dev, stream, logits.data_ptr(), _pitch(stride[0], T, E), dt, T, E, k, router,
         _flat(idx, "out: idx", i32, TK, dev), _flat(weights, "out: weights", torch.float32, TK, dev),
         _flat(offsets, "out: offsets", i32, (E + 1,), dev), _flat(rows, "out: rows", i32, P, dev),
         _flat(pairs, "out: pairs", i32, P, dev), ws, ws_bytes)
    return out


def group_route_workspace(T, E, k):
    """Bytes of workspace that group_route needs at these sizes (0 for sizes it refuses)."""
    return int(_lib().moe_group_route_workspace(T, E, k))


def grouped_workspace(m, k, groups):
    """Bytes of workspace that grouped_matmul needs for m rows of length k named by number (0 where it needs none)."""
    return int(_lib().moe_grouped_workspace(m, k, groups))


def grouped_wgrad_workspace(m, length):
    """Bytes of workspace that grouped_wgrad needs for m rows of that length named by number."""
    return int(_lib().moe_grouped_wgrad_workspace(m, length))


def debug_batch_wait(cycles=-1):
    """Bound the batch operators' device waits on the current device in SM cycles (0: their
    products wait for a flag that nothing sets, -1: the usual bound), and forget one that ran out (moe_debug_batch_wait)."""
    st = _lib().moe_debug_batch_wait(cycles)
    if st != OK:
        raise MoeError(st, "moe_debug_batch_wait")


def grouped_kernel(args, num_sms):
    """The kernel (GROUPED_FEW, GROUPED_PAIR or GROUPED_ANY; GROUPED_NONE) that a call with these GroupedArgs or
    GroupedWgradArgs takes on a device of that many SMs; host code, no device."""
    call = _lib().moe_grouped_kernel if isinstance(args, GroupedArgs) else _lib().moe_grouped_wgrad_kernel
    return call(ctypes.byref(args), num_sms)


def grouped_matmul(x, w, offsets, rows=None, out_rows=None, w_layout="nk", act=None, out=None, out_dtype=None, stream=None,
                   workspace=None):
    """The products of ragged groups of rows with their experts' weights (moe_grouped_matmul).

    x [R, k] bf16 or fp16; w [E, n, k] ("nk") or [E, k, n] ("kn") of the same type; offsets [E + 1] int32: sorted
    row i of [offsets[e], offsets[e + 1]) gives out = W_e x[rows[i]] (x[i] without rows), written to
    out[out_rows[i]] (out[i] without out_rows).  act="swiglu" ("nk" only): the first n / 2 rows of W_e are gate, the others
    up, and out = silu(gate x) * (up x) has n / 2 columns.  Rows of out that no sorted row names are left as they
    were (undefined in a new tensor).  The gradient of x is the same call on dy with the other w_layout.
    workspace (with rows): uint8 device memory of grouped_workspace(m, k, E) bytes; new memory without it."""
    torch, L = _start()
    dev = _cuda(x, "x")
    (R, k), x_stride = _dense(x, "x", 2, dev)
    dt = _type(x, "x", fp32=False)
    (E, n, kw), w_stride = _dense(w, "w", 3, dev)
    if w.dtype is not x.dtype:
        raise ValueError("w: dtype %s, x has %s" % (w.dtype, x.dtype))
    ldw = _pitch(w_stride[1], n, kw)
    if w_layout == "nk":
        layout = GROUP_NK
    elif w_layout == "kn":
        layout, n, kw = GROUP_KN, kw, n
    else:
        raise ValueError("w_layout: 'nk' or 'kn', got %r" % (w_layout,))
    if kw != k:
        raise ValueError("x has %d columns, w takes %d" % (k, kw))
    if act is None:
        n_out, act = n, ACT_NONE
    elif act == "swiglu":
        n_out, act = n // 2, ACT_SWIGLU
    else:
        raise ValueError("act: None or 'swiglu', got %r" % (act,))
    i32 = torch.int32
    m = rows.shape[0] if rows is not None else out_rows.shape[0] if out_rows is not None else R
    if out is None:
        out, = _new(stream, dev, ((m, n_out), out_dtype or x.dtype))
    (N, cols), o_stride = _dense(out, "out", 2, dev)
    if cols != n_out or (out_dtype is not None and out.dtype != out_dtype):
        raise ValueError("out: %s %s, wanted %d columns" % (tuple(out.shape), out.dtype, n_out))
    ws = ws_bytes = rows_at = 0
    if rows is not None:
        rows_at = _flat(rows, "rows", i32, (m,), dev)
        ws, ws_bytes, _held = _space(workspace, 0 if workspace is not None else _matmul_space(m, k, E), stream, dev)
    if m:
        a = _pack_matmul(
            x.data_ptr(), w.data_ptr(), _flat(offsets, "offsets", i32, (E + 1,), dev), rows_at,
            0 if out_rows is None else _flat(out_rows, "out_rows", i32, (m,), dev), out.data_ptr(), R, _pitch(x_stride[0], R, k),
            ldw, w_stride[0] if E > 1 else 0, N, _pitch(o_stride[0], N, n_out), m, E, n, k, dt, _type(out, "out"), layout, act, ws,
            ws_bytes)
        _run("moe_grouped_matmul", L.moe_grouped_matmul, dev, stream, a)
    return out


def grouped_wgrad(dy, x, offsets, dy_rows=None, x_rows=None, out=None, out_dtype=None, stream=None, workspace=None):
    """The weights' gradient of grouped_matmul (moe_grouped_wgrad): out[e] = sum over the sorted rows i of
    expert e of dy[dy_rows[i]]^T x[x_rows[i]], [E, n, k] (zeros where a group is empty).

    dy [R, n] and x [S, k] bf16 or fp16 of one type (R = S without row numbers); offsets [E + 1] int32.  For "kn" weights exchange dy and x.
    workspace (with row numbers): uint8 device memory of grouped_wgrad_workspace(m, n) bytes for dy_rows and
    grouped_wgrad_workspace(m, k) for x_rows; new memory without it."""
    torch, L = _start()
    dev = _cuda(dy, "dy")
    (R, n), dy_stride = _dense(dy, "dy", 2, dev)
    dt = _type(dy, "dy", fp32=False)
    (S, k), x_stride = _dense(x, "x", 2, dev)
    if x.dtype is not dy.dtype:
        raise ValueError("x: dtype %s, dy has %s" % (x.dtype, dy.dtype))
    if offsets.dim() != 1 or offsets.shape[0] < 2:
        raise ValueError("offsets: one more than the groups, got %s" % (tuple(offsets.shape),))
    E, i32 = offsets.shape[0] - 1, torch.int32
    if dy_rows is None and x_rows is None and R != S:
        raise ValueError("dy has %d rows, x %d, and neither's are named by number" % (R, S))
    m = dy_rows.shape[0] if dy_rows is not None else x_rows.shape[0] if x_rows is not None else R
    if out is None:
        out, = _new(stream, dev, ((E, n, k), out_dtype or dy.dtype))
    shape, o_stride = _dense(out, "out", 3, dev)
    if shape != (E, n, k) or (out_dtype is not None and out.dtype != out_dtype):
        raise ValueError("out: %s %s, wanted %s" % (tuple(shape), out.dtype, (E, n, k)))
    ldw = _pitch(o_stride[1], n, k)
    dy_at = x_at = need = 0
    if dy_rows is not None:
        dy_at = _flat(dy_rows, "dy_rows", i32, (m,), dev)
        need = _wgrad_space(m, n)
    if x_rows is not None:
        x_at = _flat(x_rows, "x_rows", i32, (m,), dev)
        need += _wgrad_space(m, k)
    ws, ws_bytes, _held = _space(workspace, need, stream, dev) if need else (0, 0, None)
    a = _pack_wgrad(
        dy.data_ptr(), x.data_ptr(), _flat(offsets, "offsets", i32, (E + 1,), dev), dy_at, x_at, out.data_ptr(), R,
        _pitch(dy_stride[0], R, n), S, _pitch(x_stride[0], S, k), ldw, _pitch(o_stride[0], E, (n - 1) * ldw + k), m, E, n, k, dt,
        _type(out, "out"), ws, ws_bytes)
    _run("moe_grouped_wgrad", L.moe_grouped_wgrad, dev, stream, a)
    return out


def verify_draft(p, draft, u, q=None, lengths=None, out=None, stream=None):
    """Which drafted tokens stand, and the token drawn after them (moe_verify_draft).

    p [B, D + 1, V]: the target's probabilities (bf16, fp16 or fp32); draft [B, D] int32; u [B, D + 1] fp32 in [0, 1);
    q [B, D, V]: the draft's probabilities, of p's type, or None for drafts given without; lengths [B] int32:
    drafts per sequence (D without it).  Returns (accepted [B] int32, tokens [B, D + 1] int32): the accepted drafts,
    the drawn token, then -1."""
    torch, L = _start()
    dev = _cuda(p, "p")
    (B, D1, V), p_stride = _dense(p, "p", 3, dev)
    dt = _type(p, "p")
    D, i32 = D1 - 1, torch.int32
    q_at = q_seq = q_row = 0
    if q is not None:
        shape, stride = _dense(q, "q", 3, dev)
        if shape != (B, D, V) or q.dtype is not p.dtype:
            raise ValueError("q: %s %s, wanted %s %s" % (tuple(shape), q.dtype, (B, D, V), p.dtype))
        if D:
            q_at, q_seq, q_row = q.data_ptr(), _pitch(stride[0], B, D * V), _pitch(stride[1], D, V)
    out_shape = (B, D1)
    if out is None:
        out = tuple(_new(stream, dev, ((B,), i32), (out_shape, i32)))
    a = _pack_verify(
        p.data_ptr(), q_at, _flat(draft, "draft", i32, (B, D), dev) if D else 0,
        0 if lengths is None else _flat(lengths, "lengths", i32, (B,), dev), _flat(u, "u", torch.float32, out_shape, dev),
        _flat(out[0], "out: accepted", i32, (B,), dev), _flat(out[1], "out: tokens", i32, out_shape, dev),
        _pitch(p_stride[0], B, D1 * V), _pitch(p_stride[1], D1, V), q_seq, q_row, B, D, V, dt)
    _run("moe_verify_draft", L.moe_verify_draft, dev, stream, a)
    return out
