"""Python binding of the batch operators on rows in include/moe.h: the root-mean-square norm with the residual's addition
and an output in 8 bits, its gradient, rows in 8 bits, the weighted sum of experts' results and its gradient.

Argument marshalling only, as in ``batch``.
"""
from __future__ import annotations

import ctypes
import functools
from typing import NamedTuple, Optional

from . import batch as B
from .batch import _cuda, _dense, _f, _flat, _i, _ll, _new, _packer, _pitch, _run, _space, _type, _vp


class NormArgs(ctypes.Structure):
    _fields_ = [(n, _vp) for n in ("x", "residual", "gain", "sum", "out", "out8", "scale", "rstd")] + \
        [(n, _ll) for n in ("ldx", "ld_residual", "ld_sum", "ldo", "ldo8")] + \
        [(n, _i) for n in ("T", "H", "dtype", "residual_dtype", "gain_dtype", "out_dtype")] + [("eps", _f)]


class NormGradArgs(ctypes.Structure):
    _fields_ = [(n, _vp) for n in ("dy", "h", "rstd", "gain", "dsum", "dh", "dgain")] + \
        [(n, _ll) for n in ("ld_dy", "ld_h", "ld_dsum", "ld_dh")] + \
        [(n, _i) for n in ("T", "H", "dy_dtype", "h_dtype", "gain_dtype", "dsum_dtype", "dh_dtype")] + \
        [("workspace", _vp), ("workspace_bytes", ctypes.c_size_t)]


class CombineArgs(ctypes.Structure):
    _fields_ = [(n, _vp) for n in ("y", "weights", "places", "residual", "out")] + \
        [(n, _ll) for n in ("y_rows", "ldy", "ld_residual", "ldo")] + [(n, _i) for n in ("T", "k", "H", "dtype", "out_dtype")]


class CombineGradArgs(ctypes.Structure):
    _fields_ = [(n, _vp) for n in ("dout", "y", "weights", "places", "dy", "dweights")] + \
        [(n, _ll) for n in ("y_rows", "ld_dout", "ldy", "ld_dy")] + [(n, _i) for n in ("T", "k", "H", "dout_dtype", "dtype")]


_pack_norm, _pack_norm_grad = _packer(NormArgs), _packer(NormGradArgs)
_pack_combine, _pack_combine_grad = _packer(CombineArgs), _packer(CombineGradArgs)


class Norm(NamedTuple):
    """What rms_norm returns; None for what was not asked for."""
    out: Optional[object]     # [T, H]
    sum: Optional[object]     # [T, H], with a residual
    rstd: Optional[object]    # [T] fp32
    out8: Optional[object]    # [T, H] float8_e4m3fn
    scale: Optional[object]   # [T] fp32, with out8


_NOTHING = Norm(None, None, None, None, None)
_WANT = frozenset(("out", "out8", "rstd"))


@functools.lru_cache(4096)
def _norm_grad_space(T, H):
    return B._lib().moe_rms_norm_backward_workspace(T, H)


def rms_norm_backward_workspace(T, H):
    """Bytes of workspace that rms_norm_backward needs for the gain's gradient at these sizes."""
    return int(B._lib().moe_rms_norm_backward_workspace(T, H))


def _rows(t, what, T, H, index):
    """(address, pitch, type) of a [T, H] tensor on the device."""
    shape, stride = _dense(t, what, 2, index)
    if shape != (T, H):
        raise ValueError("%s: %s, wanted %s" % (what, tuple(shape), (T, H)))
    return t.data_ptr(), _pitch(stride[0], T, H), _type(t, what)


def _rows8(t, what, T, H, index):
    shape, stride = _dense(t, what, 2, index)
    if shape != (T, H) or t.dtype is not B._torch.float8_e4m3fn:
        raise ValueError("%s: %s %s, wanted float8_e4m3fn %s" % (what, t.dtype, tuple(shape), (T, H)))
    return t.data_ptr(), _pitch(stride[0], T, H)


def _gain(gain, H, index):
    if gain is None:
        return 0, 0
    dt = _type(gain, "gain")
    return _flat(gain, "gain", gain.dtype, (H,), index), dt


def rms_norm(x, gain=None, residual=None, eps=1e-6, want=("out",), out_dtype=None, out=None, stream=None):
    """Root-mean-square norm of the rows of x, the residual added first (moe_rms_norm).

    x [T, H]; residual [T, H]; gain [H]; each bf16, fp16 or fp32.  h = x + residual in the residual's type is returned as sum;
    y = h / sqrt(mean h^2 + eps) * gain.  want: any of "out" (y in out_dtype, x's type without it), "out8" (y in 8 bits, float8_e4m3fn,
    with a scale for each row), "rstd" (for rms_norm_backward).  Returns a Norm.  out: a Norm whose tensors are written instead of new
    ones (for what it has; its sum may be the residual itself)."""
    torch, L = B._start()
    dev = _cuda(x, "x")
    (T, H), stride = _dense(x, "x", 2, dev)
    dt = _type(x, "x")
    f32 = torch.float32
    for w in want:
        if w not in _WANT:
            raise ValueError("want: any of 'out', 'out8', 'rstd', got %r" % (w,))
    old = out if out is not None else _NOTHING
    # what is new is made as it is passed on, so it needs no check
    new = []
    o = total = rstd = out8 = scale = None
    o_at = o_ld = o_dt = r_at = r_ld = r_dt = s_at = s_ld = d_at = q_at = q_ld = c_at = 0
    if "out" in want:
        if old.out is None:
            new.append(((T, H), out_dtype or x.dtype))
        else:
            o = old.out
            if out_dtype is not None and o.dtype != out_dtype:
                raise ValueError("out: %s, wanted %s" % (o.dtype, out_dtype))
            o_at, o_ld, o_dt = _rows(o, "out", T, H, dev)
    if residual is not None:
        r_at, r_ld, r_dt = _rows(residual, "residual", T, H, dev)
        if old.sum is None:
            new.append(((T, H), residual.dtype))
        else:
            total = old.sum
            s_at, s_ld, s_dt = _rows(total, "out: sum", T, H, dev)
            if s_dt != r_dt:
                raise ValueError("out: sum: %s, the residual has %s" % (total.dtype, residual.dtype))
    if "rstd" in want:
        if old.rstd is None:
            new.append(((T,), f32))
        else:
            rstd = old.rstd
            d_at = _flat(rstd, "out: rstd", f32, (T,), dev)
    if "out8" in want:
        if old.out8 is None:
            new.append(((T, H), torch.float8_e4m3fn))
        else:
            out8 = old.out8
            q_at, q_ld = _rows8(out8, "out: out8", T, H, dev)
        if old.scale is None:
            new.append(((T,), f32))
        else:
            scale = old.scale
            c_at = _flat(scale, "out: scale", f32, (T,), dev)
    if new:
        made = _new(stream, dev, *new)[::-1]
        if "out" in want and o is None:
            o = made.pop()
            o_at, o_ld, o_dt = o.data_ptr(), H, _type(o, "out")
        if residual is not None and total is None:
            total = made.pop()
            s_at, s_ld = total.data_ptr(), H
        if "rstd" in want and rstd is None:
            rstd = made.pop()
            d_at = rstd.data_ptr()
        if "out8" in want:
            if out8 is None:
                out8 = made.pop()
                q_at, q_ld = out8.data_ptr(), H
            if scale is None:
                scale = made.pop()
                c_at = scale.data_ptr()
    g_at, g_dt = _gain(gain, H, dev)
    if T:
        a = _pack_norm(x.data_ptr(), r_at, g_at, s_at, o_at, q_at, c_at, d_at, _pitch(stride[0], T, H), r_ld, s_ld, o_ld, q_ld, T, H, dt,
                       r_dt, g_dt, o_dt, eps)
        _run("moe_rms_norm", L.moe_rms_norm, dev, stream, a)
    return Norm(o, total, rstd, out8, scale)


def rms_norm_backward(dy, h, rstd, gain=None, dsum=None, out=None, out_dtype=None, workspace=None, stream=None):
    """The gradient of rms_norm (moe_rms_norm_backward): (dh, dgain), dh [T, H] for x and the residual both, dgain [H] fp32 (None
    without a gain).

    dy [T, H]; h: the sum that rms_norm returned (x where there was no residual); rstd [T] fp32; dsum [T, H]: the gradient that reaches
    the sum itself, added to dh.  dh has h's type unless out_dtype is given.  out: (dh, dgain) to write instead of new tensors; dh
    may be dy, h or dsum itself.  workspace (with a gain): uint8 device memory of rms_norm_backward_workspace(T, H) bytes."""
    torch, L = B._start()
    dev = _cuda(dy, "dy")
    (T, H), _ = _dense(dy, "dy", 2, dev)
    dh, dgain = out if out is not None else (None, None)
    if dh is None:
        dh, = _new(stream, dev, ((T, H), out_dtype or h.dtype))
    elif out_dtype is not None and dh.dtype != out_dtype:
        raise ValueError("out: %s, wanted %s" % (dh.dtype, out_dtype))
    if gain is None:
        dgain = None
    elif dgain is None:
        dgain, = _new(stream, dev, ((H,), torch.float32))
    y_at, y_ld, y_dt = _rows(dy, "dy", T, H, dev)
    h_at, h_ld, h_dt = _rows(h, "h", T, H, dev)
    o_at, o_ld, o_dt = _rows(dh, "out: dh", T, H, dev)
    s_at, s_ld, s_dt = _rows(dsum, "dsum", T, H, dev) if dsum is not None else (0, 0, 0)
    g_at, g_dt = _gain(gain, H, dev)
    ws, ws_bytes, _held = _space(workspace, _norm_grad_space(T, H), stream, dev) if gain is not None else (0, 0, None)
    if T or dgain is not None:
        a = _pack_norm_grad(
            y_at, h_at, _flat(rstd, "rstd", torch.float32, (T,), dev), g_at, s_at, o_at,
            0 if dgain is None else _flat(dgain, "out: dgain", torch.float32, (H,), dev), y_ld, h_ld, s_ld, o_ld, T, H, y_dt, h_dt, g_dt,
            s_dt, o_dt, ws, ws_bytes)
        _run("moe_rms_norm_backward", L.moe_rms_norm_backward, dev, stream, a)
    return dh, dgain


def quantize_rows(x, out=None, stream=None):
    """Rows in 8 bits (moe_quantize_rows): (x8 [T, H] float8_e4m3fn, scale [T] fp32) with x8 scale the nearest to x.

    x [T, H] bf16, fp16 or fp32 (weights [E, n, k] as x.view(E n, k)).  out: the two tensors to write instead of new ones."""
    torch, L = B._start()
    dev = _cuda(x, "x")
    (T, H), stride = _dense(x, "x", 2, dev)
    dt = _type(x, "x")
    if out is None:
        out = tuple(_new(stream, dev, ((T, H), torch.float8_e4m3fn), ((T,), torch.float32)))
        q_at, q_ld, scale = out[0].data_ptr(), H, out[1].data_ptr()
    else:
        q_at, q_ld = _rows8(out[0], "out: x8", T, H, dev)
        scale = _flat(out[1], "out: scale", torch.float32, (T,), dev)
    if T:
        _run("moe_quantize_rows", L.moe_quantize_rows, dev, stream, x.data_ptr(), _pitch(stride[0], T, H), dt, T, H, q_at, q_ld, scale)
    return out


def _places(places, TK, index):
    return 0 if places is None else _flat(places, "places", B._torch.int32, TK, index)


def combine_rows(y, weights, places=None, residual=None, out=None, out_dtype=None, stream=None):
    """The weighted sum of each token's k rows of y (moe_combine_rows): out[t] = sum_j weights[t, j] y[places[t, j]] (+ residual[t]).

    y [M, H] bf16, fp16 or fp32: the experts' results as the products left them; weights [T, k] fp32; places [T, k] int32
    (``balanced_route``; row t k + j without it); residual [T, H] of the output's type.  A place outside y, and a weight of 0, add
    nothing.  out [T, H] has the residual's type, else y's, unless out_dtype is given; it may be the residual itself."""
    torch, L = B._start()
    dev = _cuda(y, "y")
    (M, H), stride = _dense(y, "y", 2, dev)
    dt = _type(y, "y")
    if weights.dim() != 2:
        raise ValueError("weights: [T, k], got %s" % (tuple(weights.shape),))
    TK = tuple(weights.shape)
    T, k = TK
    if out is None:
        out, = _new(stream, dev, ((T, H), out_dtype or (y.dtype if residual is None else residual.dtype)))
        o_at, o_ld, o_dt = out.data_ptr(), H, _type(out, "out")
    else:
        if out_dtype is not None and out.dtype != out_dtype:
            raise ValueError("out: %s, wanted %s" % (out.dtype, out_dtype))
        o_at, o_ld, o_dt = _rows(out, "out", T, H, dev)
    r_at = r_ld = 0
    if residual is not None:
        r_at, r_ld, r_dt = _rows(residual, "residual", T, H, dev)
        if r_dt != o_dt:
            raise ValueError("residual: %s, the output has %s" % (residual.dtype, out.dtype))
    if T:
        a = _pack_combine(y.data_ptr(), _flat(weights, "weights", torch.float32, TK, dev), _places(places, TK, dev), r_at, o_at, M,
                          _pitch(stride[0], M, H), r_ld, o_ld, T, k, H, dt, o_dt)
        _run("moe_combine_rows", L.moe_combine_rows, dev, stream, a)
    return out


def combine_rows_backward(dout, y, weights, places=None, out=None, stream=None):
    """The gradient of combine_rows (moe_combine_rows_backward): (dy [M, H] of y's type, dweights [T, k] fp32); that of the residual is
    dout itself.  A weight of 0 has its gradient too, so masked pairs whose rows were never written want a place outside y (gradient 0),
    or their dweights is not to be used.  Rows of dy that no place names are left as they were (undefined in a new tensor).  out: the
    two tensors to write instead of new ones; dy may be y itself."""
    torch, L = B._start()
    dev = _cuda(y, "y")
    (M, H), stride = _dense(y, "y", 2, dev)
    dt = _type(y, "y")
    if weights.dim() != 2:
        raise ValueError("weights: [T, k], got %s" % (tuple(weights.shape),))
    TK = tuple(weights.shape)
    T, k = TK
    d_at, d_ld, d_dt = _rows(dout, "dout", T, H, dev)
    if out is None:
        out = tuple(_new(stream, dev, ((M, H), y.dtype), (TK, torch.float32)))
    dy, dweights = out
    dy_at, dy_ld, dy_dt = _rows(dy, "out: dy", M, H, dev)
    if dy_dt != dt:
        raise ValueError("out: dy: %s, y has %s" % (dy.dtype, y.dtype))
    if T:
        a = _pack_combine_grad(d_at, y.data_ptr(), _flat(weights, "weights", torch.float32, TK, dev), _places(places, TK, dev), dy_at,
                               _flat(dweights, "out: dweights", torch.float32, TK, dev), M, d_ld, _pitch(stride[0], M, H), dy_ld, T, k, H,
                               d_dt, dt)
        _run("moe_combine_rows_backward", L.moe_combine_rows_backward, dev, stream, a)
    return out
