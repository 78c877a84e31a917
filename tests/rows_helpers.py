"""Plain 64-bit forms of the operators around the products, and the bounds their kernels are held to."""
from __future__ import annotations

import numpy as np

from tests.batch_helpers import HALF_STEP, TINY

U = 2.0 ** -24          # half a step of fp32


def round_type(v, name):
    """fp64 values rounded to bf16, fp16 or fp32 by way of fp32 (what an fp32 sum that is stored gives)."""
    import torch
    t = torch.from_numpy(np.asarray(v, np.float32))
    return t.to({"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}[name]).double().numpy()


def norm_ref(h, gain, eps):
    """(y, rstd) of rows h [T][H], gain [H] or None."""
    rstd = 1 / np.sqrt((h * h).mean(1) + eps)
    y = h * rstd[:, None]
    return (y if gain is None else y * gain), rstd


# rstd: the squares are summed by at most 32 additions a thread and 10 across them, all positive, so the sum is within 42 U of itself
# and its root within 21; the mean, eps and rsqrtf (2 steps) add 6.  y: two products more.
RSTD_TOL = 27 * U
Y_TOL = 29 * U


def check_norm(got, y, out_type):
    """got (fp64 array of a tensor of out_type) against y."""
    tol = Y_TOL * np.abs(y) + HALF_STEP[out_type] * np.abs(y) * (1 + Y_TOL) + TINY[out_type]
    assert (np.abs(got - y) <= tol).all(), np.max(np.abs(got - y) / tol)


def check_eight(q, scale, y, rel):
    """q e4m3 values, scale as the kernel gave it; rel: how far the kernel's y may be from y."""
    top = np.abs(y).max(1) if y.shape[1] else np.zeros(len(y))
    want = np.maximum(top / 448, 2.0 ** -100)
    assert (np.abs(scale - want) <= (rel + 2 * U) * want).all()
    v = y / scale[:, None]
    # a half step of e4m3 is 2^-4 of the value at most, 2^-10 where it is subnormal; two products and an inverse before it
    tol = np.maximum(2.0 ** -4 * np.abs(v), 2.0 ** -10) * (1 + 2.0 ** -15) + (rel + 4 * U) * np.abs(v)
    assert (np.abs(q - v) <= tol).all(), np.max(np.abs(q - v) / tol)
    # and no e4m3 number is nearer, up to that error
    a = np.abs(v)
    step = 2.0 ** (np.floor(np.log2(np.maximum(a, 2.0 ** -6))) - 3)
    near = np.minimum(np.rint(a / step) * step, 448)
    assert (np.abs(np.abs(q) - a) <= np.abs(near - a) + 2 * (rel + 4 * U) * a + 1e-30).all()


def norm_grad_ref(dy, h, rstd, gain, dsum):
    """((dh, its bound), (dgain, its bound)) without the rounding of dh."""
    T, H = h.shape
    n = h * rstd[:, None]
    d = dy if gain is None else dy * gain
    dot = (d * n).mean(1, keepdims=True)
    dh = rstd[:, None] * (d - n * dot)
    # d and n are one rounding off, their products' sum 42 more, its mean one: 46 U of the mean of absolute products
    tol = rstd[:, None] * (4 * U * (np.abs(d) + np.abs(n * dot)) + np.abs(n) * 46 * U * np.abs(d * n).mean(1, keepdims=True))
    if dsum is not None:
        dh = dh + dsum
        tol = tol + U * (np.abs(dh) + np.abs(dsum))
    dg = (dy * n).sum(0)
    # rows are added one after another within a block (304 at most, 8 warps each for short rows), then the blocks'
    return (dh, tol), (dg, (-(-T // 304) + 8 + 48 + 2) * U * np.abs(dy * n).sum(0))


def combine_ref(y, weights, places, residual=None):
    """(out, bound): y [M][H], weights [T][k], places [T][k] (outside y, or a weight of 0: nothing)."""
    T, k = weights.shape
    out, tol = np.zeros((T, y.shape[1])), np.zeros((T, y.shape[1]))
    for j in range(k):
        ok = (places[:, j] >= 0) & (places[:, j] < len(y)) & (weights[:, j] != 0)
        rows = np.where(ok[:, None], y[np.where(ok, places[:, j], 0)] if len(y) else 0.0, 0.0)
        p = np.where(ok, weights[:, j], 0.0)[:, None] * rows
        out += p
        tol += np.abs(p)
    if residual is not None:
        out, tol = out + residual, tol + np.abs(residual)
    return out, (k + 1) * U * tol


def combine_grad_ref(dout, y, weights, places):
    """((dy, written), (dweights, bound)); dy fp64 before its rounding."""
    T, k = weights.shape
    dy, written = np.zeros(y.shape), np.zeros(len(y), bool)
    dw, tol = np.zeros((T, k)), np.zeros((T, k))
    H = y.shape[1]
    for t in range(T):
        for j in range(k):
            r = places[t, j]
            if 0 <= r < len(y):
                dy[r] = weights[t, j] * dout[t]
                written[r] = True
                dw[t, j] = dout[t] @ y[r]
                tol[t, j] = np.abs(dout[t]) @ np.abs(y[r])
    return (dy, written), (dw, (H / 256 + 64) * U * tol)


def scores_of(l, kind):
    """Scores and their logarithms of cleaned logits [T][E] (-inf: masked)."""
    with np.errstate(over="ignore", invalid="ignore", divide="ignore"):
        if kind == 1:
            logs = np.minimum(l, 0) - np.log1p(np.exp(-np.abs(l)))
            return np.where(np.isneginf(l), 0.0, 1 / (1 + np.exp(-l))), logs
        m = l.max(1, keepdims=True)
        m = np.where(np.isneginf(m), 0.0, m)
        p = np.exp(l - m)
        z = p.sum(1, keepdims=True)
        z = np.where(z > 0, z, 1.0)
        return p / z, l - m - np.log(z)


def clean_logits(l):
    big = float(np.finfo(np.float32).max)
    return np.where(np.isnan(l), -np.inf, np.minimum(l, big))


def balanced_ref(logits, k, kind, bias=None, groups=1, keep=1, top2=True, renorm=True, scale=1.0):
    """(idx, weights, offsets, rows, pairs, places) of logits fp64 [T][E]."""
    T, E = logits.shape
    l = clean_logits(logits)
    s, logs = scores_of(l, kind)
    c = s if bias is None else s + clean_logits(np.asarray(bias, np.float64))[None]
    c = np.where(np.isneginf(l), -np.inf, c)
    kept = np.ones((T, E), bool)
    if keep < groups:
        g = -np.sort(-c.reshape(T, groups, -1), axis=2)
        best = g[..., 0].copy()
        if top2 and g.shape[2] > 1:
            best = np.where(np.isneginf(g[..., 1]), best, best + np.where(np.isneginf(g[..., 1]), 0, g[..., 1]))
        order = np.argsort(-best, axis=1, kind="stable")[:, :keep]
        in_group = np.zeros((T, groups), bool)
        np.put_along_axis(in_group, order, True, 1)
        in_group &= ~np.isneginf(best)
        kept = np.repeat(in_group, E // groups, axis=1)
    by = l if bias is None else c
    by = np.where(kept & ~np.isneginf(c), by, -np.inf)
    order = np.argsort(-by, axis=1, kind="stable")[:, :k]
    idx = np.where(np.isneginf(np.take_along_axis(by, order, 1)), -1, order)
    sel = np.maximum(idx, 0)
    with np.errstate(invalid="ignore", over="ignore"):
        z = np.where(idx >= 0, np.take_along_axis(l if kind == 0 else logs, sel, 1), -np.inf)
        if renorm:
            top = z.max(1, keepdims=True)
            num = np.exp(z - np.where(np.isneginf(top), 0, top))
            den = num.sum(1, keepdims=True)
            w = num / np.where(den > 0, den, 1)
        else:
            w = np.exp(np.where(idx >= 0, np.take_along_axis(logs, sel, 1), -np.inf))
    flat = idx.reshape(-1)
    pairs = np.concatenate([np.flatnonzero(flat == e) for e in range(E)])
    offsets = np.concatenate([[0], np.cumsum(np.bincount(flat[flat >= 0], minlength=E))])
    places = np.full(T * k, -1)
    places[pairs] = np.arange(len(pairs))
    fill = np.full(T * k - len(pairs), -1)
    return (idx, w * scale, offsets, np.concatenate([pairs // k, fill]), np.concatenate([pairs, fill]), places.reshape(T, k))


def weights_tol(logits, idx, w, scale):
    """A weight is e^d over a sum of them: d is off by a step of logits that large, exponentials, the sum (E / 32 additions a lane) and the
    division by a few."""
    l = np.clip(clean_logits(logits), -3.5e38, None)
    sel = np.take_along_axis(l, np.maximum(idx, 0), 1)
    rel = (4 * np.abs(sel) + 4 * np.abs(l).max(1, keepdims=True) + logits.shape[1] / 32 + idx.shape[1] + 24) * 2 * U
    return np.where(np.isfinite(rel), np.minimum(rel, 1.0), 1.0) * np.maximum(np.abs(w), abs(scale) * 2.0 ** -100) + 2.0 ** -126


def balanced_grad_ref(dweights, logits, idx, kind, renorm=True, scale=1.0):
    """(dlogits, bound) without the rounding to its type."""
    T, E = logits.shape
    l = clean_logits(logits)
    s, logs = scores_of(l, kind)
    ok = (idx >= 0) & (idx < E)
    sel = np.where(ok, idx, 0)
    ok &= ~np.isneginf(np.take_along_axis(l, sel, 1))
    v = np.where(ok, dweights * scale, 0.0)
    ls = np.take_along_axis(l, sel, 1)
    rho = (4 * np.abs(np.where(np.isfinite(l), l, 0)).max(1, keepdims=True) + E / 32 + idx.shape[1] + 32) * 2 * U
    if renorm:
        z = np.where(ok, ls if kind == 0 else np.take_along_axis(logs, sel, 1), -np.inf)
        top = z.max(1, keepdims=True)
        num = np.exp(z - np.where(np.isneginf(top), 0, top))
        den = num.sum(1, keepdims=True)
        r = num / np.where(den > 0, den, 1)
        d = r * (v - (r * v).sum(1, keepdims=True))
        t = r * (np.abs(v) + (r * np.abs(v)).sum(1, keepdims=True))
        if kind == 1:
            left = 1 / (1 + np.exp(np.minimum(ls, 700)))
            d, t = d * left, t * left
        dense, dt = np.zeros((T, E)), np.zeros((T, E))
    elif kind == 1:
        p = np.take_along_axis(s, sel, 1)
        d = v / (2 + np.exp(np.minimum(ls, 700)) + np.exp(np.minimum(-ls, 700)))
        t = np.abs(d)
        dense, dt = np.zeros((T, E)), np.zeros((T, E))
        del p
    else:
        p = np.where(ok, np.take_along_axis(s, sel, 1), 0.0)
        total, mass = (p * v).sum(1, keepdims=True), (p * np.abs(v)).sum(1, keepdims=True)
        d, t = p * (v - total), p * (np.abs(v) + mass)
        dense, dt = -s * total, s * mass
    for t_ in range(T):
        for j in range(idx.shape[1]):
            if 0 <= idx[t_, j] < E:
                dense[t_, idx[t_, j]], dt[t_, idx[t_, j]] = (d[t_, j], t[t_, j]) if ok[t_, j] else (0.0, 0.0)
    return dense, 4 * rho * dt + 1e-38
