"""Plain 64-bit forms of the batch operators and the bounds their kernels are held to."""
from __future__ import annotations

import numpy as np

# half a rounding step relative to the value, and the least step of subnormal results
HALF_STEP = {"bf16": 2.0 ** -8, "fp16": 2.0 ** -11, "fp32": 2.0 ** -24}
TINY = {"bf16": 2.0 ** -133, "fp16": 2.0 ** -25, "fp32": 2.0 ** -149}


def torch_type(name):
    import torch
    return {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}[name]


def make_groups(sizes, rng, first=0):
    """offsets int32 [E + 1] of groups of the given sizes, the first starting at `first`."""
    return np.concatenate([[first], first + np.cumsum(sizes)]).astype(np.int32)


def sum_bound(length, absum):
    """How far a sum of `length` products in fp32, added in any order, may be from the exact one: each of
    at most `length` additions (and the final one to a partial sum) is off by at most one step, 2^-23, of
    a partial sum no larger than the sum of the absolute products (a tensor core may truncate)."""
    return (length + 1) * 2.0 ** -23 * absum


def grouped_ref(x, w, offsets, rows=None, kn=False, swiglu=False):
    """(values, bounds) of the sorted rows, both fp64 [m][n_out]; NaN bounds where no group has the row."""
    m = len(rows) if rows is not None else x.shape[0]
    n = w.shape[2] if kn else w.shape[1]
    n_out = n // 2 if swiglu else n
    k = x.shape[1]
    val = np.full((m, n_out), np.nan)
    tol = np.full((m, n_out), np.nan)
    for e in range(w.shape[0]):
        a, z = int(offsets[e]), int(offsets[e + 1])
        if a >= z:
            continue
        r = np.arange(a, z) if rows is None else rows[a:z]
        inside = (r >= 0) & (r < x.shape[0])
        xe = np.where(inside[:, None], x[np.clip(r, 0, max(0, x.shape[0] - 1))], 0.0)
        we = w[e] if kn else w[e].T
        y = xe @ we
        t = sum_bound(k, np.abs(xe) @ np.abs(we))
        if swiglu:
            g, u, dg, du = y[:, :n_out], y[:, n_out:], t[:, :n_out], t[:, n_out:]
            s = g / (1 + np.exp(-g))
            y = s * u
            # |silu'| <= 1.1; exp, the division and two products are each within a few steps
            t = 1.1 * dg * (np.abs(u) + du) + np.abs(s) * du + 8 * 2.0 ** -23 * np.abs(y)
        val[a:z], tol[a:z] = y, t
    return val, tol


def wgrad_ref(dy, x, offsets, dy_rows=None, x_rows=None):
    E = len(offsets) - 1
    val = np.zeros((E, dy.shape[1], x.shape[1]))
    tol = np.zeros_like(val)

    def take(v, idx, a, z):
        r = np.arange(a, z) if idx is None else idx[a:z]
        inside = (r >= 0) & (r < v.shape[0])
        return np.where(inside[:, None], v[np.clip(r, 0, max(0, v.shape[0] - 1))], 0.0)

    for e in range(E):
        a, z = int(offsets[e]), int(offsets[e + 1])
        if a < z:
            d, xe = take(dy, dy_rows, a, z), take(x, x_rows, a, z)
            val[e] = d.T @ xe
            tol[e] = sum_bound(z - a, np.abs(d).T @ np.abs(xe))
    return val, tol


def check_close(got, val, tol, out_type):
    """got (a tensor) against the 64-bit value: the bound of its sum, and half a step of its type."""
    g = got.double().cpu().numpy()
    bound = tol + HALF_STEP[out_type] * (np.abs(val) + tol) + TINY[out_type]
    err = np.abs(g - val)
    bad = ~(err <= bound)
    assert not bad.any(), "%d of %d off, worst %.3g at %s: got %r, wanted %r within %.3g" % (
        bad.sum(), bad.size, np.nanmax(err / bound), np.argwhere(bad)[0], g[tuple(np.argwhere(bad)[0])],
        val[tuple(np.argwhere(bad)[0])], bound[tuple(np.argwhere(bad)[0])])


def route_ref(logits, k, kind):
    """(idx, weights fp64, offsets, rows, pairs) of logits fp64 [T][E]."""
    T, E = logits.shape
    big = float(np.finfo(np.float32).max)
    l = np.where(np.isnan(logits), -np.inf, np.minimum(logits, big))
    order = np.argsort(-l, axis=1, kind="stable")[:, :k]
    top = np.take_along_axis(l, order, 1)
    idx = np.where(np.isneginf(top), -1, order)
    z = np.minimum(top, 0) - np.log1p(np.exp(-np.abs(top))) if kind == 1 else top
    with np.errstate(invalid="ignore"):
        num = np.where(idx >= 0, np.exp(z - z[:, :1]), 0.0)
    den = num.sum(1, keepdims=True)
    w = np.where(den > 0, num / np.where(den > 0, den, 1), 0.0)
    flat = idx.reshape(-1)
    pairs = np.concatenate([np.flatnonzero(flat == e) for e in range(E)])
    offsets = np.concatenate([[0], np.cumsum(np.bincount(flat[flat >= 0], minlength=E))])
    fill = np.full(T * k - len(pairs), -1)
    return idx, w, offsets, np.concatenate([pairs // k, fill]), np.concatenate([pairs, fill])


def verify_ref(p, draft, u, q=None, lengths=None):
    """(accepted, tokens): comparisons of drafts in fractions; weights are fp32 differences, clamped, summed in
    exact integers of 2^-60 (Python's own)."""
    from fractions import Fraction
    B, D1, V = p.shape
    D = D1 - 1

    def clean(v):
        return np.clip(np.nan_to_num(v, nan=0.0, posinf=1.0, neginf=0.0), 0.0, 1.0)

    def ints(v):   # v 2^60, rounded (half to even), as Python integers: the product is exact in fp64
        return [int(a) for a in np.rint(clean(v) * 2.0 ** 60)]

    acc, tok = np.zeros(B, int), np.full((B, D1), -1)
    for b in range(B):
        L = D if lengths is None else min(max(int(lengths[b]), 0), D)
        r = L
        for i in range(L):
            t = int(draft[b, i])
            if 0 <= t < V:
                qv = 1.0 if q is None else float(clean(q[b, i, t]))
                if Fraction(float(clean(u[b, i]))) * Fraction(qv) < Fraction(float(clean(p[b, i, t]))):
                    continue
            r = i
            break
        base = ints(p[b, r])
        w = base
        if r < L:
            if q is None:
                w = [0 if v == draft[b, r] else a for v, a in enumerate(base)]
            else:
                with np.errstate(invalid="ignore"):
                    w = ints((p[b, r].astype(np.float32) - q[b, r].astype(np.float32)).astype(np.float64))
            if sum(w) == 0:
                w = base
        total = sum(w)
        t = -1
        if total:
            uu = float(clean(u[b, D]))
            thr = total - 1 if uu >= 1 else int(Fraction(uu) * total)
            run = 0
            for v, a in enumerate(w):
                run += a
                if run > thr:
                    t = v
                    break
        acc[b] = r
        tok[b, :r] = draft[b, :r]
        tok[b, r] = t
    return acc, tok
