"""The argument checks of the operators around the products, and their plain 64-bit forms against closed forms and differences;
no GPU."""
import ctypes

import numpy as np
import pytest

from tests import rows_helpers as R
from tests.test_batch_host import M, P  # noqa: F401


def call(M, name, struct, base, over):
    a = dict(base, **over)
    return getattr(M.lib(), name)(ctypes.byref(struct(**a)), None)


NORM = dict(x=P, residual=None, gain=None, sum=None, out=P, out8=None, scale=None, rstd=None, ldx=64, ld_residual=64, ld_sum=64, ldo=64,
            ldo8=64, T=10, H=64, dtype=0, residual_dtype=0, gain_dtype=0, out_dtype=0, eps=1e-6)


@pytest.mark.parametrize("over", [
    dict(x=None), dict(out=None), dict(T=-1), dict(H=0), dict(H=32769, ldx=40000, ldo=40000), dict(dtype=3), dict(out_dtype=-1),
    dict(ldx=63), dict(ldo=63), dict(x=P + 1), dict(out=P + 1), dict(dtype=2, x=P + 2), dict(residual=P), dict(sum=P),
    dict(residual=P, sum=P, ld_residual=63), dict(residual=P, sum=P, ld_sum=63), dict(residual=P, sum=P, residual_dtype=3),
    dict(gain=P + 1), dict(gain=P, gain_dtype=5), dict(out8=P), dict(scale=P), dict(out8=P, scale=P, ldo8=63), dict(out8=P, scale=P + 2),
    dict(rstd=P + 2), dict(eps=-1.0), dict(eps=float("nan")), dict(eps=float("inf")), dict(ldx=2 ** 61)], ids=str)
def test_rms_norm_refuses(M, over):  # noqa: F811
    assert call(M, "moe_rms_norm", M.NormArgs, NORM, over) == M.EINVAL


def test_rows_calls_without_rows_do_nothing(M):  # noqa: F811
    assert call(M, "moe_rms_norm", M.NormArgs, NORM, dict(T=0, x=None, out=None)) == M.OK
    assert M.lib().moe_quantize_rows(None, 64, 0, 0, 64, None, 64, None, None) == M.OK
    assert call(M, "moe_combine_rows", M.CombineArgs, COMBINE, dict(T=0, weights=None, out=None)) == M.OK
    assert call(M, "moe_combine_rows_backward", M.CombineGradArgs, COMBINE_GRAD, dict(T=0, dout=None, dweights=None, weights=None)) == M.OK
    assert call(M, "moe_grouped_matmul8", M.Grouped8Args, PRODUCT8, dict(m=0)) == M.OK
    for name in ("moe_rms_norm", "moe_rms_norm_backward", "moe_combine_rows", "moe_combine_rows_backward", "moe_grouped_matmul8",
                 "moe_balanced_route", "moe_balanced_route_backward"):
        assert getattr(M.lib(), name)(None, None) == M.EINVAL


@pytest.mark.parametrize("over", [dict(x=None), dict(q=None), dict(s=None), dict(ld=63), dict(ldq=63), dict(dtype=4), dict(T=-1), dict(H=0),
                                  dict(H=40000, ld=40000, ldq=40000), dict(x=P + 1), dict(s=P + 1)], ids=str)
def test_quantize_rows_refuses(M, over):  # noqa: F811
    a = dict(x=P, ld=64, dtype=0, T=3, H=64, q=P, ldq=64, s=P)
    a.update(over)
    assert M.lib().moe_quantize_rows(*[a[n] for n in ("x", "ld", "dtype", "T", "H", "q", "ldq", "s")], None) == M.EINVAL


@pytest.mark.parametrize("over", [
    dict(dy=None), dict(h=None), dict(rstd=None), dict(dh=None), dict(T=-1), dict(H=0), dict(H=32769), dict(dy_dtype=3), dict(h_dtype=3),
    dict(dh_dtype=3), dict(ld_dy=63), dict(ld_h=63), dict(ld_dh=63), dict(dsum=P, ld_dsum=63), dict(dsum=P + 1), dict(gain=P + 1),
    dict(rstd=P + 1), dict(dgain=P + 2), dict(workspace=None), dict(workspace_bytes=100), dict(workspace=P + 4)], ids=str)
def test_rms_norm_backward_refuses(M, over):  # noqa: F811
    base = dict(dy=P, h=P, rstd=P, gain=P, dsum=None, dh=P, dgain=P, ld_dy=64, ld_h=64, ld_dsum=64, ld_dh=64, T=10, H=64, dy_dtype=0,
                h_dtype=0, gain_dtype=0, dsum_dtype=0, dh_dtype=0, workspace=P, workspace_bytes=1 << 20)
    assert call(M, "moe_rms_norm_backward", M.NormGradArgs, base, over) == M.EINVAL


COMBINE = dict(y=P, weights=P, places=None, residual=None, out=P, y_rows=30, ldy=64, ld_residual=64, ldo=64, T=10, k=3, H=64, dtype=0,
               out_dtype=0)


@pytest.mark.parametrize("over", [
    dict(y=None), dict(weights=None), dict(out=None), dict(T=-1), dict(k=0), dict(k=33, y_rows=1000), dict(H=0), dict(H=2 ** 24 + 1),
    dict(dtype=3), dict(out_dtype=3), dict(ldy=63), dict(ldo=63), dict(residual=P, ld_residual=63), dict(y_rows=29), dict(y_rows=-1),
    dict(y=P + 1), dict(out=P + 1), dict(residual=P + 1), dict(places=P + 2), dict(weights=P + 2), dict(T=2 ** 30, k=4, places=P)], ids=str)
def test_combine_rows_refuses(M, over):  # noqa: F811
    assert call(M, "moe_combine_rows", M.CombineArgs, COMBINE, over) == M.EINVAL


COMBINE_GRAD = dict(dout=P, y=P, weights=P, places=None, dy=P, dweights=P, y_rows=30, ld_dout=64, ldy=64, ld_dy=64, T=10, k=3, H=64,
                    dout_dtype=0, dtype=0)


@pytest.mark.parametrize("over", [
    dict(dout=None), dict(y=None), dict(weights=None), dict(dy=None), dict(dweights=None), dict(k=0), dict(k=33), dict(H=0),
    dict(dtype=3), dict(dout_dtype=3), dict(ld_dout=63), dict(ldy=63), dict(ld_dy=63), dict(y_rows=29), dict(dweights=P + 2),
    dict(places=P + 1), dict(dy=P + 1)], ids=str)
def test_combine_rows_backward_refuses(M, over):  # noqa: F811
    assert call(M, "moe_combine_rows_backward", M.CombineGradArgs, COMBINE_GRAD, over) == M.EINVAL


PRODUCT8 = dict(x=P, x_scale=P, w=P, w_scale=P, offsets=P, rows=None, out_rows=None, out=P, x_rows=10, ldx=64, ldw=64, w_stride=64 * 32,
                out_rows_n=10, ldo=32, m=10, groups=4, n=32, k=64, out_dtype=0, act=0)


@pytest.mark.parametrize("over", [
    dict(x=None), dict(x_scale=None), dict(w=None), dict(w_scale=None), dict(offsets=None), dict(out=None), dict(groups=0), dict(groups=1025),
    dict(m=-1), dict(m=11), dict(n=0), dict(k=0), dict(k=60), dict(k=72, ldx=80, ldw=80), dict(ldx=72), dict(ldw=72), dict(ldx=48),
    dict(ldw=48), dict(w_stride=64 * 32 - 16), dict(w_stride=64 * 32 + 8), dict(out_dtype=3), dict(act=2), dict(act=1, n=33), dict(ldo=31),
    dict(x=P + 8), dict(w=P + 8), dict(x_scale=P + 2), dict(w_scale=P + 2), dict(out=P + 1), dict(rows=P + 1), dict(out_rows=P + 2),
    dict(x_rows=9), dict(out_rows_n=9), dict(rows=P, workspace=P + 8, workspace_bytes=1), dict(rows=P, workspace_bytes=64)], ids=str)
def test_grouped_matmul8_refuses(M, over):  # noqa: F811
    assert call(M, "moe_grouped_matmul8", M.Grouped8Args, PRODUCT8, over) == M.EINVAL


def test_grouped_matmul8_kernels(M):  # noqa: F811
    def kernel(**over):
        return M.grouped_kernel(M.Grouped8Args(**dict(PRODUCT8, **over)), 152)
    big = dict(m=5000, x_rows=5000, out_rows_n=5000, n=512, w_stride=64 * 512, ldo=512)
    assert kernel() == M.GROUPED_FEW
    assert kernel(**big, k=4096, ldx=4096, ldw=4096) == M.GROUPED_NONE                # experts that overlap
    big.update(k=4096, ldx=4096, ldw=4096, w_stride=4096 * 512, n=2048, ldo=2048)
    big["w_stride"] = 4096 * 2048
    assert kernel(**big) == M.GROUPED_PAIR
    assert kernel(**dict(big, rows=P)) == M.GROUPED_NONE                              # rows by number want the workspace
    assert kernel(**dict(big, rows=P, workspace=P, workspace_bytes=M.grouped8_workspace(5000, 4096, 4))) == M.GROUPED_PAIR
    assert M.grouped8_workspace(100, 64, 1) == 100 * 64 and M.grouped8_workspace(8, 64, 256) == 0
    for bad in ((-1, 64, 1), (2 ** 30 + 1, 64, 1), (100, 0, 1), (100, 24, 1), (100, 64, 0), (100, 64, 1025)):
        assert M.grouped8_workspace(*bad) == 0


ROUTE = dict(logits=P, bias=None, idx=P, weights=P, offsets=P, rows=P, pairs=P, places=P, ld=8, T=1000, E=8, k=2, dtype=2, router=0, groups=4,
             keep=2, group_score=1, renormalize=1, scale=1.0, workspace=P, workspace_bytes=1 << 30)


@pytest.mark.parametrize("over", [
    dict(logits=None), dict(idx=None), dict(weights=None), dict(offsets=None), dict(rows=None), dict(pairs=None), dict(places=None),
    dict(ld=7), dict(dtype=3), dict(T=0), dict(E=0), dict(E=1025, ld=1025, groups=1, keep=1), dict(k=0), dict(k=9, keep=4), dict(k=5),
    dict(router=2), dict(groups=0), dict(groups=3), dict(groups=33, E=33, ld=33), dict(keep=0), dict(keep=5), dict(group_score=2),
    dict(scale=float("nan")), dict(scale=float("inf")), dict(logits=P + 2), dict(bias=P + 2), dict(places=P + 2), dict(workspace=None),
    dict(workspace_bytes=0), dict(workspace=P + 8), dict(T=2 ** 30, k=2)], ids=str)
def test_balanced_route_refuses(M, over):  # noqa: F811
    assert call(M, "moe_balanced_route", M.BalancedRouteArgs, ROUTE, over) == M.EINVAL


@pytest.mark.parametrize("over", [
    dict(dweights=None), dict(logits=None), dict(idx=None), dict(dlogits=None), dict(ld=7), dict(ldd=7), dict(T=0), dict(E=0), dict(k=0),
    dict(k=9), dict(dtype=3), dict(out_dtype=3), dict(router=2), dict(scale=float("inf")), dict(idx=P + 2), dict(dlogits=P + 2)], ids=str)
def test_balanced_route_backward_refuses(M, over):  # noqa: F811
    base = dict(dweights=P, logits=P, idx=P, dlogits=P, ld=8, ldd=8, T=10, E=8, k=2, dtype=2, out_dtype=2, router=0, renormalize=1, scale=1.0)
    assert call(M, "moe_balanced_route_backward", M.BalancedRouteGradArgs, base, over) == M.EINVAL


def test_packed_arguments_are_the_structures(M):  # noqa: F811
    from routed_expert_ffn_03_gb300 import batch, batch_rows as rows
    for cls, pack in ((M.Grouped8Args, batch._pack_matmul8), (M.BalancedRouteArgs, batch._pack_balanced),
                      (M.BalancedRouteGradArgs, batch._pack_balanced_grad), (M.NormArgs, rows._pack_norm),
                      (M.NormGradArgs, rows._pack_norm_grad), (M.CombineArgs, rows._pack_combine), (M.CombineGradArgs, rows._pack_combine_grad)):
        v = list(range(1, len(cls._fields_) + 1))
        assert ctypes.string_at(ctypes.byref(cls(*v)), ctypes.sizeof(cls)).startswith(pack(*v))
        assert len(pack(*v)) >= max(getattr(cls, n).offset + getattr(cls, n).size for n, _ in cls._fields_)


def test_binding_refuses_before_any_launch(M):  # noqa: F811
    import torch
    x, f = torch.zeros(4, 8, dtype=torch.bfloat16), torch.zeros(4, 2)
    for refused in (lambda: M.rms_norm(x), lambda: M.rms_norm_backward(x, x, f[:, 0]), lambda: M.quantize_rows(x),
                    lambda: M.combine_rows(x, f), lambda: M.combine_rows_backward(x, x, f), lambda: M.balanced_route(x, 2),
                    lambda: M.balanced_route_backward(f, x, f.int()),
                    lambda: M.grouped_matmul8(x, f, x, f, torch.zeros(3, dtype=torch.int32))):
        with pytest.raises(ValueError):
            refused()


# ---- the plain forms themselves

def test_plain_norm_by_hand():
    y, r = R.norm_ref(np.array([[3.0, 4.0], [0.0, 0.0]]), np.array([2.0, 1.0]), 0.5)
    np.testing.assert_allclose(r, [1 / np.sqrt(13), 1 / np.sqrt(0.5)])
    np.testing.assert_allclose(y, [[6 / np.sqrt(13), 4 / np.sqrt(13)], [0, 0]])
    R.check_eight(np.array([[448.0, -208.0, 2.0 ** -9]]), np.array([1.0]), np.array([[448.0, -207.0, 0.0016]]), 0)
    with pytest.raises(AssertionError):
        R.check_eight(np.array([[448.0, 1.125]]), np.array([1.0]), np.array([[448.0, 1.0]]), 0)
    with pytest.raises(AssertionError):
        R.check_eight(np.array([[224.0, 1.0]]), np.array([2.0]), np.array([[448.0, 2.0]]), 0)


@pytest.mark.parametrize("gain", [False, True])
def test_plain_norm_gradient_by_differences(gain):
    rng = np.random.default_rng(0)
    h, c, ds, eps = rng.normal(size=(3, 5)), rng.normal(size=(3, 5)), rng.normal(size=(3, 5)), 0.3
    g = rng.normal(size=5) if gain else None
    f = lambda h, g: float((R.norm_ref(h, g, eps)[0] * c).sum() + (h * ds).sum())  # noqa: E731
    (dh, _), (dg, _) = R.norm_grad_ref(c, h, R.norm_ref(h, g, eps)[1], g, ds)
    for i in np.ndindex(h.shape):
        d = np.zeros_like(h)
        d[i] = 1e-6
        assert abs((f(h + d, g) - f(h - d, g)) / 2e-6 - dh[i]) < 1e-8
    for i in range(5 if gain else 0):
        d = np.zeros(5)
        d[i] = 1e-6
        assert abs((f(h, g + d) - f(h, g - d)) / 2e-6 - dg[i]) < 1e-8


def test_plain_combine_and_its_gradient():
    rng = np.random.default_rng(1)
    y, w, c = rng.normal(size=(7, 3)), rng.normal(size=(2, 3)), rng.normal(size=(2, 3))
    places = np.array([[4, 0, -1], [6, 9, 2]])
    out, _ = R.combine_ref(y, w, places)
    np.testing.assert_allclose(out[0], w[0, 0] * y[4] + w[0, 1] * y[0])
    np.testing.assert_allclose(out[1], w[1, 0] * y[6] + w[1, 2] * y[2])
    (dy, written), (dw, _) = R.combine_grad_ref(c, y, w, places)
    assert written.tolist() == [True, False, True, False, True, False, True]
    f = lambda y, w: float((R.combine_ref(y, w, places)[0] * c).sum())  # noqa: E731
    for v, g in ((y, dy), (w, dw)):
        for i in np.ndindex(v.shape):
            d = np.zeros_like(v)
            d[i] = 1e-6
            a, b = (f(y + d, w), f(y - d, w)) if v is y else (f(y, w + d), f(y, w - d))
            assert abs((a - b) / 2e-6 - g[i]) < 1e-8


def test_plain_balanced_route_by_hand():
    l = np.log(np.array([[1.0, 2.0, 3.0, 4.0, 10.0, 1e-9]]))
    # without groups and bias: as group_route
    idx, w, off, rows, pairs, places = R.balanced_ref(l, 2, 0)
    assert idx.tolist() == [[4, 3]] and np.allclose(w, [[10 / 14, 4 / 14]]) and off.tolist() == [0, 0, 0, 0, 1, 2, 2]
    assert pairs.tolist() == [1, 0] and rows.tolist() == [0, 0] and places.tolist() == [[1, 0]]
    # groups of two by the sum of both: {1, 2}, {3, 4}, {10, 0}; two stay
    assert R.balanced_ref(l, 3, 0, groups=3, keep=2)[0].tolist() == [[4, 3, 2]]
    assert R.balanced_ref(l, 3, 0, groups=3, keep=2, top2=False)[0].tolist() == [[4, 3, 2]]
    assert R.balanced_ref(l, 2, 0, groups=3, keep=1)[0].tolist() == [[4, 5]]
    # a bias that lifts the first group, and does not enter the weights
    idx, w = R.balanced_ref(l, 2, 0, bias=[1, 0.9, 0, 0, 0, 0], groups=3, keep=1, renorm=False, scale=2.0)[:2]
    assert idx.tolist() == [[0, 1]] and np.allclose(w, [[2 / 20, 4 / 20]])
    # masks: a group with one expert left counts that one; everything masked
    inf = np.inf
    l = np.array([[0.0, -inf, -1.0, -1.0], [-inf] * 4])
    idx = R.balanced_ref(l, 2, 1, groups=2, keep=1)[0]
    assert idx.tolist() == [[2, 3], [-1, -1]]
    assert R.balanced_ref(l, 2, 1, groups=2, keep=1, top2=False)[0].tolist() == [[0, -1], [-1, -1]]


@pytest.mark.parametrize("kind", [0, 1])
@pytest.mark.parametrize("renorm", [True, False])
def test_plain_route_gradient_by_differences(kind, renorm):
    rng = np.random.default_rng(2)
    l, c = rng.normal(size=(3, 6)), rng.normal(size=(3, 2))
    idx = R.balanced_ref(l, 2, kind)[0]

    def f(l):
        s, logs = R.scores_of(l, kind)
        p = np.take_along_axis(s, idx, 1)
        return float(((p / p.sum(1, keepdims=True) if renorm else p) * 1.5 * c).sum())
    d, _ = R.balanced_grad_ref(c, l, idx, kind, renorm, 1.5)
    for i in np.ndindex(l.shape):
        e = np.zeros_like(l)
        e[i] = 1e-6
        assert abs((f(l + e) - f(l - e)) / 2e-6 - d[i]) < 1e-8
