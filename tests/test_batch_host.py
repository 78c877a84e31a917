"""The batch operators' argument checks, and their plain 64-bit forms against closed forms; no GPU."""
import ctypes

import numpy as np
import pytest

from tests import batch_helpers as B


@pytest.fixture(scope="module")
def M():
    from routed_expert_ffn_03_gb300 import build
    build.build()
    import routed_expert_ffn_03_gb300 as M
    M.batch._lib()
    return M


P = 4096   # an address that no refused call touches


def matmul_args(M, **over):
    a = dict(x=P, w=P, offsets=P, rows=None, out_rows=None, out=P, x_rows=10, ldx=64, ldw=64, w_stride=64 * 32,
             out_rows_n=10, ldo=32, m=10, groups=4, n=32, k=64, dtype=0, out_dtype=0, layout=0, act=0)
    a.update(over)
    return M.GroupedArgs(**a)


@pytest.mark.parametrize("over", [
    dict(x=None), dict(w=None), dict(offsets=None), dict(out=None), dict(groups=0), dict(groups=1025), dict(m=-1),
    dict(m=2 ** 30 + 1), dict(n=0), dict(k=0), dict(n=2 ** 24 + 1), dict(dtype=2), dict(dtype=7), dict(out_dtype=3),
    dict(layout=2), dict(act=2), dict(act=1, n=33, ldo=33), dict(act=1, layout=1), dict(ldx=63), dict(ldw=63),
    dict(layout=1, ldw=31), dict(ldo=31), dict(m=11), dict(x_rows=9), dict(out_rows_n=9), dict(x=P + 1), dict(w=P + 1),
    dict(out_dtype=2, out=P + 2), dict(offsets=P + 2), dict(rows=P + 1), dict(out_rows=P + 3), dict(w_stride=-1),
    dict(x_rows=-1, rows=P), dict(ldx=2 ** 61),
    dict(rows=P, workspace=P + 8, workspace_bytes=1), dict(rows=P, workspace_bytes=64)], ids=str)
def test_grouped_matmul_refuses(M, over):
    assert M.lib().moe_grouped_matmul(ctypes.byref(matmul_args(M, **over)), None) == M.EINVAL


def test_grouped_matmul_without_rows_does_nothing(M):
    assert M.lib().moe_grouped_matmul(ctypes.byref(matmul_args(M, m=0)), None) == M.OK
    assert M.lib().moe_grouped_matmul(None, None) == M.EINVAL


@pytest.mark.parametrize("over", [
    dict(dy=None), dict(x=None), dict(offsets=None), dict(dw=None), dict(groups=0), dict(groups=2000), dict(m=-1),
    dict(n=0), dict(k=0), dict(dtype=2), dict(out_dtype=5), dict(lddy=31), dict(ldx=63), dict(lddw=63), dict(m=11),
    dict(dw_stride=64 * 32 - 1), dict(dy=P + 1), dict(dw=P + 1), dict(dy_rows=P + 2), dict(x_rows=P + 1)], ids=str)
def test_grouped_wgrad_refuses(M, over):
    a = dict(dy=P, x=P, offsets=P, dy_rows=None, x_rows=None, dw=P, dy_rows_n=10, lddy=32, x_rows_n=10, ldx=64, lddw=64,
             dw_stride=64 * 32, m=10, groups=4, n=32, k=64, dtype=0, out_dtype=0)
    a.update(over)
    assert M.lib().moe_grouped_wgrad(ctypes.byref(M.GroupedWgradArgs(**a)), None) == M.EINVAL


@pytest.mark.parametrize("over", [
    dict(logits=None), dict(idx=None), dict(pairs=None), dict(ld=7), dict(dtype=3), dict(T=0), dict(E=0, ld=8),
    dict(E=1025, ld=1025), dict(k=0), dict(k=9), dict(T=2 ** 30, k=4), dict(router=2), dict(logits=P + 2), dict(idx=P + 1),
    dict(ws=None), dict(ws=P + 8), dict(ws_bytes=0)], ids=str)
def test_group_route_refuses(M, over):
    a = dict(logits=P, ld=8, dtype=2, T=1000, E=8, k=2, router=0, idx=P, weights=P, offsets=P, rows=P, pairs=P, ws=P,
             ws_bytes=1 << 30)
    a.update(over)
    assert M.group_route_workspace(2000, 8, 2) > 0
    assert M.lib().moe_group_route(*[a[n] for n in ("logits", "ld", "dtype", "T", "E", "k", "router", "idx", "weights", "offsets",
                                                    "rows", "pairs", "ws", "ws_bytes")], None) == M.EINVAL


def test_packed_arguments_are_the_structures(M):
    """The packed form that the binding passes has the structures' layout."""
    from routed_expert_ffn_03_gb300 import batch
    for cls, pack in ((M.GroupedArgs, batch._pack_matmul), (M.GroupedWgradArgs, batch._pack_wgrad), (M.VerifyArgs, batch._pack_verify)):
        v = list(range(1, len(cls._fields_) + 1))
        assert ctypes.string_at(ctypes.byref(cls(*v)), ctypes.sizeof(cls)).startswith(pack(*v))
        assert len(pack(*v)) >= max(getattr(cls, n).offset + getattr(cls, n).size for n, _ in cls._fields_)


def test_grouped_workspaces(M):
    assert M.grouped_workspace(100, 64, 1) == 100 * 64 * 2 and M.grouped_workspace(100, 65, 1) == 100 * 72 * 2
    assert M.grouped_workspace(8, 64, 256) == 0          # few rows are read where they are
    assert M.grouped_wgrad_workspace(8, 64) == 8 * 64 * 2
    for bad in ((-1, 64, 1), (2 ** 30 + 1, 64, 1), (100, 0, 1), (100, 64, 0), (100, 64, 1025)):
        assert M.grouped_workspace(*bad) == 0


def test_group_route_workspace_of_bad_sizes(M):
    for bad in ((0, 8, 2), (10, 0, 1), (10, 1025, 2), (10, 8, 9), (10, 64, 33), (2 ** 30, 8, 4)):
        assert M.group_route_workspace(*bad) == 0


@pytest.mark.parametrize("over", [
    dict(p=None), dict(u=None), dict(accepted=None), dict(tokens=None), dict(draft=None), dict(B=0), dict(D=-1), dict(D=32),
    dict(V=0), dict(V=2 ** 30 + 1), dict(dtype=3), dict(p_row=99), dict(p_seq=399), dict(q=P, q_row=99, q_seq=1000),
    dict(q=P, q_row=100, q_seq=299), dict(p=P + 2), dict(u=P + 2), dict(lengths=P + 1)], ids=str)
def test_verify_draft_refuses(M, over):
    a = dict(p=P, q=None, draft=P, lengths=None, u=P, accepted=P, tokens=P, p_seq=400, p_row=100, q_seq=0, q_row=0, B=2, D=3,
             V=100, dtype=2)
    a.update(over)
    assert M.lib().moe_verify_draft(ctypes.byref(M.VerifyArgs(**a)), None) == M.EINVAL


def test_binding_refuses_before_any_launch(M):
    import torch
    x, w = torch.zeros(4, 8, dtype=torch.bfloat16), torch.zeros(2, 6, 8, dtype=torch.bfloat16)
    o = torch.zeros(3, dtype=torch.int32)
    with pytest.raises(ValueError):
        M.grouped_matmul(x, w, o)              # not on a CUDA device
    with pytest.raises(ValueError):
        M.grouped_wgrad(x, x, o)
    with pytest.raises(ValueError):
        M.group_route(torch.zeros(2, 4), 2)
    with pytest.raises(ValueError):
        M.verify_draft(torch.zeros(1, 2, 4), torch.zeros(1, 1, dtype=torch.int32), torch.zeros(1, 2))


# ---- the plain forms themselves

def test_plain_products_against_hand_sums():
    x = np.array([[1.0, 2.0], [3.0, -1.0], [0.5, 4.0]])
    w = np.array([[[1.0, 0.0], [0.0, 1.0]], [[2.0, 1.0], [-1.0, 1.0]]])
    y, _ = B.grouped_ref(x, w, [0, 1, 3])
    np.testing.assert_array_equal(y, [[1, 2], [5, -4], [5, 3.5]])
    y, _ = B.grouped_ref(x, w, [0, 1, 3], kn=True)
    np.testing.assert_array_equal(y, [[1, 2], [7, 2], [-3, 4.5]])
    y, _ = B.grouped_ref(x, w, [0, 0, 2], rows=np.array([2, 9, 0]))
    np.testing.assert_array_equal(y[:2], [[5, 3.5], [0, 0]])
    assert np.isnan(y[2]).all()
    s = B.grouped_ref(x, w, [0, 1, 3], swiglu=True)[0]
    np.testing.assert_allclose(s[1, 0], 5 / (1 + np.exp(-5)) * -4)
    d, _ = B.wgrad_ref(np.array([[1.0], [2.0], [3.0]]), x, [0, 2, 2])
    np.testing.assert_array_equal(d, [[[7, 0]], [[0, 0]]])


def test_plain_input_gradient_by_differences():
    rng = np.random.default_rng(0)
    x, w, c = rng.normal(size=(5, 3)), rng.normal(size=(2, 4, 3)), rng.normal(size=(5, 4))
    off, h = [0, 2, 5], 1e-6
    f = lambda x, w: float((B.grouped_ref(x, w, off)[0] * c).sum())  # noqa: E731
    dx, dw = B.grouped_ref(c, w, off, kn=True)[0], B.wgrad_ref(c, x, off)[0]
    for i in np.ndindex(x.shape):
        d = np.zeros_like(x)
        d[i] = h
        assert abs((f(x + d, w) - f(x - d, w)) / (2 * h) - dx[i]) < 1e-7
    for i in np.ndindex(w.shape):
        d = np.zeros_like(w)
        d[i] = h
        assert abs((f(x, w + d) - f(x, w - d)) / (2 * h) - dw[i]) < 1e-7


def test_plain_route_masks_ties_and_weights():
    inf = np.inf
    l = np.array([[0.0, 1.0, 1.0, -inf], [-inf] * 4, [np.nan, -1.0, -inf, -inf], [inf, 5.0, inf, -0.0]])
    idx, w, off, rows, pairs = B.route_ref(l, 2, 0)
    np.testing.assert_array_equal(idx, [[1, 2], [-1, -1], [1, -1], [0, 2]])
    np.testing.assert_allclose(w, [[0.5, 0.5], [0, 0], [1, 0], [0.5, 0.5]])
    np.testing.assert_array_equal(off, [0, 1, 3, 5, 5])
    np.testing.assert_array_equal(pairs, [6, 0, 4, 1, 7, -1, -1, -1])
    np.testing.assert_array_equal(rows, [3, 0, 2, 0, 3, -1, -1, -1])
    w = B.route_ref(np.array([[-2000.0, -2000.0, -2001.0]]), 3, 1)[1]
    np.testing.assert_allclose(w[0], np.exp([0, 0, -1]) / np.exp([0, 0, -1]).sum())


def test_plain_verify_by_hand():
    p = np.array([[[0.5, 0.25, 0.25], [0.0, 1.0, 0.0]]])
    q = np.array([[[1.0, 0.0, 0.0]]])
    d = np.array([[0]])
    assert [v.tolist() for v in B.verify_ref(p, d, np.array([[0.4, 0.0]]), q)] == [[1], [[0, 1]]]
    assert [v.tolist() for v in B.verify_ref(p, d, np.array([[0.5, 0.49]]), q)] == [[0], [[1, -1]]]
    assert [v.tolist() for v in B.verify_ref(p, d, np.array([[0.5, 0.5]]), q)] == [[0], [[2, -1]]]
    # the same without probabilities, and a residual with nothing left
    assert [v.tolist() for v in B.verify_ref(p, d, np.array([[0.5, 0.5]]))] == [[0], [[2, -1]]]
    assert [v.tolist() for v in B.verify_ref(np.array([[[0.5, 0.0], [1, 0]]]), d, np.array([[0.5, 0.9]]),
                                             np.array([[[1.0, 0.0]]]))] == [[0], [[0, -1]]]


def test_plain_verify_keeps_the_target_distribution():
    """Over a grid of random numbers the first token's frequencies are the target's (the point of the method)."""
    p = np.array([0.1, 0.2, 0.3, 0.4])
    q = np.array([0.4, 0.3, 0.2, 0.1])
    n = 40
    grid = (np.arange(n) + 0.5) / n
    freq = np.zeros(4)
    for t in range(4):
        for a in grid:
            u = np.stack([np.full(n, a), grid], 1)
            acc, tok = B.verify_ref(np.tile(np.stack([p, p]), (n, 1, 1)), np.full((n, 1), t), u, np.tile(q, (n, 1, 1)))
            freq += q[t] * np.bincount(tok[:, 0], minlength=4) / n ** 2
    np.testing.assert_allclose(freq, p, atol=4 * 2 / n)   # each border cuts a grid cell: 2/n per draft at most
