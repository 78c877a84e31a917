"""balanced_route and its gradient against the plain 64-bit forms."""
import numpy as np
import pytest

from tests import batch_helpers as B
from tests import rows_helpers as R
from tests.test_gpu_grouped import M  # noqa: F401

pytestmark = pytest.mark.gpu


def check(M, logits, k, bias=None, router=0, groups=1, keep=1, group_score="top2", renormalize=True, scale=1.0, **kw):  # noqa: F811
    l = logits.double().cpu().numpy()
    ref = R.balanced_ref(l, k, router, None if bias is None else bias.double().cpu().numpy(), groups, keep, group_score == "top2",
                         renormalize, scale)
    got = [t.cpu().numpy() for t in M.balanced_route(logits, k, bias=bias, router=router, groups=groups, keep=keep, group_score=group_score,
                                                     renormalize=renormalize, scale=scale, **kw)]
    for i in (0, 2, 3, 4, 5):
        np.testing.assert_array_equal(got[i], ref[i])
    assert (np.abs(got[1] - ref[1]) <= R.weights_tol(l, ref[0], ref[1], scale)).all()
    assert (got[1][ref[0] < 0] == 0).all()
    return got


def random_logits(T, E, dtype, scale=1.5, seed=0):
    import torch
    g = torch.Generator(device="cuda").manual_seed(seed + T + E)
    return (scale * torch.randn(T, E, generator=g, device="cuda")).to(B.torch_type(dtype))


def random_bias(E, scale=0.05):
    import torch
    g = torch.Generator(device="cuda").manual_seed(E)
    return scale * torch.randn(E, generator=g, device="cuda")


CASES = [  # T, E, k, groups, keep
    (1, 256, 8, 8, 4), (1, 1, 1, 1, 1), (3, 8, 2, 1, 1), (5, 12, 3, 4, 2), (257, 160, 6, 8, 3), (1000, 64, 6, 32, 5), (33, 1024, 32, 32, 8),
    (700, 1000, 10, 8, 3), (64, 40, 32, 5, 4), (513, 256, 8, 8, 4), (2000, 256, 8, 8, 4), (200, 96, 10, 3, 2), (260, 384, 16, 1, 1),
    (100, 512, 8, 8, 8), (40, 30, 30, 30, 30), (300, 31, 5, 31, 7), (600, 768, 4, 12, 2)]


@pytest.mark.parametrize("dtype", ["fp32", "bf16", "fp16"])
@pytest.mark.parametrize("router", [0, 1])
@pytest.mark.parametrize("T,E,k,groups,keep", CASES)
def test_balanced_route(M, T, E, k, groups, keep, router, dtype):  # noqa: F811
    logits = random_logits(T, E, dtype)
    check(M, logits, k, random_bias(E), router, groups, keep, "top2", True, 2.5)
    check(M, logits, k, None, router, groups, keep, "max", False, 1.0)


@pytest.mark.parametrize("group_score", ["max", "top2"])
@pytest.mark.parametrize("renormalize", [True, False])
@pytest.mark.parametrize("with_bias", [True, False])
@pytest.mark.parametrize("router", [0, 1])
def test_balanced_route_options(M, router, with_bias, renormalize, group_score):  # noqa: F811
    for groups, keep in ((1, 1), (6, 2), (6, 6)):
        check(M, random_logits(70, 48, "fp32"), 5, random_bias(48) if with_bias else None, router, groups, keep, group_score, renormalize, -1.5)


def test_balanced_route_without_bias_or_groups_is_group_route(M):  # noqa: F811
    for router in (0, 1):
        l = random_logits(600, 200, "bf16")
        a, b = M.balanced_route(l, 7, router=router), M.group_route(l, 7, router=router)
        for i in (0, 2, 3, 4):
            assert (a[i] == b[i]).all()
        assert (a[1] - b[1]).abs().max() < 1e-6
        p, places = a[4].cpu().numpy(), a[5].cpu().numpy().reshape(-1)
        np.testing.assert_array_equal(p[places], np.arange(len(p)))


@pytest.mark.parametrize("dtype", ["fp32", "bf16", "fp16"])
@pytest.mark.parametrize("router", [0, 1])
@pytest.mark.parametrize("T,E,k,groups,keep", [(40, 64, 4, 8, 3), (1, 64, 4, 8, 3), (3000, 12, 6, 3, 2), (600, 12, 6, 1, 1)])
def test_balanced_route_ties_masks_and_extremes(M, T, E, k, groups, keep, router, dtype):  # noqa: F811
    import torch
    rng = np.random.default_rng(T)
    # ties everywhere, but no two sums of scores that are equal in the reals alone (as sigmoid(1) + sigmoid(-1) = 2 sigmoid(0))
    l = rng.choice(np.array([0.0, -0.0, 1.0, -1.5, 2.0], np.float32), (T, E))
    l[rng.random((T, E)) < 0.3] = -np.inf
    l[rng.random((T, E)) < 0.05] = np.nan
    l[rng.random((T, E)) < 0.02] = np.inf
    l[rng.random((T, E)) < 0.05] = np.finfo(np.float32).min
    l[:: 5] = -np.inf                                                                 # padding
    if T > 2:
        l[1] = np.finfo(np.float32).min
        l[2] = -2000.0                                                                # every sigmoid underflows
    logits = torch.from_numpy(l).cuda().to(B.torch_type(dtype))
    bias = torch.from_numpy(rng.choice(np.array([0.0, 0.25, -0.25, 0.25, 1.0, -3.0], np.float32), E)).cuda()
    for b in (None, torch.zeros(E, device="cuda")):
        check(M, logits, k, b, router, groups, keep, "top2")
        check(M, logits, k, b, router, groups, keep, "max", renormalize=False)
    check(M, logits, k, bias, router, groups, keep, "max")
    bias = bias + torch.from_numpy((0.01 * rng.normal(size=E)).astype(np.float32)).cuda()   # (with shared ones such sums occur)
    check(M, logits, k, bias, router, groups, keep, "top2")
    bias[3], bias[4], bias[5] = -np.inf, np.nan, np.inf
    check(M, logits, k, bias, router, groups, keep, "top2")


@pytest.mark.parametrize("router", [0, 1])
@pytest.mark.parametrize("E,k,groups,keep", [(64, 8, 1, 1), (64, 8, 8, 4), (300, 32, 1, 1), (1000, 6, 8, 2), (40, 5, 5, 2)])
def test_balanced_route_scores_a_rounding_apart(M, router, E, k, groups, keep):  # noqa: F811
    """Scores with the bias that differ by less than fp32 can tell, and some that are equal: the order of 64 bits decides."""
    import torch
    rng = np.random.default_rng(E + k)
    T = 200
    l = rng.choice(np.array([0.5, 1.0, 2.0], np.float32), (T, E)) + (rng.integers(0, 4, (T, E)) * 2.0 ** -22).astype(np.float32)
    bias = (rng.choice(np.array([0.0, 2.0 ** -24, 0.1]), E) + np.arange(E) * 2.0 ** -26).astype(np.float32)
    l[::9] = rng.normal(size=l[::9].shape)
    l[::7] -= 12.0                                  # small scores, where a bias of 2^-24 counts
    check(M, torch.from_numpy(l.astype(np.float32)).cuda(), k, torch.from_numpy(bias).cuda(), router, groups, keep, "top2")
    check(M, torch.from_numpy(l.astype(np.float32)).cuda(), k, torch.zeros(E, device="cuda"), router, groups, keep, "max")
    check(M, torch.from_numpy((l + 20).astype(np.float32)).cuda(), k, torch.from_numpy(bias).cuda(), router, groups, keep, "top2")


@pytest.mark.parametrize("router", [0, 1])
@pytest.mark.parametrize("E,k,groups,keep", [(40, 10, 4, 2), (16, 12, 8, 7), (256, 32, 8, 3), (64, 6, 32, 5)])
def test_balanced_route_biases_at_the_limits_of_fp32(M, router, E, k, groups, keep):  # noqa: F811
    """Two such biases together are past fp32; the group counts all the same, behind (or before) the others."""
    import torch
    rng = np.random.default_rng(E)
    lowest, l = float(np.finfo(np.float32).min), random_logits(64, E, "fp32")
    l[1:, : E // 2][torch.from_numpy(rng.random((63, E // 2)) < 0.8).cuda()] = -np.inf   # few of the unmasked are left
    bias = torch.zeros(E, device="cuda")
    bias[E // 2:] = lowest
    check(M, l, k, bias, router, groups, keep, "top2")
    check(M, l, k, bias.flip(0), router, groups, keep, "top2")
    check(M, l, k, -bias, router, groups, keep, "top2")
    bias[:] = torch.from_numpy((rng.choice([1.0, 0.7, 0.5, -0.4], E) * lowest).astype(np.float32)).cuda()
    check(M, l, k, bias, router, groups, keep, "top2")


def test_balanced_route_rows_apart_workspace_and_refusals(M):  # noqa: F811
    import torch
    big = random_logits(1300, 50, "bf16")
    ws = torch.empty(M.group_route_workspace(1300, 36, 4) + 64, dtype=torch.uint8, device="cuda")
    check(M, big[:, 3:39], 4, random_bias(36), 0, 4, 2, workspace=ws)
    with pytest.raises(M.MoeError):
        M.balanced_route(big, 4, workspace=ws[:16])
    with pytest.raises(M.MoeError):
        M.balanced_route(big, 4, groups=3)
    with pytest.raises(M.MoeError):
        M.balanced_route(big, 11, groups=5, keep=1)
    for bad in (dict(bias=random_bias(49)), dict(bias=random_bias(50).double()), dict(group_score="sum")):
        with pytest.raises(ValueError):
            M.balanced_route(big, 4, **bad)


def test_balanced_route_streams_and_capture(M):  # noqa: F811
    import torch
    a, bias = random_logits(2000, 96, "fp32"), random_bias(96)
    torch.cuda.synchronize()
    call = lambda **kw: M.balanced_route(a, 5, bias=bias, router=1, groups=4, keep=2, **kw)  # noqa: E731
    outs = [call(stream=s) for s in [torch.cuda.Stream() for _ in range(3)] for _ in range(2)]
    out = call()
    ws = torch.empty(M.group_route_workspace(2000, 96, 5), dtype=torch.uint8, device="cuda")
    torch.cuda.synchronize()
    for o in outs:
        assert all((x == y).all() for x, y in zip(o, out))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call(out=out, workspace=ws)
    a.copy_(random_logits(2000, 96, "fp32", seed=5))
    graph.replay()
    torch.cuda.synchronize()
    got = [t.clone() for t in out]
    assert all((x == y).all() for x, y in zip(got, call()))


def check_grad(M, logits, idx, dweights, router, renormalize, scale, out_type=None, **kw):  # noqa: F811
    got = M.balanced_route_backward(dweights, logits, idx, router=router, renormalize=renormalize, scale=scale,
                                    out_dtype=None if out_type is None else B.torch_type(out_type), **kw)
    ref = R.balanced_grad_ref(dweights.double().cpu().numpy(), logits.double().cpu().numpy(), idx.cpu().numpy(), router, renormalize, scale)
    name = {B.torch_type(n): n for n in ("bf16", "fp16", "fp32")}[got.dtype]
    B.check_close(got, *ref, name)
    return got


@pytest.mark.parametrize("dtype", ["fp32", "bf16", "fp16"])
@pytest.mark.parametrize("router", [0, 1])
@pytest.mark.parametrize("renormalize", [True, False])
@pytest.mark.parametrize("T,E,k", [(1, 1, 1), (1, 256, 8), (37, 8, 2), (100, 160, 6), (9, 1000, 32), (300, 65, 5), (20, 512, 16), (4, 1024, 3)])
def test_balanced_route_backward(M, T, E, k, renormalize, router, dtype):  # noqa: F811
    import torch
    logits = random_logits(T, E, dtype)
    idx = M.balanced_route(logits, k, bias=random_bias(E), router=router)[0]
    g = torch.Generator(device="cuda").manual_seed(3)
    check_grad(M, logits, idx, torch.randn(T, k, generator=g, device="cuda"), router, renormalize, 2.5)


@pytest.mark.parametrize("router", [0, 1])
@pytest.mark.parametrize("renormalize", [True, False])
def test_balanced_route_backward_masks_and_extremes(M, router, renormalize):  # noqa: F811
    import torch
    rng = np.random.default_rng(1)
    l = rng.normal(size=(40, 24)).astype(np.float32)
    l[rng.random(l.shape) < 0.4] = -np.inf
    l[3], l[4], l[5] = -np.inf, np.nan, -90.0
    l[6, :20] = -np.inf
    l[7] = 80.0
    logits = torch.from_numpy(l).cuda()
    idx = M.balanced_route(logits, 6, router=router, renormalize=renormalize)[0]
    dw = torch.from_numpy(rng.normal(size=(40, 6)).astype(np.float32)).cuda()
    dw[(idx < 0)] = float("nan")                   # of pairs that were masked: not used
    clean = torch.where(idx < 0, torch.zeros_like(dw), dw)
    got = M.balanced_route_backward(dw, logits, idx, router=router, renormalize=renormalize)
    assert (got == check_grad(M, logits, idx, clean, router, renormalize, 1.0)).all()
    assert (got[torch.isinf(logits) | torch.isnan(logits)] == 0).all()
    wild = idx.clone()
    wild[:, 0] = 24
    wild[:, 1] = 2 ** 31 - 1
    check_grad(M, logits, wild, clean, router, renormalize, 1.0)


def test_balanced_route_backward_rows_apart(M):  # noqa: F811
    import torch
    big = random_logits(30, 64, "bf16")
    logits = big[:, 3:50]
    idx = M.balanced_route(logits, 4)[0]
    out = torch.zeros(30, 60, device="cuda")
    check_grad(M, logits, idx, torch.randn(30, 4, device="cuda"), 0, False, 1.0, out=out[:, 5:52])
    assert (out[:, :5] == 0).all() and (out[:, 52:] == 0).all()
    with pytest.raises(ValueError):
        M.balanced_route_backward(torch.zeros(30, 5, device="cuda"), logits, idx)
    with pytest.raises(ValueError):
        M.balanced_route_backward(torch.zeros(30, 4, device="cuda"), logits, idx.long())


@pytest.mark.parametrize("router", [0, 1])
@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
def test_balanced_route_equal_logits(M, router, dtype):  # noqa: F811
    """A router that has not learned anything: every logit the same; biases all zero, all different, or of a few values."""
    import torch
    logits = torch.zeros(300, 64, device="cuda").to(B.torch_type(dtype))
    logits[7] = 3.0
    rng = np.random.default_rng(0)
    for bias in (None, torch.zeros(64, device="cuda"), random_bias(64),
                 torch.from_numpy(rng.choice(np.array([0.0, 0.125], np.float32), 64)).cuda()):
        for groups, keep in ((1, 1), (8, 3), (4, 3)):
            check(M, logits, 6, bias, router, groups, keep, "top2")
            check(M, logits, 6, bias, router, groups, keep, "max", renormalize=False)


@pytest.mark.parametrize("groups,keep", [(1, 1), (8, 4)])
@pytest.mark.parametrize("router", [0, 1])
def test_balanced_route_twins_beside_near_ones(M, router, groups, keep):  # noqa: F811
    """Experts with the same logit and bias beside one whose score differs by less than fp32 tells, above or below them."""
    import torch
    T, E = 400, 64
    rng = np.random.default_rng(3)
    l = rng.normal(size=(T, E)).astype(np.float32) - 4
    bias = np.zeros(E, np.float32)
    for t in range(T):
        g = rng.integers(0, groups) * (E // groups)
        at = g + rng.permutation(E // groups)[:5]
        l[t, at] = 1.0
        l[t, at[0]] = np.float32(1.0) + np.float32(2.0 ** -23) * rng.integers(-2, 3)
        l[t, at[1]] = np.float32(1.0) + np.float32(2.0 ** -23) * rng.integers(-2, 3)
    logits = torch.from_numpy(l).cuda()
    for k in (1, 2, 3, 4):
        check(M, logits, k, torch.from_numpy(bias).cuda(), router, groups, keep, "top2")
        check(M, logits, k, None, router, groups, keep, "top2")


@pytest.mark.parametrize("router", [0, 1])
@pytest.mark.parametrize("E", [8, 256, 300])
def test_balanced_route_best_expert_over_many_ranges(M, router, E):  # noqa: F811
    """The best score stands at the end of the range that keys are made of, another one for each token: it comes first."""
    import torch
    T = 1 << 20
    logits, bias = random_logits(T, E, "fp32"), random_bias(E)
    idx = M.balanced_route(logits, 2, bias=bias, router=router)[0]
    for t in range(0, T, 1 << 17):
        l = logits[t:t + (1 << 17)].double()
        c = (torch.sigmoid(l) if router else torch.softmax(l, 1)) + bias.double()
        top = c.topk(2, dim=1)
        # (where 64-bit scores lie closer than their own rounding, 2^-50, either is right)
        clear = top.values[:, 0] - top.values[:, 1] > 2.0 ** -45
        assert torch.equal(idx[t:t + (1 << 17), 0][clear], top.indices[:, 0][clear].int())
        assert int(clear.sum()) > (1 << 17) - 10


def test_balanced_route_without_tokens(M):  # noqa: F811
    """An empty share of a batch goes through selection, products, sum and gradient as any other."""
    import torch
    H, F, E, k = 64, 48, 8, 2
    x, wr = torch.empty(0, H, dtype=torch.bfloat16, device="cuda"), torch.randn(H, E, device="cuda")
    w1, w2 = torch.randn(E, F, H, device="cuda").bfloat16(), torch.randn(E, H, F, device="cuda").bfloat16()
    logits = x.float() @ wr
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    for stream in (None, side, side.cuda_stream):
        out = M.balanced_route(logits, k, bias=torch.zeros(E, device="cuda"), groups=4, keep=2, stream=stream)
        idx, w, offsets, rows, pairs, places = out
        torch.cuda.synchronize()
        assert [tuple(t.shape) for t in out] == [(0, k), (0, k), (E + 1,), (0,), (0,), (0, k)]
        assert [t.dtype for t in out] == [torch.int32, torch.float32] + [torch.int32] * 4 and (offsets == 0).all()
    old = tuple(torch.full_like(t, 5) for t in out)
    assert M.balanced_route(logits, k, out=old) is old and (old[2] == 0).all()
    y = M.grouped_matmul(M.grouped_matmul(x, w1, offsets, rows=rows), w2, offsets)
    assert M.combine_rows(y, w, places=places, residual=x).shape == (0, H)
    dy, dw = M.combine_rows_backward(x, y, w, places=places)
    dl = M.balanced_route_backward(dw, logits, idx)
    assert dl.shape == (0, E) and dl.dtype == torch.float32 and dy.shape == (0, H)
    with pytest.raises(ValueError):
        M.balanced_route(logits, k, out=old[:5] + (old[5].long(),))
    with pytest.raises(ValueError):
        M.balanced_route_backward(dw.double(), logits, idx)
