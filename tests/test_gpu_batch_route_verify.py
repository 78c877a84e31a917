"""group_route and verify_draft against the plain 64-bit forms, and the batch operators used together."""
import numpy as np
import pytest

from tests import batch_helpers as B
from tests.test_gpu_grouped import M, dev, values  # noqa: F401

pytestmark = pytest.mark.gpu


def check_route(M, logits, k, kind, **kw):
    """logits: a device tensor.  Whole numbers equal; weights within 16 steps of fp32 (exp and log1p within a
    few steps each of values no larger than the logits' differences, which are exact to half a step of the
    difference: see the bound)."""
    l = logits.double().cpu().numpy()
    idx, w, off, rows, pairs = B.route_ref(l, k, kind)
    g = [t.cpu().numpy() for t in M.group_route(logits, k, router=kind, **kw)]
    np.testing.assert_array_equal(g[0], idx)
    np.testing.assert_array_equal(g[2], off)
    np.testing.assert_array_equal(g[3], rows)
    np.testing.assert_array_equal(g[4], pairs)
    # a weight exp(d)/sum: d = z_j - z_0 is off by at most a step of z (|z| 2^-23), which the exponential passes on
    # relative to the weight; exp, log1p, the sum of k and the division add a few steps
    top = np.where(idx >= 0, np.take_along_axis(np.nan_to_num(l, nan=0, posinf=3.5e38, neginf=0), np.maximum(idx, 0), 1), 0)
    with np.errstate(over="ignore", invalid="ignore"):
        rel = (4 * np.abs(top) + 4 * np.abs(top[:, :1]) + k + 16) * 2.0 ** -23
        tol = np.where(w > 0, np.minimum(rel, 1.0) * np.maximum(w, w.max(1, keepdims=True) * 2.0 ** -100), 2.0 ** -126)
    assert (np.abs(g[1] - w) <= tol).all(), np.abs(g[1] - w).max()
    return g


@pytest.mark.parametrize("dtype", ["fp32", "bf16", "fp16"])
@pytest.mark.parametrize("kind", [0, 1])
@pytest.mark.parametrize("T,E,k", [(1, 256, 8), (1, 1, 1), (3, 8, 2), (4, 5, 5), (31, 33, 4), (257, 384, 16), (1000, 64, 6),
                                   (33, 1024, 32), (5000, 17, 3), (700, 1000, 10), (64, 40, 32), (65, 256, 8), (200, 96, 10),
                                   (512, 512, 4), (513, 40, 8), (256, 1000, 8), (1111, 256, 9)])
def test_route(M, T, E, k, kind, dtype):
    import torch
    g = torch.Generator(device="cuda").manual_seed(T + E)
    logits = (2 * torch.randn(T, E, generator=g, device="cuda")).to(B.torch_type(dtype))
    check_route(M, logits, k, kind)


@pytest.mark.parametrize("kind", [0, 1])
@pytest.mark.parametrize("dtype", ["fp32", "bf16", "fp16"])
@pytest.mark.parametrize("T,E,k", [(40, 64, 4), (1, 64, 4), (3000, 12, 6)])
def test_route_ties_masks_and_extremes(M, T, E, k, kind, dtype):
    import torch
    rng = np.random.default_rng(T)
    l = rng.choice(np.array([0.0, -0.0, 1.0, -1.0, 2.0], np.float32), (T, E))          # ties everywhere
    l[rng.random((T, E)) < 0.3] = -np.inf
    l[rng.random((T, E)) < 0.05] = np.nan
    l[rng.random((T, E)) < 0.02] = np.inf
    l[rng.random((T, E)) < 0.05] = np.finfo(np.float32).min
    l[:: 5] = -np.inf                                                                    # padding
    if T > 2:
        l[1] = np.finfo(np.float32).min
        l[2] = -2000.0                                                                   # every sigmoid underflows
    check_route(M, torch.from_numpy(l).cuda().to(B.torch_type(dtype)), k, kind)


@pytest.mark.parametrize("T,E,k", [(300, 64, 8), (300, 200, 9), (40, 1000, 12), (300, 300, 32), (300, 32, 32), (50, 33, 32)])
def test_route_fp32_neighbours_a_few_bits_apart(M, T, E, k):
    """fp32 logits that share their leading bits: within the selection, across its end, and equal ones."""
    import torch
    rng = np.random.default_rng(E)
    base = rng.choice(np.array([1.0, 1.0 + 2.0 ** -13, 2.5, -0.75], np.float32), (T, E))
    l = base + (rng.integers(0, 6, (T, E)) * 2.0 ** -22).astype(np.float32)
    l[::7, : E // 2] = 0.0
    l[::11] = rng.normal(size=l[::11].shape)
    check_route(M, torch.from_numpy(l.astype(np.float32)).cuda(), k, 0)


def test_route_everything_masked(M):
    import torch
    g = check_route(M, torch.full((50, 16), -np.inf, device="cuda"), 3, 0)
    assert (g[2] == 0).all() and (g[4] == -1).all()


def test_route_rows_apart_and_workspace(M):
    import torch
    g = torch.Generator(device="cuda").manual_seed(1)
    big = torch.randn(1300, 50, generator=g, device="cuda").bfloat16()
    ws = torch.empty(M.group_route_workspace(1300, 37, 4) + 64, dtype=torch.uint8, device="cuda")
    check_route(M, big[:, 3:40], 4, 0, workspace=ws)
    with pytest.raises(M.MoeError):
        M.group_route(big, 4, workspace=ws[:16])
    with pytest.raises(M.MoeError):
        M.group_route(big, 33)
    with pytest.raises(ValueError):
        M.group_route(big.double(), 4)


def test_route_streams_and_capture(M):
    import torch
    g = torch.Generator(device="cuda").manual_seed(1)
    a = torch.randn(2000, 96, generator=g, device="cuda")
    torch.cuda.synchronize()
    s = [torch.cuda.Stream() for _ in range(3)]
    outs = [M.group_route(a, 5, stream=x) for x in s for _ in range(2)]
    torch.cuda.synchronize()
    ref = B.route_ref(a.double().cpu().numpy(), 5, 0)
    for o in outs:
        np.testing.assert_array_equal(o[4].cpu().numpy(), ref[4])
    out = M.group_route(a, 5)
    ws = torch.empty(M.group_route_workspace(2000, 96, 5), dtype=torch.uint8, device="cuda")
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        M.group_route(a, 5, out=out, workspace=ws)
    a.neg_()
    graph.replay()
    torch.cuda.synchronize()
    np.testing.assert_array_equal(out[4].cpu().numpy(), B.route_ref(a.double().cpu().numpy(), 5, 0)[4])


# ---------------------------------------------------------------- verification

def check_verify(M, p, draft, u, q=None, lengths=None):
    import torch
    d = lambda t: None if t is None else t.double().cpu().numpy()  # noqa: E731
    acc, tok = B.verify_ref(d(p), draft, u, d(q), lengths)
    ga, gt = M.verify_draft(p, torch.from_numpy(draft.astype(np.int32)).cuda(), torch.from_numpy(u.astype(np.float32)).cuda(),
                            q=q, lengths=None if lengths is None else torch.from_numpy(lengths.astype(np.int32)).cuda())
    np.testing.assert_array_equal(ga.cpu().numpy(), acc)
    np.testing.assert_array_equal(gt.cpu().numpy(), tok)
    return acc, tok


def make(Bn, D, V, dtype, seed, with_q=True, sharp=2.0):
    import torch
    g = torch.Generator(device="cuda").manual_seed(seed)
    z = sharp * torch.randn(Bn, D + 1, V, generator=g, device="cuda")
    q = torch.softmax(z[:, :D] + 0.7 * torch.randn(Bn, D, V, generator=g, device="cuda"), -1)
    draft = (q / torch.empty_like(q).exponential_(generator=g)).argmax(-1).cpu().numpy().reshape(Bn, D) if D else \
        np.zeros((Bn, 0), np.int64)
    t = B.torch_type(dtype)
    u = np.random.default_rng(seed).random((Bn, D + 1), dtype=np.float32)
    return torch.softmax(z, -1).to(t), draft, u, q.to(t) if with_q else None


@pytest.mark.parametrize("dtype", ["fp32", "bf16", "fp16"])
@pytest.mark.parametrize("with_q", [True, False], ids=["q", "onehot"])
@pytest.mark.parametrize("Bn,D,V", [(1, 3, 1000), (5, 4, 33), (3, 1, 1), (40, 8, 257), (2, 31, 100), (7, 0, 501), (3, 5, 20001),
                                    (200, 2, 64)])
def test_verify(M, Bn, D, V, with_q, dtype):
    p, draft, u, q = make(Bn, D, V, dtype, Bn + D, with_q)
    rng = np.random.default_rng(Bn)
    check_verify(M, p, draft, u, q)
    check_verify(M, p, draft, u, q, rng.integers(0, D + 1, Bn))


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
def test_verify_large_vocabulary(M, dtype):
    p, draft, u, q = make(3, 3, 262145, dtype, 1)
    check_verify(M, p, draft, u, q)
    check_verify(M, p, draft, u)


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("Bn,D,V", [(640, 1, 5001), (320, 1, 20001), (160, 1, 65001), (80, 1, 121001), (2, 1, 1100003)])
def test_verify_shares(M, Bn, D, V, dtype):
    """Many sequences of short rows, few of long ones, and what lies between: other numbers of blocks to a sequence."""
    p, draft, u, q = make(Bn, D, V, dtype, V, sharp=1.0)
    check_verify(M, p, draft, u, q)
    check_verify(M, p, draft, u)


@pytest.mark.parametrize("V", [10, 999, 5000])
def test_verify_borders(M, V):
    """Random numbers at the borders: 0, the last below 1, 1, and sums that fall on a border exactly."""
    import torch
    D = 2
    p = torch.zeros(12, D + 1, V, device="cuda")
    p[:, :, 1], p[:, :, V // 2], p[:, :, V - 2] = 0.25, 0.5, 0.25
    q = torch.zeros(12, D, V, device="cuda")
    q[:, :, 1], q[:, :, 3] = 0.5, 0.5
    draft = np.tile(np.array([[1, 3]]), (12, 1))
    one = np.float32(1) - np.float32(2.0 ** -24)
    u = np.array([[0.5, 0, 0], [0.49, 0, 0], [0.5, 0, one], [0.5, 0, 1.0], [0.5, 0, 2 / 3], [0, 0, 0.25], [0, 0.5, 0.75],
                  [one, 0, 0.5], [0.499, one, 0], [0, 0, 1e-30], [np.nan, np.nan, np.nan], [7, -3, 9]], np.float32)
    check_verify(M, p, draft, u, q)
    check_verify(M, p, draft, u)
    check_verify(M, p, draft, u, q, np.array([0, 1, 2, 5, -1, 0, 1, 2, 0, 1, 2, 0]))


def test_verify_empty_residuals_and_bad_values(M):
    import torch
    V = 300
    p, draft, u, q = make(8, 3, V, "fp32", 3)
    draft[0, 0], draft[1, 1], draft[2, 2] = -1, V, 2 ** 31 - 1      # no such tokens
    u[3] = 0.999
    q[3] = 1.0                                                      # p <= q everywhere: nothing left of the residual
    p[4, 0] = 0.0                                                   # nothing at all
    u[4] = 0.5
    p[5] = float("nan")
    p[6, :, 7] = float("inf")
    p[6, :, 8] = -1.0
    q[6, :, 9] = float("nan")
    acc, tok = check_verify(M, p, draft, u, q)
    assert tok[4, 0] == -1 and tok[5, 0] == -1
    check_verify(M, p, draft, u)


def test_verify_rows_apart_and_not_read(M):
    """p and q as parts of larger tensors; rows past a sequence's length hold NaN and are not looked at."""
    import torch
    for V, lead in ((1000, 1), (1024, 8), (77, 3)):
        p, draft, u, q = make(6, 4, V, "bf16", 5)
        P = torch.full((6, 7, V + 11), float("nan"), dtype=torch.bfloat16, device="cuda")
        Q = torch.full((6, 5, V + 16), float("nan"), dtype=torch.bfloat16, device="cuda")
        P[:, 1:6, lead:lead + V], Q[:, :4, 16:] = p, q
        lengths = np.array([4, 3, 2, 1, 0, 4])
        for b, n in enumerate(lengths):
            P[b, 2 + n:], Q[b, n:] = float("nan"), float("nan")
        a = check_verify(M, P[:, 1:6, lead:lead + V], draft, u, Q[:, :4, 16:], lengths)
        b = B.verify_ref(p.double().cpu().numpy(), draft, u, q.double().cpu().numpy(), lengths)
        np.testing.assert_array_equal(a[1], b[1])


def test_verify_streams_and_capture(M):
    import torch
    p, draft, u, q = make(9, 3, 4097, "fp16", 8)
    d, uu = dev(draft.astype(np.int32)), dev(u)
    ref = B.verify_ref(p.double().cpu().numpy(), draft, u, q.double().cpu().numpy())
    torch.cuda.synchronize()
    outs = [M.verify_draft(p, d, uu, q=q, stream=s) for s in (torch.cuda.Stream(), torch.cuda.Stream()) for _ in range(3)]
    torch.cuda.synchronize()
    for o in outs:
        np.testing.assert_array_equal(o[1].cpu().numpy(), ref[1])
    out = M.verify_draft(p, d, uu, q=q)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        M.verify_draft(p, d, uu, q=q, out=out)
    u2 = 1 - u
    uu.copy_(dev(u2))
    g.replay()
    torch.cuda.synchronize()
    np.testing.assert_array_equal(out[1].cpu().numpy(),
                                  B.verify_ref(p.double().cpu().numpy(), draft, u2, q.double().cpu().numpy())[1])


def test_verify_refusals(M):
    import torch
    p, draft, u, q = make(2, 3, 50, "fp32", 1)
    d, uu = dev(draft.astype(np.int32)), dev(u)
    for bad in (dict(p=p.double()), dict(p=p[0]), dict(draft=d.long()), dict(draft=d[:, :2]), dict(u=uu.double()), dict(u=uu[:, :3]),
                dict(q=q.half()), dict(q=q[:, :2]), dict(lengths=d[:, 0].long()), dict(lengths=d[:1, 0].contiguous()), dict(u=uu.cpu())):
        with pytest.raises(ValueError):
            M.verify_draft(**{**dict(p=p, draft=d, u=uu, q=q), **bad})
    big = torch.zeros(1, 33, 4, device="cuda")
    with pytest.raises(M.MoeError):
        M.verify_draft(big, torch.zeros(1, 32, dtype=torch.int32, device="cuda"), torch.zeros(1, 33, device="cuda"))


# ---------------------------------------------------------------- together

@pytest.mark.parametrize("T", [4, 150])
def test_a_batch_through_the_layer_and_its_gradients(M, T):
    """Route, gate/up with SwiGLU, down, combine, and verify; padded tokens stay out.  Then the products'
    gradients of the same batch."""
    import torch
    H, F, E, k = 256, 512, 8, 2       # this framework's tiny layer
    x, xd = values((T, H), 1, "bf16")
    wgu, wgud = values((E, 2 * F, H), 2, "bf16", H ** -0.5)
    wd, wdd = values((E, H, F), 3, "bf16", F ** -0.5)
    wr, _ = values((E, H), 4, "bf16", H ** -0.5)
    logits = x.float() @ wr.float().T
    logits[T - 1] = -float("inf")     # a padded token
    idx, weights, offsets, rows, pairs = M.group_route(logits, k)
    h = M.grouped_matmul(x, wgu, offsets, rows=rows, act="swiglu")
    y = torch.zeros(T * k, H, device="cuda")
    M.grouped_matmul(h, wd, offsets, out_rows=pairs, out=y)
    out = (weights[..., None] * y.view(T, k, H)).sum(1)

    r = B.route_ref(logits.double().cpu().numpy(), k, 0)
    np.testing.assert_array_equal(idx.cpu().numpy(), r[0])
    n = int(r[2][-1])
    hv, ht = B.grouped_ref(xd, wgud, r[2], r[3], swiglu=True)
    B.check_close(h[:n], hv[:n], ht[:n], "bf16")
    hd = h.double().cpu().numpy()
    yv, yt = B.grouped_ref(hd, wdd, r[2])
    full = np.zeros((T * k, H))
    tol = np.zeros((T * k, H))
    full[r[4][:n]], tol[r[4][:n]] = yv[:n], yt[:n]
    w = r[1][..., None]
    ref = (w * full.reshape(T, k, H)).sum(1)
    bound = (w * tol.reshape(T, k, H)).sum(1) + (np.abs(w * full.reshape(T, k, H))).sum(1) * 128 * 2.0 ** -23 + 1e-30
    assert (np.abs(out.double().cpu().numpy() - ref) <= bound).all()
    assert bool((out[T - 1] == 0).all())

    # gradients of the down product: its input's (rows in sorted order) and its weights'
    dy, dyd = values((T * k, H), 7, "bf16")
    dh = M.grouped_matmul(dy, wd, offsets, rows=pairs, w_layout="kn")
    v, t = B.grouped_ref(dyd, wdd, r[2], r[4], kn=True)
    B.check_close(dh[:n], v[:n], t[:n], "bf16")
    dw = M.grouped_wgrad(dy, h, offsets, dy_rows=pairs, out_dtype=torch.float32)
    v, t = B.wgrad_ref(dyd, hd, r[2], dy_rows=r[4])
    B.check_close(dw, v, t, "fp32")

    # the batch's answer: four sequences' drafts against probabilities made from the layer's output
    V, D = 64, 3
    head, _ = values((V, H), 8, "bf16", 0.3)
    p = torch.softmax(out[:4].float() @ head.float().T, -1)[None]     # one sequence of three drafts
    q = torch.softmax(p[:, :D].log() * 0.5, -1)
    draft = q.argmax(-1).cpu().numpy()
    check_verify(M, p, draft, np.random.default_rng(0).random((1, D + 1), dtype=np.float32), q)
