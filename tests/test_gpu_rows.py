"""The norm, rows in 8 bits and the weighted sum of experts' results, with their gradients, against the plain 64-bit forms."""
import numpy as np
import pytest

from tests import batch_helpers as B
from tests import rows_helpers as R
from tests.test_gpu_grouped import M  # noqa: F401

pytestmark = pytest.mark.gpu


def make(shape, name, seed, scale=1.0, pitch=0, offset=0):
    """A random device tensor [T][H]; pitch > 0: rows that many elements apart, starting `offset` elements into memory."""
    import torch
    g = torch.Generator(device="cuda").manual_seed(seed)
    v = (torch.randn(*shape, generator=g, device="cuda") * scale).to(B.torch_type(name))
    if not pitch:
        return v
    big = torch.empty(offset + shape[0] * pitch, dtype=v.dtype, device="cuda")
    view = big[offset:].as_strided(shape, (pitch, 1))
    view.copy_(v)
    return view


def f64(t):
    return t.detach().double().cpu().numpy()


def check_norm_call(M, x, residual=None, gain=None, eps=1e-5, want=("out", "out8", "rstd"), out_type="bf16", out=None, **kw):  # noqa: F811
    xs, rs = f64(x), None if residual is None else f64(residual)
    res_type = None if residual is None else residual.dtype
    got = M.rms_norm(x, gain=gain, residual=residual, eps=eps, want=want, out_dtype=B.torch_type(out_type), out=out, **kw)
    name = {v: k for k, v in ((n, B.torch_type(n)) for n in ("bf16", "fp16", "fp32"))}
    h = xs
    if residual is not None:
        h = R.round_type(np.float32(xs) + np.float32(rs), name[res_type])
        np.testing.assert_array_equal(f64(got.sum), h)
        assert got.sum.dtype == res_type
    else:
        assert got.sum is None
    y, rstd = R.norm_ref(h, None if gain is None else f64(gain), np.float32(eps).astype(np.float64))
    if "out" in want:
        assert got.out.dtype == B.torch_type(out_type)
        R.check_norm(f64(got.out), y, out_type)
    if "rstd" in want:
        assert (np.abs(f64(got.rstd) - rstd) <= R.RSTD_TOL * rstd).all()
    if "out8" in want:
        R.check_eight(f64(got.out8.float()), f64(got.scale), y, R.Y_TOL)
    return got


SIZES = [(1, 1), (3, 7), (5, 8), (9, 64), (4, 100), (17, 256), (2, 264), (7, 512), (3, 1000), (10, 1024), (2, 1025), (5, 1032), (1, 4096),
         (160, 4096), (3, 4095), (2, 7168), (200, 7168), (3, 8192), (2, 8200), (153, 8200), (2, 16384), (2, 20001), (2, 32768), (155, 16392),
         (0, 64)]


@pytest.mark.parametrize("T,H", SIZES)
@pytest.mark.parametrize("dtype,res,gain,out", [("bf16", "bf16", "bf16", "bf16"), ("fp32", None, None, "fp32"),
                                                ("fp16", "fp32", "fp32", "fp16"), ("fp32", "fp16", "fp16", "bf16"),
                                                ("bf16", "fp32", None, "fp32")])
def test_rms_norm(M, T, H, dtype, res, gain, out):  # noqa: F811
    check_norm_call(M, make((T, H), dtype, H + T), None if res is None else make((T, H), res, 2, 3.0),
                    None if gain is None else make((1, H), gain, 3)[0], out_type=out)


@pytest.mark.parametrize("want", [("out",), ("out8",), ("rstd",), ("out", "out8")], ids=str)
def test_rms_norm_outputs_alone(M, want):  # noqa: F811
    got = check_norm_call(M, make((6, 520), "bf16", 1), make((6, 520), "bf16", 2), make((1, 520), "bf16", 3)[0], want=want)
    assert (got.out is None) == ("out" not in want) and (got.out8 is None) == ("out8" not in want)
    with pytest.raises(ValueError):
        M.rms_norm(make((2, 8), "bf16", 1), want=("out", "y"))


@pytest.mark.parametrize("H,pitch,offset", [(64, 72, 0), (64, 65, 0), (64, 64, 1), (1032, 1040, 8), (2048, 2056, 4), (2048, 2050, 0),
                                            (4100, 4104, 0)])
def test_rms_norm_strides_and_alignment(M, H, pitch, offset):  # noqa: F811
    import torch
    x, r = make((5, H), "bf16", 1, 1, pitch, offset), make((5, H), "fp32", 2, 1, pitch, offset)
    gain = make((1, H + 1), "bf16", 3)[0, offset % 2:][:H]
    out = torch.zeros(5 * pitch + offset, dtype=torch.bfloat16, device="cuda")
    o8 = torch.zeros(5 * pitch + offset, dtype=torch.uint8, device="cuda")
    total = torch.zeros(5 * pitch + offset, device="cuda")
    view = lambda t: t[offset:].as_strided((5, H), (pitch, 1))  # noqa: E731
    check_norm_call(M, x, r, gain, out=M.Norm(view(out), view(total), None, view(o8.view(torch.float8_e4m3fn)), None))
    for t in (out, o8, total):       # nothing between the rows or before them
        keep = torch.ones(t.numel(), dtype=torch.bool, device="cuda")
        view(keep).fill_(False)
        assert (t[keep].float() == 0).all()


def test_rms_norm_in_place_and_out_of_place_agree(M):  # noqa: F811
    x, r, g = make((40, 1000), "bf16", 1), make((40, 1000), "bf16", 2), make((1, 1000), "fp32", 3)[0]
    a = M.rms_norm(x, gain=g, residual=r)
    x2, r2 = x.clone(), r.clone()
    b = M.rms_norm(x2, gain=g, residual=r2, out=M.Norm(x2, r2, None, None, None))
    assert b.out is x2 and b.sum is r2
    assert (a.out == x2).all() and (a.sum == r2).all()


def test_rms_norm_special_values(M):  # noqa: F811
    import torch
    x = make((6, 300), "fp32", 1)
    x[0] = 0
    x[1, 5] = float("nan")
    x[2, 7] = float("inf")
    x[3] = 1e-30
    x[4] *= 1e-12
    got = M.rms_norm(x, eps=1e-6, want=("out", "out8"), gain=torch.ones(300, device="cuda"))
    y = f64(got.out)
    assert (y[0] == 0).all() and np.isnan(y[1]).all() and np.isnan(y[2, 7]) and (np.delete(y[2], 7) == 0).all()
    q = f64(got.out8.float())
    assert (q[0] == 0).all() and np.isnan(q[1]).all() and np.isnan(q[2, 7])
    ok = [0, 3, 4, 5]
    ref, _ = R.norm_ref(f64(x)[ok], None, np.float64(np.float32(1e-6)))
    R.check_norm(y[ok], ref, "fp32")
    R.check_eight(q[ok], f64(got.scale)[ok], ref, R.Y_TOL)


@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("T,H", [(1, 1), (4, 16), (33, 100), (3, 2048), (200, 2048), (9, 14336), (2, 14337), (1000, 256), (0, 8)])
def test_quantize_rows(M, T, H, dtype):  # noqa: F811
    x = make((T, H), dtype, T + H, 0.01)
    if T > 3:
        x[1] = 0
        x[2] *= 2.0 ** -10
    q, s = M.quantize_rows(x)
    R.check_eight(f64(q.float()), f64(s), f64(x), 0.0)


def test_quantize_rows_special_values(M):  # noqa: F811
    x = make((3, 64), "fp32", 1)
    x[0, 3] = float("inf")
    x[1, 4] = float("nan")
    x[2] *= 1e-38
    q, s = (f64(t.float()) for t in M.quantize_rows(x))
    assert np.isinf(s[0]) and np.isnan(q[0, 3]) and (np.delete(q[0], 3) == 0).all()
    assert np.isnan(q[1, 4]) and np.isfinite(np.delete(q[1], 4)).all()
    assert s[2] == 2.0 ** -100 and (q[2] == 0).all()


def check_grad(M, dy, h, gain, dsum, out_type, **kw):  # noqa: F811
    import torch
    rstd = (1 / torch.sqrt(h.double().square().mean(1) + 1e-6)).float()
    dh, dg = M.rms_norm_backward(dy, h, rstd, gain=gain, dsum=dsum, out_dtype=B.torch_type(out_type), **kw)
    a, b = R.norm_grad_ref(f64(dy), f64(h), f64(rstd), None if gain is None else f64(gain), None if dsum is None else f64(dsum))
    B.check_close(dh, *a, out_type)
    if gain is None:
        assert dg is None
    else:
        B.check_close(dg, *b, "fp32")
    return dh, dg


@pytest.mark.parametrize("T,H", [(1, 1), (3, 7), (9, 64), (300, 64), (4, 100), (2500, 256), (17, 520), (7, 1024), (2, 1025), (400, 1032),
                                 (1, 4096), (700, 4096), (3, 4095), (320, 4095), (305, 7168), (2, 8200), (310, 16384), (2, 20001),
                                 (306, 32768)])
@pytest.mark.parametrize("dy,h,gain,dsum,out", [("bf16", "bf16", "bf16", None, "bf16"), ("bf16", "fp32", "fp32", "fp32", "fp32"),
                                                ("fp16", "fp16", None, "fp16", "fp16"), ("fp32", "bf16", "fp16", "bf16", "fp32")])
def test_rms_norm_backward(M, T, H, dy, h, gain, dsum, out):  # noqa: F811
    check_grad(M, make((T, H), dy, 1), make((T, H), h, 2, 2.0), None if gain is None else make((1, H), gain, 3)[0],
               None if dsum is None else make((T, H), dsum, 4), out)


@pytest.mark.parametrize("H,pitch,offset", [(64, 72, 8), (64, 65, 0), (1032, 1040, 4), (2048, 2056, 8)])
def test_rms_norm_backward_strides_and_in_place(M, H, pitch, offset):  # noqa: F811
    dy, h, ds = (make((50, H), "fp32", i, 1, pitch, offset) for i in (1, 2, 3))
    gain = make((1, H), "bf16", 4)[0]
    dh, dg = check_grad(M, dy, h, gain, ds, "fp32")
    import torch
    rstd = (1 / torch.sqrt(h.double().square().mean(1) + 1e-6)).float()
    # (copies are contiguous: another order of addition than that of rows apart)
    dh, dg = check_grad(M, dy.clone(), h.clone(), gain, ds.clone(), "fp32")
    for which in range(3):
        t = [dy.clone(), h.clone(), ds.clone()]
        a, b = M.rms_norm_backward(t[0], t[1], rstd, gain=gain, dsum=t[2], out=(t[which], None))
        assert a is t[which] and (a == dh).all() and (b == dg).all()


def test_rms_norm_backward_without_rows(M):  # noqa: F811
    import torch
    e = torch.empty(0, 24, device="cuda")
    dh, dg = M.rms_norm_backward(e, e, torch.empty(0, device="cuda"), gain=torch.ones(24, device="cuda"))
    assert dh.shape == (0, 24) and (dg == 0).all()


def test_norm_gradient_is_that_of_the_norm(M):  # noqa: F811
    """Of the whole call by differences: the sum's, with the residual, in fp32."""
    x, r, g, c = make((4, 40), "fp32", 1), make((4, 40), "fp32", 2), make((1, 40), "fp32", 3)[0], make((4, 40), "fp32", 4)
    n = M.rms_norm(x, gain=g, residual=r, eps=0.1, want=("out", "rstd"))
    dh, dg = (f64(t) for t in M.rms_norm_backward(c, n.sum, n.rstd, gain=g))
    h, gg, cc = f64(x) + f64(r), f64(g), f64(c)
    f = lambda h, g: float((R.norm_ref(h, g, 0.1)[0] * cc).sum())  # noqa: E731
    # h is off by 2^-24 of itself where it was rounded: the gradient by about that times its second derivative (below 10 here)
    for i in ((0, 0), (1, 17), (3, 39)):
        d = np.zeros_like(h)
        d[i] = 1e-5
        assert abs((f(h + d, gg) - f(h - d, gg)) / 2e-5 - dh[i]) < 1e-5
    d = np.zeros(40)
    d[11] = 1e-5
    assert abs((f(h, gg + d) - f(h, gg - d)) / 2e-5 - dg[11]) < 1e-5


def make_places(T, k, M_rows, seed, masked=0.2):
    rng = np.random.default_rng(seed)
    p = rng.permutation(M_rows)[: T * k].reshape(T, k)
    p[rng.random((T, k)) < masked] = -1
    if T > 2:
        p[1] = -1
    return p


@pytest.mark.parametrize("T,k,H", [(1, 1, 1), (1, 8, 7168), (4, 8, 7168), (3, 2, 100), (5, 9, 264), (300, 2, 4096), (7, 32, 64), (2, 17, 3001),
                                   (10, 3, 20000), (0, 4, 64)])
@pytest.mark.parametrize("dtype,out,residual", [("bf16", "bf16", True), ("fp16", "fp32", False), ("fp32", "bf16", True),
                                                ("bf16", "fp16", False), ("fp32", "fp32", True)])
def test_combine_rows(M, T, k, H, dtype, out, residual):  # noqa: F811
    import torch
    rows = T * k + 3
    y, w = make((rows, H), dtype, 1), make((T, k), "fp32", 2)
    res = make((T, H), out, 3) if residual else None
    for places in (None, make_places(T, k, rows, T + k)):
        p = np.arange(T * k).reshape(T, k) if places is None else places
        dev = None if places is None else torch.from_numpy(places.astype(np.int32)).cuda()
        got = M.combine_rows(y, w, places=dev, residual=res, out_dtype=B.torch_type(out))
        assert got.dtype == B.torch_type(out)
        B.check_close(got, *R.combine_ref(f64(y), f64(w), p, None if res is None else f64(res)), out)


def test_combine_rows_masked_rows_are_not_read(M):  # noqa: F811
    """Rows of masked pairs may hold anything; places past the end or below it add nothing."""
    import torch
    y, w = make((12, 72), "bf16", 1), make((4, 3), "fp32", 2)
    w[2] = 0
    w[0, 1] = 0
    y[6:9] = float("nan")
    y[1] = float("inf")
    B.check_close(M.combine_rows(y, w), *R.combine_ref(np.nan_to_num(f64(y), posinf=0), f64(w), np.arange(12).reshape(4, 3)), "bf16")
    places = np.array([[0, 12, 3], [-1, 2 ** 31 - 1, -2 ** 31], [9, 10, 11], [4, 5, 13]])
    got = M.combine_rows(y, torch.ones(4, 3, device="cuda"), places=torch.from_numpy(places.astype(np.int32)).cuda())
    B.check_close(got, *R.combine_ref(np.nan_to_num(f64(y), posinf=0), np.ones((4, 3)), places), "bf16")
    assert (got[1] == 0).all()


@pytest.mark.parametrize("H,pitch,offset", [(64, 72, 8), (64, 65, 0), (4096, 4100, 0), (264, 264, 4)])
def test_combine_rows_strides_and_in_place(M, H, pitch, offset):  # noqa: F811
    y, w, res = make((12, H), "bf16", 1, 1, pitch, offset), make((4, 3), "fp32", 2), make((4, H), "fp32", 3, 1, pitch, offset)
    want = R.combine_ref(f64(y), f64(w), np.arange(12).reshape(4, 3), f64(res))
    got = M.combine_rows(y, w, residual=res, out=res)
    assert got is res
    B.check_close(res, *want, "fp32")


@pytest.mark.parametrize("T,k,H", [(1, 1, 1), (1, 8, 7168), (3, 2, 100), (5, 9, 264), (310, 2, 4096), (7, 32, 64), (2, 17, 3001), (4, 3, 20000),
                                   (306, 1, 1040), (0, 4, 64)])
@pytest.mark.parametrize("dtype,dout", [("bf16", "bf16"), ("fp16", "fp32"), ("fp32", "bf16")])
def test_combine_rows_backward(M, T, k, H, dtype, dout):  # noqa: F811
    import torch
    rows = T * k + 3
    y, w, d = make((rows, H), dtype, 1), make((T, k), "fp32", 2), make((T, H), dout, 3)
    for places in (None, make_places(T, k, rows, T + k)):
        p = np.arange(T * k).reshape(T, k) if places is None else places
        dev = None if places is None else torch.from_numpy(places.astype(np.int32)).cuda()
        old = make((rows, H), dtype, 9)
        dy, dw = M.combine_rows_backward(d, y, w, places=dev, out=(old.clone(), torch.empty(T, k, device="cuda")))
        (rdy, written), dws = R.combine_grad_ref(f64(d), f64(y), f64(w), p)
        B.check_close(dy[torch.from_numpy(written)], rdy[written], B.HALF_STEP["fp32"] * np.abs(rdy[written]), dtype)
        assert (dy == old)[torch.from_numpy(~written)].all()       # as they were
        B.check_close(dw, *dws, "fp32")
    if T:
        mine = y.clone()
        a, b = M.combine_rows_backward(d, mine, w, places=dev, out=(mine, torch.empty(T, k, device="cuda")))
        assert (b == dw).all() and (a[torch.from_numpy(written)] == dy[torch.from_numpy(written)]).all()


def test_rows_streams_and_capture(M):  # noqa: F811
    """On other streams, captured and replayed with new inputs: what eager calls give."""
    import torch
    x, r, g = make((50, 2048), "bf16", 1), make((50, 2048), "bf16", 2), make((1, 2048), "bf16", 3)[0]
    w = make((25, 2), "fp32", 4)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]

    def step(stream=None):
        n = M.rms_norm(x, gain=g, residual=r, want=("out", "rstd", "out8"), stream=stream)
        c = M.combine_rows(n.out, w, stream=stream)
        dy, dw = M.combine_rows_backward(c, n.out, w, stream=stream)
        dh, dg = M.rms_norm_backward(dy, n.sum, n.rstd, gain=g, stream=stream)
        return [n.out, n.sum, n.rstd, n.out8.view(torch.uint8), n.scale, c, dy, dw, dh, dg]

    ref = [t.clone() for t in step()]
    outs = [step(s) for s in streams]
    torch.cuda.synchronize()
    for o in outs:
        assert all((a == b).all() for a, b in zip(o, ref))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        captured = step()
    x.copy_(make((50, 2048), "bf16", 7))
    graph.replay()
    torch.cuda.synchronize()
    again = step()
    assert all((a == b).all() for a, b in zip(captured, again)) and not (again[0] == ref[0]).all()


@pytest.mark.parametrize("T,H", [(1, 8), (5, 16), (33, 64), (4, 64), (17, 72), (31, 120), (1, 128), (35, 128), (600, 128), (3, 136)])
def test_short_rows(M, T, H):  # noqa: F811
    """Several rows a warp, whole warps and parts of the last; nothing behind the last row is written."""
    import torch
    x, r, g = make((T, H), "bf16", T), make((T, H), "bf16", 2), make((1, H), "bf16", 3)[0]
    out, total = torch.full((T + 8, H), 7.0, device="cuda").bfloat16(), torch.full((T + 8, H), 7.0, device="cuda").bfloat16()
    o8, scale = torch.full((T + 8, H), 7, dtype=torch.uint8, device="cuda"), torch.full((T + 8,), 7.0, device="cuda")
    rstd = torch.full((T + 8,), 7.0, device="cuda")
    n = M.Norm(out[:T], total[:T], rstd[:T], o8[:T].view(torch.float8_e4m3fn), scale[:T])
    check_norm_call(M, x, r, g, out=n)
    for t in (out, total, o8, scale, rstd):
        assert (t[T:] == 7).all()
    q, s = M.quantize_rows(x)
    R.check_eight(f64(q.float()), f64(s), f64(x), 0.0)


def test_zero_rows_under_a_small_eps(M):  # noqa: F811
    import torch
    for H in (64, 2048, 7168, 100):
        x = torch.zeros(3, H, device="cuda").bfloat16()
        n = M.rms_norm(x, eps=1e-30, want=("out", "out8"))
        assert (n.out == 0).all() and (n.out8.view(torch.uint8) == 0).all() and (n.scale == 2.0 ** -100).all()
