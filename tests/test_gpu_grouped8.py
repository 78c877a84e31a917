"""The grouped products in 8 bits against the plain 64-bit form, and the operators around the products used together."""
import numpy as np
import pytest

from tests import batch_helpers as B
from tests import rows_helpers as R
from tests.test_gpu_grouped import M, RAGGED, dev  # noqa: F401

pytestmark = pytest.mark.gpu


def eight(shape, seed, scale=60.0):
    """(device tensor of e4m3 numbers, their values in fp64)"""
    import torch
    g = torch.Generator(device="cuda").manual_seed(seed)
    t = (torch.randn(*shape, generator=g, device="cuda") * scale).clamp(-448, 448).to(torch.float8_e4m3fn)
    return t, t.float().double().cpu().numpy()


def scales(shape, seed, scale):
    import torch
    g = torch.Generator(device="cuda").manual_seed(seed)
    t = (torch.rand(*shape, generator=g, device="cuda") + 0.5) * scale
    return t, t.double().cpu().numpy()


def run(M, sizes, n, k, swiglu=False, gather=False, scatter=False, out="bf16", tail=0, first=0, seed=0, kernel=None):  # noqa: F811
    """One call against the plain form, in an output with guard rows and columns that must stay as they were."""
    import torch
    rng = np.random.default_rng(seed)
    E, nw = len(sizes), n * (2 if swiglu else 1)
    offsets = B.make_groups(sizes, rng, first)
    m = int(offsets[-1]) + tail
    rows_n = max(1, m // 2 + 1) if gather else m
    x, xd = eight((rows_n, k), seed + 1)
    w, wd = eight((E, nw, k), seed + 2)
    xs, xsd = scales((rows_n,), seed + 3, 0.02)
    ws, wsd = scales((E, nw), seed + 4, 0.02 * k ** -0.5)
    rows = rng.integers(0, rows_n, m).astype(np.int32) if gather else None
    out_rows = rng.permutation(m + 3)[:m].astype(np.int32) if scatter else None
    # two scales more than a 16-bit product: their product and the sum's, a rounding each, within the bound's spare step
    val, tol = B.grouped_ref(xd * xsd[:, None], wd * wsd[:, :, None], offsets, rows, False, swiglu)
    full = torch.full((m + 3, n + (5 if seed % 2 else 8)), 7.0, dtype=B.torch_type(out), device="cuda")
    got = M.grouped_matmul8(x, xs, w, ws, dev(offsets), rows=None if rows is None else dev(rows),
                            out_rows=None if out_rows is None else dev(out_rows), act="swiglu" if swiglu else None, out=full[:, :n])
    assert got.data_ptr() == full.data_ptr()
    if kernel is not None:
        a = M.Grouped8Args(x=4096, x_scale=4096, w=4096, w_scale=4096, offsets=4096, rows=4096 if gather else None, out=4096,
                           x_rows=rows_n, ldx=k, ldw=k, w_stride=nw * k, out_rows_n=m + 3, ldo=full.shape[1], m=m, groups=E, n=nw, k=k,
                           out_dtype={"bf16": 0, "fp16": 1, "fp32": 2}[out], act=int(swiglu), out_rows=4096 if scatter else None,
                           workspace=4096 if gather else None, workspace_bytes=M.grouped8_workspace(m, k, E) if gather else 0)
        assert M.grouped_kernel(a, torch.cuda.get_device_properties(0).multi_processor_count) == kernel
    at = out_rows if scatter else np.arange(m)
    live = np.arange(int(offsets[0]), int(offsets[-1]))
    if len(live):
        B.check_close(full[torch.from_numpy(at[live].astype(np.int64)).cuda(), :n], val[live], tol[live], out)
    rest = np.setdiff1d(np.arange(m + 3), at[live])
    assert bool((full[torch.from_numpy(rest).cuda()] == 7).all()), "rows of no group were written"
    assert bool((full[:, n:] == 7).all()), "columns behind the last were written"


CASES = [
    # groups, n, k
    (RAGGED, 256, 64), (RAGGED, 136, 80), (RAGGED, 520, 1040), ([5, 0, 3], 8, 16), ([1], 1, 16), ([33, 64, 65], 33, 32),
    ([0, 0, 4], 1000, 272), ([130, 129], 48, 112), ([1, 1, 0, 1], 2048, 2064), ([700, 0, 31], 64, 512), ([1] * 40, 96, 160),
    ([17, 16, 15, 32, 33, 31, 48, 64, 63], 272, 208), ([2, 0] * 300, 40, 48), ([1, 0, 0, 2] * 256, 24, 48), ([300, 3], 1000, 2064),
    ([5, 2, 0, 1], 201, 144), ([19, 2] * 512, 9, 16)]


@pytest.mark.parametrize("swiglu", [False, True], ids=["plain", "swiglu"])
@pytest.mark.parametrize("case", range(len(CASES)))
def test_matmul8(M, case, swiglu):  # noqa: F811
    sizes, n, k = CASES[case]
    run(M, sizes, n, k, swiglu, gather=case % 2 == 1, scatter=case % 3 == 1, tail=case % 4, seed=case, out=["bf16", "fp16", "fp32"][case % 3])


PAIR = {
    "uneven": ([0, 1, 37, 600, 255, 257, 513, 385], 1056, 2064),
    "by 16": ([300, 700, 0, 64], 1000, 4240),
    "bands": ([2400, 3], 1304, 4224),
    "borders": ([256, 512, 32, 64, 96, 1, 288, 31], 1040, 4144),
    "odd columns": ([512, 511, 513], 3591, 4112),
    "long": ([300, 260, 300], 3000, 33024),
}


@pytest.mark.parametrize("out", ["bf16", "fp32"])
@pytest.mark.parametrize("form", ["plain", "gather", "scatter", "swiglu", "swiglu gather"])
@pytest.mark.parametrize("case", PAIR)
def test_matmul8_many_rows(M, case, form, out):  # noqa: F811
    sizes, n, k = PAIR[case]
    run(M, sizes, n, k, "swiglu" in form, "gather" in form, form == "scatter", out, seed=len(case), kernel=M.GROUPED_PAIR)


@pytest.mark.parametrize("sizes,n,k", [([1] * 8, 7168, 2048), ([4, 0, 9, 2], 1032, 4096), ([16, 3, 30, 17], 520, 4112), ([60, 2, 50, 40], 264, 2064)])
@pytest.mark.parametrize("form", ["plain", "gather", "scatter", "swiglu", "swiglu gather"])
def test_matmul8_few_rows(M, sizes, n, k, form):  # noqa: F811
    run(M, sizes, n, k, "swiglu" in form, "gather" in form, form == "scatter", "fp32", seed=n, kernel=M.GROUPED_FEW)


@pytest.mark.parametrize("first,tail", [(5, 0), (0, 9), (130, 70)])
def test_matmul8_rows_before_and_behind_the_groups_stay(M, first, tail):  # noqa: F811
    run(M, [40, 0, 300], 256, 128, first=first, tail=tail)
    run(M, [1, 0, 2], 256, 128, first=first, tail=tail, gather=True)
    run(M, [0, 0, 0], 64, 64, tail=4)


def test_matmul8_extremes_and_bad_numbers(M):  # noqa: F811
    """The largest numbers, zeros, NaN that stays in its row or column; row numbers and offsets outside their range."""
    import torch
    for sizes, n, k in (([3, 0, 5], 136, 144), ([700, 0, 513], 1544, 4240)):
        offsets = B.make_groups(sizes, None)
        m = int(offsets[-1])
        x, xd = eight((m, k), 1)
        w, wd = eight((3, n, k), 2)
        x[0], w[0, 3], x[1] = 448.0, 448.0, 0.0
        xs, ws = torch.ones(m, device="cuda"), torch.ones(3, n, device="cuda")
        xs[2] = float("nan")
        ws[2, 5] = float("nan")
        got = M.grouped_matmul8(x, xs, w, ws, dev(offsets), out_dtype=torch.float32).double().cpu().numpy()
        val, tol = B.grouped_ref(x.float().double().cpu().numpy(), w.float().double().cpu().numpy(), offsets)
        bad = np.zeros(got.shape, bool)
        bad[2] = True
        bad[sizes[0]:, 5] = True
        assert np.isnan(got[bad]).all()
        assert (np.abs(got - val) <= tol + B.HALF_STEP["fp32"] * np.abs(val) + 1e-30)[~bad].all()
        assert got[0, 3] == 448.0 * 448.0 * k
        rows = np.arange(m).astype(np.int32)
        rows[0], rows[4], rows[5] = -1, m, 2 ** 31 - 1
        xs[2], ws[2, 5] = 1.0, 1.0
        wild = offsets.copy()
        wild[0], wild[-1] = -7, m + 1000
        got = M.grouped_matmul8(x, xs, w, ws, dev(wild), rows=dev(rows), out_dtype=torch.float32).double().cpu().numpy()
        assert (got[[0, 4, 5]] == 0).all()
        ok = np.setdiff1d(np.arange(m), [0, 4, 5])
        assert (np.abs(got - val) <= tol + B.HALF_STEP["fp32"] * np.abs(val) + 1e-30)[ok].all()


def test_matmul8_strides_streams_and_capture(M):  # noqa: F811
    import torch
    g = torch.Generator(device="cuda").manual_seed(0)
    bytes_ = lambda *s: torch.randint(0, 120, s, generator=g, device="cuda", dtype=torch.uint8).view(torch.float8_e4m3fn)  # noqa: E731
    x, w = bytes_(900, 1040)[:, 16:1024 - 16], bytes_(3, 700, 1056)[:, 8:, 32:1024]
    xs, ws = torch.rand(900, device="cuda"), torch.rand(3, 692, device="cuda")
    offsets, rows = dev(np.array([0, 300, 310, 900], np.int32)), dev(np.random.default_rng(0).permutation(900).astype(np.int32))
    call = lambda **kw: M.grouped_matmul8(x, xs, w, ws, offsets, rows=rows, **kw)  # noqa: E731
    torch.cuda.synchronize()
    outs = [call(stream=s) for s in [torch.cuda.Stream() for _ in range(2)]]
    out = call(out_dtype=torch.float32)
    xr = x.contiguous().float().double().cpu().numpy() * xs.double().cpu().numpy()[:, None]
    val, tol = B.grouped_ref(xr, w.contiguous().float().double().cpu().numpy() * ws.double().cpu().numpy()[:, :, None],
                             offsets.cpu().numpy(), rows.cpu().numpy())
    B.check_close(out, val, tol, "fp32")
    torch.cuda.synchronize()
    assert (outs[0] == outs[1]).all()
    ws_mem = torch.empty(M.grouped8_workspace(900, 992, 3), dtype=torch.uint8, device="cuda")
    again = torch.empty_like(out)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call(out=again, workspace=ws_mem)
    graph.replay()
    torch.cuda.synchronize()
    assert (again == out).all()
    xs.mul_(2)
    graph.replay()
    torch.cuda.synchronize()
    assert (again == 2 * out).all()


def test_matmul8_refusals(M):  # noqa: F811
    import torch
    z = lambda *s: torch.zeros(*s, dtype=torch.float8_e4m3fn, device="cuda")  # noqa: E731
    f = lambda *s: torch.ones(*s, device="cuda")  # noqa: E731
    o = torch.tensor([0, 4, 4], dtype=torch.int32, device="cuda")
    M.grouped_matmul8(z(4, 32), f(4), z(2, 8, 32), f(2, 8), o)
    for bad in (lambda: M.grouped_matmul8(z(4, 32).view(torch.uint8), f(4), z(2, 8, 32), f(2, 8), o),
                lambda: M.grouped_matmul8(z(4, 32), f(5), z(2, 8, 32), f(2, 8), o),
                lambda: M.grouped_matmul8(z(4, 32), f(4), z(2, 8, 32), f(2, 9), o),
                lambda: M.grouped_matmul8(z(4, 32), f(4), z(2, 8, 48), f(2, 8), o),
                lambda: M.grouped_matmul8(z(4, 32), f(4).double(), z(2, 8, 32), f(2, 8), o),
                lambda: M.grouped_matmul8(z(4, 32), f(4), z(2, 8, 32), f(2, 8), o, act="gelu")):
        with pytest.raises(ValueError):
            bad()
    for bad in (lambda: M.grouped_matmul8(z(4, 24), f(4), z(2, 8, 24), f(2, 8), o),                       # k no multiple of 16
                lambda: M.grouped_matmul8(z(4, 40)[:, :32], f(4), z(2, 8, 32), f(2, 8), o),               # rows 40 bytes apart
                lambda: M.grouped_matmul8(z(4, 48)[:, 8:40], f(4), z(2, 8, 32), f(2, 8), o),              # 8 bytes into memory
                lambda: M.grouped_matmul8(z(4, 32), f(4), z(1, 8, 32).expand(2, 8, 32), f(2, 8), o)):     # experts on one another
        with pytest.raises(M.MoeError):
            bad()
    many = torch.tensor([0, 2000, 4000], dtype=torch.int32, device="cuda")
    with pytest.raises(M.MoeError):   # many rows by number without room for them
        M.grouped_matmul8(z(100, 4096), f(100), z(2, 2048, 4096), f(2, 2048), many, rows=torch.zeros(4000, dtype=torch.int32, device="cuda"),
                          workspace=torch.empty(16, dtype=torch.uint8, device="cuda"))


# ---- used together

def test_layer_in_8_bits(M):  # noqa: F811
    """A served layer: norm with the residual, routing from its 16-bit output, the experts on its 8-bit output, their results summed
    onto the residual; each step against 64 bits of what it was given."""
    import torch
    g = torch.Generator(device="cuda").manual_seed(0)
    normal = lambda *s, scale=1.0: torch.randn(*s, generator=g, device="cuda") * scale  # noqa: E731
    for T in (1, 5, 300):
        H, F, E, k = 512, 384, 16, 4
        x, res, gain = normal(T, H).bfloat16(), normal(T, H).bfloat16(), (1 + normal(H, scale=0.1)).bfloat16()
        up8, ups = M.quantize_rows(normal(E * 2 * F, H, scale=H ** -0.5).bfloat16())
        down8, downs = M.quantize_rows(normal(E * H, F, scale=F ** -0.5).bfloat16())
        n = M.rms_norm(x, gain=gain, residual=res, want=("out", "out8"))
        logits = n.out.float() @ normal(H, E, scale=H ** -0.5)
        idx, w, offsets, rows, pairs, places = M.balanced_route(logits, k, bias=normal(E, scale=0.1), router=M.ROUTER_SIGMOID, groups=4,
                                                                keep=2, scale=2.5)
        h = M.grouped_matmul8(n.out8, n.scale, up8.view(E, 2 * F, H), ups.view(E, 2 * F), offsets, rows=rows, act="swiglu")
        h8, hs = M.quantize_rows(h)
        y = M.grouped_matmul8(h8, hs, down8.view(E, H, F), downs.view(E, H), offsets)
        out = M.combine_rows(y, w, places=places, residual=n.sum)
        f64 = lambda t: t.float().double().cpu().numpy()  # noqa: E731
        o, r = offsets.cpu().numpy(), rows.cpu().numpy()
        val, tol = B.grouped_ref(f64(n.out8) * f64(n.scale)[:, None], (f64(up8) * f64(ups)[:, None]).reshape(E, 2 * F, H), o, r, False, True)
        B.check_close(h, val, tol, "bf16")
        val, tol = B.grouped_ref(f64(h8) * f64(hs)[:, None], (f64(down8) * f64(downs)[:, None]).reshape(E, H, F), o)
        B.check_close(y, val, tol, "bf16")
        B.check_close(out, *R.combine_ref(f64(y), f64(w), places.cpu().numpy(), f64(n.sum)), "bf16")
        # and of the whole: the same layer from the unrounded rows and weights differs by the two 8-bit roundings alone: 2^-4 at
        # most each, some 2.6% root mean square, of four operands
        full = np.zeros((T, H))
        W1, W2 = (f64(up8) * f64(ups)[:, None]).reshape(E, 2 * F, H), (f64(down8) * f64(downs)[:, None]).reshape(E, H, F)
        yn, _ = R.norm_ref(f64(n.sum), f64(gain), 1e-6)
        for t in range(T):
            for j in range(k):
                e = int(idx[t, j])
                a = W1[e] @ yn[t]
                full[t] += float(w[t, j]) * (W2[e] @ (a[:F] / (1 + np.exp(-a[:F])) * a[F:]))
        part = f64(out) - f64(n.sum)
        assert np.linalg.norm(part - full) <= 0.15 * np.linalg.norm(full)


def test_training_step_of_a_layer(M):  # noqa: F811
    """Norm, routing, 16-bit experts and the weighted sum, forward and back through every operator, against autograd in 64 bits of
    the same choice of experts and of relu's side (some 60 of the 40000 inputs lie within a rounding of 0, and one that goes the
    other way changes its token's gradient by 6%)."""
    import torch
    g = torch.Generator(device="cuda").manual_seed(1)
    normal = lambda *s, scale=1.0: torch.randn(*s, generator=g, device="cuda") * scale  # noqa: E731
    T, H, F, E, k = 70, 256, 192, 12, 3
    x, gain, bias, c = normal(T, H), 1 + normal(H, scale=0.1), normal(E, scale=0.05), normal(T, H)
    wr, w1 = normal(H, E, scale=H ** -0.5), normal(E, F, H, scale=H ** -0.5).bfloat16()
    w2 = normal(E, H, F, scale=F ** -0.5).bfloat16()
    for router, renorm in ((1, True), (0, False)):
        n = M.rms_norm(x, gain=gain, want=("out", "rstd"))
        xb = n.out.bfloat16()
        logits = n.out @ wr
        idx, w, offsets, rows, pairs, places = M.balanced_route(logits, k, bias=bias, router=router, groups=3, keep=2, renormalize=renorm,
                                                                scale=2.0)
        a = M.grouped_matmul(xb, w1, offsets, rows=rows, out_dtype=torch.float32)
        h = torch.relu(a).bfloat16()
        y = M.grouped_matmul(h, w2, offsets, out_dtype=torch.float32)
        out = M.combine_rows(y, w, places=places, residual=x)
        dy, dw = M.combine_rows_backward(c, y, w, places=places)
        dyb = dy.bfloat16()
        dw2 = M.grouped_wgrad(dyb, h, offsets, out_dtype=torch.float32)
        da = (M.grouped_matmul(dyb, w2, offsets, w_layout="kn", out_dtype=torch.float32) * (a > 0)).bfloat16()
        dw1 = M.grouped_wgrad(da, xb, offsets, x_rows=rows, out_dtype=torch.float32)
        dxr = M.grouped_matmul(da, w1, offsets, w_layout="kn", out_dtype=torch.float32)
        dn = M.combine_rows(dxr, torch.ones_like(w), places=places)
        dl = M.balanced_route_backward(dw, logits, idx, router=router, renormalize=renorm, scale=2.0)
        dn = dn + dl @ wr.T
        dx, dgain = M.rms_norm_backward(dn, x, n.rstd, gain=gain, dsum=c)
        # the same in 64 bits
        v = {q: t.double().detach().requires_grad_(True) for q, t in dict(x=x, gain=gain, w1=w1, w2=w2).items()}
        nn = v["x"] / torch.sqrt(v["x"].square().mean(1, keepdim=True) + 1e-6) * v["gain"]
        l = nn @ wr.double()
        s = torch.sigmoid(l) if router else torch.softmax(l, 1)
        sel = s.gather(1, idx.long())
        ww = 2.0 * (sel / sel.sum(1, keepdim=True) if renorm else sel)
        o64 = v["x"].clone()
        for j in range(k):
            e = idx[:, j].long()
            z = torch.einsum("tfh,th->tf", v["w1"][e], nn) * (a > 0)[places[:, j].long()]
            o64 = o64 + ww[:, j:j + 1] * torch.einsum("thf,tf->th", v["w2"][e], z)
        ref = torch.autograd.grad((o64 * c.double()).sum(), list(v.values()))
        # bf16 rounds the experts' inputs and gradients, half a step of 2^-8 each at most: some 0.2% root mean square for each of at most
        # four on the way
        for got, want in zip((out, dx, dgain, dw1, dw2), (o64.detach(), *ref)):
            assert float((got.double() - want).norm() / want.norm()) < 0.02
