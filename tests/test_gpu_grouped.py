"""The grouped products against the plain 64-bit forms, at the sizes and masks where they can go wrong.

Inputs are the 16-bit values themselves, so the references are exact; the bounds are those of fp32
sums in any order plus half a rounding step of the output (tests/batch_helpers.py)."""
import numpy as np
import pytest

from tests import batch_helpers as B

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def M():
    from routed_expert_ffn_03_gb300 import build
    build.build()
    import routed_expert_ffn_03_gb300 as M
    return M


def dev(a, dtype=None):
    import torch
    return torch.from_numpy(np.ascontiguousarray(a)).cuda().to(dtype or torch.from_numpy(a[:0]).dtype)


def values(shape, seed, dtype, scale=1.0):
    """(device tensor of a 16-bit type, its values in fp64)"""
    import torch
    g = torch.Generator(device="cuda").manual_seed(seed)
    t = (torch.randn(*shape, generator=g, device="cuda") * scale).to(B.torch_type(dtype))
    return t, t.double().cpu().numpy()


RAGGED = [0, 1, 37, 256, 0, 300, 0, 2]
CASES = [
    # groups, n, k
    (RAGGED, 256, 64), (RAGGED, 136, 72), (RAGGED, 520, 1032), ([5, 0, 3], 8, 8), ([1], 1, 1), ([33, 64, 65], 33, 7),
    ([0, 0, 4], 1000, 264), ([130, 129], 48, 100), ([1, 1, 0, 1], 2048, 2056), ([700, 0, 31], 64, 512),
    ([1] * 40, 96, 160), ([17, 16, 15, 32, 33, 31, 48, 64, 63], 272, 200), ([2, 0] * 300, 40, 48),
    ([1, 0, 0, 2] * 256, 24, 40), (RAGGED, 200, 64), ([5, 2, 0, 1], 200, 136), ([300, 3], 1000, 2064), ([40, 0, 3, 20] * 256, 24, 40), ([19, 2] * 512, 9, 15),
]


def run_matmul(M, sizes, n, k, dtype, kn=False, swiglu=False, gather=False, scatter=False, out="same", tail=0, first=0, seed=0):
    """One call against the plain form, in an output with guard rows and columns that must stay as they were."""
    import torch
    rng = np.random.default_rng(seed)
    out = dtype if out == "same" else out
    E, n_w = len(sizes), n * (2 if swiglu else 1)
    offsets = B.make_groups(sizes, rng, first)
    m = int(offsets[-1]) + tail
    R = max(1, m // 2 + 1) if gather else m
    x, xd = values((R, k), seed + 1, dtype)
    w, wd = values((E, k, n_w) if kn else (E, n_w, k), seed + 2, dtype, k ** -0.5)
    rows = rng.integers(0, R, m).astype(np.int32) if gather else None
    out_rows = rng.permutation(m + 3)[:m].astype(np.int32) if scatter else None
    val, tol = B.grouped_ref(xd, wd, offsets, rows, kn, swiglu)
    full = torch.full((m + 3, n + (5 if seed % 2 else 8)), 7.0, dtype=B.torch_type(out), device="cuda")
    got = M.grouped_matmul(x, w, dev(offsets), rows=None if rows is None else dev(rows),
                           out_rows=None if out_rows is None else dev(out_rows), w_layout="kn" if kn else "nk",
                           act="swiglu" if swiglu else None, out=full[:, :n])
    assert got.data_ptr() == full.data_ptr()
    at = out_rows if scatter else np.arange(m)
    live = np.arange(int(offsets[0]), int(offsets[-1]))
    if len(live):
        B.check_close(full[torch.from_numpy(at[live].astype(np.int64)).cuda(), :n], val[live], tol[live], out)
    rest = np.setdiff1d(np.arange(m + 3), at[live])
    assert bool((full[torch.from_numpy(rest).cuda()] == 7).all()), "rows of no group were written"
    assert bool((full[:, n:] == 7).all()), "columns behind the last were written"
    return full


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("kn", [False, True], ids=["nk", "kn"])
@pytest.mark.parametrize("case", range(len(CASES)))
def test_matmul(M, case, kn, dtype):
    sizes, n, k = CASES[case]
    run_matmul(M, sizes, n, k, dtype, kn=kn, gather=case % 2 == 1, scatter=case % 3 == 1, tail=case % 4, seed=case)


@pytest.mark.parametrize("out", ["bf16", "fp32"])
@pytest.mark.parametrize("case", range(len(CASES)))
def test_swiglu(M, case, out):
    sizes, n, k = CASES[case]
    run_matmul(M, sizes, n, k, "bf16", swiglu=True, gather=case % 2 == 0, scatter=case % 3 == 0, out=out, seed=case)


@pytest.mark.parametrize("out", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
def test_output_types(M, dtype, out):
    run_matmul(M, [3, 0, 290], 264, 192, dtype, out=out, gather=True)
    run_matmul(M, [3, 1, 2], 264, 192, dtype, out=out)
    run_matmul(M, [3, 1, 2], 21, 9, dtype, out=out)


@pytest.mark.parametrize("first,tail", [(5, 0), (0, 9), (130, 70)])
def test_rows_before_and_behind_the_groups_stay(M, first, tail):
    for n, k in ((256, 128), (19, 23)):
        run_matmul(M, [40, 0, 300], n, k, "bf16", first=first, tail=tail)
        run_matmul(M, [1, 0, 2], n, k, "bf16", first=first, tail=tail, gather=True)


def test_no_rows_in_any_group(M):
    for n, k in ((64, 64), (7, 5)):
        run_matmul(M, [0, 0, 0], n, k, "bf16", tail=4)
        run_matmul(M, [0, 0, 0], n, k, "bf16")
        run_matmul(M, [0], n, k, "fp16", tail=300)


def test_bad_offsets_and_row_numbers_stay_inside(M):
    """Row numbers outside x are zero rows, out rows outside out write nothing, offsets are clamped."""
    import torch
    for n, k in ((128, 64), (20, 12)):
        for m in (6, 200):
            x, xd = values((10, k), 3, "bf16")
            w, wd = values((2, n, k), 4, "bf16")
            rows = np.arange(m).astype(np.int32) % 10
            rows[[1, 2, 4]] = [-1, 10, 2 ** 31 - 1]
            out_rows = np.arange(m).astype(np.int32)
            out_rows[[0, 3, 5]] = [-5, m, 2 ** 31 - 1]
            full = torch.full((m, n), 7.0, device="cuda")
            off = np.array([-4, 3, 2 ** 31 - 1], np.int32)
            M.grouped_matmul(x, w, dev(off), rows=dev(rows), out_rows=dev(out_rows), out=full)
            val, tol = B.grouped_ref(xd, wd, [0, 3, m], rows.astype(np.int64))
            keep = np.setdiff1d(np.arange(m), [0, 3, 5])
            B.check_close(full[torch.from_numpy(keep).cuda()], val[keep], tol[keep], "fp32")
            assert bool((full[[0, 3, 5]] == 7).all())


def test_decreasing_offsets_stay_inside(M):
    """Offsets that go back and forth make more tiles than m rows can; nothing outside out is written, and the next call
    is right."""
    import torch
    for n, k in ((264, 64), (33, 17)):
        for m in (40, 700):
            E = 64
            off = np.array([0, m] * (E // 2) + [0], np.int32)
            x, _ = values((m, k), 1, "bf16")
            w, _ = values((E, n, k), 2, "bf16")
            full = torch.full((m + 2, n + 4), 7.0, device="cuda")
            M.grouped_matmul(x, w, dev(off), out=full[1:m + 1, :n])
            d = M.grouped_wgrad(x, x, dev(off))
            assert d.shape == (E, k, k)
            torch.cuda.synchronize()
            assert bool((full[0] == 7).all()) and bool((full[m + 1] == 7).all()) and bool((full[:, n:] == 7).all())
    run_matmul(M, [40, 0, 300], 264, 64, "bf16")


@pytest.mark.parametrize("pad", [0, 3, 8])
def test_strides_and_alignment(M, pad):
    """x, w and out as parts of larger tensors: rows and matrices further apart, odd starts."""
    import torch
    for sizes in ([3, 1, 0, 5], [130, 0, 200]):
        m, n, k = sum(sizes), 144, 80
        xs, _ = values((m + 2, k + pad + 1), 1, "fp16")
        ws, _ = values((len(sizes), n + 2, k + 2 * pad), 2, "fp16", k ** -0.5)
        for s in ((1 if pad == 3 else 0), 0):
            x = xs[1:m + 1, s:s + k] if pad != 8 else values((m, k + 8), 1, "fp16")[0][:, :k]
            w = ws[:, 1:n + 1, s:s + k]
            off = B.make_groups(sizes, None)
            val, tol = B.grouped_ref(x.double().cpu().numpy(), w.double().cpu().numpy(), off)
            big = torch.full((m, n + 1), 7.0, dtype=torch.float16, device="cuda")
            M.grouped_matmul(x, w, dev(off), out=big[:, 1:])
            B.check_close(big[:, 1:], val, tol, "fp16")
            assert bool((big[:, 0] == 7).all())
            back, btol = B.grouped_ref(val, w.double().cpu().numpy(), off, kn=True)
            dy = big[:, 1:].contiguous()
            back, btol = B.grouped_ref(dy.double().cpu().numpy(), w.double().cpu().numpy(), off, kn=True)
            B.check_close(M.grouped_matmul(dy, w, dev(off), w_layout="kn"), back, btol, "fp16")


def test_infinities_and_nan_stay_in_their_rows(M):
    """A row of NaN or infinities, of a neighbour group or behind the last, reaches no other row."""
    import torch
    for n, k in ((136, 64), (136, 72), (9, 11)):
        for sizes in ([3, 2, 4], [100, 60, 90]):
            m = sum(sizes) + 5
            x, _ = values((m, k), 5, "bf16")
            x[sizes[0] + 1] = float("nan")
            x[sizes[0]] = float("inf")
            x[sum(sizes):] = float("nan")
            w, wd = values((3, n, k), 6, "bf16")
            off = B.make_groups(sizes, None)
            bad = [sizes[0], sizes[0] + 1]
            clean = x.clone()
            clean[bad] = 0
            val, tol = B.grouped_ref(torch.nan_to_num(clean).double().cpu().numpy(), wd, off)
            got = M.grouped_matmul(x, w, dev(off), out=torch.zeros(m, n, device="cuda"))
            live = np.setdiff1d(np.arange(sum(sizes)), bad)
            B.check_close(got[torch.from_numpy(live).cuda()], val[live], tol[live], "fp32")
            assert bool(torch.isnan(got[sizes[0] + 1]).all())
            assert bool((got[sum(sizes):] == 0).all())


def test_long_offsets_pass_32_bits(M):
    """The last expert's matrix, and the last rows of x and out, start past 2^32 bytes."""
    import torch
    free = torch.cuda.mem_get_info()[0]
    if free < 40 << 30:
        pytest.skip("needs 40 GB")
    n, k, E = 8192, 4096, 80          # 5.4 GB of weights
    w = torch.zeros(E, n, k, dtype=torch.bfloat16, device="cuda")
    w[-1, -1, -1] = 2.0
    w[-1, 0, 0] = 3.0
    m = 600_000                       # 4.9 GB of x, 9.8 GB of out
    x = torch.zeros(m, k, dtype=torch.bfloat16, device="cuda")
    x[-1, -1] = 1.5
    x[-1, 0] = -1.0
    off = torch.full((E + 1,), m - 300, dtype=torch.int32, device="cuda")
    off[-1] = m
    for lay in ("nk", "kn"):
        y = torch.full((m, n if lay == "nk" else k), 7.0, dtype=torch.bfloat16, device="cuda") if lay == "nk" else None
        if lay == "nk":
            M.grouped_matmul(x, w, off, out=y)
            assert float(y[-1, -1]) == 3.0 and float(y[-1, 0]) == -3.0 and float(y[-2].abs().max()) == 0
            assert float(y[m - 301].min()) == 7.0
            del y
        else:
            dy = torch.zeros(m, n, dtype=torch.bfloat16, device="cuda")
            dy[-1, -1] = 4.0
            dx = M.grouped_matmul(dy, w, off, w_layout="kn")
            assert float(dx[-1, -1]) == 8.0 and float(dx[-1, 0]) == 0.0
            g = M.grouped_wgrad(dy, x, off)
            assert float(g[-1, -1, -1]) == 6.0 and float(g[-1, -1, 0]) == -4.0 and float(g[:-1].abs().max()) == 0


WCASES = [(RAGGED, 256, 64), (RAGGED, 136, 72), ([5, 0, 3], 8, 8), ([1], 1, 1), ([33, 64, 65], 33, 7), ([0, 0, 4], 520, 264),
          ([130, 129, 128], 48, 104), ([700, 0, 31], 64, 512), ([63, 64, 1], 264, 392), ([2, 0] * 200, 40, 48),
          ([3, 0, 130], 20, 12), ([65, 1, 40], 33, 7)]


@pytest.mark.parametrize("out", ["same", "fp32"])
@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("case", range(len(WCASES)))
def test_wgrad(M, case, dtype, out):
    import torch
    sizes, n, k = WCASES[case]
    rng = np.random.default_rng(case)
    out = dtype if out == "same" else out
    off = B.make_groups(sizes, rng, first=case % 3)
    m = int(off[-1]) + case % 2 * 7
    xr = rng.integers(0, m, m).astype(np.int32) if case % 2 else None
    dr = rng.permutation(m).astype(np.int32) if case % 4 == 1 else None
    if xr is not None and m > 6:
        xr[[2, 4]] = [-1, m]
    dy, dyd = values((m, n), case + 1, dtype)
    x, xd = values((m, k), case + 2, dtype)
    val, tol = B.wgrad_ref(dyd, xd, off, dr, xr)
    full = torch.full((len(sizes), n + 1, k + (3 if case % 3 else 8)), 7.0, dtype=B.torch_type(out), device="cuda")
    M.grouped_wgrad(dy, x, dev(off), dy_rows=None if dr is None else dev(dr), x_rows=None if xr is None else dev(xr),
                    out=full[:, :n, :k])
    B.check_close(full[:, :n, :k], val, tol, out)
    assert bool((full[:, n:] == 7).all()) and bool((full[:, :, k:] == 7).all())


def test_wgrad_without_rows_is_zero(M):
    import torch
    for n, k in ((64, 128), (5, 3)):
        for m in (0, 4):
            t = torch.full((m, n), float("nan"), dtype=torch.bfloat16, device="cuda")
            x = torch.full((m, k), float("inf"), dtype=torch.bfloat16, device="cuda")
            out = torch.full((3, n, k), 7.0, device="cuda")
            M.grouped_wgrad(t, x, dev(np.zeros(4, np.int32)), out=out)
            assert bool((out == 0).all())


def test_wgrad_neighbours_with_nan_stay_out(M):
    """Rows of other groups and behind the last, NaN in both factors, do not reach a group's sums."""
    import torch
    for n, k in ((128, 64), (136, 72), (7, 9)):
        sizes = [3, 2, 70, 61]
        m = sum(sizes) + 9
        dy, _ = values((m, n), 1, "bf16")
        x, _ = values((m, k), 2, "bf16")
        for t in (dy, x):
            t[3:5] = float("nan")
            t[sum(sizes):] = float("inf")
        off = B.make_groups(sizes, None)
        got = M.grouped_wgrad(dy, x, dev(off), out_dtype=torch.float32)
        z = lambda t: torch.nan_to_num(t, 0, 0, 0).double().cpu().numpy()  # noqa: E731
        val, tol = B.wgrad_ref(z(dy), z(x), off)
        for e in (0, 2, 3):
            B.check_close(got[e], val[e], tol[e], "fp32")
        assert bool(torch.isnan(got[1]).all())


def test_gradients_against_differences(M):
    """dx and dw of sum(c * y) agree with central differences of the 64-bit form at the same point."""
    sizes, n, k = [3, 0, 2], 16, 24
    off = B.make_groups(sizes, None)
    x, xd = values((5, k), 1, "fp16")
    w, wd = values((3, n, k), 2, "fp16")
    c, cd = values((5, n), 3, "fp16")
    dx = M.grouped_matmul(c, w, dev(off), w_layout="kn", out_dtype=B.torch_type("fp32")).double().cpu().numpy()
    dw = M.grouped_wgrad(c, x, dev(off), out_dtype=B.torch_type("fp32")).double().cpu().numpy()
    f = lambda x, w: float((B.grouped_ref(x, w, off)[0] * cd).sum())  # noqa: E731
    h = 2.0 ** -10                     # f is linear in each factor: differences are exact up to 64-bit rounding
    for i in [(0, 0), (4, 23), (2, 11)]:
        d = np.zeros_like(xd)
        d[i] = h
        assert abs((f(xd + d, wd) - f(xd - d, wd)) / (2 * h) - dx[i]) < B.sum_bound(n, n * 16.0) + 1e-9
    for i in [(0, 0, 0), (2, 15, 23), (1, 3, 3)]:
        d = np.zeros_like(wd)
        d[i] = h
        assert abs((f(xd, wd + d) - f(xd, wd - d)) / (2 * h) - dw[i]) < B.sum_bound(3, 3 * 16.0) + 1e-9


@pytest.mark.parametrize("T,n,k", [(700, 264, 1024), (9, 264, 1024), (300, 263, 77)])
def test_calls_in_a_row_give_what_calls_apart_give(M, T, n, k):
    """Routing, gathered products, their gradients and a workspace used again, launched without a pause and captured:
    each launch may start before the one in front has ended, and must not read early."""
    import torch
    E, top = 12, 3
    gen = torch.Generator(device="cuda").manual_seed(T)
    x = torch.randn(T, k, generator=gen, device="cuda").bfloat16()
    w = (torch.randn(E, n, k, generator=gen, device="cuda") * k ** -0.5).bfloat16()
    logits = torch.randn(8, T, E, generator=gen, device="cuda")
    ws = torch.empty(max(16, M.grouped_workspace(T * top, k, E), M.grouped_wgrad_workspace(T * top, k)), dtype=torch.uint8, device="cuda")

    def chain(l, pause):
        idx, _, off, rows, pairs = M.group_route(l, top)
        pause()
        y = M.grouped_matmul(x, w, off, rows=rows, workspace=ws)
        pause()
        dw = M.grouped_wgrad(y, x, off, x_rows=rows, workspace=ws)
        pause()
        dx = M.grouped_matmul(y, w, off, w_layout="kn", out_rows=pairs, out=torch.zeros(T * top, k, dtype=x.dtype, device="cuda"))
        pause()
        return idx, off, rows, y, dw, dx

    apart = [chain(l, torch.cuda.synchronize) for l in logits]
    run = [chain(l, lambda: None) for l in logits]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        captured = [chain(l, lambda: None) for l in logits]
    for _ in range(3):
        graph.replay()
    torch.cuda.synchronize()
    for a, b, c in zip(apart, run, captured):
        for p, q, r in zip(a, b, c):
            assert torch.equal(p, q) and torch.equal(p, r)


def test_other_stream_capture_and_two_at_once(M):
    """A call on a side stream, a captured call replayed on new data, and calls on two streams at once."""
    import torch
    for sizes in ([1, 0, 3, 2], [200, 1, 77]):
        n, k, m = 264, 136, sum(sizes)
        off = B.make_groups(sizes, None)
        x, xd = values((m, k), 1, "bf16")
        w, wd = values((len(sizes), n, k), 2, "bf16", k ** -0.5)
        o = dev(off)
        val, tol = B.grouped_ref(xd, wd, off)
        side = [torch.cuda.Stream() for _ in range(2)]
        torch.cuda.synchronize()
        outs = [M.grouped_matmul(x, w, o, stream=s) for s in side for _ in range(3)]
        outs.append(M.grouped_matmul(x, w, o, stream=side[0].cuda_stream))
        torch.cuda.synchronize()
        for y in outs:
            B.check_close(y, val, tol, "bf16")
        idx = np.random.default_rng(0).permutation(m).astype(np.int32)
        gathered = dev(idx)
        torch.cuda.synchronize()
        outs = [M.grouped_matmul(x, w, o, rows=gathered, stream=s) for s in side for _ in range(3)]
        dws = [M.grouped_wgrad(x, x, o, x_rows=gathered, stream=s) for s in side for _ in range(2)]
        torch.cuda.synchronize()
        v2, t2 = B.grouped_ref(xd, wd, off, idx)
        for g in outs:
            B.check_close(g, v2, t2, "bf16")
        v2, t2 = B.wgrad_ref(xd, xd, off, None, idx)
        for g in dws:
            B.check_close(g, v2, t2, "bf16")
        y = torch.zeros_like(outs[0])
        d = torch.zeros(len(sizes), n, k, dtype=torch.bfloat16, device="cuda")
        M.grouped_wgrad(y, x, o, out=d)
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            M.grouped_matmul(x, w, o, out=y)
            M.grouped_wgrad(y, x, o, out=d)
        x2, x2d = values((m, k), 9, "bf16")
        x.copy_(x2)
        g.replay()
        torch.cuda.synchronize()
        val, tol = B.grouped_ref(x2d, wd, off)
        B.check_close(y, val, tol, "bf16")
        dv, dt = B.wgrad_ref(y.double().cpu().numpy(), x2d, off)
        B.check_close(d, dv, dt, "bf16")
        again = M.grouped_matmul(x, w, o)
        assert bool((again == y).all()), "the same inputs gave other bits"


def test_binding_refusals(M):
    import torch
    x = torch.zeros(4, 8, dtype=torch.bfloat16, device="cuda")
    w = torch.zeros(2, 6, 8, dtype=torch.bfloat16, device="cuda")
    o = torch.zeros(3, dtype=torch.int32, device="cuda")
    bad = [dict(x=x.float()), dict(x=x.half()), dict(w=w[0]), dict(w=w.transpose(1, 2)), dict(offsets=o.long()),
           dict(offsets=o[:2]), dict(rows=o.long()), dict(x=x[:, :6]), dict(w_layout="xx"), dict(act="gelu"),
           dict(out=torch.zeros(4, 5, device="cuda")), dict(out=torch.zeros(4, 6, dtype=torch.float64, device="cuda")),
           dict(w=w.cpu()), dict(offsets=o.cpu())]
    for b in bad:
        with pytest.raises(ValueError):
            M.grouped_matmul(**{**dict(x=x, w=w, offsets=o), **b})
    with pytest.raises(M.MoeError):
        M.grouped_matmul(x, w, o, out=torch.zeros(3, 6, device="cuda"))      # fewer rows than x
    with pytest.raises(M.MoeError):
        M.grouped_matmul(x, w.transpose(1, 2).contiguous(), o, w_layout="kn", act="swiglu")
    with pytest.raises(M.MoeError):
        M.grouped_matmul(x[:1].expand(4, 8), w, o)                             # rows on top of one another
    with pytest.raises(ValueError):
        M.grouped_wgrad(x, x.half(), o)
    with pytest.raises(ValueError):
        M.grouped_wgrad(x, x, o, out=torch.zeros(2, 8, 9, device="cuda"))
    assert M.grouped_matmul(x[:0], w, o).shape == (0, 6)
