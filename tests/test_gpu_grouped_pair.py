"""The kernel for pairs of SMs in forward products, against the plain 64-bit forms, on random numbers.  Each case is held
to reach that kernel (and, with sizes that the host test knows, to go on reaching it)."""
import numpy as np
import pytest

from tests import batch_helpers as B
from tests import grouped_cases as G
from tests.test_gpu_grouped import M, dev, run_matmul, values  # noqa: F401

pytestmark = pytest.mark.gpu


def reaches(M, *case, **kw):
    import torch
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    assert M.grouped_kernel(G.args(M, *case, **kw), sms) == M.GROUPED_PAIR


# form, type, result, gathered, scattered, seed (odd: an output pitch that is odd too), first row of the groups, rows behind them
FORMS = [("nk", "bf16", "bf16", False, False, 0, 0, 0), ("nk", "fp16", "fp16", True, True, 1, 3, 2), ("nk", "bf16", "fp32", True, False, 2, 0, 9),
         ("nk", "fp16", "fp32", False, True, 3, 5, 0), ("kn", "bf16", "bf16", True, True, 4, 0, 0), ("kn", "fp16", "fp16", False, False, 5, 1, 70),
         ("kn", "fp16", "fp32", True, True, 7, 0, 0), ("swiglu", "bf16", "bf16", True, False, 8, 0, 5), ("swiglu", "fp16", "fp16", False, True, 9, 2, 0),
         ("swiglu", "bf16", "fp32", True, True, 11, 0, 0), ("swiglu", "fp16", "fp32", False, False, 12, 0, 0), ("swiglu", "bf16", "bf16", True, True, 13, 0, 0)]


@pytest.mark.parametrize("form,dtype,out,gather,scatter,seed,first,tail", FORMS, ids=lambda v: str(v))
@pytest.mark.parametrize("name", G.PAIR)
def test_forms(M, name, form, dtype, out, gather, scatter, seed, first, tail):
    sizes, n, k = G.PAIR[name]
    kn, swiglu = form == "kn", form == "swiglu"
    reaches(M, sizes, n, k, kn=kn, swiglu=swiglu, gather=gather, scatter=scatter, out=out, dtype=dtype,
            pitch=5 if seed % 2 else 8, m=sum(sizes) + first + tail)
    run_matmul(M, sizes, n, k, dtype, kn=kn, swiglu=swiglu, gather=gather, scatter=scatter, out=out, tail=tail, first=first,
               seed=seed)


@pytest.mark.parametrize("out", ["bf16", "fp32"])
@pytest.mark.parametrize("form", ["nk", "kn", "swiglu"])
def test_bad_row_numbers_and_neighbours(M, form, out):
    """Row numbers outside x are zero rows, out rows outside out write nothing; a row of NaN or infinities stays in its own."""
    import torch
    sizes, n, k = G.PAIR["uneven"]
    kn, sw = form == "kn", form == "swiglu"
    m, nw = sum(sizes) + 6, n * (2 if sw else 1)
    reaches(M, sizes, n, k, kn=kn, swiglu=sw, gather=True, scatter=True, out=out, m=m)
    rng = np.random.default_rng(1)
    x, xd = values((m, k), 1, "bf16")
    w, wd = values((8, k, nw) if kn else (8, nw, k), 2, "bf16", k ** -0.5)
    off = B.make_groups(sizes, None)
    rows = rng.permutation(m).astype(np.int32)
    out_rows = rng.permutation(m).astype(np.int32)
    bad = np.array([0, 40, 700, 1000, 2047])
    x[torch.from_numpy(rows[bad].astype(np.int64)).cuda()] = float("nan")
    x[int(rows[41])] = float("inf")
    rows[[3, 300, 1500, 2046]] = [-1, m, 2 ** 31 - 1, -2 ** 31]
    out_rows[[7, 301, 1501]] = [-1, m, 2 ** 31 - 1]
    full = torch.full((m, n), 7.0, dtype=B.torch_type(out), device="cuda")
    M.grouped_matmul(x, w, dev(off), rows=dev(rows), out_rows=dev(out_rows), w_layout="kn" if kn else "nk",
                     act="swiglu" if sw else None, out=full)
    val, tol = B.grouped_ref(xd, wd, off, rows.astype(np.int64), kn, sw)
    live = np.setdiff1d(np.arange(sum(sizes)), np.concatenate([bad, [41, 7, 301, 1501]]))
    to = torch.from_numpy(out_rows.astype(np.int64)).cuda()
    B.check_close(full[to[live]], val[live], tol[live], out)
    assert bool(torch.isnan(full[to[bad]]).all())
    left = np.setdiff1d(np.arange(m), out_rows[: sum(sizes)])
    assert len(left) >= 6 and bool((full[torch.from_numpy(left).cuda()] == 7).all())


@pytest.mark.parametrize("form", ["nk", "kn", "swiglu"])
def test_offsets_that_decrease(M, form):
    """More tiles than m rows can make: nothing is written outside out, and the next call is right."""
    import torch
    E, m, n, k = 64, 1400, 264, 2112
    kn, sw = form == "kn", form == "swiglu"
    reaches(M, [m // E] * E, n, k, kn=kn, swiglu=sw, m=m)
    x, _ = values((m, k), 1, "bf16")
    nw = n * (2 if sw else 1)
    w, _ = values((E, k, nw) if kn else (E, nw, k), 2, "bf16")
    for off in ([0, m] * (E // 2) + [0], [m] * E + [0], [0] * 20 + [m, 5] * 22 + [m]):
        full = torch.full((m + 2, n + 8), 7.0, dtype=torch.bfloat16, device="cuda")
        M.grouped_matmul(x, w, dev(np.array(off, np.int32)), w_layout="kn" if kn else "nk", act="swiglu" if sw else None,
                         out=full[1:m + 1, :n])
        torch.cuda.synchronize()
        assert bool((full[0] == 7).all()) and bool((full[m + 1] == 7).all()) and bool((full[:, n:] == 7).all())
    sizes, n, k = G.PAIR["short k"]
    run_matmul(M, sizes, n, k, "bf16", kn=kn, swiglu=sw)


def test_streams_and_capture(M):
    """Gathered and scattered products on streams of their own, and captured with the routing's kind of workspace."""
    import torch
    sizes, n, k = G.PAIR["short k"]
    E, m = len(sizes), sum(sizes)
    reaches(M, sizes, n, k, gather=True, scatter=True, m=m)
    rng = np.random.default_rng(3)
    x, xd = values((m, k), 1, "bf16")
    w, wd = values((E, n, k), 2, "bf16", k ** -0.5)
    rows, out_rows = (rng.permutation(m).astype(np.int32) for _ in range(2))
    off = B.make_groups(sizes, None)
    o, r, d = dev(off), dev(rows), dev(out_rows)
    torch.cuda.synchronize()

    def check(y, xd):
        val, tol = B.grouped_ref(xd, wd, off, rows)
        B.check_close(y[torch.from_numpy(out_rows.astype(np.int64)).cuda()], val, tol, "bf16")

    outs = [M.grouped_matmul(x, w, o, rows=r, out_rows=d, stream=s) for s in [torch.cuda.Stream() for _ in range(3)] for _ in range(2)]
    torch.cuda.synchronize()
    for y in outs:
        check(y, xd)
    y = torch.empty_like(outs[0])
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        M.grouped_matmul(x, w, o, rows=r, out_rows=d, out=y)
    x2, x2d = values((m, k), 9, "bf16")
    x.copy_(x2)
    g.replay()
    torch.cuda.synchronize()
    check(y, x2d)
    assert torch.equal(y, M.grouped_matmul(x, w, o, rows=r, out_rows=d)), "the same inputs gave other bits"
