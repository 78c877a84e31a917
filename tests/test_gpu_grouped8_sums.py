"""Sums and scales of the 8-bit products that leave no room for a coarser one."""
import numpy as np
import pytest

from tests import batch_helpers as B
from tests.test_gpu_grouped import M, dev  # noqa: F401

pytestmark = pytest.mark.gpu


def numbers(values):
    """(e4m3 tensor of them, which hold them all)"""
    import torch
    t = torch.from_numpy(np.asarray(values, np.float32)).cuda()
    q = t.to(torch.float8_e4m3fn)
    assert (q.float() == t).all()
    return q


@pytest.mark.parametrize("xs,ws", [(2e-28, 1e-18), (1e-18, 2e-28), (1e-20, 1e-21), (5e27, 1e11), (2e11, 3e27), (1e25, 1e-30)])
@pytest.mark.parametrize("swiglu", [False, True], ids=["plain", "swiglu"])
@pytest.mark.parametrize("sizes,n,k", [([1, 2], 256, 512), ([700, 600], 1024, 4096)])
def test_scales_whose_product_leaves_fp32(M, sizes, n, k, swiglu, xs, ws):  # noqa: F811
    """The sums, of one number's square, are exact; each scale then costs a rounding, 2^-24 of the value."""
    import torch
    m, v = sum(sizes), 448.0 if xs * ws < 1 else 2.0 ** -9
    x, w = numbers(np.full((m, k), v)), torch.empty(2, n, k, dtype=torch.float8_e4m3fn, device="cuda")
    w.copy_(numbers([v])[0])
    x_scale, w_scale = torch.full((m,), xs, device="cuda"), torch.full((2, n), ws, device="cuda")
    if swiglu:   # a gate of 32, which is its own SiLU (e^-32 is below fp32's last bit)
        w[:, : n // 2] = numbers([1])[0]
        w_scale[:, : n // 2] = float(32 / (v * k * xs))
    got = M.grouped_matmul8(x, x_scale, w, w_scale, dev(B.make_groups(sizes, None)), act="swiglu" if swiglu else None,
                            out_dtype=torch.float32).double()
    want = v * v * k * float(x_scale[0]) * float(w_scale[0, -1])
    if swiglu:
        want *= v * k * float(x_scale[0]) * float(w_scale[0, 0])
    assert 2.0 ** -126 < want < 3e38
    # two products of each sum, and SiLU's exponential, division and two products of a few steps each
    assert float((got - want).abs().max()) <= (4 + 16 if swiglu else 2) * 2.0 ** -24 * want


# few rows a group, tiles that stand at once, many rows, odd widths; contractions that end on a stage of 128, 16 before and behind it, and
# around the 32768 elements that 16-bit results are summed over in one go
WHOLE = [([1, 0, 3, 2], 264, 2064), ([4, 0, 9, 2], 1032, 32784), ([40, 0, 300], 264, 192), ([0, 1, 37, 600, 255, 257, 513, 385], 1056, 2064),
         ([130, 33], 261, 2032), ([300, 260, 300], 3000, 32752), ([300, 260, 300], 3000, 32768), ([300, 260, 300], 2999, 32784),
         ([300, 260, 300], 1500, 33024)]


@pytest.mark.parametrize("out", ["fp32", "bf16", "fp16"])
@pytest.mark.parametrize("form", ["plain", "gather", "scatter"])
@pytest.mark.parametrize("case", range(len(WHOLE)))
def test_products_of_whole_numbers_are_rounded_once(M, case, form, out):  # noqa: F811
    """|sum| <= 64 k < 2^24, and scales are powers of two: the only rounding is the result's own, so a stage that is missing, repeated
    or read at the wrong place shows."""
    import torch
    sizes, n, k = WHOLE[case]
    rng = np.random.default_rng(case)
    E, m = len(sizes), sum(sizes)
    R = m // 2 + 1 if form == "gather" else m
    x, w = (torch.from_numpy(rng.integers(-8, 9, s).astype(np.float32)).cuda() for s in ((R, k), (E, n, k)))
    xs, ws = (torch.from_numpy(2.0 ** rng.integers(-4, 2, s).astype(np.float32)).cuda() for s in ((R,), (E, n)))
    offsets = B.make_groups(sizes, None)
    rows = rng.integers(0, R, m) if form == "gather" else np.arange(m)
    at = rng.permutation(m) if form == "scatter" else np.arange(m)
    got = M.grouped_matmul8(x.to(torch.float8_e4m3fn), xs, w.to(torch.float8_e4m3fn), ws, dev(offsets),
                            rows=dev(rows.astype(np.int32)) if form == "gather" else None,
                            out_rows=dev(at.astype(np.int32)) if form == "scatter" else None, out_dtype=B.torch_type(out))
    r, at = torch.from_numpy(rows).cuda(), torch.from_numpy(at).cuda()
    for e in range(E):
        a, z = int(offsets[e]), int(offsets[e + 1])
        val = (x[r[a:z]].double() @ w[e].double().T) * xs[r[a:z]].double()[:, None] * ws[e].double()
        assert torch.equal(got[at[a:z]], val.to(B.torch_type(out)))


def bound(k, out, kernel_part):
    """The header's, relative to the sum of the absolute products: steps of 32 in a part, and as many additions as parts."""
    steps = min(k, 1024 if out == "fp32" else 32768) // 32
    return (steps + -(-k // kernel_part)) * 2.0 ** -23


@pytest.mark.parametrize("out", ["fp32", "fp16"])
@pytest.mark.parametrize("k", [512, 1024, 4096, 16384, 32768, 32896, 131072])
@pytest.mark.parametrize("sizes,n,part", [([1, 2], 256, 512), ([300, 500], 2048, 1024)])
def test_sums_whose_steps_lose_all_that_they_can(M, sizes, n, part, k, out):  # noqa: F811
    """A sum of 1.28e7, whose steps are 1, then 63/64 every 32 elements, each of which is cut off while that sum stands, and in the
    end its negative: what remains is small, so 16-bit results hide nothing."""
    import torch
    a, b = np.zeros(k), np.zeros(k)
    a[:64] = a[-64:] = b[:64] = 448
    b[-64:] = -448
    a[64:-64:32], b[64:-64:32] = 1.125, 0.875
    want, absum = float((a * b).sum()), float(np.abs(a * b).sum())
    x, w = numbers(a).expand(sum(sizes), k).contiguous(), numbers(b).expand(len(sizes), n, k).contiguous()
    one = torch.ones(sum(sizes), device="cuda")
    got = M.grouped_matmul8(x, one, w, torch.ones(len(sizes), n, device="cuda"), dev(B.make_groups(sizes, None)),
                            out_dtype=B.torch_type(out)).double()
    assert float((got - want).abs().max()) <= bound(k, out, part) * absum + B.HALF_STEP[out] * (want + bound(k, out, part) * absum)


@pytest.mark.parametrize("k", [512, 14336, 32768, 131072])
@pytest.mark.parametrize("sizes,n,part", [([1, 2], 256, 512), ([300, 500], 2048, 1024)])
def test_long_sums_of_one_sign(M, sizes, n, part, k):  # noqa: F811
    import torch
    g = torch.Generator(device="cuda").manual_seed(k)
    r = lambda *s: ((1 + torch.rand(*s, generator=g, device="cuda")) * 2.0 ** torch.randint(  # noqa: E731
        -3, 6, s, generator=g, device="cuda")).to(torch.float8_e4m3fn)
    x, w = r(sum(sizes), k), r(len(sizes), n, k)
    offsets = B.make_groups(sizes, None)
    got = M.grouped_matmul8(x, torch.ones(sum(sizes), device="cuda"), w, torch.ones(len(sizes), n, device="cuda"), dev(offsets),
                            out_dtype=torch.float32).double()
    for e in range(len(sizes)):
        a, z = int(offsets[e]), int(offsets[e + 1])
        val = x[a:z].double() @ w[e].double().T
        assert bool(((got[a:z] - val).abs() <= (bound(k, "fp32", part) + 2.0 ** -24) * val).all())
