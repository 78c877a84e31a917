"""Sums of the grouped products that leave no room for a coarser one: whole numbers, whose fp32 sums are exact in any
order, and long contractions that a running sum cut off at each step would lose."""
import numpy as np
import pytest

from tests import batch_helpers as B
from tests.test_gpu_grouped import M, dev  # noqa: F401

pytestmark = pytest.mark.gpu

BIG = 4096.0    # its square is 2^24: the next larger fp32 is two further


def whole(shape, seed, dtype, top=8):
    """Whole numbers in [-top, top]: (device tensor, its values in fp64)"""
    v = np.random.default_rng(seed).integers(-top, top + 1, shape).astype(np.float64)
    return dev(v, B.torch_type(dtype)), v


# few rows a group, tiles that stand at once, many rows, odd widths: the kernels that the sizes lead to
WHOLE = [([1, 0, 3, 2], 264, 2056), ([40, 0, 300], 264, 192), ([0, 1, 37, 600, 255, 257, 513, 385], 1056, 2056),
         ([130, 33], 261, 2055), ([1, 0, 3, 2], 1024, 14336)]


@pytest.mark.parametrize("out", ["fp32", "bf16", "fp16"])
@pytest.mark.parametrize("kn", [False, True], ids=["nk", "kn"])
@pytest.mark.parametrize("case", range(len(WHOLE)))
def test_products_of_whole_numbers_are_rounded_once(M, case, kn, out):
    """|sum| <= 64 k < 2^24, so the only rounding is the result's own."""
    import torch
    sizes, n, k = WHOLE[case]
    t = out if out != "fp32" else "bf16"
    x, xd = whole((sum(sizes), k), case, t)
    w, wd = whole((len(sizes), k, n) if kn else (len(sizes), n, k), case + 1, t)
    off = B.make_groups(sizes, None)
    got = M.grouped_matmul(x, w, dev(off), w_layout="kn" if kn else "nk", out_dtype=B.torch_type(out))
    val, _ = B.grouped_ref(xd, wd, off, None, kn)
    assert torch.equal(got.cpu(), torch.from_numpy(val).to(B.torch_type(out)))


@pytest.mark.parametrize("out", ["fp32", "bf16", "fp16"])
@pytest.mark.parametrize("sizes,n,k", [([700, 0, 31, 64], 264, 520), ([1025, 3], 33, 47), ([0, 4000], 264, 136)])
def test_weight_gradients_of_whole_numbers_are_rounded_once(M, sizes, n, k, out):
    import torch
    t = out if out != "fp32" else "fp16"
    dy, dyd = whole((sum(sizes), n), 1, t)
    x, xd = whole((sum(sizes), k), 2, t)
    off = B.make_groups(sizes, None)
    got = M.grouped_wgrad(dy, x, dev(off), out_dtype=B.torch_type(out))
    assert torch.equal(got.cpu(), torch.from_numpy(B.wgrad_ref(dyd, xd, off)[0]).to(B.torch_type(out)))


def far_sum(length):
    """Two factors of `length` numbers: 2^24 at first, then one 1 in every 16 from element 512 on, and in the end -2^24 with
    nothing beside it in its part of 512; and how many ones.  A sum held in fp32 over parts of at most 512 elements is exact;
    one that runs on over the whole length stands at 2^24, where a 1 is below half of its step, and loses them all."""
    a, b = np.zeros(length), np.zeros(length)
    a[0], b[0] = BIG, BIG
    a[-1], b[-1] = BIG, -BIG
    end = (length - 1) // 512 * 512
    a[512:end:16], b[512:end:16] = 1, 1
    return a, b, (end - 512) // 16


@pytest.mark.parametrize("out", ["fp16", "bf16", "fp32"])
@pytest.mark.parametrize("form", ["nk", "kn", "swiglu"])
@pytest.mark.parametrize("sizes,n,k", [([300, 290], 2560, 20480), ([300, 290], 1280, 33288), ([2, 1], 256, 20480),
                                       ([33, 2], 33, 20481)])
def test_long_contractions_lose_nothing(M, sizes, n, k, form, out):
    import torch
    a, b, ones = far_sum(k)
    t = B.torch_type(out if out != "fp32" else "fp16")
    E, sw = len(sizes), form == "swiglu"
    x = dev(a, t).expand(sum(sizes), k).contiguous()
    w = torch.zeros(E, n * (2 if sw else 1), k, dtype=t, device="cuda")
    w[:, -n:] = dev(b, t)
    want = float(ones)
    if sw:
        w[:, :n, 512] = 1        # a gate of one
        want = ones / (1 + np.exp(-1.0))
    if form == "kn":
        w = w.transpose(1, 2).contiguous()
    y = M.grouped_matmul(x, w, dev(B.make_groups(sizes, None)), w_layout="kn" if form == "kn" else "nk",
                         act="swiglu" if sw else None, out_dtype=B.torch_type(out))
    # exact but for SwiGLU's exponential, division and products (a few steps each), and the result's own rounding
    tol = (8 * 2.0 ** -23 if sw else 0) * want + (B.HALF_STEP[out] * want if sw or out != "fp32" else 0)
    assert float((y.double() - want).abs().max()) <= tol, (float(y.min()), float(y.max()), want)


@pytest.mark.parametrize("out", ["fp16", "bf16", "fp32"])
@pytest.mark.parametrize("n,k", [(264, 520), (40, 8), (33, 7)])
def test_long_groups_of_a_weight_gradient_lose_nothing(M, n, k, out):
    """Groups longer and shorter than what is summed in one go, in one call."""
    import torch
    sizes = [20485, 40, 0, 16384, 65536]
    t = B.torch_type(out if out != "fp32" else "fp16")
    cols = [far_sum(s) if s > 20000 else (np.ones(s), np.ones(s), s) for s in sizes if s]
    a, b = (np.concatenate([c[i] for c in cols]) for i in (0, 1))
    want = np.array([cols[0][2], 40, 0, 16384, cols[-1][2]], float)
    dy = dev(a, t)[:, None].expand(-1, n).contiguous()
    x = dev(b, t)[:, None].expand(-1, k).contiguous()
    g = M.grouped_wgrad(dy, x, dev(B.make_groups(sizes, None)), out_dtype=B.torch_type(out)).double().cpu().numpy()
    tol = (B.HALF_STEP[out] if out != "fp32" else 0) * want
    assert (np.abs(g - want[:, None, None]) <= tol[:, None, None]).all(), (g.min((1, 2)), g.max((1, 2)), want)


@pytest.mark.parametrize("sizes,n,k", [([3, 2], 1024, 64), ([512, 700, 33, 800], 1536, 192), ([70, 2], 999, 65)])
def test_swiglu_over_the_range_of_its_gate(M, sizes, n, k):
    """Gates from deep in the exponential's underflow to past its overflow, with factors that bring the product back."""
    import torch
    E, m = len(sizes), sum(sizes)
    g = np.concatenate([np.linspace(-104, 104, n - 8), [-87.5, -88, -88.5, -0.0, 0.0, -1e-30, 30000.0, -30000.0]])
    u = np.where(np.arange(n) % 2 == 0, 2.0 ** 60, -1.5)
    w = torch.zeros(E, 2 * n, k, dtype=torch.bfloat16, device="cuda")
    w[:, :n, 0], w[:, n:, 0] = dev(g, torch.bfloat16), dev(u, torch.bfloat16)
    x = torch.zeros(m, k, dtype=torch.bfloat16, device="cuda")
    x[:, 0] = 1
    y = M.grouped_matmul(x, w, dev(B.make_groups(sizes, None)), act="swiglu", out_dtype=torch.float32).double().cpu().numpy()
    g, u = w[0, :n, 0].double().cpu().numpy(), w[0, n:, 0].double().cpu().numpy()
    with np.errstate(over="ignore"):
        want = g / (1 + np.exp(-g)) * u
    # the exponential, two products, a sum and a division, each within a step or two; below 2^-126 the exponential and the
    # quotient have steps of 2^-149 each, which the gate and the factor multiply, and so has the result
    tol = 8 * 2.0 ** -23 * np.abs(want) + 2 * 2.0 ** -149 * (np.abs(g * u) + 1)
    bad = np.argwhere(~(np.abs(y - want) <= tol))
    assert not len(bad), [(g[c], u[c], y[r, c], want[c]) for r, c in bad[:3]]


def test_a_group_that_takes_longer_than_a_wait(M):
    """300 million rows in one group of one tile: more than a second of steps in front of the one that ends the group.  They
    are summed, and the next call finds nothing wrong."""
    import torch
    if torch.cuda.mem_get_info()[0] < 24 << 30:
        pytest.skip("needs 24 GB")
    m = 300_000_037
    t = torch.ones(m, 8, dtype=torch.bfloat16, device="cuda")
    o = torch.tensor([0, m - 3, m], dtype=torch.int32, device="cuda")
    for out in (torch.bfloat16, torch.float32):
        g = M.grouped_wgrad(t, t, o, out_dtype=out)
        torch.cuda.synchronize()
        # parts of 512 ones are exact, and so is their sum up to the last one (below 2^29 fp32 has steps of 32)
        assert float((g[0].double() - (m - 3)).abs().max()) <= 32 + (B.HALF_STEP["bf16"] * m if out == torch.bfloat16 else 0)
        assert bool((g[1] == 3).all())
    assert float(M.grouped_wgrad(t[:70], t[:70], torch.tensor([0, 70], dtype=torch.int32, device="cuda")).max()) == 70


@pytest.mark.parametrize("out", ["fp16", "bf16", "fp32"])
def test_long_group_into_rows_of_an_odd_pitch(M, out):
    """The same in a result that leaves the kernel element by element."""
    import torch
    sizes, n, k = [20485, 40], 264, 520
    a, b, ones = far_sum(sizes[0])
    t = B.torch_type(out if out != "fp32" else "bf16")
    dy = torch.ones(sum(sizes), n, dtype=t, device="cuda")
    x = torch.ones(sum(sizes), k, dtype=t, device="cuda")
    scale = 1 + np.arange(n) % 4             # each row of the gradient its own multiple
    dy[:sizes[0]] = dev(a[:, None] * np.where(a[:, None] == 1, scale, 1), t)
    x[:sizes[0]] = dev(b, t)[:, None]
    full = torch.full((2, n + 1, k + 3), 7.0, dtype=B.torch_type(out), device="cuda")
    M.grouped_wgrad(dy, x, dev(B.make_groups(sizes, None)), out=full[:, :n, :k])
    want = np.stack([ones * scale, np.full(n, 40)])[:, :, None]
    g = full[:, :n, :k].double().cpu().numpy()
    assert (np.abs(g - want) <= (B.HALF_STEP[out] * want if out != "fp32" else 0)).all(), (g.min((1, 2)), g.max((1, 2)))
    assert bool((full[:, n:] == 7).all()) and bool((full[:, :, k:] == 7).all())
