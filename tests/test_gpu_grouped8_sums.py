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
