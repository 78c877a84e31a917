"""Grouped products whose rows are named by number in a tensor without rows: each of them is a row of zeros."""
import pytest

from tests.test_gpu_grouped import M  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("n,k", [(64, 64), (7, 5), (1056, 2056)])
@pytest.mark.parametrize("m", [3, 600])
def test_no_rows_in_x(M, m, n, k):
    import torch
    new = lambda *s: torch.ones(*s, dtype=torch.bfloat16, device="cuda")  # noqa: E731
    rows = torch.zeros(m, dtype=torch.int32, device="cuda")
    o = torch.tensor([0, m // 3, m // 3, m], dtype=torch.int32, device="cuda")
    for lay, w in (("nk", new(3, n, k)), ("kn", new(3, k, n))):
        y = M.grouped_matmul(new(0, k), w, o, rows=rows, w_layout=lay, out=new(m, n))
        assert y.shape == (m, n) and bool((y == 0).all())
    y = M.grouped_matmul(new(0, k), new(3, 2 * n, k), o, rows=rows, act="swiglu", out=new(m, n))
    assert bool((y == 0).all())
    for dy, x, kw in ((new(0, n), new(m, k), dict(dy_rows=rows)), (new(m, n), new(0, k), dict(x_rows=rows)),
                      (new(0, n), new(0, k), dict(dy_rows=rows, x_rows=rows))):
        assert bool((M.grouped_wgrad(dy, x, o, out=new(3, n, k), **kw) == 0).all())
