"""Calls of the grouped products that the binding refuses."""
import pytest

from tests.test_gpu_grouped import M  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("R,S", [(6, 4), (4, 6), (0, 3)])
def test_wgrad_of_factors_with_different_rows(M, R, S):
    """Without row numbers a weight gradient of dy and x of different lengths is a mistake (a forgotten x_rows), not a
    gradient of the rows that both have."""
    import torch
    dy, x = (torch.zeros(r, 8, dtype=torch.bfloat16, device="cuda") for r in (R, S))
    o = torch.zeros(3, dtype=torch.int32, device="cuda")
    with pytest.raises(ValueError, match="rows"):
        M.grouped_wgrad(dy, x, o)
    rows = torch.arange(4, dtype=torch.int32, device="cuda") % max(1, S)
    if R >= 4:
        assert M.grouped_wgrad(dy, x, o, x_rows=rows).shape == (2, 8, 8)
    assert M.grouped_wgrad(dy, x, o, x_rows=rows, dy_rows=rows).shape == (2, 8, 8)
