"""What numbers that are none, and pairs that were masked, do to the operators on rows."""
import numpy as np
import pytest

from tests import batch_helpers as B
from tests import rows_helpers as R
from tests.test_gpu_grouped import M  # noqa: F401
from tests.test_gpu_rows import f64, make

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("H", [64, 300, 2047, 2048, 7168])
def test_gain_that_is_no_number(M, H):  # noqa: F811
    """A NaN of the gain makes its column NaN.  An infinity makes its column infinite; in 8 bits every row with something in that
    column gets an infinite scale, under which it is 0, and NaN in the column."""
    import torch
    x, gain = make((5, H), "bf16", 1), make((1, H), "fp32", 3)[0]
    x[3, 7] = 0
    y, _ = R.norm_ref(f64(x), f64(gain), np.float64(np.float32(1e-6)))
    rest = np.delete(np.arange(H), 7)
    gain[7] = float("nan")
    n = M.rms_norm(x, gain=gain, want=("out", "out8"), out_dtype=torch.float32)
    assert np.isnan(f64(n.out)[:, 7]).all() and np.isnan(f64(n.out8.float())[:, 7]).all()
    R.check_norm(f64(n.out)[:, rest], y[:, rest], "fp32")
    R.check_eight(f64(n.out8.float())[:, rest], f64(n.scale), y[:, rest], R.Y_TOL)
    gain[7] = float("inf")
    n = M.rms_norm(x, gain=gain, want=("out", "out8"), out_dtype=torch.float32)
    o, q, s = f64(n.out), f64(n.out8.float()), f64(n.scale)
    R.check_norm(o[:, rest], y[:, rest], "fp32")
    has = [0, 1, 2, 4]
    assert np.isinf(o[has, 7]).all() and np.isnan(o[3, 7])            # 0 times infinity
    assert np.isinf(s[has]).all() and (q[has][:, rest] == 0).all() and np.isnan(q[has, 7]).all()
    assert np.isfinite(s[3]) and np.isnan(q[3, 7])
    R.check_eight(q[3:4, rest], s[3:4], y[3:4, rest], R.Y_TOL)


def test_combine_rows_backward_of_masked_pairs(M):  # noqa: F811
    """A weight of 0 has its gradient, the product with its row, as any other; a masked pair whose row was never written is named by
    a place outside y, and has none."""
    import torch
    y, w, d = make((12, 72), "bf16", 1), make((4, 3), "fp32", 2), make((4, 72), "bf16", 3)
    w[0, 1], w[2] = 0, 0
    dy, dw = M.combine_rows_backward(d, y, w)
    (rdy, written), dws = R.combine_grad_ref(f64(d), f64(y), f64(w), np.arange(12).reshape(4, 3))
    B.check_close(dw, *dws, "fp32")
    assert (f64(dw)[2] != 0).all() and (dy[6:9] == 0).all() and (dy[1] == 0).all()
    y[6:9] = float("nan")                                             # never written
    places = np.arange(12).reshape(4, 3)
    places[2] = -1
    dy, dw = M.combine_rows_backward(d, y, w, places=torch.from_numpy(places.astype(np.int32)).cuda(),
                                     out=(torch.full_like(y, 7), torch.empty(4, 3, device="cuda")))
    (rdy, written), dws = R.combine_grad_ref(f64(d), np.nan_to_num(f64(y)), f64(w), places)
    B.check_close(dw, *dws, "fp32")
    assert (dw[2] == 0).all() and (dy[6:9] == 7).all()
