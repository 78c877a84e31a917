"""Which kernel a grouped product takes: the rule on sizes, types and alignment, without a GPU."""
import pytest

from tests import grouped_cases as G
from tests.test_batch_host import M  # noqa: F401


@pytest.mark.parametrize("sms", [148, 152])
@pytest.mark.parametrize("out", ["bf16", "fp32"])
@pytest.mark.parametrize("form", ["nk", "kn", "swiglu"])
@pytest.mark.parametrize("name", G.PAIR)
def test_cases_of_the_pair_kernel_reach_it(M, name, form, out, sms):
    for more in (dict(), dict(gather=True), dict(scatter=True), dict(pitch=5)):
        a = G.args(M, *G.PAIR[name], kn=form == "kn", swiglu=form == "swiglu", out=out, **more)
        assert M.grouped_kernel(a, sms) == M.GROUPED_PAIR, more


def test_few_rows(M):
    for sizes, n, k in (([1] * 8, 2048, 7168), ([16] * 4, 4096, 4096), ([24] * 32, 512, 512), ([100, 28], 4096, 2048)):
        assert M.grouped_kernel(G.args(M, sizes, n, k), 152) == M.GROUPED_FEW
        assert M.grouped_kernel(G.args(M, sizes, n, k, gather=True), 152) == M.GROUPED_FEW
    # 16 rows a group that m rows can reach, and one more row
    assert M.grouped_kernel(G.args(M, [16] * 64, 4096, 4096), 152) == M.GROUPED_FEW
    assert M.grouped_kernel(G.args(M, [16] * 63 + [17], 4096, 4096), 152) == M.GROUPED_PAIR


def test_operands_that_tensor_maps_cannot_take(M):
    sizes, n, k = G.PAIR["uneven"]
    for field, value in (("x", 4098), ("w", 4104), ("ldx", k + 4), ("ldw", k + 1), ("w_stride", n * k + 2), ("w_stride", 0),
                         ("w", 4096 + 2)):
        a = G.args(M, sizes, n, k)
        setattr(a, field, value)
        assert M.grouped_kernel(a, 152) == M.GROUPED_ANY, field
    a = G.args(M, sizes, n, k, gather=True)
    a.workspace_bytes -= 1
    assert M.grouped_kernel(a, 152) == M.GROUPED_ANY
    a.x_rows = 0
    assert M.grouped_kernel(a, 152) == M.GROUPED_ANY
    one = G.args(M, [2000], 1056, 2056)
    one.w_stride = 0       # of a single expert it does not matter
    assert M.grouped_kernel(one, 152) == M.GROUPED_PAIR
    few = G.args(M, [1] * 8, 2048, 7168)
    few.ldx = 7169
    assert M.grouped_kernel(few, 152) == M.GROUPED_ANY


def test_weight_gradients(M):
    assert M.grouped_kernel(G.wgrad_args(M, [5, 0, 3], 8, 8), 152) == M.GROUPED_PAIR
    assert M.grouped_kernel(G.wgrad_args(M, [5, 0, 3], 264, 520, dy_rows=True, x_rows=True, out="fp32"), 152) == M.GROUPED_PAIR
    assert M.grouped_kernel(G.wgrad_args(M, [5, 0, 3], 8, 7), 152) == M.GROUPED_ANY
    a = G.wgrad_args(M, [5, 0, 3], 264, 520, dy_rows=True, x_rows=True)
    a.workspace_bytes -= 16
    assert M.grouped_kernel(a, 152) == M.GROUPED_ANY
    a = G.wgrad_args(M, [5, 0, 3], 8, 8)
    a.lddw, a.dw = 9, 4098                      # the result's pitch and start do not count
    a.dw_stride = 72
    assert M.grouped_kernel(a, 152) == M.GROUPED_PAIR
    a.m = 0
    assert M.grouped_kernel(a, 152) == M.GROUPED_ANY


def test_calls_that_launch_nothing(M):
    assert M.grouped_kernel(G.args(M, [1, 2], 64, 64, m=0), 152) == M.GROUPED_NONE
    a = G.args(M, [1, 2], 64, 64)
    a.n = 0
    assert M.grouped_kernel(a, 152) == M.GROUPED_NONE
    assert M.grouped_kernel(G.args(M, [1, 2], 64, 64), 0) == M.GROUPED_NONE
    w = G.wgrad_args(M, [1, 2], 64, 64)
    w.groups = 0
    assert M.grouped_kernel(w, 152) == M.GROUPED_NONE


def test_an_empty_x_may_have_no_address(M):
    """Rows named by number of an x without rows are rows of zeros."""
    a = G.args(M, [4, 3], 64, 64, gather=True)
    a.x, a.x_rows = None, 0
    assert M.grouped_kernel(a, 152) == M.GROUPED_ANY
    a.x_rows = 1
    assert M.grouped_kernel(a, 152) == M.GROUPED_NONE
    a.x_rows, a.rows = 0, None       # rows by their place would stand outside it
    assert M.grouped_kernel(a, 152) == M.GROUPED_NONE
    w = G.wgrad_args(M, [4, 3], 64, 64, dy_rows=True)
    w.dy, w.dy_rows_n = None, 0
    assert M.grouped_kernel(w, 152) == M.GROUPED_ANY
    w.dy_rows = None
    assert M.grouped_kernel(w, 152) == M.GROUPED_NONE


def test_waits_stay_bounded(M):
    with pytest.raises(M.MoeError) as e:
        M.debug_batch_wait(2 ** 36 + 1)
    assert e.value.status == M.EINVAL
