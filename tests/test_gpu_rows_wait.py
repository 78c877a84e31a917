"""Device waits of the 8-bit products and the norm's gradient that run out, on a flag that nothing sets: the call ends by itself and the
ones after it say so, until that is forgotten; then everything works as before."""
import pytest

from tests import batch_helpers as B
from tests.test_gpu_grouped import M, dev  # noqa: F401
from tests.test_gpu_grouped8 import PAIR

pytestmark = pytest.mark.gpu


def product(M, sizes, n, k, act):  # noqa: F811
    import torch
    nw = n * (2 if act else 1)
    one = lambda *s: torch.full(s, 0x38, dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn)  # noqa: E731
    return M.grouped_matmul8(one(sum(sizes), k), torch.ones(sum(sizes), device="cuda"), one(len(sizes), nw, k),
                             torch.ones(len(sizes), nw, device="cuda"), dev(B.make_groups(sizes, None)), act=act)


def gradient(M, T, H, dtype):  # noqa: F811
    import torch
    x = torch.ones(T, H, dtype=dtype, device="cuda")
    return M.rms_norm_backward(x, x, torch.ones(T, device="cuda"), gain=torch.ones(H, device="cuda"), dsum=x)[0]


def calls(M):  # noqa: F811
    import torch
    return {"few": lambda: product(M, [3, 1, 2], 1024, 4096, None), "few swiglu": lambda: product(M, [3, 1, 2], 1024, 4096, "swiglu"),
            "pair": lambda: product(M, *PAIR["borders"], None), "pair swiglu": lambda: product(M, *PAIR["borders"], "swiglu"),
            "gradient, two blocks an SM": lambda: gradient(M, 500, 4096, torch.bfloat16),
            "gradient, one block an SM": lambda: gradient(M, 200, 8192, torch.float32)}


@pytest.mark.parametrize("name", ["few", "few swiglu", "pair", "pair swiglu", "gradient, two blocks an SM", "gradient, one block an SM"])
def test_a_wait_that_runs_out(M, name):  # noqa: F811
    import torch
    call = calls(M)[name]
    good = call()
    torch.cuda.synchronize()
    M.debug_batch_wait(0)
    try:
        call()
        torch.cuda.synchronize()              # ends, without an error of the device
        x, f = torch.zeros(4, 64, device="cuda"), torch.zeros(4, 2, device="cuda")
        for after in (call, lambda: M.rms_norm(x), lambda: M.quantize_rows(x), lambda: M.combine_rows(x, f[:2]),
                      lambda: M.combine_rows_backward(x[:2], x, f[:2]), lambda: M.balanced_route(x, 2),
                      lambda: M.balanced_route_backward(f, x, f.int())):
            with pytest.raises(M.MoeError) as e:
                after()
            assert e.value.status == M.ETIMEOUT
    finally:
        torch.cuda.synchronize()
        M.debug_batch_wait()
    assert torch.equal(call(), good)
