"""Rows whose elements lie past 2^31 and 2^32 from the start, of every operator on rows; the last rows against the plain forms."""
import numpy as np
import pytest

from tests import batch_helpers as B
from tests import rows_helpers as R
from tests.test_gpu_grouped import M, dev  # noqa: F401
from tests.test_gpu_rows import f64

pytestmark = pytest.mark.gpu

T, H = 140000, 32768          # 4.6e9 elements
LAST = [0, 65536, 65537, 131072, T - 2, T - 1]


@pytest.fixture(scope="module")
def x():
    import torch
    g = torch.Generator(device="cuda").manual_seed(0)
    x = torch.empty(T, H, dtype=torch.bfloat16, device="cuda").fill_(0.5)
    x[LAST] = torch.randn(len(LAST), H, generator=g, device="cuda").bfloat16()
    yield x
    del x
    torch.cuda.empty_cache()


def test_norm_and_its_gradient(M, x):  # noqa: F811
    import torch
    gain = torch.randn(H, device="cuda")
    n = M.rms_norm(x, gain=gain, want=("out", "out8", "rstd"))
    y, rstd = R.norm_ref(f64(x[LAST]), f64(gain), np.float64(np.float32(1e-6)))
    R.check_norm(f64(n.out[LAST]), y, "bf16")
    R.check_eight(f64(n.out8[LAST].float()), f64(n.scale[LAST]), y, R.Y_TOL)
    dh, _ = M.rms_norm_backward(n.out, x, n.rstd, gain=gain, out=(n.out, None))
    (ref, tol), _ = R.norm_grad_ref(f64(M.rms_norm(x[LAST], gain=gain).out), f64(x[LAST]), f64(n.rstd[LAST]), f64(gain), None)
    B.check_close(dh[LAST], ref, tol, "bf16")


def test_quantised(M, x):  # noqa: F811
    q, s = M.quantize_rows(x)
    R.check_eight(f64(q[LAST].float()), f64(s[LAST]), f64(x[LAST]), 0.0)


def test_combined(M, x):  # noqa: F811
    import torch
    places = torch.tensor([[T - 1, 0], [65537, 131072], [T - 2, 65536]], dtype=torch.int32, device="cuda")
    w, d = torch.randn(3, 2, device="cuda"), torch.randn(3, H, device="cuda").bfloat16()
    rows = f64(x[LAST])
    at = {r: i for i, r in enumerate(LAST)}
    p = np.vectorize(at.get)(places.cpu().numpy())
    B.check_close(M.combine_rows(x, w, places=places), *R.combine_ref(rows, f64(w), p), "bf16")
    dy = torch.empty_like(x)
    _, dw = M.combine_rows_backward(d, x, w, places=places, out=(dy, torch.empty(3, 2, device="cuda")))
    (ref, _), dws = R.combine_grad_ref(f64(d), rows, f64(w), p)
    B.check_close(dy[LAST], ref, B.HALF_STEP["fp32"] * np.abs(ref), "bf16")
    B.check_close(dw, *dws, "fp32")


def test_products_of_far_rows_and_experts(M):  # noqa: F811
    """Experts' weights past 2^32 bytes, rows named past 2^31."""
    import torch
    E, n, k = 40, 4096, 32768                                       # 5.4e9 bytes
    g = torch.Generator(device="cuda").manual_seed(1)
    w = torch.empty(E, n, k, dtype=torch.uint8, device="cuda").fill_(0x30)
    few = [0, 31, 32, 39]
    w[few] = torch.randint(0, 0x40, (4, n, k), generator=g, device="cuda", dtype=torch.uint8)
    rows_n = 70000
    x = torch.empty(rows_n, k, dtype=torch.uint8, device="cuda").fill_(0x30)
    used = [0, 65535, 65536, rows_n - 1]
    x[used] = torch.randint(0, 0x40, (4, k), generator=g, device="cuda", dtype=torch.uint8)
    ws, xs = torch.rand(E, n, generator=g, device="cuda") * 1e-3, torch.rand(rows_n, generator=g, device="cuda")
    for per in (1, 300):
        sizes = [per if e in few else 0 for e in range(E)]
        rows = np.concatenate([np.full(per, r) for r in used]).astype(np.int32)
        out = M.grouped_matmul8(x.view(torch.float8_e4m3fn), xs, w.view(torch.float8_e4m3fn), ws, dev(B.make_groups(sizes, None)),
                                rows=dev(rows), out_dtype=torch.float32)
        for i, e in enumerate(few):
            xv = x[used[i]].view(torch.float8_e4m3fn).double() * xs[used[i]].double()
            wv = w[e].view(torch.float8_e4m3fn).double() * ws[e].double()[:, None]
            got = out[i * per: (i + 1) * per].double()
            tol = B.sum_bound(k, wv.abs() @ xv.abs()) + B.HALF_STEP["fp32"] * (wv @ xv).abs()
            assert ((got - wv @ xv).abs() <= tol).all()


@pytest.mark.parametrize("H", [64, 1000, 1024, 2047, 4096, 7168, 8192])
@pytest.mark.parametrize("sign", [False, True], ids=["random", "one sign"])
def test_gain_gradient_over_many_rows(M, H, sign):  # noqa: F811
    """Each block adds its rows in fp32, one after another: 921 of them at most (152 blocks), 8 warps' and 32 blocks' sums behind that, with a
    product's two roundings each: (921 + 8 + 10 + 32 + 2) 2^-24 of the sum of the absolute products."""
    import torch
    rows = 140000
    g = torch.Generator(device="cuda").manual_seed(H)
    dy, h = (torch.randn(rows, H, generator=g, device="cuda").bfloat16() for _ in range(2))
    if sign:
        dy, h = dy.abs(), h.abs()
    rstd = torch.rsqrt(h.float().square().mean(1) + 1e-6)
    _, dgain = M.rms_norm_backward(dy, h, rstd, gain=torch.ones(H, device="cuda"))
    want, absum = torch.zeros(H, dtype=torch.float64, device="cuda"), torch.zeros(H, dtype=torch.float64, device="cuda")
    for t in range(0, rows, 20000):
        p = dy[t:t + 20000].double() * h[t:t + 20000].double() * rstd[t:t + 20000, None].double()
        want += p.sum(0)
        absum += p.abs().sum(0)
    assert bool(((dgain.double() - want).abs() <= 973 * R.U * absum + R.U * want.abs()).all())
