"""A device wait of a grouped product that runs out, on a flag that nothing sets: the call ends by itself and the ones after it say
so, until that is forgotten; then everything works as before."""
import pytest

from tests import batch_helpers as B
from tests import grouped_cases as G
from tests.test_gpu_grouped import M, dev, run_matmul  # noqa: F401

pytestmark = pytest.mark.gpu

FEW, ODD = ([3, 1, 2], 1024, 4096), ([70, 0, 33], 261, 135)
CASES = {"few": FEW, "pair": G.PAIR["short k"], "any": ODD}


def run(M, form, case):
    import torch
    sizes, n, k = case
    E, m = len(sizes), sum(sizes)
    x = torch.ones(m, k, dtype=torch.bfloat16, device="cuda")
    o = dev(B.make_groups(sizes, None))
    if form == "wgrad":
        return M.grouped_wgrad(torch.ones(m, n, dtype=torch.bfloat16, device="cuda"), x, o, out_dtype=torch.float32)
    nw = n * (2 if form == "swiglu" else 1)
    w = torch.ones(*((E, k, nw) if form == "kn" else (E, nw, k)), dtype=torch.bfloat16, device="cuda")
    return M.grouped_matmul(x, w, o, w_layout="kn" if form == "kn" else "nk", act="swiglu" if form == "swiglu" else None)


@pytest.mark.parametrize("name,form", [(n, f) for n in CASES for f in ("nk", "kn", "swiglu", "wgrad") if (n, f) != ("few", "wgrad")])
def test_a_wait_that_runs_out(M, name, form):
    import torch
    case = CASES[name]
    good = run(M, form, case)
    torch.cuda.synchronize()
    M.debug_batch_wait(0)
    try:
        run(M, form, case)
        torch.cuda.synchronize()              # ends, without an error of the device
        logits = torch.zeros(4, 8, device="cuda")
        p = torch.full((1, 2, 4), 0.25, device="cuda")
        for call in (lambda: run(M, form, case), lambda: M.group_route(logits, 2),
                     lambda: M.verify_draft(p, torch.zeros(1, 1, dtype=torch.int32, device="cuda"), torch.zeros(1, 2, device="cuda"))):
            with pytest.raises(M.MoeError) as e:
                call()
            assert e.value.status == M.ETIMEOUT
    finally:
        torch.cuda.synchronize()
        M.debug_batch_wait()
    assert torch.equal(run(M, form, case), good)
    if form != "wgrad":
        run_matmul(M, *case, "bf16", kn=form == "kn", swiglu=form == "swiglu")


def test_a_bound_that_is_long_enough(M):
    import torch
    M.debug_batch_wait(500_000_000)
    try:
        a = run(M, "nk", G.PAIR["short k"])
        torch.cuda.synchronize()
    finally:
        M.debug_batch_wait()
    assert torch.equal(a, run(M, "nk", G.PAIR["short k"]))
