"""verify_draft on views (one sequence of a larger tensor, sequences row by row), and on drafts whose probabilities are at the
bottom of fp32's range."""
import numpy as np
import pytest

from tests.test_gpu_batch_route_verify import check_verify, make
from tests.test_gpu_grouped import M  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("D", [0, 1, 4])
@pytest.mark.parametrize("with_q", [True, False], ids=["q", "onehot"])
def test_one_sequence_of_a_time_major_tensor(M, D, with_q):
    """Rows of [D + 1, sequences, V] tensors: rows of one sequence lie further apart than V, and the sequence's own pitch is
    that of the neighbours."""
    import torch
    V, others = 300, 5
    p, draft, u, q = make(1, D, V, "fp32", 3 + D, with_q)
    P = torch.full((D + 1, others, V), float("nan"), device="cuda")
    Q = torch.full((D, others, V), float("nan"), device="cuda")
    for b in (0, others - 1):
        P[:, b] = p[0]
        if with_q:
            Q[:, b] = q[0]
        check_verify(M, P[:, b:b + 1].transpose(0, 1), draft, u, Q[:, b:b + 1].transpose(0, 1) if with_q else None)


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
def test_sequences_of_time_major_tensors(M, dtype):
    """[D + 1, B, V] and [D, B, V] tensors as they come from a model that runs step by step; and one of each kind."""
    for Bn, D, V in ((5, 3, 301), (40, 1, 1000), (2, 0, 64)):
        p, draft, u, q = make(Bn, D, V, dtype, V)
        step = lambda t: t.transpose(0, 1).contiguous().transpose(0, 1)  # noqa: E731
        check_verify(M, step(p), draft, u, step(q))
        check_verify(M, step(p), draft, u, q)
        check_verify(M, p, draft, u, step(q))
        check_verify(M, step(p), draft, u)


def test_drafts_of_the_least_probabilities(M):
    """u q below fp32's least step, where it rounds up to p or down to 0: the comparison is exact."""
    import torch
    V, tiny = 64, 2.0 ** -149
    cases = [(u, q, p) for u in (2.0 ** -24, 0.25, 0.5, 0.75, 1 - 2.0 ** -24, 1e-40, tiny, 0.0) for q in (tiny, 2 * tiny, 3 * tiny, 1e-38, 0.5, 1.0)
             for p in (0.0, tiny, 2 * tiny, 3 * tiny, 1e-39)]
    n = len(cases)
    uu = np.zeros((n, 2), np.float32)
    P, Q = np.zeros((n, 2, V), np.float32), np.zeros((n, 1, V), np.float32)
    P[:, :, 5], Q[:, :, 6] = 0.5, 0.5
    for i, (u, q, p) in enumerate(cases):
        uu[i, 0], P[i, 0, 9], Q[i, 0, 9] = u, p, q
    uu[:, 1] = 0.3
    d = np.full((n, 1), 9)
    acc, _ = check_verify(M, torch.from_numpy(P).cuda(), d, uu, torch.from_numpy(Q).cuda())
    assert 0 < acc.sum() < n
