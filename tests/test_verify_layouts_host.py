"""Which layouts of p and q the verification takes, without a GPU: refusals come before anything is launched."""
import ctypes

import pytest

from tests.test_batch_host import M, P  # noqa: F401


def status(M, **over):
    a = dict(p=P, q=P, draft=P, lengths=None, u=P, accepted=P, tokens=P, p_seq=400, p_row=100, q_seq=300, q_row=100, B=2,
             D=3, V=100, dtype=2)
    a.update(over)
    return M.lib().moe_verify_draft(ctypes.byref(M.VerifyArgs(**a)), None)


@pytest.mark.parametrize("over", [
    dict(p_seq=399), dict(p_seq=100, p_row=199), dict(p_seq=99, p_row=400), dict(p_row=99), dict(q_seq=299), dict(q_seq=99, q_row=500),
    dict(q_seq=100, q_row=199), dict(B=3, p_seq=100, p_row=299), dict(B=1, p_row=99), dict(B=2 ** 31 - 1, p_seq=2 ** 39, p_row=2 ** 39),
    dict(p_row=2 ** 61), dict(p_seq=-1)], ids=str)
def test_rows_on_one_another_are_refused(M, over):
    assert status(M, **over) == M.EINVAL


def test_layouts_that_are_taken(M):
    """The call behind the checks fails for want of a device."""
    import torch
    if torch.cuda.is_available():
        pytest.skip("would launch")
    for over in (dict(), dict(p_seq=100, p_row=200), dict(q_seq=100, q_row=200), dict(B=1, p_seq=0, q_seq=0),
                 dict(B=1, p_seq=100, p_row=500, q_seq=100, q_row=500), dict(D=0, p_seq=100, q=None)):
        assert status(M, **over) == M.ECUDA, over
