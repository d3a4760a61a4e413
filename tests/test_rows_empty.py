"""Calls on no rows at all: pointers of empty tensors are null, and every call accepts them."""
import pytest

from test_rows_abi import INVALID, OK, distill, embed, embed_grad, logprobs, logprobs_grad


@pytest.mark.parametrize("grad", [False, True])
def test_distill_of_no_rows_takes_null_pointers(grad):
    null = dict(z=None, ids=None, t=None, labels=None, weights=None, d_loss=None, loss=None, accept=None, dz=None)
    assert distill(grad, N=0, **null) == OK
    assert distill(grad, N=0, K=0, **null) == OK
    # what does not depend on the rows is still checked
    assert distill(grad, N=0, tau=0.0, **null) == INVALID
    assert distill(grad, N=0, ws=None, **null) == INVALID
    assert distill(grad, N=0, **(null | dict(ids=0x10000002))) == INVALID
    # with rows the teacher is required as before
    assert distill(grad, N=1, ids=None, t=None) == INVALID


def test_the_other_calls_on_no_rows_take_null_pointers():
    assert logprobs(N=0, z=None, tokens=None, logprob=None, entropy=None, rank=None, row_max=None,
                    row_sumexp=None, ids=None, top=None) == OK
    assert logprobs_grad(N=0, z=None, tokens=None, row_max=None, row_sumexp=None, entropy=None, d_logprob=None,
                         d_entropy=None, dz=None) == OK
    assert embed(N=0, ids=None, out=None) == OK
    assert embed_grad(N=0, ids=None, d_out=None, accumulate=1) == OK
