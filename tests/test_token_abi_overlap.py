"""Which gradients the distillation takes beside its logits: any that shares no
element with them, rows of the two that lie in between one another among them.
Host checks only; device pointers are fake and never dereferenced."""
import pytest

from test_token_abi import FAKE, _api, mat, teacher

ROWS, COLS = 5000, 16


def _refused(logits, grad):
    """Status of a call without a workspace: 1 where the matrices are taken."""
    L, te = _api()._lib(), teacher()
    a = L.tbe_distill_backward(logits, te, FAKE, None, 1.0, grad, None, 0, None, None)
    b = L.tbe_distill_loss_grad(logits, te, None, 1.0, FAKE, FAKE, grad, None, 0, None, None, None)
    assert a == b
    return a


# bytes from the logits to the gradient, stride in elements, columns
@pytest.mark.parametrize("off,stride,cols", [(4 * 16, 32, 16), (-4 * 16, 32, 16), (4 * 17, 40, 16), (4 * 24, 40, 16),
                                             (4 * (40 * 70 + 16), 40, 16), (4 * (24 - 40 * 3), 40, 16), (4, 2, 1)])
def test_rows_between_one_another_are_taken(off, stride, cols):
    assert _refused(mat(ROWS, cols, stride), mat(ROWS, cols, stride, data=FAKE + off)) == 1


@pytest.mark.parametrize("off,stride,grad_stride", [(4 * 15, 32, 32), (4 * 17, 32, 32), (-4 * 15, 32, 32), (4 * 25, 40, 40),
                                                    (4 * 16, 31, 31), (4 * 16, 32, 33), (4 * 16, 32, 48), (4 * 32, 32, 32),
                                                    (4 * 16, 16, 32)])
def test_rows_that_share_elements_are_refused(off, stride, grad_stride):
    assert _refused(mat(ROWS, COLS, stride), mat(ROWS, COLS, grad_stride, data=FAKE + off)) == 2


def test_in_place_and_apart_are_taken():
    assert _refused(mat(ROWS), mat(ROWS)) == 1
    assert _refused(mat(ROWS), mat(ROWS, data=FAKE + 4 * ROWS * COLS)) == 1
