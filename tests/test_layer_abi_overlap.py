"""Results that share an element with what else a call of the layer operators reads
or writes are refused: in place, rows that reach into one another, a tensor of an
AdamW step that is listed twice.  Host checks only: every call here is refused, and
the fake device pointers are never dereferenced."""
import ctypes

import pytest

from test_layer_abi import _api, experts, options, tensor
from test_token_abi import FAKE, mat, route

FAR = FAKE + (1 << 30)
# where a result of 8 rows of 16 lies beside a matrix of as many at FAKE: offset in bytes, strides of both
SHARED = [(0, 16, 16), (4 * 15, 16, 16), (-4 * 127, 16, 16), (4 * 15, 32, 32), (-4 * 15, 32, 32), (4 * 16, 31, 31),
          (4 * 16, 32, 33), (4 * 32, 16, 32), (4 * 15, 32, 0)]


@pytest.mark.parametrize("off,ours,theirs", SHARED)
def test_rows_that_share_elements_are_refused(off, ours, theirs):
    L, r = _api()._lib(), route()
    out, x, far = mat(8, 16, ours, data=FAKE + off), mat(8, 16, theirs), mat(8, 16, data=FAR)
    w = experts(data=FAR + (1 << 28))
    assert L.tbe_expert_forward(r, x, w, out, None, None, None) == 2
    assert L.tbe_expert_backward(r, x, w, None, 0, out, None, None, None) == 2
    assert L.tbe_expert_backward(r, far, experts(cols=8, data=FAR + (1 << 28)), x, 0, out, None, None, None) == 2
    assert L.tbe_expert_gated_forward(r, x, experts(rows=32, data=FAR + (1 << 28)), 0, out, None, None, None, None) == 2
    assert L.tbe_expert_gated_forward(r, x, w, 0, mat(8, 8, data=FAR), out, None, None, None) == 2
    assert L.tbe_layer_norm_forward(x, None, None, 0, 1e-5, out, None, None, None, None) == 2
    for dy, y in ((x, far), (far, x)):
        assert L.tbe_layer_norm_backward(dy, y, None, 0, FAKE, FAKE, out, None, None, 0, None, 0, None, None) == 2


def test_a_block_s_results_and_weights():
    L, r = _api()._lib(), route()
    # hidden inside gate_up; results and gradients in the weights' memory
    assert L.tbe_expert_gated_forward(r, mat(8, data=FAR), experts(), 0, mat(8, 8, 16, data=FAKE + (1 << 20)),
                                      mat(8, data=FAKE + (1 << 20)), None, None, None) == 2
    for off in (0, 4 * 255, 4 * 256, 4 * (3 * 256 - 1), -4 * 127):
        assert L.tbe_expert_forward(r, mat(8, data=FAR), experts(), mat(8, data=FAKE + off), None, None, None) == 2
    for dy, x in ((mat(8), mat(8, data=FAR)), (mat(8, data=FAR), mat(8))):
        assert L.tbe_expert_weight_backward(r, dy, x, experts(data=FAKE - 4), 0, FAKE, 1 << 40, None, None, None) == 2


# two tensors of 100 elements, whose memory lies apart but for what is named
def _two(**second):
    at = [dict(zip(("param", "grad", "m", "v"), (FAKE + 4096 * (4 * i + k) for k in range(4)))) for i in range(2)]
    at[1].update(second)
    return (_api().tbe_adamw_tensor * 2)(*(tensor(**a) for a in at))


@pytest.mark.parametrize("second", [
    dict(param=FAKE), dict(param=FAKE + 396), dict(param=FAKE - 396), dict(m=FAKE), dict(v=FAKE + 4096 * 2), dict(grad=FAKE + 4),
    dict(grad=FAKE + 4096 * 3), dict(param=FAKE + 4096), dict(copy=FAKE + 4096 * 2 + 398, copy_dtype=1), dict(m=FAKE + 4096 * 4),
    dict(grad=FAKE + 4096 * 4), dict(state=1, scales=FAKE + 4096 * 2 + 396), dict(state=1, scales=FAKE + 4096 * 7 + 96)])
def test_tensors_of_a_step_lie_apart(second):
    assert _api()._lib().tbe_adamw_step(ctypes.byref(_two(**second)), 2, options(), None, 0, None, None) == 2


def test_a_tensor_listed_twice_is_refused():
    t = (_api().tbe_adamw_tensor * 40)(*(tensor(param=FAKE + 4096 * (i % 39), grad=FAKE + (1 << 20) + 4096 * i, m=FAKE + (2 << 20) + 4096 * i,
                                                v=FAKE + (3 << 20) + 4096 * i) for i in range(40)))
    assert _api()._lib().tbe_adamw_step(ctypes.byref(t), 40, options(), None, 0, None, None) == 2
