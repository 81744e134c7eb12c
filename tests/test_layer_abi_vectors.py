"""The vectors, scalars and workspaces of the layer operators' calls: what a call
writes shares no byte with what else it writes or reads.  Host checks only: every
call here is refused or has no rows, and the fake device pointers are never
dereferenced."""
import pytest

from test_layer_abi import _api
from test_token_abi import FAKE, mat

ROWS, COLS = 8, 16


def at(i):
    """Places that lie 1 MB apart."""
    return FAKE + (i << 20)


def _forward(**kw):
    a = dict(x=mat(data=at(0)), weight=at(1), bias=at(2), out=mat(data=at(3)), mean=at(4), rstd=at(5)) | kw
    return _api()._lib().tbe_layer_norm_forward(a["x"], a["weight"], a["bias"], 0, 1e-5, a["out"], a["mean"], a["rstd"], None, None)


@pytest.mark.parametrize("kw", [
    dict(rstd=at(4)), dict(rstd=at(4) + 4 * (ROWS - 1)), dict(rstd=at(4) - 4 * (ROWS - 1)), dict(mean=at(0)),
    dict(mean=at(0) + 4 * (ROWS * COLS - 1)), dict(rstd=at(0) - 4), dict(mean=at(3) + 64), dict(rstd=at(3)), dict(mean=at(1)),
    dict(rstd=at(2) + 4 * (COLS - 1)), dict(weight=at(3)), dict(bias=at(3) + 4), dict(weight=at(3) - 4 * (COLS - 1)),
    # in the columns between the rows of x, but for the last value
    dict(x=mat(stride=2 * COLS, data=at(0)), mean=at(0) + 4 * (2 * COLS - ROWS + 1))], ids=str)
def test_layer_norm_forward(kw):
    assert _forward(**kw) == 2


def _backward(**kw):
    a = dict(dy=mat(data=at(0)), x=mat(data=at(1)), weight=at(2), mean=at(3), rstd=at(4), dx=mat(data=at(5)), dw=at(6), db=at(7),
             ws=at(8)) | kw
    return _api()._lib().tbe_layer_norm_backward(a["dy"], a["x"], a["weight"], 0, a["mean"], a["rstd"], a["dx"], a["dw"], a["db"], 0,
                                                 a["ws"], 1 << 20, None, None)


@pytest.mark.parametrize("kw", [
    dict(db=at(6)), dict(db=at(6) + 4 * (COLS - 1)), dict(dw=at(0)), dict(db=at(1) + 4), dict(dw=at(2)), dict(db=at(2) - 4),
    dict(dw=at(3)), dict(db=at(4) + 4 * (ROWS - 1)), dict(dw=at(5)), dict(db=at(5) + 4 * (ROWS * COLS - 1)), dict(dw=at(8)),
    dict(db=at(8) + 256), dict(weight=at(5)), dict(mean=at(5)), dict(rstd=at(5) + 8), dict(ws=at(0)), dict(ws=at(1)),
    dict(ws=at(2)), dict(ws=at(3)), dict(ws=at(4)), dict(ws=at(5)), dict(dx=None, db=at(6)), dict(dx=None, dw=None, db=at(0))], ids=str)
def test_layer_norm_backward(kw):
    assert _backward(**kw) == 2


def test_sums_over_no_rows_lie_apart():
    none = mat(rows=0, data=None)
    assert _backward(dy=none, x=none, dx=none, db=at(6)) == 2


def test_nothing_is_compared_that_is_not_used():
    # no rows: mean and rstd have no values, the weight's memory is free
    none = mat(rows=0, data=None)
    assert _forward(x=none, out=none, mean=at(4), rstd=at(4)) == 0
    assert _backward(dy=none, x=none, dx=none, dw=None, db=None) == 0


def _weights(**kw):
    """The weights' gradient of 8192 rows in one group, whose sums lie in the workspace first."""
    from test_layer_abi import experts
    a = dict(dy=mat(8192, data=at(0)), x=mat(8192, data=at(1)), dw=experts(E=1, data=at(2)), ws=at(3)) | kw
    L = _api()._lib()
    need = L.tbe_expert_workspace_bytes(8192, 1, COLS, COLS)
    assert 0 < need <= 1 << 20
    return L.tbe_expert_weight_backward(None, a["dy"], a["x"], a["dw"], 0, a["ws"], need, None, None, None)


@pytest.mark.parametrize("place", [0, 1, 2], ids=["grad_out", "rows", "grad_weight"])
def test_workspace_of_the_weights_gradient(place):
    assert _weights(ws=at(place)) == 2
    assert _weights(ws=at(place) + 256) == 2
    assert _weights(ws=at(place) - 256) == 2


@pytest.mark.parametrize("words", ["offset", "status"])
def test_results_over_the_route_and_the_status_words(words):
    from test_layer_abi import experts
    from test_token_abi import route
    L = _api()._lib()
    # the route of 3 experts has 4 words, the status 4: all but the last lie before the results
    r, st = (route(offset=at(5) - 12), None) if words == "offset" else (route(offset=at(8)), at(5) - 12)
    x, w, out, z = mat(data=at(0)), experts(data=at(1)), mat(data=at(5)), mat(cols=2 * COLS, data=at(5))
    assert L.tbe_expert_forward(r, x, w, out, st, None, None) == 2
    assert L.tbe_expert_gated_forward(r, x, experts(rows=2 * COLS, data=at(1)), 0, out, None, st, None, None) == 2
    assert L.tbe_expert_gated_forward(r, x, experts(rows=2 * COLS, data=at(1)), 0, mat(data=at(3)), z, st, None, None) == 2
    assert L.tbe_expert_backward(r, x, w, None, 0, out, st, None, None) == 2
    assert L.tbe_expert_backward(r, x, w, mat(cols=2 * COLS, data=at(3)), 0, z, st, None, None) == 2
    assert L.tbe_expert_weight_backward(r, x, mat(data=at(2)), experts(data=at(5)), 0, None, 0, st, None, None) == 2
    # ... and the workspace
    many, rows = route(tokens=8192, K=1, experts=1, offset=r.offset), mat(8192, data=at(0))
    dw = experts(E=1, data=at(9))
    need = L.tbe_expert_workspace_bytes(8192, 1, COLS, COLS)
    assert L.tbe_expert_weight_backward(many, rows, mat(8192, data=at(2)), dw, 0, at(5) - 256, need, st, None, None) == 2


def _step(ws=at(9), **opts):
    """A step of one tensor of 100 elements, at places 0 to 5, whose numbers lie at 6 to 8 and come to the workspace."""
    import ctypes
    from test_layer_abi import options, tensor
    t = tensor(param=at(0), grad=at(1), m=at(2), v=at(3), scales=at(4), copy=at(5), copy_dtype=1, state=1)
    o = options(**(dict(step_device=at(6), lr_device=at(7), grad_scale=at(8)) | opts))
    return _api()._lib().tbe_adamw_step(ctypes.byref(t), 1, o, ws, 256, None, None)


@pytest.mark.parametrize("name", ["step_device", "lr_device", "grad_scale"])
@pytest.mark.parametrize("place", [at(0), at(0) + 392, at(2), at(3) + 96, at(4), at(5) + 192, at(9), at(9) + 8], ids=hex)
def test_numbers_of_a_step_in_what_it_writes(name, place):
    assert _step(**{name: place}) == 2


@pytest.mark.parametrize("place", range(9))
def test_workspace_of_a_step(place):
    assert _step(ws=at(place)) == 2
