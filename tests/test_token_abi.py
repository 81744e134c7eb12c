"""Host-side checks of the token operators' C entry points that need no GPU:
sizes, pointers, alignment and limits are refused before anything is
enqueued.  Device pointers are fake and never dereferenced."""
import ctypes
import math

import pytest

FAKE = 0x7f0000000000


def _api():
    from recsys_table_embedding_gb300 import tokens
    return tokens


def mat(rows=8, cols=16, stride=None, dtype=0, data=FAKE):
    return _api().tbe_matrix(data, rows, cols, cols if stride is None else stride, dtype)


def test_every_entry_point_is_declared_and_bound():
    from test_abi import header_functions
    t = _api()
    names = [n for n in header_functions() if n.startswith(("tbe_token_", "tbe_route_", "tbe_distill_"))]
    assert sorted(names) == sorted(t.TOKEN_EXPORTED) == sorted(t._ARGS)
    t._lib()


def test_workspace_sizes():
    L = _api()._lib()
    assert L.tbe_token_workspace_bytes(100, 50, 64) == 0      # few tokens need none
    small, large = L.tbe_token_workspace_bytes(3000, 50, 64), L.tbe_token_workspace_bytes(100000, 50, 64)
    assert 16 * 3000 <= small < large
    for bad in ((-1, 5, 5), (5, 0, 5), (5, 5, 0), (1 << 30, 5, 5), (5, 2 ** 31 - 1, 5), (5, 5, (1 << 20) + 1)):
        assert L.tbe_token_workspace_bytes(*bad) == 0
    assert L.tbe_route_workspace_bytes(5000, 4, 16) > 0 and L.tbe_route_workspace_bytes(10, 4, 16) == 0
    assert L.tbe_distill_workspace_bytes(1000, 4) > 0 and L.tbe_distill_workspace_bytes(4, 4) == 0
    for bad in ((-1, 4), (4, 0), (4, 1025), (1 << 30, 4)):
        assert L.tbe_distill_workspace_bytes(*bad) == 0
    for bad in ((-1, 4, 4), (4, 0, 4), (4, 1025, 4), (4, 4, 0), (4, 4, 4097), (1 << 28, 4, 4)):
        assert L.tbe_route_workspace_bytes(*bad) == 0


# (status, changes to the arguments)
FORWARD = [(1, dict(ids=None)), (1, dict(table=mat(data=None))), (2, dict(table=mat(cols=15))), (2, dict(itype=2)),
           (2, dict(table=mat(rows=0))), (2, dict(table=mat(rows=2 ** 31 - 1, stride=0))), (2, dict(table=mat(stride=-16))),
           (2, dict(out=mat(stride=8))), (2, dict(out=mat(rows=1 << 30))), (4, dict(table=mat(dtype=3))),
           (4, dict(out=mat(dtype=1))), (5, dict(table=mat(data=FAKE + 2))), (5, dict(ids=FAKE + 4, itype=1)),
           (5, dict(status=FAKE + 2)), (2, dict(table=mat(cols=(1 << 20) + 1), out=mat(cols=(1 << 20) + 1))),
           (0, dict(out=mat(rows=0, data=None), ids=None))]


@pytest.mark.parametrize("code,kw", FORWARD)
def test_token_forward_refuses(code, kw):
    a = dict(table=mat(rows=100), ids=FAKE, itype=0, out=mat(), status=None) | kw
    L = _api()._lib()
    assert L.tbe_token_forward(a["table"], a["ids"], a["itype"], 1.0, a["out"], a["status"], None, None) == code


def test_null_matrices():
    L = _api()._lib()
    assert L.tbe_token_forward(None, FAKE, 0, 1.0, mat(), None, None, None) == 1
    assert L.tbe_token_forward(mat(), FAKE, 0, 1.0, None, None, None, None) == 1
    assert L.tbe_distill_forward(mat(), None, FAKE, FAKE, FAKE, 1 << 20, None, None, None) == 1
    assert L.tbe_route_sort(None, FAKE, 0, FAKE, 1 << 20, None, None) == 1


BACKWARD = [(1, dict(ids=None)), (1, dict(ws=None)), (5, dict(ws=FAKE + 128)), (7, dict(n=1000)), (2, dict(acc=2)),
            (2, dict(dw=mat(rows=100, stride=0))), (2, dict(dw=mat(rows=100, cols=20))), (4, dict(dw=mat(rows=100, dtype=2))),
            (4, dict(g=mat(rows=5000, dtype=5))), (2, dict(g=mat(rows=-1))), (5, dict(dw=mat(rows=100, data=FAKE + 1)))]


@pytest.mark.parametrize("code,kw", BACKWARD)
def test_token_backward_refuses(code, kw):
    a = dict(g=mat(rows=5000), ids=FAKE, itype=1, dw=mat(rows=100), acc=0, ws=FAKE, n=1 << 30) | kw
    assert _api()._lib().tbe_token_backward(a["g"], a["ids"], a["itype"], -1, 1.0, a["dw"], a["acc"], a["ws"], a["n"],
                                            None, None, None) == code


def route(tokens=4, K=2, experts=3, slot=FAKE, source=FAKE, offset=FAKE):
    return _api().tbe_route(tokens, K, experts, slot, source, offset)


ROUTE = [(1, dict(slot=None)), (1, dict(source=None)), (1, dict(offset=None)), (5, dict(offset=FAKE + 1)), (2, dict(K=0)),
         (2, dict(K=1025)), (2, dict(experts=0)), (2, dict(experts=4097)), (2, dict(tokens=-1)), (2, dict(tokens=1 << 29))]


@pytest.mark.parametrize("code,kw", ROUTE)
def test_routes_are_refused(code, kw):
    L, r = _api()._lib(), route(**kw)
    assert L.tbe_route_sort(r, FAKE, 0, FAKE, 1 << 30, None, None) == code
    assert L.tbe_route_dispatch(r, mat(4), mat(8), None, None) == code
    assert L.tbe_route_sort_dispatch(r, FAKE, 0, mat(4), mat(8), FAKE, 1 << 30, None, None) == code
    assert L.tbe_route_combine(r, mat(8), FAKE, 0, mat(4), None, None) == code
    assert L.tbe_route_dispatch_backward(r, mat(8), mat(4), None, None) == code
    assert L.tbe_route_combine_backward(r, mat(4), mat(8), FAKE, 0, mat(8), FAKE, None, None) == code


def test_route_arguments():
    L, r = _api()._lib(), route()
    assert L.tbe_route_sort(r, None, 0, FAKE, 1 << 30, None, None) == 1
    assert L.tbe_route_sort(r, FAKE, 7, FAKE, 1 << 30, None, None) == 2
    assert L.tbe_route_sort(r, FAKE + 4, 1, FAKE, 1 << 30, None, None) == 5
    assert L.tbe_route_sort(r, FAKE, 0, FAKE + 4, 1 << 30, None, None) == 5
    many = route(tokens=4000)
    assert L.tbe_route_sort(many, FAKE, 0, FAKE, L.tbe_route_workspace_bytes(4000, 2, 3) - 1, None, None) == 7
    assert L.tbe_route_sort(many, FAKE, 0, None, 1 << 30, None, None) == 1
    for x, rows, code in ((mat(5), mat(8), 2), (mat(4), mat(9), 2), (mat(4, 8), mat(8), 2), (mat(4, dtype=1), mat(8), 4),
                          (mat(4), mat(8, stride=0), 2), (mat(4, data=None), mat(8), 1)):
        assert L.tbe_route_dispatch(r, x, rows, None, None) == code
    assert L.tbe_route_combine(r, mat(8), None, 0, mat(4), None, None) == 1
    assert L.tbe_route_combine(r, mat(8), FAKE, 9, mat(4), None, None) == 4
    assert L.tbe_route_combine(r, mat(8), FAKE + 2, 0, mat(4), None, None) == 5
    assert L.tbe_route_combine(r, mat(8), FAKE, 0, mat(4, stride=1), None, None) == 2
    assert L.tbe_route_combine_backward(r, mat(4), mat(8), FAKE, 0, mat(8), None, None, None) == 1
    assert L.tbe_route_combine_backward(r, mat(4), mat(8), FAKE, 0, mat(7), FAKE, None, None) == 2


def teacher(**kw):
    a = dict(ids=FAKE, logits=FAKE, index_type=0, dtype=0, K=4, temperature=1.0) | kw
    return _api().tbe_teacher(*a.values())


@pytest.mark.parametrize("code,kw", [(1, dict(ids=None)), (1, dict(logits=None)), (2, dict(index_type=2)), (4, dict(dtype=3)),
                                     (2, dict(K=0)), (2, dict(K=1025)), (2, dict(temperature=0.0)), (2, dict(temperature=-1.0)),
                                     (2, dict(temperature=math.nan)), (2, dict(temperature=math.inf)),
                                     (5, dict(ids=FAKE + 4, index_type=1)), (5, dict(logits=FAKE + 2))])
def test_teachers_are_refused(code, kw):
    L, te, z, dz = _api()._lib(), teacher(**kw), mat(rows=5000), mat(rows=5000, data=FAKE + (1 << 24))
    assert L.tbe_distill_forward(z, te, FAKE, FAKE, FAKE, 1 << 20, None, None, None) == code
    assert L.tbe_distill_backward(z, te, FAKE, None, 1.0, dz, FAKE, 1 << 20, None, None) == code
    assert L.tbe_distill_loss_grad(z, te, None, 1.0, FAKE, FAKE, dz, FAKE, 1 << 20, None, None, None) == code


def test_distill_arguments():
    L, te, z = _api()._lib(), teacher(), mat(rows=5000)
    assert L.tbe_distill_forward(z, te, None, FAKE, FAKE, 1 << 20, None, None, None) == 1
    assert L.tbe_distill_forward(z, te, FAKE, None, FAKE, 1 << 20, None, None, None) == 1
    assert L.tbe_distill_forward(z, te, FAKE + 2, FAKE, FAKE, 1 << 20, None, None, None) == 5
    assert L.tbe_distill_loss_grad(z, te, None, 1.0, None, FAKE, mat(rows=5000, data=FAKE + (1 << 24)), FAKE, 1 << 20, None, None, None) == 1
    assert L.tbe_distill_forward(mat(rows=0, data=None), te, None, None, FAKE, 1 << 20, None, None, None) == 0
    for dz, code in ((mat(7, data=FAKE + (1 << 24)), 2), (mat(rows=5000, cols=15, data=FAKE + (1 << 24)), 2), (mat(rows=5000, dtype=1, data=FAKE + (1 << 24)), 4),
                     (mat(rows=5000, data=None), 1), (mat(rows=5000, stride=3, data=FAKE + (1 << 24)), 2), (mat(rows=5000, data=FAKE + 64), 2), (mat(rows=5000, data=FAKE - 64), 2),
                     (mat(rows=5000, stride=32), 2)):
        assert L.tbe_distill_backward(z, te, FAKE, None, 1.0, dz, FAKE, 1 << 20, None, None) == code
        assert L.tbe_distill_loss_grad(z, te, None, 1.0, FAKE, FAKE, dz, FAKE, 1 << 20, None, None, None) == code
    assert L.tbe_distill_backward(z, te, FAKE, FAKE + 1, 1.0, mat(rows=5000, data=FAKE + (1 << 24)), FAKE, 1 << 20, None, None) == 5
    dz = mat(rows=5000, data=FAKE + (1 << 24))
    for ws, n, code in ((None, 1 << 20, 1), (FAKE + 4, 1 << 20, 5), (FAKE, 100, 7)):
        assert L.tbe_distill_forward(z, te, FAKE, FAKE, ws, n, None, None, None) == code
        assert L.tbe_distill_backward(z, te, FAKE, None, 1.0, dz, ws, n, None, None) == code
        assert L.tbe_distill_loss_grad(z, te, None, 1.0, FAKE, FAKE, dz, ws, n, None, None, None) == code
