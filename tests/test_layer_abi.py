"""Host-side checks of the layer operators' C entry points and their binding that
need no GPU: sizes, pointers, alignment, types and limits are refused before
anything is enqueued.  Device pointers are fake and never dereferenced."""
import ctypes
import math

import pytest
import torch

from test_token_abi import FAKE, mat, route
from test_token_binding import OnDevice, SomeRoute


def _api():
    from recsys_table_embedding_gb300 import layers
    return layers


def test_every_entry_point_is_declared_and_bound():
    from test_abi import header_functions
    t = _api()
    names = [n for n in header_functions() if n.startswith(("tbe_expert_", "tbe_layer_norm_", "tbe_adamw_"))]
    assert sorted(names) == sorted(t.LAYER_EXPORTED) == sorted(t._ARGS)
    t._lib()


def test_records_have_the_header_s_sizes():
    t = _api()
    assert (ctypes.sizeof(t.tbe_experts), ctypes.sizeof(t.tbe_adamw_tensor), ctypes.sizeof(t.tbe_adamw_options)) == (56, 72, 80)


def test_workspace_sizes():
    L = _api()._lib()
    assert L.tbe_layer_norm_workspace_bytes(1, 64) == 0 and L.tbe_layer_norm_workspace_bytes(1000, 64) > 0
    for bad in ((0, 5), (-1, 5), (5, 0), (5, (1 << 20) + 1), (1 << 30, 5)):
        assert L.tbe_layer_norm_workspace_bytes(*bad) == 0
    assert L.tbe_layer_norm_workspace_bytes((1 << 30) - 1, 1 << 20) <= 1 << 25
    assert L.tbe_adamw_workspace_bytes() > 0
    for bad in ((-1, 4, 8, 8), (8, 0, 8, 8), (8, 4097, 8, 8), (8, 4, 0, 8), (8, 4, 8, 0), (1 << 30, 1, 8, 8),
                (8, 1, (1 << 20) + 1, 8)):
        assert L.tbe_expert_workspace_bytes(*bad) == 0


def experts(E=3, rows=16, cols=16, expert_stride=None, stride=None, dtype=0, data=FAKE):
    stride = cols if stride is None else stride
    return _api().tbe_experts(data, E, rows, cols, rows * stride if expert_stride is None else expert_stride, stride, dtype)


# what is wrong with the weight; (status)
WEIGHTS = [(1, dict(data=None)), (2, dict(E=0)), (2, dict(E=4097)), (2, dict(E=4)), (2, dict(rows=0)), (2, dict(cols=0)),
           (2, dict(rows=(1 << 20) + 1)), (2, dict(cols=(1 << 20) + 1)), (2, dict(stride=-1)), (2, dict(expert_stride=-1)),
           (2, dict(stride=1 << 40)), (2, dict(cols=15)), (4, dict(dtype=3)), (4, dict(dtype=1)), (5, dict(data=FAKE + 2))]


@pytest.mark.parametrize("code,kw", WEIGHTS)
def test_weights_are_refused(code, kw):
    L, w, r = _api()._lib(), experts(**kw), route()
    assert L.tbe_expert_gated_forward(r, mat(8), w, 0, mat(8, 8), None, None, None, None) == code
    assert L.tbe_expert_forward(r, mat(8), w, mat(8), None, None, None) == code
    if kw != dict(cols=15):
        assert L.tbe_expert_backward(r, mat(8), w, None, 0, mat(8), None, None, None) == code
    if kw != dict(dtype=1):
        assert L.tbe_expert_weight_backward(r, mat(8), mat(8), w, 0, FAKE, 1 << 40, None, None, None) == code


@pytest.mark.parametrize("code,kw", [(1, dict(offset=None)), (5, dict(offset=FAKE + 2)), (2, dict(tokens=5)), (2, dict(K=0)),
                                     (2, dict(experts=2)), (2, dict(tokens=-1)), (2, dict(tokens=1 << 40))])
def test_routes_are_refused(code, kw):
    L, r = _api()._lib(), route(**kw)
    assert L.tbe_expert_gated_forward(r, mat(8), experts(), 0, mat(8, 8), None, None, None, None) == code
    assert L.tbe_expert_forward(r, mat(8), experts(), mat(8), None, None, None) == code
    assert L.tbe_expert_backward(r, mat(8), experts(), None, 0, mat(8), None, None, None) == code
    assert L.tbe_expert_weight_backward(r, mat(8), mat(8), experts(), 0, FAKE, 1 << 40, None, None, None) == code


def test_one_group_without_a_route():
    L = _api()._lib()
    assert L.tbe_expert_forward(None, mat(8), experts(E=3), mat(8), None, None, None) == 2
    assert L.tbe_expert_forward(None, mat(0, data=None), experts(E=1), mat(0, data=None), None, None, None) == 0


def test_products_arguments():
    L, r, w = _api()._lib(), route(), experts()
    for x, out, code in ((mat(8, 15), mat(8), 2), (mat(7), mat(8), 2), (mat(8), mat(7), 2), (mat(8), mat(8, 15), 2),
                         (mat(8), mat(8, dtype=1), 4), (mat(8), mat(8, stride=0), 2), (mat(8, data=None), mat(8), 1),
                         (mat(8), mat(8, data=None), 1), (mat(8), None, 1), (None, mat(8), 1), (mat(8, data=FAKE + 1), mat(8), 5)):
        assert L.tbe_expert_forward(r, x, w, out, None, None, None) == code
    assert L.tbe_expert_forward(r, mat(8), w, mat(8), FAKE + 1, None, None) == 5
    for hidden, z, act, code in ((mat(8), None, 0, 2), (mat(8, 8), mat(8, 8), 0, 2), (mat(8, 8), mat(7), 0, 2),
                                 (mat(8, 8), mat(8, dtype=2), 0, 4), (mat(8, 8), None, 2, 2), (mat(8, 8), mat(8, stride=1), 0, 2)):
        assert L.tbe_expert_gated_forward(r, mat(8), w, act, hidden, z, None, None, None) == code
    for z, dx, act, code in ((None, mat(8, 32), 0, 2), (mat(8, 32), mat(8), 0, 2), (mat(8), mat(8, 32), 0, 2),
                             (mat(8, 32), mat(8, 32), 7, 2), (mat(8, 32, dtype=1), mat(8, 32), 0, 4), (mat(7, 32), mat(8, 32), 0, 2)):
        assert L.tbe_expert_backward(r, mat(8), w, z, act, dx, None, None, None) == code
    for dy, x, dw, acc, code in ((mat(8), mat(7), w, 0, 2), (mat(8, 15), mat(8), w, 0, 2), (mat(8), mat(8), w, 2, 2),
                                 (mat(8, dtype=1), mat(8), w, 0, 4), (mat(8), mat(8), experts(dtype=1), 0, 4),
                                 (mat(8), mat(8), experts(stride=15), 0, 2), (mat(8), mat(8), experts(expert_stride=255), 0, 2)):
        assert L.tbe_expert_weight_backward(r, dy, x, dw, acc, FAKE, 1 << 40, None, None, None) == code
    assert L.tbe_expert_weight_backward(r, mat(8), mat(8), w, 0, FAKE + 4, 1 << 40, None, None, None) == 5
    many = route(tokens=1 << 20, K=1, experts=1)
    need = L.tbe_expert_workspace_bytes(1 << 20, 1, 16, 16)
    if need:
        args = many, mat(1 << 20), mat(1 << 20), experts(E=1), 0
        assert L.tbe_expert_weight_backward(*args, None, 1 << 40, None, None, None) == 1
        assert L.tbe_expert_weight_backward(*args, FAKE, need - 1, None, None, None) == 7


def test_layer_norm_arguments():
    L = _api()._lib()
    fwd = lambda x=mat(), w=FAKE, b=FAKE, wt=0, eps=1e-5, out=mat(), mean=FAKE, rstd=FAKE: L.tbe_layer_norm_forward(  # noqa: E731
        x, w, b, wt, eps, out, mean, rstd, None, None)
    for kw, code in ((dict(x=None), 1), (dict(out=None), 1), (dict(x=mat(data=None)), 1), (dict(x=mat(cols=15)), 2),
                     (dict(x=mat(rows=7)), 2), (dict(x=mat(dtype=1)), 4), (dict(x=mat(dtype=5)), 4), (dict(wt=3), 4),
                     (dict(w=FAKE + 2), 5), (dict(b=FAKE + 1, wt=1), 5), (dict(mean=FAKE + 2), 5), (dict(rstd=FAKE + 1), 5),
                     (dict(eps=-1e-9), 2), (dict(eps=math.nan), 2), (dict(eps=math.inf), 2), (dict(out=mat(stride=0)), 2),
                     (dict(x=mat(cols=(1 << 20) + 1), out=mat(cols=(1 << 20) + 1)), 2),
                     (dict(x=mat(rows=1 << 30, stride=0), out=mat(rows=1 << 30)), 2),
                     (dict(x=mat(rows=0, data=None), out=mat(rows=0, data=None)), 0)):
        assert fwd(**kw) == code, kw
    bwd = lambda dy=mat(), x=mat(), w=FAKE, wt=0, mean=FAKE, rstd=FAKE, dx=mat(), dw=FAKE, db=FAKE, gt=0, ws=FAKE, n=1 << 30: \
        L.tbe_layer_norm_backward(dy, x, w, wt, mean, rstd, dx, dw, db, gt, ws, n, None, None)  # noqa: E731
    for kw, code in ((dict(dy=None), 1), (dict(x=None), 1), (dict(mean=None), 1), (dict(rstd=None), 1), (dict(dy=mat(cols=15)), 2),
                     (dict(dy=mat(dtype=1)), 4), (dict(dx=mat(rows=7)), 2), (dict(dx=mat(dtype=2)), 4), (dict(wt=-1), 4),
                     (dict(gt=3), 4), (dict(dw=FAKE + 2), 5), (dict(db=FAKE + 1, gt=2), 5), (dict(ws=FAKE + 128), 5),
                     (dict(ws=None), 1), (dict(n=100), 7), (dict(mean=FAKE + 2), 5), (dict(dx=mat(stride=3)), 2),
                     (dict(dx=None, dw=None, db=None, ws=None, n=0), 0)):
        assert bwd(**kw) == code, kw


def tensor(**kw):
    a = dict(param=FAKE, grad=FAKE, m=FAKE, v=FAKE, scales=None, copy=None, n=100, param_dtype=0, grad_dtype=0, copy_dtype=0,
             state=0) | kw
    return _api().tbe_adamw_tensor(*a.values())


def options(**kw):
    a = dict(lr=1e-3, beta1=0.9, beta2=0.999, eps=1e-8, weight_decay=0.0, step=1, step_device=None, lr_device=None,
             grad_scale=None, seed=0) | kw
    return _api().tbe_adamw_options(*a.values())


def _step(t, o, count=1, ws=None, n=0):
    return _api()._lib().tbe_adamw_step(ctypes.byref(t) if t is not None else None, count, o, ws, n, None, None)


@pytest.mark.parametrize("code,kw", [(1, dict(param=None)), (1, dict(grad=None)), (1, dict(m=None)), (1, dict(v=None)), (1, dict(state=1)),
                                     (2, dict(n=-1)), (2, dict(n=(1 << 40) + 1)), (4, dict(param_dtype=3)), (4, dict(grad_dtype=-1)),
                                     (4, dict(state=2)), (4, dict(copy=FAKE)), (4, dict(copy=FAKE, copy_dtype=3)), (5, dict(param=FAKE + 2)),
                                     (5, dict(grad=FAKE + 1, grad_dtype=1)), (5, dict(m=FAKE + 1)), (5, dict(v=FAKE + 2)),
                                     (5, dict(state=1, scales=FAKE + 2)), (5, dict(copy=FAKE + 1, copy_dtype=1)), (0, dict(n=0, param=None))])
def test_tensors_of_a_step_are_refused(code, kw):
    assert _step(tensor(**kw), options()) == code


@pytest.mark.parametrize("code,kw", [(2, dict(lr=-1.0)), (2, dict(lr=math.nan)), (2, dict(lr=math.inf)), (2, dict(beta1=1.0)), (2, dict(beta1=-0.1)),
                                     (2, dict(beta2=1.0)), (2, dict(beta2=math.nan)), (2, dict(eps=-1.0)), (2, dict(weight_decay=-1.0)),
                                     (2, dict(step=0)), (2, dict(step=-3)), (5, dict(step_device=FAKE + 4)), (5, dict(lr_device=FAKE + 2)),
                                     (5, dict(grad_scale=FAKE + 1)), (1, dict(step_device=FAKE)), (1, dict(lr_device=FAKE))])
def test_options_of_a_step_are_refused(code, kw):
    assert _step(tensor(), options(**kw)) == code
    assert _step(tensor(n=0), options(**kw)) == code


def test_step_arguments():
    assert _step(None, options()) == 1 and _step(tensor(), None) == 1 and _step(None, options(), count=0) == 0
    assert _step(tensor(), options(), count=-1) == 2
    assert _step(tensor(), options(step_device=FAKE), ws=FAKE, n=255) == 7
    assert _step(tensor(), options(step_device=FAKE), ws=FAKE + 16, n=256) == 5


def test_tensors_that_require_a_gradient_are_refused():
    t = _api()
    on = OnDevice
    calls = [(t.tbe_expert_gated_forward, [on, on], {"hidden": on, "gate_up": on}), (t.tbe_expert_forward, [on, on], {"out": on}),
             (t.tbe_expert_backward, [on, on], {"gate_up": on, "grad_rows": on}),
             (t.tbe_expert_weight_backward, [on, on], {"grad_weight": on, "workspace": on}),
             (t.tbe_layer_norm_forward, [on], {"weight": on, "bias": on, "out": on, "mean": on, "rstd": on}),
             (t.tbe_layer_norm_backward, [on, on, on, on], {"weight": on, "grad_x": on, "grad_weight": on, "grad_bias": on})]
    for fn, args, more in calls:
        for i in range(len(args)):
            with pytest.raises(t._refuse.__globals__["TbeError"], match="requires a gradient"):
                fn(*[on(requires_grad=i == j) for j in range(len(args))])
        for name in more:
            with pytest.raises(t._refuse.__globals__["TbeError"], match="requires a gradient"):
                fn(*[on() for _ in args], **{name: on(requires_grad=True)})
            with pytest.raises(t._refuse.__globals__["TbeError"], match="one device"):
                fn(*[on() for _ in args], **{name: on(1)})


def test_a_route_lies_on_the_calls_device():
    t = _api()
    with pytest.raises(RuntimeError, match="one device"):
        t.tbe_expert_forward(OnDevice(), OnDevice(), SomeRoute(device=1))


def test_lists_of_a_step():
    t, x = _api(), torch.zeros(4)
    with pytest.raises(RuntimeError, match="one entry"):
        t.tbe_adamw_step([x], [x, x], [x], [x], 1)
    with pytest.raises(RuntimeError, match="CUDA"):
        t.tbe_adamw_step([x], [x], [x], [x], 1)
    assert t.tbe_adamw_step([x, x], [None, None], [x, x], [x, x], 1) is None and t.tbe_adamw_step([], [], [], [], 1) is None
