"""Checks of the token operators' binding that need no GPU: stand-ins for device
tensors are refused before anything of them is used."""
import pytest
import torch


def _api():
    from recsys_table_embedding_gb300 import tokens
    return tokens


class OnDevice:
    """What the binding's first checks see of a tensor."""

    def __init__(self, device=0, requires_grad=False, **more):
        self.device_index, self.requires_grad = device, requires_grad
        self.__dict__.update(more)

    def get_device(self):
        return self.device_index


@pytest.mark.parametrize("name", ["tbe_route_sort", "tbe_route_sort_dispatch"])
def test_a_callers_route_lies_on_the_calls_device(name):
    t = _api()
    route = t.Route(torch.zeros(2 * 8 + 5 + 1, dtype=torch.int32), 4, 2, 5)        # a CPU buffer
    args = (OnDevice(),) if name == "tbe_route_sort" else (OnDevice(), OnDevice())
    with pytest.raises(t.TbeError, match="one device"):
        getattr(t, name)(*args, 5, route=route)
    route.buffer = OnDevice(1)
    with pytest.raises(t.TbeError, match="one device"):
        getattr(t, name)(*args, 5, route=route)


class SomeRoute:
    def __init__(self, **kw):
        self.buffer = OnDevice(**kw)


def _calls(t):
    """Every function, with the places of its tensors' arguments."""
    on = OnDevice
    return [(t.tbe_token_forward, [on, on], {"out": on}), (t.tbe_token_backward, [on, on], {"grad_table": on}),
            (t.tbe_route_sort_dispatch, [on, on, 5], {"rows": on}), (t.tbe_route_dispatch, [on, SomeRoute], {"rows": on}),
            (t.tbe_route_dispatch_backward, [on, SomeRoute], {"grad_x": on}),
            (t.tbe_route_combine, [on, SomeRoute, on], {"out": on}),
            (t.tbe_route_combine_backward, [on, on, SomeRoute, on], {"grad_rows": on, "grad_weights": on}),
            (t.tbe_distill_forward, [on, on, on], {"loss": on, "lse": on}),
            (t.tbe_distill_backward, [on, on, on, on], {"grad_logits": on}),
            (t.tbe_distill_loss_grad, [on, on, on], {"loss": on, "lse": on, "grad_logits": on})]


def test_tensors_that_require_a_gradient_are_refused():
    # the functions are not recorded: torch would lose their gradients without a word
    t = _api()
    make = lambda a, **kw: a(**kw) if isinstance(a, type) else a  # noqa: E731
    for fn, args, more in _calls(t):
        for i, a in enumerate(args):
            if a is not OnDevice:
                continue
            with pytest.raises(t.TbeError, match="requires a gradient"):
                fn(*[make(b, requires_grad=i == j) if b is OnDevice else make(b) for j, b in enumerate(args)])
        for name, a in more.items():
            with pytest.raises(t.TbeError, match="requires a gradient"):
                fn(*[make(b) for b in args], **{name: make(a, requires_grad=True)})
    with torch.no_grad():
        assert t._device_of(OnDevice(3, requires_grad=True), None, OnDevice(3)) == 3
    assert t._device_of(OnDevice(3), None, OnDevice(3)) == 3


@pytest.mark.parametrize("given", [None, -1, 1 << 64, (1 << 64) + 3, 1 << 63, -(1 << 63) - 1, -(1 << 64)])
def test_padding_ids_beyond_64_bits_are_no_row(given):
    # "any value outside the table": not the row that its low 64 bits name
    padding = _api()._padding(given)
    assert -(1 << 63) <= padding < 0 or padding >= (1 << 31) - 1


def test_padding_ids_of_rows():
    assert [_api()._padding(x) for x in (0, 5, (1 << 31) - 2, (1 << 63) - 1)] == [0, 5, (1 << 31) - 2, (1 << 63) - 1]


@pytest.mark.parametrize("experts", [(1 << 32) + 5, 1 << 31, 0, -3])
def test_numbers_of_experts_beyond_32_bits_are_refused(experts):
    t = _api()
    with pytest.raises(t.TbeError, match="expert"):
        t._sort_args(t._lib(), None, torch.zeros(4, 2, dtype=torch.int32), experts, None, None)
