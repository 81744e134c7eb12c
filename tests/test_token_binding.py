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
