"""The token operators beside autograd: what a call writes into the caller's
tensors counts as a change of them, so a tensor that autograd has saved is not
overwritten unseen; calls under no_grad take parameters."""
import pytest
import torch

from test_gpu_tokens import _api, _distill_case, _ids, _rand

pytestmark = pytest.mark.gpu


def _results(api):
    """(call with the caller's tensors, those tensors) for every result."""
    table, ids, g = _rand(0, (50, 16), "f32"), _ids(1, 40, 50, bad=0), _rand(2, (40, 16), "f32")
    out, dtable = torch.empty_like(g), torch.zeros_like(table)
    yield lambda: api.tbe_token_forward(table, ids, out=out), [out]
    yield lambda: api.tbe_token_backward(g, ids, grad_table=dtable), [dtable]
    yield lambda: api.tbe_token_backward(g, ids, grad_table=dtable, accumulate=True), [dtable]
    eids = torch.randint(0, 5, (40, 2), device="cuda", dtype=torch.int32)
    route = api.tbe_route_sort(eids, 5)
    rows, back, w, dw = _rand(3, (80, 16), "f32"), torch.empty(80, 16, device="cuda"), _rand(4, (40, 2), "f32"), torch.empty(40, 2, device="cuda")
    yield lambda: api.tbe_route_sort(eids, 5, route=route), [route.buffer, route.slot]
    yield lambda: api.tbe_route_sort_dispatch(g, eids, 5, route=route, rows=back), [route.buffer, back]
    yield lambda: api.tbe_route_dispatch(g, route, rows=back), [back]
    yield lambda: api.tbe_route_dispatch_backward(rows, route, grad_x=out), [out]
    yield lambda: api.tbe_route_combine(rows, route, w, out=out), [out]
    yield lambda: api.tbe_route_combine_backward(g, rows, route, w, grad_rows=back, grad_weights=dw), [back, dw]
    z, tid, top, gl = _distill_case(5, 6, 90, 4, "f32")
    loss, lse, dz = torch.empty(6, device="cuda"), torch.empty(6, device="cuda"), torch.empty_like(z)
    yield lambda: api.tbe_distill_forward(z, tid, top, loss=loss, lse=lse), [loss, lse]
    yield lambda: api.tbe_distill_backward(z, tid, top, lse, gl, grad_logits=dz), [dz]
    yield lambda: api.tbe_distill_loss_grad(z, tid, top, gl, loss=loss, lse=lse, grad_logits=dz), [loss, lse, dz]
    yield lambda: api.tbe_distill_loss_grad(z, tid, top, gl, grad_logits=z), [z]


def test_results_count_as_changes_of_the_callers_tensors():
    for call, written in _results(_api()):
        before = [t._version for t in written]
        call()
        assert all(t._version > b for t, b in zip(written, before))


def test_a_saved_tensor_is_not_overwritten_unseen():
    z, tid, top, gl = _distill_case(5, 6, 90, 4, "f32")
    w = torch.ones(90, device="cuda", requires_grad=True)
    y = (z * w).sum()                                        # saves z
    _api().tbe_distill_loss_grad(z, tid, top, gl, grad_logits=z)
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        y.backward()


def test_parameters_without_gradient_mode():
    api = _api()
    table, ids = torch.nn.Parameter(_rand(0, (50, 16), "f32")), _ids(1, 40, 50, bad=0)
    with pytest.raises(api.TbeError, match="requires a gradient"):
        api.tbe_token_forward(table, ids)
    with torch.no_grad():
        h = api.tbe_token_forward(table, ids)
        table.grad = api.tbe_token_backward(_rand(2, (40, 16), "f32"), ids, 50)
    assert torch.equal(h, table.detach()[ids]) and not h.requires_grad
    api.tbe_token_backward(_rand(2, (40, 16), "f32"), ids, grad_table=table.grad, accumulate=True)
