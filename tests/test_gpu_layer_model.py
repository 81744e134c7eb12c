"""The layer operators together, with the token operators around them: the example
model's loss and gradients against torch's automatic differentiation in 64 bits,
its update against AdamW in 64 bits, and a short training run."""
import pytest
import torch

import layer_oracle as o

pytestmark = pytest.mark.gpu


def _norm(x, w, b):
    c = x - x.mean(1, keepdim=True)
    return c * ((c * c).mean(1, keepdim=True) + 1e-5).rsqrt() * w + b


def _reference(model, ids, teacher_ids, teacher_logits, padding_id=0):
    """The model's loss in 64 bits, differentiated by torch."""
    p = {n: v.double().requires_grad_() for n, v in model.parameters.items()}
    h = p["table"][ids] * model.scale
    # padding tokens' rows have no gradient through the lookup
    h = torch.where((ids == padding_id)[:, None], h.detach(), h)
    x = _norm(h, p["norm1_weight"], p["norm1_bias"])
    scores = x @ p["router"]
    top, experts = torch.topk(scores, model.K, dim=1)
    weights = torch.softmax(top, 1)
    weights = torch.where((ids == padding_id)[:, None], 0.0, weights)
    gate, up = torch.einsum("nd,nkfd->nkf", x, p["w_in"][experts]).chunk(2, 2)
    value = gate * torch.sigmoid(gate) if model.activation == "silu" else gate * torch.special.ndtr(gate)
    y = torch.einsum("nkf,nkdf->nkd", value * up, p["w_out"][experts])
    z = _norm(h + (weights[:, :, None] * y).sum(1), p["norm2_weight"], p["norm2_bias"])
    c = model.temperature
    logq = torch.log_softmax(z @ p["table"].t() / c, 1)
    valid = teacher_ids >= 0
    logp = torch.log_softmax((teacher_logits.double() / c).masked_fill(~valid, -1e300), 1)
    terms = torch.where(valid, logp.exp() * (logp - logq.gather(1, teacher_ids.clamp(min=0))), 0.0)
    loss = c * c * terms.sum() / int(valid.any(1).sum())
    loss.backward()
    return float(loss.detach()), {n: v.grad for n, v in p.items()}


@pytest.mark.parametrize("D,F,activation", [(32, 24, "silu"), (33, 27, "gelu")])
def test_gradients_against_automatic_differentiation(D, F, activation):
    from examples.layer_model import LayerModel
    from examples.token_model import synthetic_batch
    model = LayerModel(V=120, D=D, F=F, experts=5, K=2, activation=activation)
    batch = synthetic_batch(120, 300, 4, seed=3)
    torch.backends.cuda.matmul.allow_tf32 = False
    loss, grads = model.step(*batch)
    want_loss, want = _reference(model, *batch)
    # chains of 32-bit sums of up to 300 terms through eight products and two norms:
    # 1e-4 of each gradient's size
    assert abs(float(loss) - want_loss) <= 1e-4 * abs(want_loss)
    assert set(grads) == set(want)
    for name, g in grads.items():
        assert float((g.double() - want[name]).norm()) <= 1e-4 * float(want[name].norm()), name


def test_update_against_64_bits():
    from examples.layer_model import LayerModel
    from examples.token_model import synthetic_batch
    model = LayerModel(V=120, D=32, F=24, experts=5, K=2, dtype=torch.bfloat16)
    _, grads = model.step(*synthetic_batch(120, 300, 4, seed=5))
    before = {n: p.clone() for n, p in model.master.items()}
    model.update(grads, 1e-3, weight_decay=0.1)
    for n, p in model.master.items():
        zero = torch.zeros_like(p)
        want, bound = o.adamw(before[n], grads[n], zero, zero, 1, 1e-3, 0.9, 0.999, 1e-8, 0.1)
        o.close(p, want[0], bound[0])
        assert torch.equal(model.copies[n], p.to(torch.bfloat16))


@pytest.mark.parametrize("dtype,states", [(torch.float32, "f32"), (torch.bfloat16, "f8"), (torch.float16, "f8")])
def test_example_runs(dtype, states):
    from examples.layer_model import train
    losses = train(steps=6, V=100, N=512, dtype=dtype, states=states)
    assert all(x == x and x > 0 for x in losses)
