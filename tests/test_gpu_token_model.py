"""The token operators together: the example model's loss and gradients against
torch's automatic differentiation in 64 bits, and a short training run."""
import pytest
import torch

pytestmark = pytest.mark.gpu


def _reference(model, ids, teacher_ids, teacher_logits, padding_id=0):
    """The model's loss in 64 bits, differentiated by torch."""
    p = {n: getattr(model, n).double().requires_grad_() for n in ("table", "router", "experts")}
    h = p["table"][ids] * model.scale
    # padding tokens' rows have no gradient through the lookup
    h = torch.where((ids == padding_id)[:, None], h.detach(), h)
    scores = h @ p["router"]
    top, experts = torch.topk(scores, model.K, dim=1)
    weights = torch.softmax(top, 1)
    weights = torch.where((ids == padding_id)[:, None], 0.0, weights)
    y = torch.einsum("nd,nkde->nke", h, p["experts"][experts])
    hidden = h + (weights[:, :, None] * y).sum(1)
    c = model.temperature
    logq = torch.log_softmax(hidden @ p["table"].t() / c, 1)
    valid = teacher_ids >= 0
    t = (teacher_logits.double() / c).masked_fill(~valid, -1e300)
    logp = torch.log_softmax(t, 1)
    terms = torch.where(valid, logp.exp() * (logp - logq.gather(1, teacher_ids.clamp(min=0))), 0.0)
    rows = int(valid.any(1).sum())
    loss = c * c * terms.sum() / rows
    loss.backward()
    return float(loss.detach()), {n: v.grad for n, v in p.items()}


def test_gradients_against_automatic_differentiation():
    from examples.token_model import TokenModel, synthetic_batch
    model = TokenModel(V=120, D=32, experts=5, K=2)
    batch = synthetic_batch(120, 300, 4, seed=3)
    torch.backends.cuda.matmul.allow_tf32 = False
    loss, grads = model.step(*batch)
    want_loss, want = _reference(model, *batch)
    # chains of 32-bit sums of up to 300 terms through five products: 1e-4 of
    # each gradient's size
    assert abs(float(loss) - want_loss) <= 1e-4 * abs(want_loss)
    for name, g in grads.items():
        assert float((g.double() - want[name]).norm()) <= 1e-4 * float(want[name].norm()), name


def test_a_small_step_lowers_the_loss_by_the_gradients_square():
    # L(p - e g) = L(p) - e |g|^2 + O(e^2): with e so that the first-order
    # change is 1e-3 of the loss, the second-order rest is far below half of it
    from examples.token_model import TokenModel, synthetic_batch
    model = TokenModel(V=120, D=32, experts=5, K=2)
    torch.backends.cuda.matmul.allow_tf32 = False
    ids, teacher_ids, teacher_logits = synthetic_batch(120, 300, 4, seed=5)
    keep = ids != 0                        # the padding row has no gradient through the lookup
    batch = ids[keep].contiguous(), teacher_ids[keep].contiguous(), teacher_logits[keep].contiguous()
    before, grads = model.step(*batch)
    square = sum(float(g.double().square().sum()) for g in grads.values())
    e = 1e-3 * float(before) / square
    model.update(grads, e)
    after, _ = model.step(*batch)
    change = float(before) - float(after)
    assert abs(change - e * square) <= 0.5 * e * square


def test_example_runs():
    from examples.token_model import train
    losses = train(steps=6, V=100, N=512)
    assert all(x == x and x > 0 for x in losses) and losses[-1] < losses[0]
