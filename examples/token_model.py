"""A small model over tokens, trained by distillation with the token operators.

One embedding table is the input and the output layer: tokens are looked up
(scaled), routed to the best K of E experts (a linear layer each), combined,
and scored against all rows of the table.  A teacher gives its top logits for
every position.  ``TokenModel.step`` runs the forward pass and all gradients;
the matrix products are torch's, everything between them is the library's.

    python -m examples.token_model
"""
from __future__ import annotations

import torch

import recsys_table_embedding_gb300 as tbe


class TokenModel:
    """Parameters: table [V, D], router [D, E], experts [E, D, D]."""

    def __init__(self, V: int, D: int, experts: int, K: int, temperature: float = 2.0, dtype=torch.float32,
                 seed: int = 0, device="cuda"):
        g = torch.Generator(device=device)
        g.manual_seed(seed)
        new = lambda *shape: torch.randn(shape, generator=g, device=device).mul_(shape[-2] ** -0.5).to(dtype)  # noqa: E731
        self.table = torch.randn((V, D), generator=g, device=device).mul_(D ** -0.5).to(dtype)
        self.router, self.experts = new(D, experts), new(experts, D, D)
        self.K, self.scale, self.temperature = K, D ** 0.5, temperature

    def step(self, ids: torch.Tensor, teacher_ids: torch.Tensor, teacher_logits: torch.Tensor,
             padding_id: int = 0):
        """(mean loss, gradients by name) for ids [N] and the teacher's top
        entries [N, k] (-1 fills short lists; a row of -1 has no loss)."""
        E = self.experts.shape[0]
        # forward
        h = tbe.tbe_token_forward(self.table, ids, scale=self.scale)
        scores = h @ self.router
        top, experts = torch.topk(scores, self.K, dim=1)
        experts = torch.where((ids == padding_id)[:, None], -1, experts)    # padding goes to no expert
        weights = torch.softmax(top.float(), dim=1)
        x, route = tbe.tbe_route_sort_dispatch(h, experts, E)
        bounds = route.offset.tolist()
        y = torch.zeros_like(x)
        for e in range(E):
            s = slice(bounds[e], bounds[e + 1])
            y[s] = x[s] @ self.experts[e]
        hidden = h + tbe.tbe_route_combine(y, route, weights)
        logits = hidden @ self.table.t()
        # loss, and the gradient in the logits' place
        rows = max(1, int((teacher_ids >= 0).any(1).sum()))
        loss, _, dlogits = tbe.tbe_distill_loss_grad(logits, teacher_ids, teacher_logits, 1.0 / rows,
                                                     temperature=self.temperature, grad_logits=logits)
        # backward
        dhidden = dlogits @ self.table
        dy, dweights = tbe.tbe_route_combine_backward(dhidden, y, route, weights)
        dexperts, dx = torch.empty_like(self.experts), torch.zeros_like(x)
        for e in range(E):
            s = slice(bounds[e], bounds[e + 1])
            dexperts[e] = x[s].t() @ dy[s]
            dx[s] = dy[s] @ self.experts[e].t()
        dh = dhidden + tbe.tbe_route_dispatch_backward(dx, route)
        dtop = weights * (dweights - (weights * dweights).sum(1, keepdim=True))
        kept = torch.where(experts >= 0, dtop, 0.0).to(scores.dtype)
        dscores = torch.zeros_like(scores).scatter_add_(1, experts.clamp(min=0), kept)
        dh = dh + dscores @ self.router.t()
        # the table's two gradients in one matrix: output layer, then tokens
        dtable = dlogits.t() @ hidden
        tbe.tbe_token_backward(dh, ids, scale=self.scale, padding_id=padding_id, grad_table=dtable, accumulate=True)
        return loss.sum() / rows, dict(table=dtable, router=h.t() @ dscores, experts=dexperts)

    def update(self, gradients, lr: float):
        for name, g in gradients.items():
            getattr(self, name).sub_(g, alpha=lr)


def synthetic_batch(V: int, N: int, k: int, seed: int, device="cuda"):
    """Tokens in a cycle with some padding, and a teacher that knows the next
    tokens of the cycle."""
    g = torch.Generator(device=device)
    g.manual_seed(seed)
    start = torch.randint(1, V, (N,), generator=g, device=device)
    ids = torch.where(torch.rand(N, generator=g, device=device) < 0.1, 0, start)
    following = 1 + (ids[:, None] + torch.arange(k, device=device)) % (V - 1)
    teacher_logits = (4.0 - torch.arange(k, device=device, dtype=torch.float32)).expand(N, k).contiguous()
    return ids, torch.where((ids == 0)[:, None], -1, following), teacher_logits


def train(steps: int = 60, V: int = 200, D: int = 64, N: int = 2048, lr: float = 2.0):
    """Losses of a short run."""
    model = TokenModel(V, D, experts=8, K=2)
    losses = []
    for i in range(steps):
        loss, gradients = model.step(*synthetic_batch(V, N, 5, seed=i))
        model.update(gradients, lr)
        losses.append(float(loss))
    return losses


if __name__ == "__main__":
    got = train()
    print("loss:", " ".join(f"{x:.3f}" for x in got[::10] + got[-1:]))
