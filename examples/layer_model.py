"""A small model over tokens whose layers are the library's: norm, experts, AdamW.

A token's row of the table is normalised, goes through the best K of E experts
(a gated feed-forward block each), is added to itself, normalised again and scored
against all rows of the table.  A teacher gives its top logits for every position.
``LayerModel.step`` runs the forward pass and all gradients and ``update`` one AdamW
step of every parameter, with states in 32 or in 8 bits; what is left to torch are
the router's products and those with the table.

    python -m examples.layer_model
"""
from __future__ import annotations

import torch

import recsys_table_embedding_gb300 as tbe
from examples.token_model import synthetic_batch


class LayerModel:
    """Parameters: table [V, D], two norms' weights and biases [D], router [D, E],
    experts' matrices [E, 2F, D] and [E, D, F]; with ``dtype`` 16 bits wide each has
    a 32-bit master that the step updates."""

    def __init__(self, V: int, D: int, F: int, experts: int, K: int, temperature: float = 2.0, dtype=torch.float32,
                 states: str = "f32", activation: str = "silu", seed: int = 0, device="cuda"):
        g = torch.Generator(device=device)
        g.manual_seed(seed)
        new = lambda *shape: torch.randn(shape, generator=g, device=device).mul_(shape[-1] ** -0.5)  # noqa: E731
        self.master = dict(table=new(V, D), router=new(experts, D).t().contiguous(), w_in=new(experts, 2 * F, D),
                           w_out=new(experts, D, F))
        for n in ("norm1", "norm2"):
            self.master[n + "_weight"], self.master[n + "_bias"] = torch.ones(D, device=device), torch.zeros(D, device=device)
        self.copies = {n: p.to(dtype) for n, p in self.master.items()} if dtype != torch.float32 else None
        self.K, self.scale, self.temperature, self.activation, self.t = K, D ** 0.5, temperature, activation, 0
        kind = torch.float32 if states == "f32" else torch.float8_e4m3fn
        zeros = lambda: [torch.zeros(p.shape, dtype=torch.uint8 if states != "f32" else kind, device=device).view(kind)  # noqa: E731
                         for p in self.master.values()]
        self.m, self.v = zeros(), zeros()
        self.scales = None if states == "f32" else \
            [torch.zeros((-(-p.numel() // 256), 2), device=device) for p in self.master.values()]

    @property
    def parameters(self):
        return self.copies or self.master

    def step(self, ids: torch.Tensor, teacher_ids: torch.Tensor, teacher_logits: torch.Tensor, padding_id: int = 0):
        """(mean loss, gradients by name) for ids [N] and the teacher's top entries [N, k]."""
        p = self.parameters
        E = p["w_in"].shape[0]
        # forward
        h = tbe.tbe_token_forward(p["table"], ids, scale=self.scale)
        x, mean1, rstd1 = tbe.tbe_layer_norm_forward(h, p["norm1_weight"], p["norm1_bias"])
        scores = x @ p["router"]
        top, experts = torch.topk(scores, self.K, dim=1)
        experts = torch.where((ids == padding_id)[:, None], -1, experts)    # padding goes to no expert
        weights = torch.softmax(top.float(), dim=1)
        rows, route = tbe.tbe_route_sort_dispatch(x, experts, E)
        hidden, gate_up = tbe.tbe_expert_gated_forward(rows, p["w_in"], route, activation=self.activation, keep=True)
        y = tbe.tbe_expert_forward(hidden, p["w_out"], route)
        r = h + tbe.tbe_route_combine(y, route, weights)
        z, mean2, rstd2 = tbe.tbe_layer_norm_forward(r, p["norm2_weight"], p["norm2_bias"])
        logits = z @ p["table"].t()
        # loss, and the gradient in the logits' place
        count = max(1, int((teacher_ids >= 0).any(1).sum()))
        loss, _, dlogits = tbe.tbe_distill_loss_grad(logits, teacher_ids, teacher_logits, 1.0 / count,
                                                     temperature=self.temperature, grad_logits=logits)
        # backward
        grads = {}
        dz = dlogits @ p["table"]
        dr, grads["norm2_weight"], grads["norm2_bias"] = tbe.tbe_layer_norm_backward(dz, r, mean2, rstd2, p["norm2_weight"])
        dy, dweights = tbe.tbe_route_combine_backward(dr, y, route, weights)
        grads["w_out"] = tbe.tbe_expert_weight_backward(dy, hidden, route)
        dgate_up = tbe.tbe_expert_backward(dy, p["w_out"], route, gate_up=gate_up, activation=self.activation)
        grads["w_in"] = tbe.tbe_expert_weight_backward(dgate_up, rows, route)
        dx = tbe.tbe_route_dispatch_backward(tbe.tbe_expert_backward(dgate_up, p["w_in"], route), route)
        dtop = weights * (dweights - (weights * dweights).sum(1, keepdim=True))
        kept = torch.where(experts >= 0, dtop, 0.0).to(scores.dtype)
        dscores = torch.zeros_like(scores).scatter_add_(1, experts.clamp(min=0), kept)
        grads["router"] = x.t() @ dscores
        dx += dscores @ p["router"].t()
        dh, grads["norm1_weight"], grads["norm1_bias"] = tbe.tbe_layer_norm_backward(dx, h, mean1, rstd1, p["norm1_weight"])
        # the table's two gradients in one matrix: output layer, then tokens
        grads["table"] = dlogits.t() @ z
        tbe.tbe_token_backward(dh + dr, ids, scale=self.scale, padding_id=padding_id, grad_table=grads["table"], accumulate=True)
        return loss.sum() / count, grads

    def update(self, gradients, lr: float, weight_decay: float = 0.0):
        self.t += 1
        names = list(self.master)
        tbe.tbe_adamw_step([self.master[n] for n in names], [gradients[n].contiguous() for n in names], self.m, self.v, self.t,
                           lr=lr, weight_decay=weight_decay, scales=self.scales,
                           copies=[self.copies[n] for n in names] if self.copies else None, seed=self.t)


def train(steps: int = 60, V: int = 200, D: int = 64, F: int = 96, N: int = 2048, lr: float = 3e-3, dtype=torch.bfloat16,
          states: str = "f8"):
    """Losses of a short run."""
    model = LayerModel(V, D, F, experts=8, K=2, dtype=dtype, states=states)
    losses = []
    for i in range(steps):
        loss, gradients = model.step(*synthetic_batch(V, N, 5, seed=i))
        model.update(gradients, lr)
        losses.append(float(loss))
    return losses


if __name__ == "__main__":
    got = train()
    print("loss:", " ".join(f"{x:.3f}" for x in got[::10] + got[-1:]))
