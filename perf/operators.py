"""Measured cases of the token operators: the token embedding and its gradient,
the expert routing and its gradients, and the distillation loss.

``own`` selects what ``run`` computes: the framework's operators where it is
true, their plain form in elementary torch operations (32-bit, rounded once at
the end) where it is false.  ``exact`` states each operator in 64 bits.
"""
from __future__ import annotations

import math

import numpy as np
import torch

own = False

_TYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
_BYTES = {"f32": 4, "f16": 2, "bf16": 2}
_INDEX = {"i32": torch.int32, "i64": torch.int64}


# ---------------------------------------------------------------------------
# cases

def _token_forward(N, V, D, type, out="", zipf=0.0, index="i64", bad=0.0):
    return dict(op="token_forward", N=N, V=V, D=D, type=type, out=out or type, zipf=zipf,
                index=index, bad=bad)


def _token_backward(N, V, D, type, out="", zipf=0.0, index="i64", bad=0.0, pad=0.0):
    return dict(op="token_backward", N=N, V=V, D=D, type=type, out=out or type, zipf=zipf,
                index=index, bad=bad, pad=pad)


def _route(op, T, K, E, H, type, weight="f32", index="i32", drop=0.0):
    return dict(op=op, T=T, K=K, E=E, H=H, type=type, weight=weight, index=index, drop=drop)


def _distill(op, N, V, K, type, temperature=1.0, index="i32", teacher="f32", empty=0.0):
    return dict(op=op, N=N, V=V, K=K, type=type, temperature=temperature, index=index,
                teacher=teacher, empty=empty)


def listed():
    cases = {
        # the newest token of one sequence being generated
        "lookup one token": _token_forward(1, 65536, 1024, "bf16"),
        # a packed batch of long histories over a million-row item table
        "lookup long batch": _token_forward(131_072, 1_000_000, 512, "f16", zipf=1.05, index="i32",
                                            bad=0.01),
        # fine-tuning on a few hundred tokens; sizes that fit no tile
        "token gradient small": _token_backward(300, 10_007, 99, "f32", zipf=0.8),
        # a training step over a tied table, gradient kept in 32 bits, padded sequences
        "token gradient step": _token_backward(16_384, 131_072, 1024, "bf16", out="f32", zipf=1.0,
                                               pad=0.15),
        # a long step over the item table, gradient in the table's type
        "token gradient long": _token_backward(262_144, 1_000_000, 256, "f16", zipf=1.05, index="i32",
                                               bad=0.01),
        # one generated token through the experts of a layer
        "route one token": _route("route_forward", 1, 8, 64, 2048, "bf16"),
        # a small ragged batch in 32 bits, forward and gradients
        "route odd batch": _route("route_step", 1001, 3, 37, 501, "f32", index="i64", drop=0.1),
        # a training step's routing, forward and gradients
        "route training step": _route("route_step", 32_768, 8, 128, 1024, "bf16", drop=0.02),
        # a handful of drafted positions against an odd vocabulary
        "distill few rows": _distill("distill_loss_grad", 7, 32_003, 10, "f32", empty=0.2),
        # 16-bit logits of an odd vocabulary: rows start at every alignment
        "distill odd vocabulary": _distill("distill_loss_grad", 1000, 50_021, 32, "f16",
                                           temperature=2.0, index="i64", teacher="f16", empty=0.1),
        # a training step's logits, gradient wanted at once
        "distill training step": _distill("distill_loss_grad", 4096, 131_072, 64, "bf16",
                                          temperature=1.5, teacher="bf16", empty=0.05),
        # loss first, gradient later from an upstream gradient
        "distill two calls": _distill("distill_two_calls", 2048, 65_536, 128, "f32",
                                      temperature=3.0, empty=0.05),
    }
    return [dict(name=k, **c) for k, c in cases.items()]


def _log(rng, lo, hi):
    """An integer in [lo, hi], spread over its logarithm, often of no round size."""
    v = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))
    if rng.random() < 0.4 and v >= 64:
        v = v // 32 * 32
    v = min(hi, max(lo, v))
    return v if v != 3072 else v - 32


def draw(rng):
    op = rng.choice(["token_forward", "token_backward", "route_forward", "route_step",
                     "distill_loss_grad", "distill_two_calls"])
    type = rng.choice(["f32", "f16", "bf16"])
    index = rng.choice(["i32", "i64"])
    if op.startswith("token"):
        D = _log(rng, 16, 4096)
        V = min(_log(rng, 500, 1_000_000), 134_217_728 // D)
        N = min(_log(rng, 1, 262_144), 67_108_864 // D)
        zipf = rng.choice([0.0, 0.8, 1.0, 1.05, 1.2])
        bad = rng.choice([0.0, 0.01])
        out = rng.choice([type, "f32"])
        if op == "token_forward":
            return _token_forward(N, V, D, type, out, zipf, index, bad)
        return _token_backward(N, V, D, type, out, zipf, index, bad, rng.choice([0.0, 0.15]))
    if op.startswith("route"):
        K = rng.randint(1, 8)
        E = _log(rng, 8, 256)
        H = _log(rng, 64, 4096)
        T = min(_log(rng, 1, 32_768), 33_554_432 // (H * (2 if type == "f32" else 1)))
        return _route(op, T, K, E, H, type, rng.choice(["f32", type]), index,
                      rng.choice([0.0, 0.02, 0.3]))
    V = _log(rng, 1000, 200_000)
    N = min(_log(rng, 1, 8192), 268_435_456 // V)
    return _distill(op, N, V, min(_log(rng, 1, 256), V), type, rng.choice([1.0, 1.5, 2.0, 4.0]), index,
                    rng.choice(["f32", type]), rng.choice([0.0, 0.05, 0.3]))


# ---------------------------------------------------------------------------
# inputs

def _normal(gen, shape, type, std=1.0):
    x = torch.empty(shape, dtype=_TYPES[type], device="cuda")
    return x.normal_(0.0, std, generator=gen)


def _uniform(gen, shape):
    return torch.rand(shape, generator=gen, device="cuda")


def _tokens(case, gen):
    """N ids: uniform or Zipf over a permuted table, a share of them out of range."""
    N, V = case["N"], case["V"]
    if case["zipf"] > 0:
        w = torch.arange(1, V + 1, device="cuda", dtype=torch.float64).pow(-case["zipf"])
        cdf = torch.cumsum(w, 0)
        u = torch.rand(N, generator=gen, device="cuda", dtype=torch.float64) * cdf[-1]
        rank = torch.searchsorted(cdf, u).clamp_(max=V - 1)
        ids = torch.randperm(V, generator=gen, device="cuda")[rank]
    else:
        ids = torch.randint(0, V, (N,), generator=gen, device="cuda")
    if case["bad"] > 0:
        ids = torch.where(_uniform(gen, N) < case["bad"], torch.where(_uniform(gen, N) < 0.5, -1, V), ids)
    return ids


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    op = case["op"]
    s = dict(case)
    if op.startswith("token"):
        ids = _tokens(case, gen)
        s["scale"] = math.sqrt(case["D"])
        if op == "token_forward":
            s["table"] = _normal(gen, (case["V"], case["D"]), case["type"], 0.02)
        else:
            s["padding"] = None
            if case["pad"] > 0:
                s["padding"] = 0
                ids = torch.where(_uniform(gen, case["N"]) < case["pad"], 0, ids)
            s["grad"] = _normal(gen, (case["N"], case["D"]), case["type"], 1e-3 if case["type"] != "f16" else 0.05)
        s["ids"] = ids.to(_INDEX[case["index"]])
        return s
    if op.startswith("route"):
        T, K, E, H = case["T"], case["K"], case["E"], case["H"]
        score = _normal(gen, (T, E), "f32") + torch.linspace(0.8, -0.8, E, device="cuda")
        top, ids = torch.topk(score, min(K, E), dim=1)
        weight = torch.softmax(top, dim=1)
        if case["drop"] > 0:
            ids = torch.where(_uniform(gen, (T, K)) < case["drop"], -1, ids)
            ids = torch.where(_uniform(gen, (T, 1)) < case["drop"] / 4, -1, ids)
        s["ids"] = ids.to(_INDEX[case["index"]])
        s["weight"] = weight.to(_TYPES[case["weight"]])
        s["x"] = _normal(gen, (T, H), case["type"])
        s["y"] = _normal(gen, (T * K, H), case["type"])
        if op == "route_step":
            s["dout"] = _normal(gen, (T, H), case["type"], 0.1)
            s["drows"] = _normal(gen, (T * K, H), case["type"], 0.1)
        return s
    N, V, K = case["N"], case["V"], case["K"]
    z = _normal(gen, (N, V), case["type"], 2.5)
    s["logits"] = z
    ids = torch.empty((N, K), dtype=torch.int64, device="cuda")
    top = torch.empty((N, K), dtype=torch.float32, device="cuda")
    rows = max(1, 134_217_728 // V)
    for a in range(0, N, rows):      # a teacher that agrees with the student in part
        t = z[a:a + rows].float() + _normal(gen, (min(rows, N - a), V), "f32", 1.5)
        top[a:a + rows], ids[a:a + rows] = torch.topk(t, K, dim=1)
    kept = torch.randint(1, K + 1, (N, 1), generator=gen, device="cuda")   # ragged lists
    kept = torch.where(_uniform(gen, (N, 1)) < 0.3, kept, K)
    kept = torch.where(_uniform(gen, (N, 1)) < case["empty"], 0, kept)     # padding positions
    ids = torch.where(torch.arange(K, device="cuda") < kept, ids, -1)
    s["ids"] = ids.to(_INDEX[case["index"]])
    s["top"] = top.to(_TYPES[case["teacher"]])
    # half precision is trained with a scaled loss: its gradients would underflow
    s["grad_loss"] = (_uniform(gen, N) + 0.5) * ((1024.0 if case["type"] == "f16" else 1.0) / N)
    return s


# ---------------------------------------------------------------------------
# the plain forms

def _plain_token_forward(s):
    V = s["V"]
    ids = s["ids"].long()
    inside = (ids >= 0) & (ids < V)
    rows = s["table"][torch.where(inside, ids, 0)].float() * s["scale"]
    return torch.where(inside[:, None], rows, 0.0).to(_TYPES[s["out"]])


def _plain_token_backward(s):
    V = s["V"]
    ids = s["ids"].long()
    inside = (ids >= 0) & (ids < V)
    if s["padding"] is not None:
        inside &= ids != s["padding"]
    rows = torch.where(inside[:, None], s["grad"].float() * s["scale"], 0.0)
    total = torch.zeros((V, s["D"]), dtype=torch.float32, device=rows.device)
    total.index_add_(0, torch.where(inside, ids, 0), rows)
    return total.to(_TYPES[s["out"]])


def _plain_sort(s):
    E = s["E"]
    e = s["ids"].long().reshape(-1)
    e = torch.where((e >= 0) & (e < E), e, E)
    ordered, source = torch.sort(e, stable=True)
    slot = torch.empty_like(source)
    slot[source] = torch.arange(source.numel(), device=source.device)
    offset = (e[None, :] < torch.arange(E + 1, device=e.device)[:, None]).sum(1) if e.numel() * E < 1 << 22 else \
        torch.searchsorted(ordered, torch.arange(E + 1, device=e.device))
    source = torch.where(ordered < E, source, -1)
    slot = torch.where(e < E, slot, -1).reshape(s["ids"].shape)
    return slot, source, offset


def _plain_gather_sum(rows, slot, weight):
    """sum_k weight[t,k] * rows[slot[t,k]] in 32 bits, dropped pairs left out."""
    inside = (slot >= 0)[:, :, None]
    picked = torch.where(inside, rows[slot.clamp(min=0)].float() * weight[:, :, None], 0.0)
    return picked.sum(1)


def _plain_route(s):
    K, kind = s["K"], _TYPES[s["type"]]
    slot, source, offset = _plain_sort(s)
    used = (source >= 0)[:, None]
    token = source.clamp(min=0) // K
    weight = s["weight"].float()
    r = dict(slot=slot.int(), source=source.int(), offset=offset.int())
    r["rows"] = torch.where(used, s["x"][token], 0)
    r["out"] = _plain_gather_sum(s["y"], slot, weight).to(kind)
    if s["op"] == "route_step":
        dout = s["dout"].float()
        flat = weight.reshape(-1)[source.clamp(min=0)]
        r["drows"] = torch.where(used, dout[token] * flat[:, None], 0.0).to(kind)
        dot = (dout[:, None, :] * s["y"][slot.clamp(min=0)].float()).sum(2)
        r["dweight"] = torch.where(slot >= 0, dot, 0.0).to(s["weight"].dtype)
        r["dx"] = _plain_gather_sum(s["drows"], slot, torch.ones_like(weight)).to(kind)
    return r


def _plain_distill(s):
    c = s["temperature"]
    z = s["logits"].float() / c
    ids = s["ids"].long()
    valid = (ids >= 0) & (ids < s["V"])
    some = valid.any(1, keepdim=True)
    at = torch.where(valid, ids, 0)
    t = torch.where(valid, s["top"].float() / c, -math.inf)
    e = torch.where(valid, (t - t.max(1, keepdim=True).values).exp(), 0.0)
    p = e / torch.where(some, e.sum(1, keepdim=True), 1.0)
    high = z.max(1, keepdim=True).values
    ez = (z - high).exp()
    total = ez.sum(1, keepdim=True)
    lse = high + total.log()
    terms = torch.where(p > 0, p * (p.log() - (z.gather(1, at) - lse)), 0.0)
    loss = torch.where(some[:, 0], c * c * terms.sum(1), 0.0)
    g = s["grad_loss"][:, None] * c
    dz = ez.div_(total).scatter_add_(1, at, -p).mul_(g)
    dz = torch.where(some, dz, 0.0).to(_TYPES[s["type"]])
    return dict(loss=loss, lse=torch.where(some, lse, 0.0)[:, 0], grad=dz)


# ---------------------------------------------------------------------------
# the framework's operators

def _own(s):
    import recsys_table_embedding_gb300 as tbe
    op = s["op"]
    if op == "token_forward":
        return tbe.tbe_token_forward(s["table"], s["ids"], scale=s["scale"], dtype=_TYPES[s["out"]])
    if op == "token_backward":
        return tbe.tbe_token_backward(s["grad"], s["ids"], s["V"], scale=s["scale"],
                                      padding_id=s["padding"], dtype=_TYPES[s["out"]])
    if op.startswith("route"):
        rows, route = tbe.tbe_route_sort_dispatch(s["x"], s["ids"], s["E"])
        r = dict(slot=route.slot, source=route.source, offset=route.offset, rows=rows)
        r["out"] = tbe.tbe_route_combine(s["y"], route, s["weight"])
        if op == "route_step":
            r["drows"], r["dweight"] = tbe.tbe_route_combine_backward(s["dout"], s["y"], route, s["weight"])
            r["dx"] = tbe.tbe_route_dispatch_backward(s["drows"], route)
        return r
    if op == "distill_loss_grad":
        loss, lse, grad = tbe.tbe_distill_loss_grad(s["logits"], s["ids"], s["top"], s["grad_loss"],
                                                    temperature=s["temperature"])
    else:
        loss, lse = tbe.tbe_distill_forward(s["logits"], s["ids"], s["top"], temperature=s["temperature"])
        grad = tbe.tbe_distill_backward(s["logits"], s["ids"], s["top"], lse, s["grad_loss"],
                                        temperature=s["temperature"])
    return dict(loss=loss, lse=lse, grad=grad)


def run(state):
    if own:
        return _own(state)
    op = state["op"]
    if op == "token_forward":
        return _plain_token_forward(state)
    if op == "token_backward":
        return _plain_token_backward(state)
    if op.startswith("route"):
        return _plain_route(state)
    return _plain_distill(state)


# ---------------------------------------------------------------------------
# what a pass cannot do without

def _unique(case):
    """Expected number of different rows among a case's N tokens."""
    N, V, a = case["N"], case["V"], case["zipf"]
    p = np.arange(1, V + 1, dtype=np.float64) ** -a
    p /= p.sum()
    return float(np.sum(-np.expm1(N * np.log1p(-np.minimum(p, 1 - 1e-12)))))


def work(case):
    op = case["op"]
    i = 4 if case["index"] == "i32" else 8
    b = _BYTES[case["type"]]
    if op == "token_forward":
        N, D = case["N"], case["D"]
        return {"bytes": N * i + _unique(case) * D * b + N * D * _BYTES[case["out"]], "flops": N * D}
    if op == "token_backward":
        N, V, D = case["N"], case["V"], case["D"]
        kept = N * (1 - case["pad"])
        return {"bytes": N * i + kept * D * b + V * D * _BYTES[case["out"]], "flops": 2 * kept * D}
    if op.startswith("route"):
        T, K, E, H = case["T"], case["K"], case["E"], case["H"]
        P = T * K
        n = P * (i + 8) + (E + 1) * 4 + P * _BYTES[case["weight"]]      # ids, slot, source, offset, weights
        n += (2 * T * H + 2 * P * H) * b                                # x, out; rows, y
        f = 2 * P * H
        if op == "route_step":
            n += (2 * T * H + 2 * P * H) * b + P * _BYTES[case["weight"]]   # dout, dx; both gradients of rows
            f += 4 * P * H
        return {"bytes": n, "flops": f}
    N, V, K = case["N"], case["V"], case["K"]
    n = 2 * N * V * b + N * K * (i + _BYTES[case["teacher"]]) + 12 * N
    return {"bytes": n, "flops": 6 * N * V}


# ---------------------------------------------------------------------------
# the definitions in 64 bits

def _exact_token(s):
    V = s["V"]
    ids = s["ids"].cpu().numpy().astype(np.int64)
    n = np.flatnonzero((ids >= 0) & (ids < V))
    if s["op"] == "token_forward":
        out = torch.zeros((s["N"], s["D"]), dtype=torch.float64, device="cuda")
        at = torch.from_numpy(n).cuda()
        out[at] = s["table"].index_select(0, torch.from_numpy(ids[n]).cuda()).double() * s["scale"]
        return out
    if s["padding"] is not None:
        n = n[ids[n] != s["padding"]]
    n = n[np.argsort(ids[n], kind="stable")]
    at = torch.from_numpy(n).cuda()
    grad = torch.zeros((V, s["D"]), dtype=torch.float64, device="cuda")
    step = max(1, 33_554_432 // s["D"])
    for a in range(0, len(n), step):
        part = at[a:a + step]
        grad.index_put_((s["ids"][part].long(),), s["grad"][part].double(), accumulate=True)
    return grad.mul_(s["scale"])


def _exact_route(s):
    T, K, E, H = s["T"], s["K"], s["E"], s["H"]
    ids = s["ids"].cpu().numpy().reshape(-1).astype(np.int64)
    pairs = np.concatenate([np.flatnonzero(ids == e) for e in range(E)])
    slot = np.full(T * K, -1, np.int64)
    slot[pairs] = np.arange(len(pairs))
    slot = torch.from_numpy(slot.reshape(T, K)).cuda()
    pairs = torch.from_numpy(pairs).cuda()
    w = s["weight"].double()
    M = len(pairs)
    r = dict(slot=None, source=None, offset=None)
    r["rows"] = torch.zeros((T * K, H), dtype=torch.float64, device="cuda")
    r["rows"][:M] = s["x"].double()[pairs // K]
    out = torch.zeros((T, H), dtype=torch.float64, device="cuda")
    dx = torch.zeros_like(out)
    dw = torch.zeros((T, K), dtype=torch.float64, device="cuda")
    step = s["op"] == "route_step"
    for k in range(K):
        t = torch.nonzero(slot[:, k] >= 0)[:, 0]
        at = slot[t, k]
        y = s["y"][at].double()
        out[t] += y * w[t, k, None]
        if step:
            dx[t] += s["drows"][at].double()
            dw[t, k] = torch.einsum("th,th->t", s["dout"][t].double(), y)
    r["out"] = out
    if step:
        r["drows"] = torch.zeros((T * K, H), dtype=torch.float64, device="cuda")
        r["drows"][:M] = s["dout"].double()[pairs // K] * w.reshape(-1)[pairs, None]
        r["dweight"], r["dx"] = dw, dx
    return r


def _exact_distill(s):
    N, V, c = s["N"], s["V"], s["temperature"]
    loss = torch.zeros(N, dtype=torch.float64, device="cuda")
    lse = torch.zeros(N, dtype=torch.float64, device="cuda")
    grad = torch.zeros((N, V), dtype=torch.float64, device="cuda")
    step = max(1, 33_554_432 // V)
    for a in range(0, N, step):
        ids = s["ids"][a:a + step].long()
        valid = (ids >= 0) & (ids < V)
        keep = torch.nonzero(valid.any(1))[:, 0]
        if keep.numel() == 0:
            continue
        ids, valid = ids[keep], valid[keep]
        z = s["logits"][a:a + step][keep].double() / c
        logp = torch.log_softmax((s["top"][a:a + step][keep].double() / c).masked_fill(~valid, -1e300), 1)
        p = logp.exp().masked_fill(~valid, 0.0)
        lse[a + keep] = torch.logsumexp(z, 1)
        logq = z - lse[a + keep, None]
        diff = (logp - logq.gather(1, ids.masked_fill(~valid, 0))).masked_fill(~valid, 0.0)
        loss[a + keep] = c * c * torch.einsum("nk,nk->n", p, diff)
        dense = torch.zeros_like(z).scatter_add_(1, ids.masked_fill(~valid, 0), p)
        grad[a + keep] = (logq.exp() - dense) * (c * s["grad_loss"][a + keep, None].double())
    return dict(loss=loss, lse=lse, grad=grad)


def exact(case, seed):
    s = prepare(case, seed)
    if s["op"].startswith("token"):
        return _exact_token(s)
    if s["op"].startswith("route"):
        return _exact_route(s)
    return _exact_distill(s)
