"""The token operators' definitions in 64 bits (plain torch, any device), and
the error bounds that 32-bit sums and one rounding to the result's type allow.

Bounds.  u(type) is half the distance between neighbouring values over the
value: 2^-24, 2^-11, 2^-8 for f32, f16, bf16.  A sum of n products held in 32
bits is off by at most (n + 2) u(f32) sum |terms|; rounding the result adds
u(type) |result|, and half the smallest step (2^-25) where f16 goes subnormal.
"""
import math

import torch

TYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
U = {torch.float32: 2.0 ** -24, torch.float16: 2.0 ** -11, torch.bfloat16: 2.0 ** -8}
U32 = 2.0 ** -24


def rounding(value: torch.Tensor, dtype) -> torch.Tensor:
    return U[dtype] * value.abs() + (2.0 ** -25 if dtype == torch.float16 else 0.0)


def close(got: torch.Tensor, want: torch.Tensor, bound: torch.Tensor):
    """|got - want| <= bound everywhere, infinities and NaN in the same places."""
    got = got.double()
    finite = torch.isfinite(want)
    assert torch.equal(torch.isnan(got), torch.isnan(want))
    other = ~finite & ~torch.isnan(want)
    assert torch.equal(got[other], want[other])
    off = ((got - want).abs() - bound)[finite]
    assert off.numel() == 0 or float(off.max()) <= 0, \
        f"off by {float(off.max())} over a bound of {float(bound[finite].max())}"


def token_forward(table, ids, scale):
    V = table.shape[0]
    inside = (ids >= 0) & (ids < V)
    out = torch.zeros((*ids.shape, table.shape[1]), dtype=torch.float64, device=table.device)
    out[inside] = table.double()[ids[inside].long()] * scale
    return out


def token_backward(grad, ids, V, scale, padding=None):
    """(gradient, sum of |terms|, tokens per row)"""
    keep = (ids >= 0) & (ids < V)
    if padding is not None:
        keep &= ids != padding
    at = ids[keep].long()
    rows = grad.double()[keep] * scale
    z = torch.zeros((V, grad.shape[-1]), dtype=torch.float64, device=grad.device)
    n = torch.zeros(V, dtype=torch.float64, device=grad.device)
    n.index_add_(0, at, torch.ones_like(at, dtype=torch.float64))
    return z.index_add(0, at, rows), z.index_add(0, at, rows.abs()), n[:, None]


def route(ids, E):
    """slot, source, offset by a plain loop over the experts."""
    flat = ids.reshape(-1).tolist()
    places = [p for e in range(E) for p, x in enumerate(flat) if x == e] if len(flat) * E < 1 << 20 else None
    if places is None:
        key = torch.tensor([x if 0 <= x < E else E for x in flat])
        order = sorted(range(len(flat)), key=lambda p: (int(key[p]), p))
        places = [p for p in order if key[p] < E]
    slot = [-1] * len(flat)
    for s, p in enumerate(places):
        slot[p] = s
    source = places + [-1] * (len(flat) - len(places))
    count = [0] * (E + 1)
    for p in places:
        count[flat[p] + 1] += 1
    offset = torch.tensor(count).cumsum(0)
    return (torch.tensor(slot).reshape(ids.shape).int(), torch.tensor(source, dtype=torch.int32), offset.int())


def combine(rows, slot, weight=None):
    """(out, sum of |terms|)"""
    T, K = slot.shape
    out = torch.zeros((T, rows.shape[1]), dtype=torch.float64, device=rows.device)
    mag = torch.zeros_like(out)
    for k in range(K):
        t = torch.nonzero(slot[:, k] >= 0)[:, 0]
        v = rows[slot[t, k].long()].double()
        if weight is not None:
            v = v * weight[t, k, None].double()
        out[t] += v
        mag[t] += v.abs()
    return out, mag


def combine_backward(dout, rows, slot, weight):
    """(drows, dweight, sum of |terms| of dweight)"""
    T, K = slot.shape
    drows = torch.zeros(rows.shape, dtype=torch.float64, device=rows.device)
    dw = torch.zeros((T, K), dtype=torch.float64, device=rows.device)
    mag = torch.zeros_like(dw)
    for k in range(K):
        t = torch.nonzero(slot[:, k] >= 0)[:, 0]
        s = slot[t, k].long()
        terms = dout[t].double() * rows[s].double()
        dw[t, k], mag[t, k] = terms.sum(1), terms.abs().sum(1)
        drows[s] = dout[t].double() * weight[t, k, None].double()
    return drows, dw, mag


def distill(logits, ids, top, g, c):
    """(loss, lse, grad, p per column) with a row at a time."""
    N, V = logits.shape
    z = logits.double() / c
    loss = torch.zeros(N, dtype=torch.float64, device=logits.device)
    lse = torch.zeros_like(loss)
    grad = torch.zeros((N, V), dtype=torch.float64, device=logits.device)
    dense = torch.zeros_like(grad)
    for n in range(N):
        keep = (ids[n] >= 0) & (ids[n] < V)
        t = top[n][keep].double() / c
        if t.numel() == 0 or bool((t == -math.inf).all()):
            continue
        at = ids[n][keep].long()
        logp = t - torch.logsumexp(t, 0)
        p = logp.exp()
        lse[n] = torch.logsumexp(z[n], 0)
        logq = z[n] - lse[n]
        terms = torch.where(p == 0, torch.zeros_like(p), p * (logp - logq[at]))
        loss[n] = c * c * terms.sum()
        dense[n].index_add_(0, at, p)
        grad[n] = g[n].double() * c * (logq.exp() - dense[n])
    return loss, lse, grad, dense


def distill_bounds(logits, ids, top, g, c, want, stored_lse):
    """Bounds of (loss, lse, grad).  The sum of a row's exponentials is a chain
    of at most V/256 + 64 additions; an exponent d = (z - m)/c carries 4
    roundings of its size and 2^x another 2^-21; sizes |d| beyond 40 have
    exponentials below the others' rounding.  ``stored_lse``: the gradient is
    computed from lse as it is rounded to 32 bits."""
    loss, lse, grad, dense = want
    V = logits.shape[1]
    z = logits.double() / c
    m = z.max(1).values
    rel_sum = (V / 256 + 64 + 160) * U32 + 2.0 ** -21
    b_lse = rel_sum + 4 * U32 * (m.abs() + lse.abs())
    K = ids.shape[1]
    d = (m[:, None] - torch.where((ids >= 0) & (ids < V), z.gather(1, ids.clamp(0, V - 1).long()), m[:, None]))
    d = torch.nan_to_num(d, posinf=0.0)
    t = top.double() / c
    t = torch.where((ids >= 0) & (ids < V) & torch.isfinite(t), t, torch.nan)
    spread = torch.nan_to_num(torch.nan_to_num(t, nan=-1e30).max(1).values - torch.nan_to_num(t, nan=1e30).min(1).values).clamp(0, 1e4)
    b_p = (K + 64) * U32 + 8 * U32 * spread[:, None] + 2.0 ** -21      # relative, of p
    log_size = d.max(1).values + (lse - m).abs() + spread + math.log(K + 1)
    b_loss = c * c * (b_p[:, 0] * log_size + rel_sum + 8 * U32 * log_size + (K + 8) * U32 * log_size)
    q = torch.where(dense.sum(1, keepdim=True) > 0, (z - lse[:, None]).exp(), torch.zeros_like(z))
    rel_q = rel_sum + 160 * U32 + (4 * U32 * lse.abs()[:, None] if stored_lse else 0.0)
    b = (g.double() * c).abs()[:, None] * (q * rel_q + dense * b_p + 4 * U32 * (q + dense))
    return b_loss, b_lse, b + rounding(grad, logits.dtype) + b * U[logits.dtype] + 2.0 ** -125
