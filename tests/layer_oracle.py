"""The layer operators' definitions in 64 bits (plain torch, any device), and the
error bounds that 32-bit sums and one rounding to the result's type allow.

Bounds (u = 2^-24).  An addition into a 32-bit sum is off by at most 2 u of the
sum's terms (a tensor core's accumulator may cut off instead of rounding), so a
sum of n products by 2 (n + 2) u sum |terms|.  The activations: expf, a division
and erfcf are off by a few u relative each, an argument's rounding moves a normal
tail by its square: 16 u (1 + g^2) of every term covers them.  |a'| <= 1.13.
"""
import math

import torch

from token_oracle import U, U32, close, rounding  # noqa: F401  (what the tests use of it)

SQRT2 = math.sqrt(2.0)


def groups(offset, rows):
    """(expert, first row, end) of each group, from the offsets as the library takes them."""
    if offset is None:
        return [(0, 0, rows)]
    o = [min(max(x, 0), rows) for x in offset.tolist()]
    o[0] = 0
    return [(e, a, max(a, b)) for e, (a, b) in enumerate(zip(o[:-1], o[1:]))]


def product(x, w, offset, transposed=False):
    """(x_s W_e^T or x_s W_e, bound of a 32-bit sum); rows of no group are zero."""
    P = x.shape[0]
    out = torch.zeros((P, w.shape[2 if transposed else 1]), dtype=torch.float64, device=x.device)
    mag = torch.zeros_like(out)
    for e, a, b in groups(offset, P):
        m = w[e].double() if transposed else w[e].double().t()
        out[a:b] = x[a:b].double() @ m
        mag[a:b] = x[a:b].double().abs() @ m.abs()
    return out, 2 * (x.shape[1] + 2) * U32 * mag


def weight_gradient(dy, x, offset, experts):
    out = torch.zeros((experts, dy.shape[1], x.shape[1]), dtype=torch.float64, device=x.device)
    mag = torch.zeros_like(out)
    for e, a, b in groups(offset, x.shape[0]):
        d, v = dy[a:b].double(), x[a:b].double()
        out[e] = d.t() @ v
        mag[e] = 2 * (b - a + 2) * U32 * (d.abs().t() @ v.abs())
    return out, mag


def activation(g, kind):
    """(a, a', bound of a, bound of a') for g in 64 bits."""
    loose = 16 * U32 * (1 + g * g)
    if kind == "silu":
        s = torch.sigmoid(g)
        slope = s * (1 + g * torch.sigmoid(-g))
        return g * s, slope, loose * (g * s).abs(), 16 * U32 * s * (1 + g.abs())
    c = 0.5 * torch.special.erfc(-g / SQRT2)
    d = g * torch.exp(-0.5 * g * g) / math.sqrt(2 * math.pi)
    return g * c, c + d, loose * (g * c).abs(), loose * (c + d.abs())


def gated(z, bound, kind):
    """(hidden, its bound before rounding) of [g | u] = z off by at most `bound`."""
    F = z.shape[1] // 2
    g, u = z[:, :F], z[:, F:]
    a, _, ba, _ = activation(g, kind)
    ba = ba + 1.13 * bound[:, :F]
    return a * u, ba * (u.abs() + bound[:, F:]) + a.abs() * bound[:, F:] + 2 * U32 * (a * u).abs()


def gate_gradient(dh, bound, z, kind):
    """([dg | du], bound before rounding) for dh off by at most `bound`, [g | u] = z exactly."""
    F = z.shape[1] // 2
    g, u = z[:, :F].double(), z[:, F:].double()
    a, slope, ba, bs = activation(g, kind)
    dg, du = dh * u * slope, dh * a
    bg = bound * (u * slope).abs() + (dh.abs() + bound) * u.abs() * bs + 4 * U32 * dg.abs()
    bu = bound * a.abs() + (dh.abs() + bound) * ba + 4 * U32 * du.abs()
    return torch.cat([dg, du], 1), torch.cat([bg, bu], 1)


def rounded(bound, want, dtype):
    """A bound of a result before its rounding, and that rounding."""
    return bound * (1 + U[dtype]) + rounding(want, dtype) + 2.0 ** -140


def norm(x, w, b, eps):
    """((out, mean, rstd), their bounds before rounding).  A thread adds D/1024 + 32
    terms at most, then come ten steps of a tree."""
    D = x.shape[1]
    n = D / 1024 + 64
    x = x.double()
    w = torch.ones(D, dtype=torch.float64, device=x.device) if w is None else w.double()
    b = torch.zeros(D, dtype=torch.float64, device=x.device) if b is None else b.double()
    mean = x.mean(1)
    c = x - mean[:, None]
    var = (c * c).mean(1)
    rstd = (var + eps).rsqrt()
    off = n * U32 * c.abs().mean(1)              # of the corrected mean
    first = n * U32 * x.abs().mean(1)            # of the mean before its correction
    rel = (n + 16) * U32 + (off * off + n * U32 * first * first) / (var + eps)
    out = c * rstd[:, None] * w + b
    bound = (off[:, None] + 4 * U32 * c.abs()) * rstd[:, None] * w.abs() + rel[:, None] * (out - b).abs() + \
        4 * U32 * (b.abs() + (out - b).abs())
    # where eps is 0 and a row constant: rstd is infinite and out NaN, in both
    return (out, mean, rstd), (bound, off + 2 * U32 * mean.abs() + U32 * first, rel * rstd)


def norm_backward(dy, x, mean, rstd, w):
    """((dx, dw, db), bounds before rounding), from mean and rstd as they are."""
    N, D = x.shape
    n = D / 512 + 64
    dy, x, mean, r = dy.double(), x.double(), mean.double()[:, None], rstd.double()[:, None]
    w = torch.ones(D, dtype=torch.float64, device=x.device) if w is None else w.double()
    h, d = (x - mean) * r, dy * w
    s1, s2 = d.mean(1, keepdim=True), (d * h).mean(1, keepdim=True)
    dx = r * (d - s1 - h * s2)
    b1, b2 = n * U32 * d.abs().mean(1, keepdim=True), (n + 4) * U32 * (d * h).abs().mean(1, keepdim=True)
    bx = r * (b1 + h.abs() * b2 + 6 * U32 * (d.abs() + s1.abs() + (h * s2).abs()))
    bw = (N + 24) * U32 * (dy * h).abs().sum(0)
    return (dx, (dy * h).sum(0), dy.sum(0)), (bx, bw, (N + 24) * U32 * dy.abs().sum(0))


# ---------------------------------------------------------------------------
# AdamW

def mix(h):
    """The finalising mix of MurmurHash3 on 32 bits, for ints and int64 tensors."""
    h = ((h ^ (h >> 16)) * 0x85EBCA6B) & 0xFFFFFFFF
    h = ((h ^ (h >> 13)) * 0xC2B2AE35) & 0xFFFFFFFF
    return h ^ (h >> 16)


def random16(seed, step, index, n, device):
    """The two 16-bit numbers of each element."""
    key = mix((mix((seed + step * 0x9E3779B9) & 0xFFFFFFFF) + index) & 0xFFFFFFFF)
    i = torch.arange(n, device=device)
    h = mix((mix((i // 256 + key) & 0xFFFFFFFF) + (i % 256) * 0x9E3779B9) & 0xFFFFFFFF)
    return h & 0xFFFF, h >> 16


def adamw(p, g, m, v, t, lr, b1, b2, eps, wd):
    """((p, m, v), bounds before rounding) in 64 bits; m and v as values."""
    p, g, m, v = (x.double() for x in (p, g, m, v))
    m1, v1 = b1 * m + (1 - b1) * g, b2 * v + (1 - b2) * g * g
    bm = 3 * U32 * ((b1 * m).abs() + ((1 - b1) * g).abs())
    bv = 5 * U32 * v1
    rate, root = lr / (1 - b1 ** t), 1 / math.sqrt(1 - b2 ** t)
    below = v1.sqrt() * root + eps
    change = rate * m1 / below
    bc = rate * bm / below + 12 * U32 * change.abs()
    p1 = p * (1 - lr * wd) - change
    return (p1, m1, v1), (bc + 3 * U32 * p.abs() + U32 * p1.abs(), bm, bv)


def in_blocks(x):
    return torch.nn.functional.pad(x, (0, -x.numel() % 256)).view(-1, 256)


def encode(x, bound, bits, floor):
    """(codes' values, scales, whether the code is the only one that 32-bit
    arithmetic can give) of x in 64 bits, which 32 bits hold to `bound`.  The sum t
    of at most 17 that is cut off carries that bound in steps of the code (a
    moment that two terms nearly cancel in is small, and so is its step, while the
    bound goes by the terms), the scale's bound likewise, and four roundings of t:
    4 * 17 * 2^-24 < 2^-17."""
    n = x.numel()
    a = x.abs()
    most = in_blocks(a).amax(1)
    scale = torch.where(most < 2.0 ** -100, torch.zeros_like(most), most / 448)
    wide = lambda v: v.repeat_interleave(256)[:n]  # noqa: E731
    s = wide(scale)
    y = torch.where(s > 0, a / s.clamp(min=1e-300), torch.zeros_like(a))
    step = torch.exp2(torch.floor(torch.log2(y.clamp(min=2.0 ** -30))).clamp(min=-6) - 3)
    t = y / step + bits.double() / 65536
    q = (t.floor() * step).clamp(max=448)
    if floor:
        q = torch.where((y > 0) & (q == 0), torch.full_like(q, 2.0 ** -9), q)
    off = 2.0 ** -17 + torch.where(s > 0, (bound + a * wide(in_blocks(bound).amax(1) / most.clamp(min=1e-300))) /
                                   (s.clamp(min=1e-300) * step), torch.zeros_like(a))
    sure = ((t - t.round()).abs() > off) & ((a > bound) | (y == 0))
    # a value at a binade's border may be taken with either step
    sure &= ((y / step - 8).abs() > off) & ((y / step - 16).abs() > off) | (step == 2.0 ** -9) & (y / step < 7)
    return torch.copysign(q, x), scale, sure
