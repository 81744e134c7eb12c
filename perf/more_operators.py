"""Measured cases of the layer operators: the experts' products (gated block,
plain product, gradients of rows and of weights), layer norm with its gradients,
and the AdamW step over many tensors.

``own`` selects what ``run`` computes: the framework's operators where it is
true, their plain form in elementary torch operations (32-bit, rounded once at
the end) where it is false.  ``exact`` states each operator in 64 bits.
"""
from __future__ import annotations

import math

import torch

own = False

_TYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
_BYTES = {"f32": 4, "f16": 2, "bf16": 2}
_BLOCK = 256        # elements that share a scale in 8-bit states
_BETA1, _BETA2, _EPS, _DECAY, _LR, _STEP = 0.9, 0.999, 1e-8, 0.1, 1e-3, 10


# ---------------------------------------------------------------------------
# cases

def _experts(op, T, K, E, H, F, type, grad="", act="silu", drop=0.0):
    """K = 0: a dense block, every row in the one group."""
    return dict(op=op, T=T, K=K, E=E, H=H, F=F, type=type, grad_type=grad or type, act=act, drop=drop)


def _norm(op, N, D, type, weight=""):
    return dict(op=op, N=N, D=D, type=type, weight=weight or type)


def _adamw(layers, D, F, param, grad, copy="", state="f32", odd=False):
    """The parameters of ``layers`` blocks: a norm's weight and bias, a router
    of 16 experts, the matrices of a gated block."""
    return dict(op="adamw", layers=layers, D=D, F=F, param=param, grad=grad, copy=copy, state=state, odd=odd)


def listed():
    cases = {
        # one generated token through 8 of a layer's 64 experts
        "experts one token": _experts("experts_forward", 1, 8, 64, 2048, 1024, "bf16"),
        # a decoding batch: every expert gets a few rows, the weights are read once
        "experts decoding batch": _experts("experts_forward", 64, 8, 64, 2048, 1024, "f16", drop=0.02),
        # a small ragged batch in 32 bits whose sizes fit no tile, forward and gradients
        "experts odd batch": _experts("experts_step", 1001, 3, 37, 501, 203, "f32", act="gelu", drop=0.1),
        # a training step's experts, forward and gradients
        "experts training step": _experts("experts_step", 32_768, 8, 128, 1024, 768, "bf16", drop=0.02),
        # a dense block's training step, weights' gradient kept in 32 bits
        "dense block step": _experts("experts_step", 8192, 0, 1, 2048, 5504, "bf16", grad="f32"),
        # the newest token before a layer
        "norm one token": _norm("norm_forward", 1, 2048, "bf16"),
        # odd rows in 32 bits, forward and gradients
        "norm odd batch": _norm("norm_step", 1001, 501, "f32"),
        # a training step's rows, forward and gradients
        "norm training step": _norm("norm_step", 32_768, 4096, "bf16", "f32"),
        # wide rows of a long prompt
        "norm wide rows": _norm("norm_forward", 8192, 16_384, "f16"),
        # a small model whose tensors lie back to back at odd places
        "adamw small": _adamw(4, 63, 99, "f32", "f32", odd=True),
        # 32-bit parameters and states, 16-bit gradients and copies for the next forward pass
        "adamw training step": _adamw(8, 2048, 2752, "f32", "bf16", copy="bf16"),
        # the same with states in 8 bits
        "adamw 8-bit states": _adamw(8, 2048, 2752, "f32", "bf16", copy="bf16", state="f8"),
    }
    return [dict(name=k, **c) for k, c in cases.items()]


def _log(rng, lo, hi):
    """An integer in [lo, hi], spread over its logarithm, often of no round size."""
    v = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))
    if rng.random() < 0.4 and v >= 64:
        v = v // 32 * 32
    return min(hi, max(lo, v))


def draw(rng):
    op = rng.choice(["experts_forward", "experts_step", "norm_forward", "norm_step", "adamw", "adamw"])
    type = rng.choice(["f32", "f16", "bf16"])
    if op.startswith("experts"):
        H, F = _log(rng, 32, 4096), _log(rng, 32, 4096)
        dense = rng.random() < 0.3
        E = 1 if dense else min(_log(rng, 2, 128), max(2, 50_000_000 // (H * F)))
        K = 0 if dense else min(E, rng.randint(1, 8))
        # at most a tenth of the training step's products in 32 bits, half of them in 16
        most = (4 if type == "f32" else 20) * 5_000_000_000 // (H * F)
        T = max(1, min(_log(rng, 1, 32_768), most // max(K, 1), 400_000_000 // (max(K, 1) * (H + F))))
        return _experts(op, T, K, E, H, F, type, rng.choice([type, "f32"]), rng.choice(["silu", "gelu"]),
                        0.0 if dense else rng.choice([0.0, 0.02, 0.3]))
    if op.startswith("norm"):
        D = _log(rng, 16, 32_768)
        return _norm(op, min(_log(rng, 1, 65_536), 67_108_864 // D), D, type, rng.choice([type, "f32"]))
    D, F = _log(rng, 16, 2048), _log(rng, 16, 4096)
    layers = max(1, min(rng.randint(1, 24), 100_000_000 // (3 * D * F)))
    param = rng.choice(["f32", "f32", "bf16", "f16"])
    return _adamw(layers, D, F, param, rng.choice(["f32", "bf16", "f16"]) if param == "f32" else param,
                  rng.choice(["", "bf16", "f16"]) if param == "f32" else "", rng.choice(["f32", "f8"]),
                  rng.random() < 0.4)


# ---------------------------------------------------------------------------
# inputs

def _normal(gen, shape, type, std=1.0):
    x = torch.empty(shape, dtype=_TYPES[type], device="cuda")
    return x.normal_(0.0, std, generator=gen)


def _uniform(gen, shape):
    return torch.rand(shape, generator=gen, device="cuda")


def _route(case, gen):
    """The pairs of T tokens with K of E experts, sorted: slot, source and
    offset one after the other (int32), and the offsets on the host."""
    T, K, E = case["T"], case["K"], case["E"]
    score = _normal(gen, (T, E), "f32") + torch.linspace(0.8, -0.8, E, device="cuda")
    ids = torch.topk(score, K, dim=1).indices
    ids = torch.where(_uniform(gen, (T, K)) < case["drop"], E, ids).reshape(-1)
    ordered, source = torch.sort(ids, stable=True)
    slot = torch.empty_like(source)
    slot[source] = torch.arange(T * K, device="cuda")
    offset = torch.searchsorted(ordered, torch.arange(E + 1, device="cuda"))
    route = torch.cat([torch.where(ids < E, slot, -1), torch.where(ordered < E, source, -1), offset])
    return route.int(), offset.tolist()


def _sizes(case):
    D, F = case["D"], case["F"]
    return [D, D, 16 * D, 2 * F * D, F * D] * case["layers"]


def _places(case):
    """(start of each tensor in the flat buffers, elements of a flat buffer)"""
    starts, at = [], 0
    for n in _sizes(case):
        starts.append(at)
        at += n if case["odd"] else -(-n // 64) * 64
    return starts, at


def _blocks(case):
    """(start of each tensor's scales, scales of all)"""
    starts, at = [], 0
    for n in _sizes(case):
        starts.append(at)
        at += -(-n // _BLOCK)
    return starts, at


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    op = case["op"]
    s = dict(case)
    if op.startswith("experts"):
        T, K, E, H, F = (case[k] for k in ("T", "K", "E", "H", "F"))
        P = T * max(K, 1)
        s["route"], s["bounds"] = _route(case, gen) if K else (None, [0, P])
        M = s["bounds"][-1]
        s["rows"] = _normal(gen, (P, H), case["type"])
        s["rows"][M:] = 0
        s["w_in"] = _normal(gen, (E, 2 * F, H), case["type"], H ** -0.5)
        s["w_out"] = _normal(gen, (E, H, F), case["type"], F ** -0.5)
        if op == "experts_step":      # what the forward pass kept, and the gradient that comes back
            s["gate_up"] = _normal(gen, (P, 2 * F), case["type"])
            s["kept"] = _normal(gen, (P, F), case["type"], 0.6)
            s["grad"] = _normal(gen, (P, H), case["type"], 0.1)
            s["grad_gate_up"] = _normal(gen, (P, 2 * F), case["type"], 0.1)
        else:
            s["kept"] = _normal(gen, (P, F), case["type"], 0.6)
        return s
    if op.startswith("norm"):
        N, D = case["N"], case["D"]
        # a residual stream: rows of different size, an offset, a few columns far off the others
        x = _normal(gen, (N, D), "f32") * torch.exp(0.5 * _normal(gen, (N, 1), "f32")) + 0.3
        x += 20.0 * (_uniform(gen, (1, D)) < 0.01)
        s["x"] = x.to(_TYPES[case["type"]])
        s["weight"] = (1.0 + 0.2 * _normal(gen, (D,), "f32")).to(_TYPES[case["weight"]])
        s["bias"] = _normal(gen, (D,), case["weight"], 0.2)
        if op == "norm_step":
            s["grad"] = _normal(gen, (N, D), case["type"], 0.1)
        return s
    starts, total = _places(case)
    sizes = _sizes(case)
    for n in ("param", "grad"):
        s[n + "_flat"] = _normal(gen, (total,), case[n], 0.02 if n == "param" else 1e-3)
    s["seed"] = int(seed) & 0x7fffffff
    views = lambda flat, at=starts, n=sizes: [flat[a:a + k] for a, k in zip(at, n)]  # noqa: E731
    s["copy_flat"] = torch.zeros(total, dtype=_TYPES[case["copy"]], device="cuda") if case["copy"] else None
    if case["state"] == "f32":
        s["m_flat"] = _normal(gen, (total,), "f32", 3e-4)
        s["v_flat"] = _normal(gen, (total,), "f32", 1e-3).square_()
        s["scale_flat"] = None
    else:
        at, blocks = _blocks(case)
        s["m_flat"] = _normal(gen, (total,), "f32", 80.0).clamp_(-448, 448).to(torch.float8_e4m3fn)
        s["v_flat"] = _normal(gen, (total,), "f32", 100.0).abs_().clamp_(2.0 ** -9, 448).to(torch.float8_e4m3fn)
        scale = torch.exp(_normal(gen, (blocks, 2), "f32", 0.3)) * torch.tensor([3e-4 / 80, 1e-3 / 100], device="cuda")
        s["scale_flat"] = scale
        s["scales"] = [scale[a:a + -(-n // _BLOCK)] for a, n in zip(at, sizes)]
    for n in ("param", "grad", "m", "v"):
        s[n + "s"] = views(s[n + "_flat"])
    s["copies"] = views(s["copy_flat"]) if case["copy"] else None
    return s


# ---------------------------------------------------------------------------
# the plain forms

def _activation(g, act):
    """(act(g), act'(g))"""
    if act == "silu":
        sig = 1.0 / (1.0 + torch.exp(-g))
        return g * sig, sig * (1.0 + g * (1.0 - sig))
    phi = 0.5 * (1.0 + torch.erf(g * 0.5 ** 0.5))
    return g * phi, phi + g * torch.exp(-0.5 * g * g) * (0.5 / math.pi) ** 0.5


def _groups(bounds):
    return [(e, a, b) for e, (a, b) in enumerate(zip(bounds[:-1], bounds[1:])) if b > a]


def _rows_product(x, w, bounds, transposed=False):
    """x_s W_e^T (or x_s W_e) for the rows of each group, in 32 bits."""
    out = torch.zeros((x.shape[0], w.shape[2 if transposed else 1]), dtype=torch.float32, device=x.device)
    for e, a, b in _groups(bounds):
        torch.matmul(x[a:b].float(), w[e].float() if transposed else w[e].float().t(), out=out[a:b])
    return out


def _weights_product(dy, x, bounds):
    out = torch.zeros((len(bounds) - 1, dy.shape[1], x.shape[1]), dtype=torch.float32, device=x.device)
    for e, a, b in _groups(bounds):
        torch.matmul(dy[a:b].float().t(), x[a:b].float(), out=out[e])
    return out


def _plain_experts(s):
    kind, F, bounds = _TYPES[s["type"]], s["F"], s["bounds"]
    z = _rows_product(s["rows"], s["w_in"], bounds)
    hidden = (_activation(z[:, :F], s["act"])[0] * z[:, F:]).to(kind)
    r = dict(hidden=hidden, out=_rows_product(s["kept"], s["w_out"], bounds).to(kind))
    if s["op"] == "experts_step":
        r["gate_up"] = z.to(kind)
        dh = _rows_product(s["grad"], s["w_out"], bounds, transposed=True)
        a, da = _activation(s["gate_up"][:, :F].float(), s["act"])
        r["grad_gate_up"] = torch.cat([dh * s["gate_up"][:, F:].float() * da, dh * a], 1).to(kind)
        r["grad_rows"] = _rows_product(s["grad_gate_up"], s["w_in"], bounds, transposed=True).to(kind)
        r["grad_w_in"] = _weights_product(s["grad_gate_up"], s["rows"], bounds).to(_TYPES[s["grad_type"]])
        r["grad_w_out"] = _weights_product(s["grad"], s["kept"], bounds).to(_TYPES[s["grad_type"]])
    return r


def _plain_norm(s):
    x = s["x"].float()
    w, b = s["weight"].float(), s["bias"].float()
    mean = x.mean(1)
    xc = x - mean[:, None]
    rstd = 1.0 / torch.sqrt((xc * xc).mean(1) + 1e-5)
    xh = xc * rstd[:, None]
    r = dict(out=(xh * w + b).to(s["x"].dtype), mean=mean, rstd=rstd)
    if s["op"] == "norm_step":
        dy = s["grad"].float()
        d = dy * w
        dx = (d - d.mean(1, keepdim=True) - xh * (d * xh).mean(1, keepdim=True)) * rstd[:, None]
        r["grad_x"] = dx.to(s["x"].dtype)
        r["grad_weight"] = (dy * xh).sum(0).to(s["weight"].dtype)
        r["grad_bias"] = dy.sum(0).to(s["bias"].dtype)
    return r


def _mix(h):
    """The finalising mix of MurmurHash3 on 32 bits: an int, or a tensor of int64."""
    h = ((h ^ (h >> 16)) * 0x85EBCA6B) & 0xFFFFFFFF
    h = ((h ^ (h >> 13)) * 0xC2B2AE35) & 0xFFFFFFFF
    return h ^ (h >> 16)


def _random16(s, index, n):
    """Two 16-bit numbers for each of tensor ``index``'s n elements, from the
    seed, the step and the element's place."""
    key = _mix((_mix((s["seed"] + _STEP * 0x9E3779B9) & 0xFFFFFFFF) + index) & 0xFFFFFFFF)
    i = torch.arange(n, device="cuda")
    block = _mix((torch.arange(-(-n // _BLOCK), device="cuda") + key) & 0xFFFFFFFF)
    h = _mix((block.repeat_interleave(_BLOCK)[:n] + (i % _BLOCK) * 0x9E3779B9) & 0xFFFFFFFF)
    return h & 0xFFFF, h >> 16


def _in_blocks(x):
    n = x.numel()
    return torch.nn.functional.pad(x, (0, -n % _BLOCK)).view(-1, _BLOCK)


def _encode(x, bits, floor):
    """(codes, scale of each block): |x| over the block's scale rounded to a
    neighbouring e4m3 value, up with the probability of the rest; ``floor``:
    positive values do not become 0."""
    n = x.numel()
    most = _in_blocks(x.abs()).amax(1)
    scale = torch.where(most < 2.0 ** -100, 0.0, most * (1.0 / 448.0))
    inv = torch.where(scale > 0, 1.0 / scale, 0.0)
    y = torch.clamp(x.abs() * inv.repeat_interleave(_BLOCK)[:n], max=448.0)
    exponent = (y.view(torch.int32) >> 23).clamp_(min=121)      # biased; codes below 2^-6 are 2^-9 apart
    t = torch.floor(y * ((257 - exponent) << 23).view(torch.float32) + bits.float() * 2.0 ** -16)
    q = torch.clamp(t * ((exponent - 3) << 23).view(torch.float32), max=448.0)
    if floor:
        q = torch.where((y > 0) & (q == 0), 2.0 ** -9, q)
    return torch.copysign(q, x), scale


def _decode(codes, scale):
    return codes.float() * scale.repeat_interleave(_BLOCK)[:codes.numel()]


def _adamw_factors():
    """(1 - lr wd, lr / (1 - b1^t), 1 / sqrt(1 - b2^t)), in 64 bits"""
    return 1.0 - _LR * _DECAY, _LR / (1.0 - _BETA1 ** _STEP), 1.0 / math.sqrt(1.0 - _BETA2 ** _STEP)


def _adamw_tensor(s, i):
    """(parameter, m, v or their codes, scales) of tensor i after a step."""
    keep, rate, root = _adamw_factors()
    p, g = s["params"][i].float(), s["grads"][i].float()
    if s["state"] == "f32":
        m, v = s["ms"][i], s["vs"][i]
    else:
        m = _decode(s["ms"][i], s["scales"][i][:, 0])
        v = _decode(s["vs"][i], s["scales"][i][:, 1]).square()
    m = m * _BETA1 + g * (1.0 - _BETA1)
    v = v * _BETA2 + (g * g) * (1.0 - _BETA2)
    r = torch.sqrt(v)
    p = p * keep - (m * rate) / (r * root + _EPS)
    if s["state"] == "f32":
        return p, m, v, None
    low, high = _random16(s, i, p.numel())
    m, ms = _encode(m, low, False)
    v, vs = _encode(r, high, True)
    return p, m, v, torch.stack([ms, vs], 1)


def _plain_adamw(s):
    for i in range(len(s["params"])):
        p, m, v, scale = _adamw_tensor(s, i)
        s["params"][i].copy_(p)
        s["ms"][i].copy_(m)
        s["vs"][i].copy_(v)
        if scale is not None:
            s["scales"][i].copy_(scale)
        if s["copies"] is not None:
            s["copies"][i].copy_(p)
    return _adamw_outputs(s)


def _adamw_outputs(s):
    return {n: s[n + "_flat"] for n in ("param", "m", "v", "scale", "copy") if s[n + "_flat"] is not None}


# ---------------------------------------------------------------------------
# the framework's operators

def _own(s):
    import recsys_table_embedding_gb300 as tbe
    op = s["op"]
    if op.startswith("experts"):
        route = tbe.Route(s["route"], s["T"], s["K"], s["E"]) if s["K"] else None
        step = op == "experts_step"
        hidden, gate_up = tbe.tbe_expert_gated_forward(s["rows"], s["w_in"], route, activation=s["act"], keep=step)
        r = dict(hidden=hidden, out=tbe.tbe_expert_forward(s["kept"], s["w_out"], route))
        if step:
            r["gate_up"] = gate_up
            r["grad_gate_up"] = tbe.tbe_expert_backward(s["grad"], s["w_out"], route, gate_up=s["gate_up"],
                                                        activation=s["act"])
            r["grad_rows"] = tbe.tbe_expert_backward(s["grad_gate_up"], s["w_in"], route)
            kind = _TYPES[s["grad_type"]]
            r["grad_w_in"] = tbe.tbe_expert_weight_backward(s["grad_gate_up"], s["rows"], route, dtype=kind)
            r["grad_w_out"] = tbe.tbe_expert_weight_backward(s["grad"], s["kept"], route, dtype=kind)
            if route is None:       # one matrix each
                r["grad_w_in"], r["grad_w_out"] = r["grad_w_in"][None], r["grad_w_out"][None]
        return r
    if op.startswith("norm"):
        out, mean, rstd = tbe.tbe_layer_norm_forward(s["x"], s["weight"], s["bias"], eps=1e-5)
        r = dict(out=out, mean=mean, rstd=rstd)
        if op == "norm_step":
            r["grad_x"], r["grad_weight"], r["grad_bias"] = tbe.tbe_layer_norm_backward(
                s["grad"], s["x"], mean, rstd, s["weight"])
        return r
    tbe.tbe_adamw_step(s["params"], s["grads"], s["ms"], s["vs"], _STEP, lr=_LR, beta1=_BETA1, beta2=_BETA2, eps=_EPS,
                       weight_decay=_DECAY, scales=s["scales"] if s["state"] == "f8" else None, copies=s["copies"],
                       seed=s["seed"])
    return _adamw_outputs(s)


def run(state):
    if own:
        return _own(state)
    op = state["op"]
    if op.startswith("experts"):
        return _plain_experts(state)
    if op.startswith("norm"):
        return _plain_norm(state)
    return _plain_adamw(state)


# ---------------------------------------------------------------------------
# what a pass cannot do without

def work(case):
    op = case["op"]
    if op.startswith("experts"):
        T, K, E, H, F = (case[k] for k in ("T", "K", "E", "H", "F"))
        b, P = _BYTES[case["type"]], T * max(K, 1)
        M = P * (1 - case["drop"])
        used = E * -math.expm1(M * math.log1p(-1 / E)) if E > 1 else 1      # experts that have rows
        used = min(E, max(used, K * (1 - case["drop"])))
        n = (M * (H + F) + P * (F + H) + used * 3 * F * H) * b              # rows, kept; hidden, out; weights
        f = 6 * M * H * F
        if op == "experts_step":
            g = _BYTES[case["grad_type"]]
            n += P * 2 * F * b                                              # gate_up
            n += (M * (H + 4 * F) + P * (2 * F + H)) * b + E * 3 * F * H * g
            f += 12 * M * H * F
        return {"bytes": n, "flops": f}
    if op.startswith("norm"):
        N, D, b, w = case["N"], case["D"], _BYTES[case["type"]], _BYTES[case["weight"]]
        n, f = 2 * N * D * b + 2 * D * w + 8 * N, 8 * N * D
        if op == "norm_step":
            n += 2 * N * D * b + 2 * D * w
            f += 14 * N * D
        return {"bytes": n, "flops": f}
    total = sum(_sizes(case))
    each = 2 * _BYTES[case["param"]] + _BYTES[case["grad"]] + (_BYTES[case["copy"]] if case["copy"] else 0)
    each += 16 if case["state"] == "f32" else 4 + 16 / _BLOCK
    return {"bytes": total * each, "flops": 16 * total}


# ---------------------------------------------------------------------------
# the definitions in 64 bits

def _exact_experts(s):
    E, F, H, act = s["E"], s["F"], s["H"], s["act"]
    P = s["rows"].shape[0]
    step = s["op"] == "experts_step"
    new = lambda *shape: torch.zeros(shape, dtype=torch.float64, device="cuda")  # noqa: E731
    r = dict(hidden=new(P, F), out=new(P, H))
    if step:
        r |= dict(gate_up=new(P, 2 * F), grad_gate_up=new(P, 2 * F), grad_rows=new(P, H),
                  grad_w_in=new(E, 2 * F, H), grad_w_out=new(E, H, F))
    for e in range(E):
        at = slice(s["bounds"][e], s["bounds"][e + 1])
        if at.start == at.stop:
            continue
        x, kept = s["rows"][at].double(), s["kept"][at].double()
        w_in, w_out = s["w_in"][e].double(), s["w_out"][e].double()
        gate, up = torch.einsum("sh,cfh->csf", x, w_in.view(2, F, H)).unbind(0)
        value = gate * torch.sigmoid(gate) if act == "silu" else gate * torch.special.ndtr(gate)
        r["hidden"][at] = value * up
        r["out"][at] = torch.einsum("sf,hf->sh", kept, w_out)
        if not step:
            continue
        r["gate_up"][at, :F], r["gate_up"][at, F:] = gate, up
        dy, dz = s["grad"][at].double(), s["grad_gate_up"][at].double()
        dh = torch.einsum("sh,hf->sf", dy, w_out)
        g, u = s["gate_up"][at].double().split(F, 1)
        if act == "silu":
            value, slope = g * torch.sigmoid(g), torch.sigmoid(g) + g * torch.sigmoid(g) * torch.sigmoid(-g)
        else:
            value = g * torch.special.ndtr(g)
            slope = torch.special.ndtr(g) + g * torch.exp(-g * g / 2) / math.sqrt(2 * math.pi)
        r["grad_gate_up"][at, :F], r["grad_gate_up"][at, F:] = dh * u * slope, dh * value
        r["grad_rows"][at] = torch.einsum("sf,fh->sh", dz, w_in)
        r["grad_w_in"][e] = torch.einsum("sf,sh->fh", dz, x)
        r["grad_w_out"][e] = torch.einsum("sh,sf->hf", dy, kept)
    return r


def _exact_norm(s):
    N, D = s["x"].shape
    step = s["op"] == "norm_step"
    w, b = s["weight"].double(), s["bias"].double()
    new = lambda *shape: torch.zeros(shape, dtype=torch.float64, device="cuda")  # noqa: E731
    r = dict(out=new(N, D), mean=new(N), rstd=new(N))
    if step:
        r |= dict(grad_x=new(N, D), grad_weight=new(D), grad_bias=new(D))
    rows = max(1, 67_108_864 // D)
    for a in range(0, N, rows):
        at = slice(a, min(N, a + rows))
        x = s["x"][at].double()
        var, mean = torch.var_mean(x, 1, correction=0)
        rstd = (var + 1e-5).rsqrt()
        xh = torch.einsum("nd,n->nd", x - mean[:, None], rstd)
        r["mean"][at], r["rstd"][at], r["out"][at] = mean, rstd, torch.addcmul(b, xh, w)
        if step:
            dy = s["grad"][at].double()
            d = dy * w
            along = torch.einsum("nd,nd->n", d, xh) / D
            r["grad_x"][at] = (d - d.sum(1, keepdim=True) / D - along[:, None] * xh) * rstd[:, None]
            r["grad_weight"] += torch.einsum("nd,nd->d", dy, xh)
            r["grad_bias"] += torch.einsum("nd->d", dy)
    return r


def _exact_adamw(s):
    f8 = s["state"] == "f8"
    r = {n: s[n + "_flat"].double() for n in ("param", "m", "v", "scale", "copy") if s[n + "_flat"] is not None}
    blocks, starts = _blocks(s)[0], _places(s)[0]
    for i, (n, a) in enumerate(zip(_sizes(s), starts)):
        at = slice(a, a + n)
        own_blocks = torch.arange(n, device="cuda") // _BLOCK + blocks[i]
        p, g = s["param_flat"][at].double(), s["grad_flat"][at].double()
        m, v = s["m_flat"][at].double(), s["v_flat"][at].double()
        if f8:
            m, v = m * s["scale_flat"][own_blocks, 0].double(), (v * s["scale_flat"][own_blocks, 1].double()) ** 2
        m, v = torch.lerp(m, g, 1.0 - _BETA1), torch.lerp(v, g * g, 1.0 - _BETA2)
        m_hat, v_hat = m / (1.0 - _BETA1 ** _STEP), v / (1.0 - _BETA2 ** _STEP)
        p = p - _LR * (m_hat / (v_hat.sqrt() + _EPS) + _DECAY * p)
        r["param"][at] = p
        if s["copy"]:
            r["copy"][at] = p
        if not f8:
            r["m"][at], r["v"][at] = m, v
            continue
        bits = _random16(s, i, n)
        for k, (name, x) in enumerate((("m", m), ("v", v.sqrt()))):
            top = torch.zeros(-(-n // _BLOCK), dtype=torch.float64, device="cuda")
            top.scatter_reduce_(0, torch.arange(n, device="cuda") // _BLOCK, x.abs(), "amax")
            r["scale"][blocks[i]:blocks[i] + len(top), k] = top / 448
            y = x.abs() / r["scale"][own_blocks, k]
            step = torch.exp2(torch.clamp(torch.floor(torch.log2(torch.clamp(y, min=2.0 ** -20))), min=-6) - 3)
            q = torch.clamp((y / step + bits[k] / 65536.0).floor() * step, max=448)
            r[name][at] = torch.sign(x) * (q if k == 0 else torch.clamp(q, min=2.0 ** -9))
    return r


def exact(case, seed):
    s = prepare(case, seed)
    if s["op"].startswith("experts"):
        return _exact_experts(s)
    if s["op"].startswith("norm"):
        return _exact_norm(s)
    return _exact_adamw(s)
