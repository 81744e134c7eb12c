"""Binding of the layer operators of the C ABI (include/tbe.h): the experts'
products, layer norm and the AdamW step, each with its gradients.

Argument marshalling only, in the manner of ``tokens.py``: the functions keep
the C names; results and workspaces are allocated by torch unless the caller
passes them, on the tensors' device; what a call writes shares no memory with
what else it reads or writes (it is refused otherwise); everything is enqueued on ``stream``
(default: the device's current stream); tensors that require a gradient are
taken under torch.no_grad() only, and what a call writes into the caller's
tensors counts as a change of them.  ``status`` (int32[4], optional) receives
FLAG_MMA_TIMEOUT in its second word where a wait of the products gave up, whose
results are then NaN.
"""
from __future__ import annotations

import ctypes
from typing import Optional, Sequence, Union

import torch

from .tbe import _TORCH_DTYPE, P, i32, i64, lib, tbe_config
from .tokens import Route, _device_of, _f32_rows, _matrix, _On, _refuse, _status, tbe_matrix, tbe_route

f32, f64, size_t = ctypes.c_float, ctypes.c_double, ctypes.c_size_t
ACTIVATIONS = {"silu": 0, "gelu": 1}
STATE_BLOCK = 256       # elements that share a scale in 8-bit states

LAYER_EXPORTED = ("tbe_expert_gated_forward", "tbe_expert_forward", "tbe_expert_backward",
                  "tbe_expert_workspace_bytes", "tbe_expert_weight_backward", "tbe_layer_norm_forward",
                  "tbe_layer_norm_workspace_bytes", "tbe_layer_norm_backward", "tbe_adamw_workspace_bytes",
                  "tbe_adamw_step")


class tbe_experts(ctypes.Structure):
    _fields_ = [("data", P), ("experts", i64), ("rows", i64), ("cols", i64), ("expert_stride", i64),
                ("stride", i64), ("dtype", i32)]


class tbe_adamw_tensor(ctypes.Structure):
    _fields_ = [("param", P), ("grad", P), ("m", P), ("v", P), ("scales", P), ("copy", P), ("n", i64),
                ("param_dtype", i32), ("grad_dtype", i32), ("copy_dtype", i32), ("state", i32)]


class tbe_adamw_options(ctypes.Structure):
    _fields_ = [("lr", f64), ("beta1", f64), ("beta2", f64), ("eps", f64), ("weight_decay", f64), ("step", i64),
                ("step_device", P), ("lr_device", P), ("grad_scale", P), ("seed", ctypes.c_uint32)]


_M, _R, _E, _C = (ctypes.POINTER(tbe_matrix), ctypes.POINTER(tbe_route), ctypes.POINTER(tbe_experts),
                  ctypes.POINTER(tbe_config))
_ARGS = {
    "tbe_expert_gated_forward": [_R, _M, _E, i32, _M, _M, P, _C, P],
    "tbe_expert_forward": [_R, _M, _E, _M, P, _C, P],
    "tbe_expert_backward": [_R, _M, _E, _M, i32, _M, P, _C, P],
    "tbe_expert_workspace_bytes": [i64, i64, i64, i64],
    "tbe_expert_weight_backward": [_R, _M, _M, _E, i32, P, size_t, P, _C, P],
    "tbe_layer_norm_forward": [_M, P, P, i32, f32, _M, P, P, _C, P],
    "tbe_layer_norm_workspace_bytes": [i64, i64],
    "tbe_layer_norm_backward": [_M, _M, P, i32, P, P, _M, P, P, i32, P, size_t, _C, P],
    "tbe_adamw_workspace_bytes": [],
    "tbe_adamw_step": [P, i64, ctypes.POINTER(tbe_adamw_options), P, size_t, _C, P],
}
_bound = None


def _lib():
    """The library with the layer operators' argument types set."""
    global _bound
    if _bound is None:
        L = lib()
        for name, args in _ARGS.items():
            fn = getattr(L, name)
            fn.argtypes = args
            fn.restype = size_t if name.endswith("_bytes") else i32
        _bound = L
    return _bound


# ---------------------------------------------------------------------------
# the experts' products

def _experts(t: torch.Tensor, name: str, route: Optional[Route]) -> tbe_experts:
    """A tensor [experts, rows, cols] ([rows, cols] without a route) as experts, without a copy."""
    dt = _TORCH_DTYPE.get(t.dtype)
    if dt is None:
        _refuse(f"{name} is float32, float16 or bfloat16: got {t.dtype}")
    shape, strides = tuple(t.shape), t.stride()
    if len(shape) == 2 and route is None:
        shape, strides = (1, *shape), (0, *strides)
    if len(shape) != 3:
        _refuse(f"{name} is [experts, rows, columns]: got shape {tuple(t.shape)}")
    E, rows, cols = shape
    if strides[2] != 1 and cols > 1:
        _refuse(f"{name}'s columns are not contiguous")
    return tbe_experts(t.data_ptr() or None, E, rows, cols, strides[0] if E > 1 else 0,
                       strides[1] if rows > 1 else cols, dt)


def _route(route: Optional[Route], rows: int, experts: int):
    if route is None:
        if experts != 1:
            _refuse(f"without a route there is one group: got {experts} experts")
        return None
    if route.tokens * route.K != rows or route.experts != experts:
        _refuse(f"route is of {route.tokens * route.K} rows and {route.experts} experts: got {rows} rows and "
                f"{experts} experts")
    return route.c


def _activation(name: str) -> int:
    kind = ACTIVATIONS.get(name)
    if kind is None:
        _refuse(f"activation is one of {', '.join(ACTIVATIONS)}: got {name!r}")
    return kind


def _cols(got: int, want: int, what: str):
    if got != want:
        _refuse(f"{what}: got {got} for {want}")


def tbe_expert_gated_forward(rows: torch.Tensor, weight: torch.Tensor, route: Optional[Route] = None,
                             activation: str = "silu", keep: bool = False, hidden: Optional[torch.Tensor] = None,
                             gate_up: Optional[torch.Tensor] = None, status: Optional[torch.Tensor] = None,
                             cfg: Optional[tbe_config] = None, stream=None):
    """(hidden [P, F], gate_up [P, 2F] or None): act(gate) * up with [gate | up]
    = rows @ weight[e].T, for rows [P, H] sorted by expert (``route``; None: one
    group, weight [2F, H] or [1, 2F, H]) and weight [E, 2F, H].  ``keep`` or a
    ``gate_up`` to write into: gate_up is kept for the backward pass."""
    L = _lib()
    on = _On(_device_of(rows, weight, hidden, gate_up, status, route and route.buffer), stream)
    kind, mx, we = _activation(activation), _matrix(rows, "rows"), _experts(weight, "weight", route)
    r = _route(route, mx.rows, we.experts)
    _cols(mx.cols, we.cols, "rows' and weight's columns")
    if we.rows % 2:
        _refuse(f"weight's rows are the gate's and as many others: got {we.rows}")
    lead = rows.shape[:-1]
    hidden, mh = on.result(hidden, (*lead, we.rows // 2), mx.rows, we.rows // 2, rows.dtype, "hidden")
    mg = None
    if keep or gate_up is not None:
        gate_up, mg = on.result(gate_up, (*lead, we.rows), mx.rows, we.rows, rows.dtype, "gate_up")
    on.call(L.tbe_expert_gated_forward, r, mx, we, kind, mh, mg, _status(status), cfg)
    return hidden, gate_up


def tbe_expert_forward(rows: torch.Tensor, weight: torch.Tensor, route: Optional[Route] = None,
                       out: Optional[torch.Tensor] = None, status: Optional[torch.Tensor] = None,
                       cfg: Optional[tbe_config] = None, stream=None) -> torch.Tensor:
    """rows @ weight[e].T: [P, N] for rows [P, K] sorted by expert and weight
    [E, N, K] (no route: one group, weight [N, K] or [1, N, K])."""
    L = _lib()
    on = _On(_device_of(rows, weight, out, status, route and route.buffer), stream)
    mx, we = _matrix(rows, "rows"), _experts(weight, "weight", route)
    r = _route(route, mx.rows, we.experts)
    _cols(mx.cols, we.cols, "rows' and weight's columns")
    out, mo = on.result(out, (*rows.shape[:-1], we.rows), mx.rows, we.rows, rows.dtype, "out")
    on.call(L.tbe_expert_forward, r, mx, we, mo, _status(status), cfg)
    return out


def tbe_expert_backward(grad_out: torch.Tensor, weight: torch.Tensor, route: Optional[Route] = None,
                        gate_up: Optional[torch.Tensor] = None, activation: str = "silu",
                        grad_rows: Optional[torch.Tensor] = None, status: Optional[torch.Tensor] = None,
                        cfg: Optional[tbe_config] = None, stream=None) -> torch.Tensor:
    """Gradient of tbe_expert_forward's rows, grad_out @ weight[e]: [P, K].  With
    ``gate_up`` [P, 2K] those rows were tbe_expert_gated_forward's hidden, and
    the gradient is that of gate_up: [P, 2K]."""
    L = _lib()
    on = _On(_device_of(grad_out, weight, gate_up, grad_rows, status, route and route.buffer), stream)
    kind, md, we = _activation(activation), _matrix(grad_out, "grad_out"), _experts(weight, "weight", route)
    r = _route(route, md.rows, we.experts)
    _cols(md.cols, we.rows, "grad_out's columns and weight's rows")
    cols, mg = we.cols, None
    if gate_up is not None:
        cols, mg = 2 * we.cols, _matrix(gate_up, "gate_up")
        if (mg.rows, mg.cols) != (md.rows, cols):
            _refuse(f"gate_up is [{md.rows}, {cols}]: got {tuple(gate_up.shape)}")
    grad_rows, mr = on.result(grad_rows, (*grad_out.shape[:-1], cols), md.rows, cols, grad_out.dtype, "grad_rows")
    on.call(L.tbe_expert_backward, r, md, we, mg, kind, mr, _status(status), cfg)
    return grad_rows


def tbe_expert_weight_backward(grad_out: torch.Tensor, rows: torch.Tensor, route: Optional[Route] = None,
                               grad_weight: Optional[torch.Tensor] = None, dtype: Optional[torch.dtype] = None,
                               accumulate: bool = False, workspace: Optional[torch.Tensor] = None,
                               status: Optional[torch.Tensor] = None, cfg: Optional[tbe_config] = None,
                               stream=None) -> torch.Tensor:
    """Gradient of the weights, grad_out[s].T @ rows[s] summed over the rows of
    each expert: [E, N, K] ([N, K] without a route) of the rows' dtype or float32
    (``dtype``).  With ``accumulate`` it is added to ``grad_weight``."""
    L = _lib()
    on = _On(_device_of(grad_out, rows, grad_weight, workspace, status, route and route.buffer), stream)
    md, mx = _matrix(grad_out, "grad_out"), _matrix(rows, "rows")
    _cols(mx.rows, md.rows, "rows and rows of grad_out")
    if accumulate and grad_weight is None:
        _refuse("accumulate adds to a given grad_weight")
    E = route.experts if route is not None else 1
    r = _route(route, mx.rows, E)
    if grad_weight is None:
        grad_weight = on.empty((E, md.cols, mx.cols) if route is not None else (md.cols, mx.cols), dtype or rows.dtype)
    else:
        shape = (E, md.cols, mx.cols)
        if tuple(grad_weight.shape) not in ((shape,) if route is not None else (shape, shape[1:])) or \
                dtype not in (None, grad_weight.dtype):
            _refuse(f"grad_weight is {dtype or 'a tensor'} of shape {shape}: got {grad_weight.dtype} of "
                    f"{tuple(grad_weight.shape)}")
        on.changes(grad_weight)
    wg = _experts(grad_weight, "grad_weight", route)
    ws, n, _keep = on.workspace(workspace, L.tbe_expert_workspace_bytes(mx.rows, E, md.cols, mx.cols))
    on.call(L.tbe_expert_weight_backward, r, md, mx, wg, int(accumulate), ws, n, _status(status), cfg)
    return grad_weight


# ---------------------------------------------------------------------------
# layer norm

def _param(t: Optional[torch.Tensor], name: str, cols: int):
    """(pointer, type) of a vector of one value per column, or (None, None)."""
    if t is None:
        return None, None
    dt = _TORCH_DTYPE.get(t.dtype)
    if dt is None:
        _refuse(f"{name} is float32, float16 or bfloat16: got {t.dtype}")
    if tuple(t.shape) != (cols,) or not t.is_contiguous():
        _refuse(f"{name} is contiguous with one value per column ({cols}): got {tuple(t.shape)}")
    return t.data_ptr(), dt


def _one_type(a, b, names: str) -> int:
    if a is not None and b is not None and a != b:
        _refuse(f"{names} have one dtype")
    return a if a is not None else b if b is not None else 0


def tbe_layer_norm_forward(x: torch.Tensor, weight: Optional[torch.Tensor] = None,
                           bias: Optional[torch.Tensor] = None, eps: float = 1e-5, out: Optional[torch.Tensor] = None,
                           mean: Optional[torch.Tensor] = None, rstd: Optional[torch.Tensor] = None,
                           cfg: Optional[tbe_config] = None, stream=None):
    """(out, mean, rstd): the rows of x [..., D] less their mean, over their
    deviation, times weight plus bias [D]; mean and rstd are float32 of
    x.shape[:-1], for the backward pass."""
    L = _lib()
    on = _On(_device_of(x, weight, bias, out, mean, rstd), stream)
    mx = _matrix(x, "x")
    (pw, tw), (pb, tb) = _param(weight, "weight", mx.cols), _param(bias, "bias", mx.cols)
    dt = _one_type(tw, tb, "weight and bias")
    out, mo = on.result(out, x.shape, mx.rows, mx.cols, x.dtype, "out")
    on.changes(mean, rstd)
    mean = on.empty(x.shape[:-1], torch.float32) if mean is None else mean
    rstd = on.empty(x.shape[:-1], torch.float32) if rstd is None else rstd
    on.call(L.tbe_layer_norm_forward, mx, pw, pb, dt, eps, mo, _f32_rows(mean, "mean", mx.rows),
            _f32_rows(rstd, "rstd", mx.rows), cfg)
    return out, mean, rstd


def tbe_layer_norm_backward(grad_out: torch.Tensor, x: torch.Tensor, mean: torch.Tensor, rstd: torch.Tensor,
                            weight: Optional[torch.Tensor] = None, grad_x: Optional[torch.Tensor] = None,
                            grad_weight: Optional[torch.Tensor] = None, grad_bias: Optional[torch.Tensor] = None,
                            dtype: Optional[torch.dtype] = None, workspace: Optional[torch.Tensor] = None,
                            cfg: Optional[tbe_config] = None, stream=None):
    """(grad_x, grad_weight, grad_bias) of tbe_layer_norm_forward, from its mean
    and rstd.  grad_weight and grad_bias [D] have the weight's dtype, ``dtype`` or
    that of the tensors given (without any of these: float32)."""
    L = _lib()
    on = _On(_device_of(grad_out, x, mean, rstd, weight, grad_x, grad_weight, grad_bias, workspace), stream)
    md, mx = _matrix(grad_out, "grad_out"), _matrix(x, "x")
    if tuple(grad_out.shape) != tuple(x.shape):
        _refuse(f"grad_out has the shape of x: got {tuple(grad_out.shape)} for {tuple(x.shape)}")
    pw, tw = _param(weight, "weight", mx.cols)
    pm, pr = _f32_rows(mean, "mean", mx.rows), _f32_rows(rstd, "rstd", mx.rows)
    grad_x, mo = on.result(grad_x, x.shape, mx.rows, mx.cols, x.dtype, "grad_x")
    kind = dtype or (grad_weight.dtype if grad_weight is not None else grad_bias.dtype if grad_bias is not None else
                     weight.dtype if weight is not None else torch.float32)
    on.changes(grad_weight, grad_bias)
    grad_weight = on.empty((mx.cols,), kind) if grad_weight is None else grad_weight
    grad_bias = on.empty((mx.cols,), kind) if grad_bias is None else grad_bias
    (pgw, tgw), (pgb, tgb) = _param(grad_weight, "grad_weight", mx.cols), _param(grad_bias, "grad_bias", mx.cols)
    dt = _one_type(tgw, tgb, "grad_weight and grad_bias")
    if dt != _TORCH_DTYPE.get(kind):
        _refuse(f"grad_weight and grad_bias are {kind}")
    ws, n, _keep = on.workspace(workspace, L.tbe_layer_norm_workspace_bytes(mx.rows, mx.cols))
    on.call(L.tbe_layer_norm_backward, md, mx, pw, tw or 0, pm, pr, mo, pgw, pgb, dt, ws, n, cfg)
    return grad_x, grad_weight, grad_bias


# ---------------------------------------------------------------------------
# AdamW

_CODES = torch.float8_e4m3fn
_COPY_TYPE = {torch.float16: 1, torch.bfloat16: 2}


def tbe_adamw_step(params: Sequence[torch.Tensor], grads: Sequence[Optional[torch.Tensor]],
                   exp_avgs: Sequence[torch.Tensor], exp_avg_sqs: Sequence[torch.Tensor],
                   step: Union[int, torch.Tensor], lr: Union[float, torch.Tensor] = 1e-3, beta1: float = 0.9,
                   beta2: float = 0.999, eps: float = 1e-8, weight_decay: float = 0.01,
                   scales: Optional[Sequence[Optional[torch.Tensor]]] = None,
                   copies: Optional[Sequence[Optional[torch.Tensor]]] = None,
                   grad_scale: Optional[torch.Tensor] = None, seed: int = 0,
                   workspace: Optional[torch.Tensor] = None, cfg: Optional[tbe_config] = None, stream=None) -> None:
    """One AdamW step of every tensor of the lists, in place: params, exp_avgs
    (m), exp_avg_sqs (v), scales and copies change.

    All tensors are contiguous.  States are float32, or float8_e4m3fn codes (of m,
    and of v's square root) with ``scales`` [ceil(n / 256), 2] in float32.
    ``copies`` receive the new parameters in 16 bits.  A tensor whose gradient is
    None is left out (it keeps its place in the lists, which the random numbers of
    8-bit states go by).  ``step`` (1 for the first) is a number or an int64
    tensor on the device, ``lr`` a number or a float32 tensor there, for steps
    captured into a graph; ``grad_scale`` (float32, on the device) multiplies the
    gradients.  The random numbers are a hash of (``seed``, step, place in the
    lists, place in the tensor): groups of parameters that are stepped by calls of
    their own take another seed each."""
    L = _lib()
    count = len(params)
    for name, them in (("grads", grads), ("exp_avgs", exp_avgs), ("exp_avg_sqs", exp_avg_sqs), ("scales", scales),
                       ("copies", copies)):
        if them is not None and len(them) != count:
            _refuse(f"{name} has one entry for each of {count} params: got {len(them)}")
    some = next((i for i, g in enumerate(grads) if g is not None), None)
    if some is None:
        return
    dev_step = step if isinstance(step, torch.Tensor) else None
    dev_lr = lr if isinstance(lr, torch.Tensor) else None
    dev = _device_of(params[some], dev_step, dev_lr, grad_scale, workspace)
    for name, t, dt in (("step", dev_step, torch.int64), ("lr", dev_lr, torch.float32),
                        ("grad_scale", grad_scale, torch.float32)):
        if t is not None and (t.dtype != dt or t.numel() != 1):
            _refuse(f"{name} on the device is one {dt}")
    if dev_step is None and not 1 <= int(step) < 1 << 63:
        _refuse(f"step counts from 1: got {step}")
    follow = torch.is_grad_enabled()
    words, changed = [], []
    kinds, f32_type = _TORCH_DTYPE, torch.float32
    no = (None,) * count
    for p, g, m, v, s, c in zip(params, grads, exp_avgs, exp_avg_sqs, scales or no, copies or no):
        if g is None:
            words += (0,) * 9
            continue
        shape, n, st = p.shape, p.numel(), m.dtype
        pt, gt = kinds.get(p.dtype), kinds.get(g.dtype)
        if pt is None or gt is None:
            _refuse(f"params and grads are float32, float16 or bfloat16: got {p.dtype} and {g.dtype}")
        if (st is not f32_type and st is not _CODES) or v.dtype is not st:
            _refuse(f"states are float32 or float8_e4m3fn, both of one type: got {st} and {v.dtype}")
        if g.shape != shape or m.shape != shape or v.shape != shape:
            _refuse(f"gradient and states have their param's shape: got {tuple(g.shape)}, {tuple(m.shape)} and "
                    f"{tuple(v.shape)} for {tuple(shape)}")
        if not (p.is_contiguous() and g.is_contiguous() and m.is_contiguous() and v.is_contiguous()):
            _refuse("params, grads and states are contiguous")
        if not p.get_device() == g.get_device() == m.get_device() == v.get_device() == dev:
            _refuse("the tensors of a call lie on one device")
        if follow and (p.requires_grad or g.requires_grad or m.requires_grad or v.requires_grad or
                       (c is not None and c.requires_grad)):
            _refuse("a tensor of the call requires a gradient, which autograd does not follow through the step: call "
                    "it under torch.no_grad()")
        changed += (p, m, v)
        ps = pc = ct = 0
        if st is _CODES:
            if s is None or s.dtype is not f32_type or s.numel() != 2 * -(-n // STATE_BLOCK) or \
                    not s.is_contiguous() or s.get_device() != dev:
                _refuse(f"8-bit states have scales: contiguous float32 [{-(-n // STATE_BLOCK)}, 2] on their device")
            ps = s.data_ptr()
            changed.append(s)
        if c is not None:
            ct = _COPY_TYPE.get(c.dtype)
            if ct is None or c.shape != shape or not c.is_contiguous() or c.get_device() != dev:
                _refuse("copies are contiguous float16 or bfloat16 tensors of their param's shape, on its device")
            pc = c.data_ptr()
            changed.append(c)
        words += (p.data_ptr(), g.data_ptr(), m.data_ptr(), v.data_ptr(), ps, pc, n, pt | gt << 32,
                  ct | (1 << 32 if st is _CODES else 0))
    on = _On(dev, stream)
    on.changes(*changed)
    table = (ctypes.c_uint64 * len(words))(*words)
    options = tbe_adamw_options(0.0 if dev_lr is not None else float(lr), beta1, beta2, eps, weight_decay,
                                1 if dev_step is not None else int(step),
                                dev_step.data_ptr() if dev_step is not None else None,
                                dev_lr.data_ptr() if dev_lr is not None else None,
                                grad_scale.data_ptr() if grad_scale is not None else None, seed & 0xffffffff)
    ws, nbytes, _keep = on.workspace(workspace, 0 if dev_step is None and dev_lr is None else
                                     L.tbe_adamw_workspace_bytes())
    on.call(L.tbe_adamw_step, ctypes.addressof(table), count, options, ws, nbytes, cfg)
