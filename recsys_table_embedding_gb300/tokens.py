"""Binding of the token operators of the C ABI (include/tbe.h): the token
embedding and its gradient, tokens sorted by expert and back, and the
distillation loss, each with its gradients.

Argument marshalling only, as in ``tbe.py``: the functions keep the C names.
Results and workspaces are allocated by torch unless the caller passes them
(``out`` arguments), on the tensors' device; everything is enqueued on
``stream`` (default: the device's current stream).  What a call allocates for
a stream other than the current one is recorded on that stream, so torch does
not hand the memory out while the call uses it; tensors that the caller passes
are the caller's to keep until the stream is done with them.

The functions are not recorded by autograd: each operator's gradient is a
function of its own, and a tensor that requires a gradient is refused unless
torch.no_grad() is on.

What a call writes into the caller's tensors counts as a change of them.

Matrices have contiguous columns and any row stride; leading dimensions are
flattened.  ``status`` (int32[4], optional) collects the C status words.
"""
from __future__ import annotations

import ctypes
from typing import Optional

import torch

from .tbe import _TORCH_DTYPE, P, TbeError, _check, i32, i64, lib, tbe_config

f32, size_t = ctypes.c_float, ctypes.c_size_t
_INDEX_TYPE = {torch.int32: 0, torch.int64: 1}

TOKEN_EXPORTED = ("tbe_token_forward", "tbe_token_workspace_bytes", "tbe_token_backward",
                  "tbe_route_workspace_bytes", "tbe_route_sort", "tbe_route_dispatch",
                  "tbe_route_sort_dispatch", "tbe_route_dispatch_backward", "tbe_route_combine",
                  "tbe_route_combine_backward", "tbe_distill_workspace_bytes", "tbe_distill_forward",
                  "tbe_distill_backward", "tbe_distill_loss_grad")


class tbe_matrix(ctypes.Structure):
    _fields_ = [("data", P), ("rows", i64), ("cols", i64), ("stride", i64), ("dtype", i32)]


class tbe_route(ctypes.Structure):
    _fields_ = [("tokens", i64), ("K", i32), ("experts", i32), ("slot", P), ("source", P), ("offset", P)]


class tbe_teacher(ctypes.Structure):
    _fields_ = [("ids", P), ("logits", P), ("index_type", i32), ("dtype", i32), ("K", i32),
                ("temperature", f32)]


_M, _R, _T, _C = (ctypes.POINTER(tbe_matrix), ctypes.POINTER(tbe_route), ctypes.POINTER(tbe_teacher),
                  ctypes.POINTER(tbe_config))
_ARGS = {
    "tbe_token_forward": [_M, P, i32, f32, _M, P, _C, P],
    "tbe_token_workspace_bytes": [i64, i64, i64],
    "tbe_token_backward": [_M, P, i32, i64, f32, _M, i32, P, size_t, P, _C, P],
    "tbe_route_workspace_bytes": [i64, i32, i32],
    "tbe_route_sort": [_R, P, i32, P, size_t, _C, P],
    "tbe_route_dispatch": [_R, _M, _M, _C, P],
    "tbe_route_sort_dispatch": [_R, P, i32, _M, _M, P, size_t, _C, P],
    "tbe_route_dispatch_backward": [_R, _M, _M, _C, P],
    "tbe_route_combine": [_R, _M, P, i32, _M, _C, P],
    "tbe_route_combine_backward": [_R, _M, _M, P, i32, _M, P, _C, P],
    "tbe_distill_workspace_bytes": [i64, i32],
    "tbe_distill_forward": [_M, _T, P, P, P, size_t, P, _C, P],
    "tbe_distill_backward": [_M, _T, P, P, f32, _M, P, size_t, _C, P],
    "tbe_distill_loss_grad": [_M, _T, P, f32, P, P, _M, P, size_t, P, _C, P],
}
_bound = None


def _lib():
    """The library with the token operators' argument types set."""
    global _bound
    if _bound is None:
        L = lib()
        for name, args in _ARGS.items():
            fn = getattr(L, name)
            fn.argtypes = args
            fn.restype = size_t if name.endswith("_bytes") else i32
        _bound = L
    return _bound


# the raw handle of a device's current stream, and the current device: the
# small calls of serving are bound by the host
_current_stream = torch._C._cuda_getCurrentRawStream
_current_device = torch._C._cuda_getDevice


def _refuse(message: str):
    raise TbeError(message)


def _device_of(t: torch.Tensor, *others) -> int:
    """The one CUDA device of a call's tensors, none of which autograd follows."""
    dev = t.get_device()
    if dev < 0:
        _refuse("the token operators take CUDA tensors")
    follows = t.requires_grad
    for o in others:
        if o is not None:
            if o.get_device() != dev:
                _refuse("the tensors of a call lie on one device")
            follows = follows or o.requires_grad
    if follows and torch.is_grad_enabled():
        _refuse("a tensor of the call requires a gradient, which autograd does not follow through the token "
                "operators: detach it, or call them under torch.no_grad() and pass their gradients on")
    return dev


def _matrix(t: torch.Tensor, name: str) -> tbe_matrix:
    """A tensor [..., cols] as a matrix, without a copy."""
    dt = _TORCH_DTYPE.get(t.dtype)
    if dt is None:
        _refuse(f"{name} is float32, float16 or bfloat16: got {t.dtype}")
    shape = t.shape
    if len(shape) != 2:
        if len(shape) < 2:
            _refuse(f"{name} has rows and columns: got shape {tuple(shape)}")
        if t.numel() == 0:
            t = t.reshape(-1, shape[-1]) if shape[-1] else t.reshape(0, 0)
        else:
            try:
                t = t.view(-1, shape[-1])
            except RuntimeError:
                _refuse(f"{name}'s leading dimensions do not flatten without a copy")
        shape = t.shape
    rows, cols = shape
    stride, step = t.stride()
    if step != 1 and cols > 1 and rows > 0:
        _refuse(f"{name}'s columns are not contiguous")
    return tbe_matrix(t.data_ptr() or None, rows, cols, stride if rows > 1 else cols, dt)


def _index(t: torch.Tensor, name: str) -> int:
    it = _INDEX_TYPE.get(t.dtype)
    if it is None:
        _refuse(f"{name} are int32 or int64: got {t.dtype}")
    if not t.is_contiguous():
        _refuse(f"{name} are not contiguous")
    return it


def _float(t: torch.Tensor, name: str, shape=None) -> int:
    dt = _TORCH_DTYPE.get(t.dtype)
    if dt is None:
        _refuse(f"{name} is float32, float16 or bfloat16: got {t.dtype}")
    if not t.is_contiguous():
        _refuse(f"{name} is not contiguous")
    if shape is not None and tuple(t.shape) != tuple(shape):
        _refuse(f"{name} has shape {tuple(shape)}: got {tuple(t.shape)}")
    return dt


def _f32_rows(t: Optional[torch.Tensor], name: str, rows: int):
    """Pointer of a contiguous float32 tensor of one value per row, or None."""
    if t is None:
        return None
    if t.dtype != torch.float32 or not t.is_contiguous() or t.numel() != rows:
        _refuse(f"{name} is contiguous float32 with one value per row")
    return t.data_ptr()


def _status(status: Optional[torch.Tensor]):
    if status is None:
        return None
    if status.dtype != torch.int32 or status.numel() < 4 or not status.is_contiguous():
        _refuse("status is int32 with 4 words")
    return status.data_ptr()


class _On:
    """The stream of one call, with the device made current for it, and the
    allocations of the call."""

    __slots__ = ("index", "given", "handle", "changed")

    def __init__(self, index: int, stream):
        self.index, self.given, self.changed = index, None, None
        current = _current_stream(index)
        if stream is None:
            self.handle = current
        else:
            self.handle = stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)
            if self.handle != current:
                self.given = stream if hasattr(stream, "cuda_stream") else \
                    torch.cuda.ExternalStream(self.handle, device=index)

    def empty(self, shape, dtype) -> torch.Tensor:
        t = torch.empty(shape, dtype=dtype, device=self.index)
        if self.given is not None:
            # the memory's former uses are on the current stream, its next on `given`
            self.given.wait_stream(torch.cuda.current_stream(self.index))
            t.record_stream(self.given)
        return t

    def changes(self, *tensors: Optional[torch.Tensor]):
        """The caller's tensors (or None) that the call writes results into."""
        for t in tensors:
            if t is not None:
                if self.changed is None:
                    self.changed = []
                self.changed.append(t)

    def result(self, out: Optional[torch.Tensor], shape, rows: int, cols: int, dtype: torch.dtype, name: str):
        """(tensor, matrix) of a result of `rows` x `cols`: the caller's, checked, or a new one."""
        if out is None:
            out = self.empty(shape, dtype)
            return out, tbe_matrix(out.data_ptr() or None, rows, cols, cols, _TORCH_DTYPE[dtype])
        if tuple(out.shape) != tuple(shape) or out.dtype != dtype:
            _refuse(f"{name} is {dtype} of shape {tuple(shape)}: got {out.dtype} of {tuple(out.shape)}")
        self.changes(out)
        return out, _matrix(out if len(shape) > 1 else out.view(1, -1), name)

    def workspace(self, given: Optional[torch.Tensor], nbytes: int):
        """(pointer, bytes, tensor) of the workspace of a call."""
        if given is None:
            if nbytes == 0:
                return None, 0, None
            given = self.empty(nbytes, torch.uint8)
        return given.data_ptr(), given.numel() * given.element_size(), given

    def call(self, fn, *args):
        if _current_device() == self.index:
            status = fn(*args, self.handle)
        else:
            with torch.cuda.device(self.index):
                status = fn(*args, self.handle)
        if status != 0:
            _check(status)
        if self.changed is not None:
            # autograd, which does not see the call, learns that their values changed
            torch.autograd.graph.increment_version(self.changed)


# ---------------------------------------------------------------------------
# token embedding

def tbe_token_forward(table: torch.Tensor, ids: torch.Tensor, scale: float = 1.0,
                      out: Optional[torch.Tensor] = None, dtype: Optional[torch.dtype] = None,
                      status: Optional[torch.Tensor] = None, cfg: Optional[tbe_config] = None,
                      stream=None) -> torch.Tensor:
    """scale * table[ids]: [*ids.shape, D] of the table's dtype or float32
    (``dtype``); an id outside the table gives zeros."""
    L = _lib()
    dev = _device_of(table, ids, out, status)
    it, mt = _index(ids, "ids"), _matrix(table, "table")
    on = _On(dev, stream)
    out, mo = on.result(out, (*ids.shape, mt.cols), ids.numel(), mt.cols,
                        dtype or (table.dtype if out is None else out.dtype), "out")
    on.call(L.tbe_token_forward, mt, ids.data_ptr(), it, scale, mo, _status(status), cfg)
    return out


def _padding(padding_id: Optional[int]) -> int:
    """The padding id as 64 bits hold it; -1, which is no row, for one that they do not."""
    return -1 if padding_id is None or not -1 << 63 <= padding_id < 1 << 63 else int(padding_id)


def tbe_token_backward(grad_out: torch.Tensor, ids: torch.Tensor, rows: Optional[int] = None,
                       scale: float = 1.0, padding_id: Optional[int] = None,
                       grad_table: Optional[torch.Tensor] = None, dtype: Optional[torch.dtype] = None,
                       accumulate: bool = False, workspace: Optional[torch.Tensor] = None,
                       status: Optional[torch.Tensor] = None, cfg: Optional[tbe_config] = None,
                       stream=None) -> torch.Tensor:
    """Gradient of ``tbe_token_forward`` with respect to a table of ``rows``
    rows: [rows, D] of grad_out's dtype or float32.  With ``accumulate`` it is
    added to ``grad_table``.  Tokens of ``padding_id`` contribute nothing."""
    L = _lib()
    dev = _device_of(grad_out, ids, grad_table, workspace, status)
    it = _index(ids, "ids")
    D = grad_out.shape[-1]
    if tuple(grad_out.shape[:-1]) != tuple(ids.shape):
        _refuse(f"grad_out is [*ids.shape, D]: got {tuple(grad_out.shape)} for ids of {tuple(ids.shape)}")
    if grad_table is None and (accumulate or rows is None):
        _refuse("the gradient's rows come from `rows` or `grad_table` (which accumulate adds to)")
    if rows is None:
        rows = grad_table.shape[0]
    on = _On(dev, stream)
    mg = _matrix(grad_out if grad_out.dim() != 1 else grad_out.view(1, -1), "grad_out")
    grad_table, mt = on.result(grad_table, (rows, D), rows, D,
                               dtype or (grad_out.dtype if grad_table is None else grad_table.dtype), "grad_table")
    ws, ws_bytes, _keep = on.workspace(workspace, L.tbe_token_workspace_bytes(mg.rows, rows, D))
    on.call(L.tbe_token_backward, mg, ids.data_ptr(), it, _padding(padding_id), scale, mt, int(accumulate), ws,
            ws_bytes, _status(status), cfg)
    return grad_table


# ---------------------------------------------------------------------------
# tokens by expert

class Route:
    """Tokens sorted by expert (tbe_route): int32 tensors slot [T, K], source
    [T*K] and offset [experts+1]; offset[experts] pairs are not dropped.  The
    three lie in one buffer; their views are made when they are asked for."""

    __slots__ = ("buffer", "tokens", "K", "experts", "c", "_views")

    def __init__(self, buffer: torch.Tensor, tokens: int, K: int, experts: int):
        P = tokens * K
        if buffer.dtype != torch.int32 or buffer.numel() < 2 * P + experts + 1 or not buffer.is_contiguous():
            _refuse("a route's buffer is contiguous int32 of 2*T*K + experts + 1 words")
        self.buffer, self.tokens, self.K, self.experts, self._views = buffer, tokens, K, experts, None
        at = buffer.data_ptr()
        self.c = tbe_route(tokens, K, experts, at, at + 4 * P, at + 8 * P)

    def views(self):
        if self._views is None:
            P = self.tokens * self.K
            flat = self.buffer.as_strided
            self._views = (flat((self.tokens, self.K), (self.K, 1)), flat((P,), (1,), self.buffer.storage_offset() + P),
                           flat((self.experts + 1,), (1,), self.buffer.storage_offset() + 2 * P))
        return self._views

    @property
    def slot(self) -> torch.Tensor:
        return self.views()[0]

    @property
    def source(self) -> torch.Tensor:
        return self.views()[1]

    @property
    def offset(self) -> torch.Tensor:
        return self.views()[2]


def _new_route(on: _On, tokens: int, K: int, experts: int, route: Optional[Route]) -> Route:
    if route is not None:
        if (route.tokens, route.K, route.experts) != (tokens, K, experts):
            _refuse("route was made for other sizes")
        on.changes(route.buffer)
        return route
    return Route(on.empty(2 * tokens * K + experts + 1, torch.int32), tokens, K, experts)


def _sort_args(L, on, expert_ids, experts, route, workspace):
    if expert_ids.dim() != 2:
        _refuse(f"expert_ids are [T, K]: got {tuple(expert_ids.shape)}")
    it = _index(expert_ids, "expert_ids")
    if experts < 1:
        _refuse("there is at least one expert")
    if experts > 0x7fffffff:
        _refuse(f"the number of experts fits 32 bits: got {experts}")
    T, K = expert_ids.shape
    route = _new_route(on, T, K, int(experts), route)
    ws = on.workspace(workspace, L.tbe_route_workspace_bytes(T, K, experts))
    return it, route, ws


def tbe_route_sort(expert_ids: torch.Tensor, experts: int, route: Optional[Route] = None,
                   workspace: Optional[torch.Tensor] = None, cfg: Optional[tbe_config] = None,
                   stream=None) -> Route:
    """Sort the pairs of expert_ids [T, K] by expert; ids outside [0, experts)
    are dropped."""
    L = _lib()
    on = _On(_device_of(expert_ids, workspace, route and route.buffer), stream)
    it, route, (ws, n, _keep) = _sort_args(L, on, expert_ids, experts, route, workspace)
    on.call(L.tbe_route_sort, route.c, expert_ids.data_ptr(), it, ws, n, cfg)
    return route


def tbe_route_dispatch(x: torch.Tensor, route: Route, rows: Optional[torch.Tensor] = None,
                       cfg: Optional[tbe_config] = None, stream=None) -> torch.Tensor:
    """rows[slot[t,k]] = x[t] for x [T, H]: [T*K, H], zeros beyond the last pair."""
    L = _lib()
    on = _On(_device_of(x, route.buffer, rows), stream)
    mx = _matrix(x, "x")
    P = route.tokens * route.K
    rows, mr = on.result(rows, (P, mx.cols), P, mx.cols, x.dtype, "rows")
    on.call(L.tbe_route_dispatch, route.c, mx, mr, cfg)
    return rows


def tbe_route_sort_dispatch(x: torch.Tensor, expert_ids: torch.Tensor, experts: int,
                            route: Optional[Route] = None, rows: Optional[torch.Tensor] = None,
                            workspace: Optional[torch.Tensor] = None,
                            cfg: Optional[tbe_config] = None, stream=None):
    """(rows, route): tbe_route_sort and tbe_route_dispatch in one call."""
    L = _lib()
    on = _On(_device_of(x, expert_ids, rows, workspace, route and route.buffer), stream)
    it, route, (ws, n, _keep) = _sort_args(L, on, expert_ids, experts, route, workspace)
    mx = _matrix(x, "x")
    P = route.tokens * route.K
    rows, mr = on.result(rows, (P, mx.cols), P, mx.cols, x.dtype, "rows")
    on.call(L.tbe_route_sort_dispatch, route.c, expert_ids.data_ptr(), it, mx, mr, ws, n, cfg)
    return rows, route


def tbe_route_dispatch_backward(grad_rows: torch.Tensor, route: Route,
                                grad_x: Optional[torch.Tensor] = None,
                                cfg: Optional[tbe_config] = None, stream=None) -> torch.Tensor:
    """Gradient of tbe_route_dispatch: grad_x[t] = sum_k grad_rows[slot[t,k]]."""
    L = _lib()
    on = _On(_device_of(grad_rows, route.buffer, grad_x), stream)
    mr = _matrix(grad_rows, "grad_rows")
    grad_x, mx = on.result(grad_x, (route.tokens, mr.cols), route.tokens, mr.cols, grad_rows.dtype, "grad_x")
    on.call(L.tbe_route_dispatch_backward, route.c, mr, mx, cfg)
    return grad_x


def tbe_route_combine(rows: torch.Tensor, route: Route, weights: torch.Tensor,
                      out: Optional[torch.Tensor] = None, cfg: Optional[tbe_config] = None,
                      stream=None) -> torch.Tensor:
    """out[t] = sum_k weights[t,k] * rows[slot[t,k]]: [T, H]."""
    L = _lib()
    on = _On(_device_of(rows, route.buffer, weights, out), stream)
    mr = _matrix(rows, "rows")
    wt = _float(weights, "weights", (route.tokens, route.K))
    out, mo = on.result(out, (route.tokens, mr.cols), route.tokens, mr.cols, rows.dtype, "out")
    on.call(L.tbe_route_combine, route.c, mr, weights.data_ptr(), wt, mo, cfg)
    return out


def tbe_route_combine_backward(grad_out: torch.Tensor, rows: torch.Tensor, route: Route,
                               weights: torch.Tensor, grad_rows: Optional[torch.Tensor] = None,
                               grad_weights: Optional[torch.Tensor] = None,
                               cfg: Optional[tbe_config] = None, stream=None):
    """(grad_rows [T*K, H], grad_weights [T, K]) of tbe_route_combine."""
    L = _lib()
    on = _On(_device_of(grad_out, rows, route.buffer, weights, grad_rows, grad_weights), stream)
    mg, mr = _matrix(grad_out, "grad_out"), _matrix(rows, "rows")
    wt = _float(weights, "weights", (route.tokens, route.K))
    grad_rows, md = on.result(grad_rows, rows.shape, mr.rows, mr.cols, rows.dtype, "grad_rows")
    if grad_weights is None:
        grad_weights = on.empty(weights.shape, weights.dtype)
    elif _float(grad_weights, "grad_weights", weights.shape) != wt:
        _refuse("grad_weights has the weights' type")
    else:
        on.changes(grad_weights)
    on.call(L.tbe_route_combine_backward, route.c, mg, mr, weights.data_ptr(), wt,
            md, grad_weights.data_ptr(), cfg)
    return grad_rows, grad_weights


# ---------------------------------------------------------------------------
# distillation

def _teacher(ids: torch.Tensor, logits: torch.Tensor, rows: int, temperature: float) -> tbe_teacher:
    it, dt = _index(ids, "teacher_ids"), _float(logits, "teacher_logits", ids.shape)
    if ids.dim() < 1 or ids.numel() != rows * ids.shape[-1]:
        _refuse(f"teacher_ids are [rows, K] for {rows} rows: got {tuple(ids.shape)}")
    return tbe_teacher(ids.data_ptr() or None, logits.data_ptr() or None, it, dt, ids.shape[-1], temperature)


def _loss_and_lse(on: _On, shape, loss, lse):
    """The two results per row that the caller did not pass."""
    if loss is None and lse is None:
        return on.empty((2, *shape), torch.float32).unbind()
    on.changes(loss, lse)
    return (on.empty(shape, torch.float32) if loss is None else loss,
            on.empty(shape, torch.float32) if lse is None else lse)


def tbe_distill_forward(logits: torch.Tensor, teacher_ids: torch.Tensor, teacher_logits: torch.Tensor,
                        temperature: float = 1.0, loss: Optional[torch.Tensor] = None,
                        lse: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None,
                        status: Optional[torch.Tensor] = None, cfg: Optional[tbe_config] = None, stream=None):
    """(loss, lse), float32 of logits.shape[:-1], for logits [..., V] and the
    teacher's top entries [..., K] (ids below 0 are no entries)."""
    L = _lib()
    on = _On(_device_of(logits, teacher_ids, teacher_logits, loss, lse, workspace, status), stream)
    ml = _matrix(logits, "logits")
    te = _teacher(teacher_ids, teacher_logits, ml.rows, temperature)
    shape = logits.shape[:-1]
    loss, lse = _loss_and_lse(on, shape, loss, lse)
    ws, n, _keep = on.workspace(workspace, L.tbe_distill_workspace_bytes(ml.rows, te.K))
    on.call(L.tbe_distill_forward, ml, te, _f32_rows(loss, "loss", ml.rows), _f32_rows(lse, "lse", ml.rows),
            ws, n, _status(status), cfg)
    return loss, lse


def _grad_loss(grad_loss, rows: int):
    """(pointer or None, factor) of the gradient of the rows' losses."""
    if grad_loss is None:
        return None, 1.0
    if isinstance(grad_loss, torch.Tensor):
        return _f32_rows(grad_loss, "grad_loss", rows), 1.0
    return None, float(grad_loss)


def tbe_distill_backward(logits: torch.Tensor, teacher_ids: torch.Tensor, teacher_logits: torch.Tensor,
                         lse: torch.Tensor, grad_loss=None, temperature: float = 1.0,
                         grad_logits: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None,
                         cfg: Optional[tbe_config] = None, stream=None) -> torch.Tensor:
    """Gradient of the logits from the rows' loss gradients: a float32 tensor
    of one value per row, one number for all rows, or None for 1.
    ``grad_logits`` may be ``logits`` itself."""
    L = _lib()
    gl_tensor = grad_loss if isinstance(grad_loss, torch.Tensor) else None
    on = _On(_device_of(logits, teacher_ids, teacher_logits, lse, grad_logits, workspace, gl_tensor), stream)
    ml = _matrix(logits, "logits")
    te = _teacher(teacher_ids, teacher_logits, ml.rows, temperature)
    grad_logits, mg = on.result(grad_logits, logits.shape, ml.rows, ml.cols, logits.dtype, "grad_logits")
    gl, factor = _grad_loss(grad_loss, ml.rows)
    ws, n, _keep = on.workspace(workspace, L.tbe_distill_workspace_bytes(ml.rows, te.K))
    on.call(L.tbe_distill_backward, ml, te, _f32_rows(lse, "lse", ml.rows), gl, factor,
            mg, ws, n, cfg)
    return grad_logits


def tbe_distill_loss_grad(logits: torch.Tensor, teacher_ids: torch.Tensor, teacher_logits: torch.Tensor,
                          grad_loss=None, temperature: float = 1.0, loss: Optional[torch.Tensor] = None,
                          lse: Optional[torch.Tensor] = None, grad_logits: Optional[torch.Tensor] = None,
                          workspace: Optional[torch.Tensor] = None, status: Optional[torch.Tensor] = None,
                          cfg: Optional[tbe_config] = None, stream=None):
    """(loss, lse, grad_logits) in one call, for a training step that knows
    the loss's gradient beforehand (1/rows for a mean)."""
    L = _lib()
    gl_tensor = grad_loss if isinstance(grad_loss, torch.Tensor) else None
    on = _On(_device_of(logits, teacher_ids, teacher_logits, loss, lse, grad_logits, workspace, status,
                        gl_tensor), stream)
    ml = _matrix(logits, "logits")
    te = _teacher(teacher_ids, teacher_logits, ml.rows, temperature)
    shape = logits.shape[:-1]
    loss, lse = _loss_and_lse(on, shape, loss, lse)
    grad_logits, mg = on.result(grad_logits, logits.shape, ml.rows, ml.cols, logits.dtype, "grad_logits")
    gl, factor = _grad_loss(grad_loss, ml.rows)
    ws, n, _keep = on.workspace(workspace, L.tbe_distill_workspace_bytes(ml.rows, te.K))
    on.call(L.tbe_distill_loss_grad, ml, te, gl, factor, _f32_rows(loss, "loss", ml.rows),
            _f32_rows(lse, "lse", ml.rows), mg, ws, n, _status(status), cfg)
    return loss, lse, grad_logits
