"""Binding of the experts' operators: tokens sorted by expert and back, and
products over groups of rows with bias, activation and residual, with their
gradients (``expert_*`` and ``linear_*`` of ``include/muon_mi355x.h``).

Argument marshalling only, like the rest of the package.  Rows may be strided
(``stride(1) == 1``); everything else is contiguous.  Calls are asynchronous
on ``stream`` (the current stream if None) and can be captured into a graph.
"""

from __future__ import annotations

import ctypes
from dataclasses import dataclass
from typing import Optional, Tuple

import torch

from . import (_DT_CODE, _check, _check_workspace, _gpu_device, _ptr, _torch_stream, _workspace_on, load_library)

ACTIVATIONS = {"none": 0, "relu": 1, "gelu": 2, "gelu_tanh": 3, "silu": 4}


class ExpertRoutesC(ctypes.Structure):
    _fields_ = [("offsets", ctypes.c_void_p), ("order", ctypes.c_void_p), ("place", ctypes.c_void_p),
                ("tokens", ctypes.c_int64), ("top", ctypes.c_int32), ("experts", ctypes.c_int32)]


class LinearArgs(ctypes.Structure):
    _fields_ = [("rows", ctypes.c_int64), ("in_", ctypes.c_int64), ("out", ctypes.c_int64),
                ("groups", ctypes.c_int64), ("offsets", ctypes.c_void_p), ("dtype", ctypes.c_int32),
                ("activation", ctypes.c_int32), ("x", ctypes.c_void_p), ("x_stride", ctypes.c_int64),
                ("w", ctypes.c_void_p), ("w_stride", ctypes.c_int64), ("w_group_stride", ctypes.c_int64),
                ("bias", ctypes.c_void_p), ("residual", ctypes.c_void_p), ("residual_stride", ctypes.c_int64),
                ("y", ctypes.c_void_p), ("y_stride", ctypes.c_int64), ("pre", ctypes.c_void_p),
                ("pre_stride", ctypes.c_int64)]


class LinearGradArgs(ctypes.Structure):
    _fields_ = [("rows", ctypes.c_int64), ("in_", ctypes.c_int64), ("out", ctypes.c_int64),
                ("groups", ctypes.c_int64), ("offsets", ctypes.c_void_p), ("dtype", ctypes.c_int32),
                ("grad_dtype", ctypes.c_int32), ("activation", ctypes.c_int32), ("x_activation", ctypes.c_int32),
                ("accumulate", ctypes.c_int32), ("reserved0", ctypes.c_int32),
                ("dy", ctypes.c_void_p), ("dy_stride", ctypes.c_int64),
                ("pre", ctypes.c_void_p), ("pre_stride", ctypes.c_int64),
                ("x", ctypes.c_void_p), ("x_stride", ctypes.c_int64),
                ("w", ctypes.c_void_p), ("w_stride", ctypes.c_int64), ("w_group_stride", ctypes.c_int64),
                ("x_pre", ctypes.c_void_p), ("x_pre_stride", ctypes.c_int64),
                ("dx", ctypes.c_void_p), ("dx_stride", ctypes.c_int64),
                ("dw", ctypes.c_void_p), ("dw_stride", ctypes.c_int64), ("dw_group_stride", ctypes.c_int64),
                ("db", ctypes.c_void_p)]


def bind(lib):
    """Argument types of the library's entry points (load_library calls it)."""
    vp, i64, i32, size = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int32, ctypes.c_size_t
    routes = ctypes.POINTER(ExpertRoutesC)
    for name, args in (("expert_sort_workspace_bytes", [i64, i32, i32, ctypes.POINTER(size)]),
                       ("expert_sort", [vp, i32, routes, vp, size, vp]),
                       ("expert_gather", [vp, i64, i64, i32, routes, vp, i64, vp]),
                       ("expert_combine", [vp, i64, i64, i32, routes, vp, i32, vp, i64, vp, i64, vp]),
                       ("expert_combine_grad", [vp, i64, vp, i64, i64, i32, routes, vp, i32, vp, i64, vp, vp]),
                       ("linear_forward", [ctypes.POINTER(LinearArgs), vp]),
                       ("linear_grad_workspace_bytes", [ctypes.POINTER(LinearGradArgs), ctypes.POINTER(size)]),
                       ("linear_grad", [ctypes.POINTER(LinearGradArgs), vp, size, vp])):
        fn = getattr(lib, name)
        fn.argtypes, fn.restype = args, ctypes.c_int


# ---------------------------------------------------------------------------
# Checks
# ---------------------------------------------------------------------------
def _tensor(t, name, device, shape, dtype):
    """A tensor argument: on the call's device, of this shape and one of these
    dtypes, its rows' elements consecutive."""
    if not isinstance(t, torch.Tensor):
        raise ValueError(f"{name} must be a tensor, got {type(t).__name__}")
    if device is not None and t.device != device:
        raise ValueError(f"{name} is on {t.device}, the call's tensors on {device}")
    if shape is not None and tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")
    dtypes = dtype if isinstance(dtype, tuple) else (dtype,)
    if t.dtype not in dtypes:
        raise ValueError(f"{name} is {t.dtype}, expected {' or '.join(str(d) for d in dtypes)}")


def _rows(t, name, device, shape, dtype) -> int:
    """Row stride of a 2-D argument."""
    _tensor(t, name, device, shape, dtype)
    if t.dim() != 2:
        raise ValueError(f"{name} must have rows and columns, got shape {tuple(t.shape)}")
    if t.shape[1] > 1 and t.stride(1) != 1:
        raise ValueError(f"{name}: a row's elements must be consecutive")
    if t.shape[0] > 1 and t.stride(0) < t.shape[1]:
        raise ValueError(f"{name}: rows overlap (stride {t.stride(0)} for {t.shape[1]} columns)")
    return t.stride(0) if t.shape[0] > 1 else max(1, t.shape[1])


def _dense(t, name, device, shape, dtype):
    _tensor(t, name, device, shape, dtype)
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


def _output(t, name, device, shape, dtype, ts) -> torch.Tensor:
    """The caller's output, or a new one on the launch stream."""
    if t is None:
        with torch.cuda.stream(ts):
            t = torch.empty(shape, dtype=dtype, device=device)
    return t


_FLOATS = tuple(_DT_CODE)
_INTS = (torch.int32, torch.int64)


# ---------------------------------------------------------------------------
# Tokens sorted by expert and back
# ---------------------------------------------------------------------------
@dataclass
class ExpertRoutes:
    """Where every token's rows are (expert_routes_t): int32 tensors
    ``offsets`` (experts + 1), ``order`` (tokens * top) and ``place`` (tokens,
    top)."""
    offsets: torch.Tensor
    order: torch.Tensor
    place: torch.Tensor

    @property
    def experts(self) -> int:
        return self.offsets.numel() - 1

    @property
    def tokens(self) -> int:
        return self.place.shape[0]

    @property
    def top(self) -> int:
        return self.place.shape[1]

    def to_c(self) -> ExpertRoutesC:
        device = self.place.device if isinstance(self.place, torch.Tensor) else None
        _dense(self.place, "routes.place", device, None, torch.int32)
        if self.place.dim() != 2:
            raise ValueError(f"routes.place must be (tokens, top), got {tuple(self.place.shape)}")
        _dense(self.offsets, "routes.offsets", device, None, torch.int32)
        if self.offsets.dim() != 1 or self.offsets.numel() < 2:
            raise ValueError(f"routes.offsets must hold experts + 1 numbers, got shape {tuple(self.offsets.shape)}")
        _dense(self.order, "routes.order", device, (self.place.numel(),), torch.int32)
        return ExpertRoutesC(self.offsets.data_ptr(), self.order.data_ptr(), self.place.data_ptr(), self.tokens,
                             self.top, self.experts)


def _routes(routes) -> ExpertRoutesC:
    if not isinstance(routes, ExpertRoutes):
        raise ValueError(f"routes must be ExpertRoutes, got {type(routes).__name__}")
    return routes.to_c()


def expert_sort(ids: torch.Tensor, experts: int, routes: Optional[ExpertRoutes] = None,
                workspace: Optional[torch.Tensor] = None, stream=None) -> ExpertRoutes:
    """Sorts the choices of a batch by expert: ``ids`` (tokens, top), int32 or
    int64, each 0..experts-1, or another number for a choice that is not
    routed.  Returns (fills, if given) ``routes``.  The sort is stable."""
    _dense(ids, "ids", None, None, _INTS)
    if ids.dim() != 2 or ids.shape[1] < 1:
        raise ValueError(f"ids must be (tokens, top), got {tuple(ids.shape)}")
    lib, nbytes = load_library(), ctypes.c_size_t(0)
    tokens, top = ids.shape
    _check(lib.expert_sort_workspace_bytes(tokens, top, experts, ctypes.byref(nbytes)))
    _check_workspace(workspace, ids.device)
    device = _gpu_device(ids.device)
    ts = _torch_stream(stream, device)
    if routes is None:
        flat = _output(None, "routes", device, (experts + 1 + 2 * tokens * top,), torch.int32, ts)
        n = tokens * top
        routes = ExpertRoutes(flat[2 * n:], flat[:n], flat[n:2 * n].view(tokens, top))
    c = _routes(routes)
    _tensor(routes.place, "routes.place", device, (tokens, top), torch.int32)
    if c.experts != experts:
        raise ValueError(f"routes are of {c.experts} experts, the call of {experts}")
    if workspace is None and nbytes.value:
        workspace = _workspace_on(None, nbytes.value, device, ts)
    with torch.cuda.device(device):
        _check(lib.expert_sort(ids.data_ptr(), ids.element_size(), ctypes.byref(c), _ptr(workspace),
                               0 if workspace is None else workspace.numel(), ts.cuda_stream))
    return routes


def expert_gather(x: torch.Tensor, routes: ExpertRoutes, out: Optional[torch.Tensor] = None,
                  stream=None) -> torch.Tensor:
    """Every token's row to its sorted rows: (tokens, width) to (tokens * top,
    width).  Rows behind the last routed one are left as they were (undefined
    in a new ``out``).  The gradient is ``expert_combine`` without weights."""
    c = _routes(routes)
    device = _gpu_device(routes.place.device)
    ld = _rows(x, "x", device, None, _FLOATS)
    _tensor(x, "x", device, (c.tokens, x.shape[1]), _FLOATS)
    ts = _torch_stream(stream, device)
    shape = (c.tokens * c.top, x.shape[1])
    out = _output(out, "out", device, shape, x.dtype, ts)
    ld_out = _rows(out, "out", device, shape, x.dtype)
    with torch.cuda.device(device):
        _check(load_library().expert_gather(x.data_ptr(), ld, x.shape[1], _DT_CODE[x.dtype], ctypes.byref(c),
                                            out.data_ptr(), ld_out, ts.cuda_stream))
    return out


def _weights(weights, device, c):
    _dense(weights, "weights", device, (c.tokens, c.top), _FLOATS)
    return weights.data_ptr(), _DT_CODE[weights.dtype]


def expert_combine(ys: torch.Tensor, routes: ExpertRoutes, weights: Optional[torch.Tensor] = None,
                   residual: Optional[torch.Tensor] = None, out: Optional[torch.Tensor] = None,
                   stream=None) -> torch.Tensor:
    """Sorted rows back to their tokens: ``residual`` + the sum over a token's
    choices of ``weights`` * row (``weights`` (tokens, top), float32 or
    bfloat16).  ``out`` may be the residual itself."""
    c = _routes(routes)
    device = _gpu_device(routes.place.device)
    ld = _rows(ys, "ys", device, None, _FLOATS)
    _tensor(ys, "ys", device, (c.tokens * c.top, ys.shape[1]), _FLOATS)
    shape = (c.tokens, ys.shape[1])
    w, w_dt = (None, 0) if weights is None else _weights(weights, device, c)
    ld_res = 0 if residual is None else _rows(residual, "residual", device, shape, ys.dtype)
    ts = _torch_stream(stream, device)
    out = _output(out, "out", device, shape, ys.dtype, ts)
    ld_out = _rows(out, "out", device, shape, ys.dtype)
    with torch.cuda.device(device):
        _check(load_library().expert_combine(ys.data_ptr(), ld, ys.shape[1], _DT_CODE[ys.dtype], ctypes.byref(c), w,
                                             w_dt, _ptr(residual), ld_res, out.data_ptr(), ld_out, ts.cuda_stream))
    return out


def expert_combine_grad(dy: torch.Tensor, ys: torch.Tensor, weights: torch.Tensor, routes: ExpertRoutes,
                        dys: Optional[torch.Tensor] = None, dweights: Optional[torch.Tensor] = None,
                        stream=None) -> Tuple[torch.Tensor, torch.Tensor]:
    """Gradient of ``expert_combine`` with weights: (dys, dweights).  The
    residual's is dy itself."""
    c = _routes(routes)
    device = _gpu_device(routes.place.device)
    ld = _rows(ys, "ys", device, None, _FLOATS)
    shape = (c.tokens * c.top, ys.shape[1])
    _tensor(ys, "ys", device, shape, _FLOATS)
    ld_dy = _rows(dy, "dy", device, (c.tokens, ys.shape[1]), ys.dtype)
    w, w_dt = _weights(weights, device, c)
    ts = _torch_stream(stream, device)
    dys = _output(dys, "dys", device, shape, ys.dtype, ts)
    ld_dys = _rows(dys, "dys", device, shape, ys.dtype)
    dweights = _output(dweights, "dweights", device, weights.shape, weights.dtype, ts)
    _dense(dweights, "dweights", device, weights.shape, weights.dtype)
    with torch.cuda.device(device):
        _check(load_library().expert_combine_grad(dy.data_ptr(), ld_dy, ys.data_ptr(), ld, ys.shape[1],
                                                  _DT_CODE[ys.dtype], ctypes.byref(c), w, w_dt, dys.data_ptr(),
                                                  ld_dys, dweights.data_ptr(), ts.cuda_stream))
    return dys, dweights


# ---------------------------------------------------------------------------
# Products over groups of rows
# ---------------------------------------------------------------------------
def _activation(name) -> int:
    if name not in ACTIVATIONS:
        raise ValueError(f"activation must be one of {sorted(ACTIVATIONS)}, got {name!r}")
    return ACTIVATIONS[name]


def _weight(w, name, device, shape, dtype):
    """(groups, out, in, row stride, group stride) of a weight: (out, in), or
    (groups, out, in)."""
    _tensor(w, name, device, shape, dtype)
    if w.dim() not in (2, 3):
        raise ValueError(f"{name} must be (out, in) or (groups, out, in), got {tuple(w.shape)}")
    groups, (out, inn) = (w.shape[0] if w.dim() == 3 else 1), w.shape[-2:]
    if inn > 1 and w.stride(-1) != 1:
        raise ValueError(f"{name}: a row's elements must be consecutive")
    ld = w.stride(-2) if out > 1 else max(1, inn)
    return groups, out, inn, ld, (w.stride(0) if groups > 1 else out * ld)


def _groups(offsets, w, groups, device):
    if offsets is None:
        if groups != 1:
            raise ValueError(f"{groups} groups need offsets")
        return None
    _dense(offsets, "offsets", device, (groups + 1,), torch.int32)
    return offsets.data_ptr()


def linear(x: torch.Tensor, w: torch.Tensor, bias: Optional[torch.Tensor] = None, activation: str = "none",
           residual: Optional[torch.Tensor] = None, offsets: Optional[torch.Tensor] = None,
           pre: Optional[torch.Tensor] = None, out: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """``act(x w^T + bias) + residual``: x (rows, in), w (out, in) and bias
    (out).  With ``offsets`` (groups + 1, int32 on the device, as
    ``ExpertRoutes`` has them) w is (groups, out, in), bias (groups, out), and
    group g takes the rows offsets[g] .. offsets[g+1]-1; rows of no group are
    left as they were (undefined in a new ``out``).  ``pre``, if given,
    receives x w^T + bias, which ``linear_grad`` wants where there is an
    activation.  ``out`` may be the residual itself."""
    act = _activation(activation)
    ld = _rows(x, "x", None, None, _FLOATS)
    groups, n, k, ld_w, group_w = _weight(w, "w", x.device, None, x.dtype)
    rows = x.shape[0]
    _tensor(x, "x", None, (rows, k), x.dtype)
    device, shape = x.device, (rows, n)
    if bias is not None:
        _dense(bias, "bias", device, w.shape[:-1], x.dtype)
    off = _groups(offsets, w, groups, device)
    ld_res = 0 if residual is None else _rows(residual, "residual", device, shape, x.dtype)
    ld_pre = 0 if pre is None else _rows(pre, "pre", device, shape, x.dtype)
    if out is not None:
        _rows(out, "out", device, shape, x.dtype)
    device = _gpu_device(device)
    ts = _torch_stream(stream, device)
    out = _output(out, "out", device, shape, x.dtype, ts)
    a = LinearArgs(rows, k, n, groups, off, _DT_CODE[x.dtype], act, x.data_ptr(), ld, w.data_ptr(), ld_w, group_w,
                   _ptr(bias), _ptr(residual), ld_res, out.data_ptr(), _rows(out, "out", device, shape, x.dtype),
                   _ptr(pre), ld_pre)
    with torch.cuda.device(device):
        _check(load_library().linear_forward(ctypes.byref(a), ts.cuda_stream))
    return out


def linear_grad(dy: torch.Tensor, x: Optional[torch.Tensor] = None, w: Optional[torch.Tensor] = None,
                activation: str = "none", pre: Optional[torch.Tensor] = None,
                offsets: Optional[torch.Tensor] = None, dx: Optional[torch.Tensor] = None,
                dw: Optional[torch.Tensor] = None, db: Optional[torch.Tensor] = None, accumulate: bool = False,
                x_activation: str = "none", x_pre: Optional[torch.Tensor] = None,
                workspace: Optional[torch.Tensor] = None, stream=None):
    """Gradients of ``linear``, into the buffers that are given: ``dx`` (needs
    w), ``dw`` (needs x; float32 or bfloat16, the very buffer that ``Param.g``
    names, or one of several groups) and ``db`` (of dw's dtype, if both are
    given).  ``accumulate`` adds to dw and db.  ``pre`` is what ``linear``
    left there (with an activation).  ``x_activation`` and ``x_pre`` carry dx
    through the activation that made x, so that dx becomes the gradient of
    x_pre.  Returns (dx, dw, db)."""
    act, x_act = _activation(activation), _activation(x_activation)
    if dx is None and dw is None and db is None:
        raise ValueError("give at least one of dx, dw and db")
    ld_dy = _rows(dy, "dy", None, None, _FLOATS)
    rows, n = dy.shape
    device, dt = dy.device, dy.dtype
    weight = w if w is not None else dw
    if weight is not None:
        groups, out, k, _, _ = _weight(weight, "w" if w is not None else "dw", device, None, _FLOATS)
        if out != n:
            raise ValueError(f"the weight has {out} rows, dy {n} columns")
    else:
        groups, k = (db.shape[0] if db.dim() == 2 else 1), 1
    a = LinearGradArgs(rows=rows, in_=k, out=n, groups=groups, dtype=_DT_CODE[dt], activation=act,
                       x_activation=x_act, accumulate=1 if accumulate else 0, dy=dy.data_ptr(), dy_stride=ld_dy)
    grouped = weight.dim() == 3 if weight is not None else db.dim() == 2
    a.offsets = _groups(offsets, weight, groups, device)
    if act:
        if pre is None:
            raise ValueError(f"the gradient through {activation} needs pre")
        a.pre_stride = _rows(pre, "pre", device, (rows, n), dt)
        a.pre = pre.data_ptr()
    if dx is not None:
        if w is None:
            raise ValueError("dx needs w")
        _, _, _, a.w_stride, a.w_group_stride = _weight(w, "w", device, None, dt)
        a.w = w.data_ptr()
        a.dx_stride = _rows(dx, "dx", device, (rows, k), dt)
        a.dx = dx.data_ptr()
        if x_act:
            if x_pre is None:
                raise ValueError(f"dx through {x_activation} needs x_pre")
            a.x_pre_stride = _rows(x_pre, "x_pre", device, (rows, k), dt)
            a.x_pre = x_pre.data_ptr()
    grad_dt = None
    if dw is not None:
        if x is None:
            raise ValueError("dw needs x")
        a.x_stride = _rows(x, "x", device, (rows, k), dt)
        a.x = x.data_ptr()
        _, _, _, a.dw_stride, a.dw_group_stride = _weight(dw, "dw", device, weight.shape, _FLOATS)
        a.dw, grad_dt = dw.data_ptr(), dw.dtype
    if db is not None:
        _dense(db, "db", device, (groups, n) if grouped else (n,), _FLOATS if grad_dt is None else grad_dt)
        a.db, grad_dt = db.data_ptr(), db.dtype
    a.grad_dtype = _DT_CODE[grad_dt] if grad_dt is not None else a.dtype
    lib, nbytes = load_library(), ctypes.c_size_t(0)
    _check(lib.linear_grad_workspace_bytes(ctypes.byref(a), ctypes.byref(nbytes)))
    _check_workspace(workspace, device)
    device = _gpu_device(device)
    ts = _torch_stream(stream, device)
    if workspace is None and nbytes.value:
        workspace = _workspace_on(None, nbytes.value, device, ts)
    with torch.cuda.device(device):
        _check(lib.linear_grad(ctypes.byref(a), _ptr(workspace), 0 if workspace is None else workspace.numel(),
                               ts.cuda_stream))
    return dx, dw, db


def linear_grad_workspace(rows: int, w: torch.Tensor, activation: str = "none", dw: bool = True, db: bool = False,
                          dtype: Optional[torch.dtype] = None) -> torch.Tensor:
    """A workspace for ``linear_grad`` over up to ``rows`` rows, to be used
    again and again (calls that share one must be ordered)."""
    groups, n, k, _, _ = _weight(w, "w", None, None, _FLOATS)
    dt = _DT_CODE[w.dtype if dtype is None else dtype]
    nbytes = ctypes.c_size_t(0)
    a = LinearGradArgs(rows=rows, in_=k, out=n, groups=groups, offsets=1, dtype=dt, activation=_activation(activation))
    a.dw, a.db = (1 if dw else None), (1 if db else None)
    _check(load_library().linear_grad_workspace_bytes(ctypes.byref(a), ctypes.byref(nbytes)))
    return torch.empty(max(nbytes.value, 256), dtype=torch.uint8, device=w.device)
