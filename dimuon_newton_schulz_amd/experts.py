"""Binding of the experts' operators: tokens sorted by expert and back, and
products over groups of rows with bias, activation and residual, with their
gradients (``expert_*`` and ``linear_*`` of ``include/muon_mi355x.h``).

Argument marshalling only, like the rest of the package.  Rows may be strided
(``stride(1) == 1``); everything else is contiguous.  Calls are asynchronous
on ``stream`` (the current stream if None) and can be captured into a graph.

Autograd records none of these calls: each gradient is a call of its own.  An
input that requires a gradient is therefore refused while autograd is on (as
torch's functions with ``out=`` do); call under ``torch.no_grad()``, or from
the forward and backward of a ``torch.autograd.Function``.
"""

from __future__ import annotations

import ctypes
import sys
import warnings
from dataclasses import dataclass
from typing import Optional, Tuple

import torch

from . import (_DT_CODE, _check, _check_workspace, _current_raw_stream, _ptr, _stream_handle, _torch_stream,
               _workspace_on, load_library)

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


# The ordinary case of a call (current GPU and stream, tensors as expected) is
# marshalled natively: csrc/binding.cpp.  None from it: not that case, and the
# Python code goes on.
_fast = None


class _NoBinding:
    """In the extension module's place where there is none: every call goes on
    in Python, which takes 7 to 10 us more of host time."""
    sort = gather = combine = combine_grad = linear = linear_grad = staticmethod(lambda *args: None)


def _load_binding(lib):
    """The extension module, or _NoBinding if it is missing or was built for
    another torch or Python: nothing else in the package needs it."""
    try:
        from . import _binding
        made_for = _binding.torch_version, _binding.python_version
        here = torch.__version__.split("+")[0], f"{sys.version_info.major}.{sys.version_info.minor}"
        if made_for != here:
            raise ImportError(f"built for torch {made_for[0]} and Python {made_for[1]}, not {here[0]} and {here[1]}")
    except (ImportError, AttributeError) as e:
        warnings.warn(f"{__package__}._binding cannot be used ({e}): short calls take longer on the host; build it with "
                      f"`python -m {__package__}.build`", RuntimeWarning, stacklevel=4)
        return _NoBinding
    _binding.bind(*(ctypes.cast(getattr(lib, name), ctypes.c_void_p).value for name in
                    ("expert_sort", "expert_gather", "expert_combine", "expert_combine_grad", "linear_forward",
                     "linear_grad_workspace_bytes", "linear_grad")))
    return _binding


def _native():
    global _fast
    if _fast is None:
        _fast = _load_binding(load_library())
    return _fast


def _done(result):
    """What a native call made, or its failing status."""
    if result.__class__ is int:
        _check(result)
    return result


# ---------------------------------------------------------------------------
# Checks.  A short call's host time is these, so the common case of each takes
# a few attribute reads; the function behind it says what is wrong.
# ---------------------------------------------------------------------------
_MAX_STRIDE = 1 << 20
_FLOATS = tuple(_DT_CODE)
_INTS = (torch.int32, torch.int64)


def _tensor(t, name, index, shape, dtype):
    """A tensor argument: on GPU `index` (None: anywhere), of this shape and
    one of these dtypes."""
    if not isinstance(t, torch.Tensor):
        raise ValueError(f"{name} must be a tensor, got {type(t).__name__}")
    if index is not None and t.get_device() != index:
        raise ValueError(f"{name} is on {t.device}, the call's tensors on {_device_name(index)}")
    if shape is not None and t.shape != shape:
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")
    if t.dtype not in (dtype if isinstance(dtype, tuple) else (dtype,)):
        raise ValueError(f"{name} is {t.dtype}, expected one of {dtype}")


def _device_name(index):
    return "the CPU" if index < 0 else f"GPU {index}"


def _rows(t, name, index, shape, dtype) -> int:
    """Row stride of a 2-D argument whose rows' elements are consecutive."""
    try:
        if t.dtype is dtype and t.shape == shape and t.get_device() == index:
            a, b = t.stride()
            if b == 1 and shape[1] <= a <= _MAX_STRIDE:
                return a
    except (AttributeError, TypeError, ValueError):
        pass
    _tensor(t, name, index, shape, dtype)
    if t.dim() != 2:
        raise ValueError(f"{name} must have rows and columns, got shape {tuple(t.shape)}")
    if t.shape[1] > 1 and t.stride(1) != 1:
        raise ValueError(f"{name}: a row's elements must be consecutive")
    if t.shape[0] > 1 and t.stride(0) < t.shape[1]:
        raise ValueError(f"{name}: rows overlap (stride {t.stride(0)} for {t.shape[1]} columns)")
    return t.stride(0) if t.shape[0] > 1 else max(1, t.shape[1])


def _dense(t, name, index, shape, dtype):
    try:
        if t.dtype is dtype and t.shape == shape and t.get_device() == index and t.is_contiguous():
            return
    except AttributeError:
        pass
    _tensor(t, name, index, shape, dtype)
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


def _matrix(t, name):
    """Shape and dtype of a call's leading 2-D argument."""
    _tensor(t, name, None, None, _FLOATS)
    if t.dim() != 2:
        raise ValueError(f"{name} must have rows and columns, got shape {tuple(t.shape)}")
    return t.shape, t.dtype


def _unrecorded(call, gradient, **tensors):
    """Refuses a call that autograd would have to record."""
    if torch.is_grad_enabled():
        for name, t in tensors.items():
            if isinstance(t, torch.Tensor) and t.requires_grad:
                raise ValueError(f"{name} requires a gradient, but autograd does not record {call} ({gradient}): call it "
                                 "under torch.no_grad() or on detached tensors")


class _Launch:
    """Where a call runs: the GPU of its tensors and the launch stream."""
    __slots__ = ("index", "stream", "given")

    def __init__(self, index, stream):
        if index < 0:
            raise ValueError("the tensors are on the CPU: they must be on the GPU")
        self.index, self.given = index, stream
        if stream is None and _current_raw_stream is not None:
            self.stream = _current_raw_stream(index)
        else:
            self.stream = _stream_handle(stream, torch.device("cuda", index))

    def empty(self, shape, dtype):
        """A new tensor that belongs to the launch stream."""
        if self.given is None:
            return torch.empty(shape, dtype=dtype, device=torch.device("cuda", self.index))
        with torch.cuda.stream(_torch_stream(self.given, torch.device("cuda", self.index))):
            return torch.empty(shape, dtype=dtype, device=torch.device("cuda", self.index))

    def workspace(self, given, nbytes):
        """The caller's workspace, or one that the allocator keeps until the
        launch stream is done with it: (pointer, bytes, tensor)."""
        if given is None:
            if not nbytes:
                return None, 0, None
            device = torch.device("cuda", self.index)
            given = _workspace_on(None, nbytes, device, _torch_stream(self.given, device))
        return given.data_ptr(), given.numel(), given

    def call(self, fn, *args):
        if torch.cuda.current_device() == self.index:
            status = fn(*args, self.stream)
        else:
            with torch.cuda.device(self.index):
                status = fn(*args, self.stream)
        if status:
            _check(status)


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
        place, offsets, order = self.place, self.offsets, self.order
        try:
            index, (tokens, top), n = place.get_device(), place.shape, offsets.numel()
        except (AttributeError, ValueError):
            raise ValueError("routes.place must be (tokens, top), routes.offsets a tensor") from None
        _dense(place, "routes.place", index, place.shape, torch.int32)
        _dense(offsets, "routes.offsets", index, (n,), torch.int32)
        _dense(order, "routes.order", index, (tokens * top,), torch.int32)
        if n < 2:
            raise ValueError(f"routes.offsets must hold experts + 1 numbers, got {n}")
        return ExpertRoutesC(offsets.data_ptr(), order.data_ptr(), place.data_ptr(), tokens, top, n - 1)


def _routes(routes):
    """(expert_routes_t, its address for a call, GPU)."""
    if not isinstance(routes, ExpertRoutes):
        raise ValueError(f"routes must be ExpertRoutes, got {type(routes).__name__}")
    c = routes.to_c()
    return c, ctypes.byref(c), routes.place.get_device()


def expert_sort(ids: torch.Tensor, experts: int, routes: Optional[ExpertRoutes] = None,
                workspace: Optional[torch.Tensor] = None, stream=None) -> ExpertRoutes:
    """Sorts the choices of a batch by expert: ``ids`` (tokens, top), int32 or
    int64, each 0..experts-1, or another number for a choice that is not
    routed.  Returns (fills, if given) ``routes``.  The sort is stable."""
    if routes is None and workspace is None and stream is None:
        done = _native().sort(ids, experts)
        if done is not None:
            return ExpertRoutes(*_done(done))
    _tensor(ids, "ids", None, None, _INTS)
    if ids.dim() != 2 or ids.shape[1] < 1:
        raise ValueError(f"ids must be (tokens, top), got {tuple(ids.shape)}")
    if not ids.is_contiguous():
        raise ValueError("ids must be contiguous")
    lib, (tokens, top) = load_library(), ids.shape
    nbytes = 0
    if tokens * top > _SORT_ALONE or not 0 < experts <= _MAX_EXPERTS:   # otherwise none is needed
        size = ctypes.c_size_t(0)
        _check(lib.expert_sort_workspace_bytes(tokens, top, experts, ctypes.byref(size)))
        nbytes = size.value
    _check_workspace(workspace, ids.device)
    on = _Launch(ids.get_device(), stream)
    if routes is None:
        n = tokens * top
        offsets, order, place = on.empty(experts + 1 + 2 * n, torch.int32).split((experts + 1, n, n))
        c = ExpertRoutesC(offsets.data_ptr(), order.data_ptr(), place.data_ptr(), tokens, top, experts)
        routes = ExpertRoutes(offsets, order, place.view(tokens, top))
    else:
        c, _, _ = _routes(routes)
        _dense(routes.place, "routes.place", on.index, (tokens, top), torch.int32)
        if c.experts != experts:
            raise ValueError(f"routes are of {c.experts} experts, the call of {experts}")
    ws, ws_bytes, _keep = on.workspace(workspace, nbytes)
    on.call(lib.expert_sort, ids.data_ptr(), ids.element_size(), ctypes.byref(c), ws, ws_bytes)
    return routes


_SORT_ALONE, _MAX_EXPERTS = 8192, 1024   # a sort of that many slots needs no workspace


def expert_gather(x: torch.Tensor, routes: ExpertRoutes, out: Optional[torch.Tensor] = None,
                  stream=None) -> torch.Tensor:
    """Every token's row to its sorted rows: (tokens, width) to (tokens * top,
    width).  Rows behind the last routed one are left as they were (undefined
    in a new ``out``).  The gradient is ``expert_combine`` without weights."""
    if stream is None and routes.__class__ is ExpertRoutes:
        done = _native().gather(x, routes.offsets, routes.order, routes.place, out)
        if done is not None:
            return _done(done)
    _unrecorded("expert_gather", "its gradient is expert_combine without weights", x=x, out=out)
    c, ref, index = _routes(routes)
    (_, width), dt = _matrix(x, "x")
    ld = _rows(x, "x", index, (c.tokens, width), dt)
    on, shape = _Launch(index, stream), (c.tokens * c.top, width)
    if out is None:
        out = on.empty(shape, dt)
    ld_out = _rows(out, "out", index, shape, dt)
    on.call(load_library().expert_gather, x.data_ptr(), ld, width, _DT_CODE[dt], ref, out.data_ptr(), ld_out)
    return out


def _weights(weights, index, c):
    _tensor(weights, "weights", index, (c.tokens, c.top), _FLOATS)
    if not weights.is_contiguous():
        raise ValueError("weights must be contiguous")
    return weights.data_ptr(), _DT_CODE[weights.dtype]


def expert_combine(ys: torch.Tensor, routes: ExpertRoutes, weights: Optional[torch.Tensor] = None,
                   residual: Optional[torch.Tensor] = None, out: Optional[torch.Tensor] = None,
                   stream=None) -> torch.Tensor:
    """Sorted rows back to their tokens: ``residual`` + the sum over a token's
    choices of ``weights`` * row (``weights`` (tokens, top), float32 or
    bfloat16).  ``out`` may be the residual itself."""
    if stream is None and routes.__class__ is ExpertRoutes:
        done = _native().combine(ys, routes.offsets, routes.order, routes.place, weights, residual, out)
        if done is not None:
            return _done(done)
    _unrecorded("expert_combine", "its gradient is expert_combine_grad", ys=ys, weights=weights, residual=residual, out=out)
    c, ref, index = _routes(routes)
    (_, width), dt = _matrix(ys, "ys")
    ld = _rows(ys, "ys", index, (c.tokens * c.top, width), dt)
    shape = (c.tokens, width)
    w, w_dt = (None, 0) if weights is None else _weights(weights, index, c)
    res, ld_res = (None, 0) if residual is None else (residual.data_ptr(), _rows(residual, "residual", index, shape, dt))
    on = _Launch(index, stream)
    if out is None:
        out = on.empty(shape, dt)
    ld_out = _rows(out, "out", index, shape, dt)
    on.call(load_library().expert_combine, ys.data_ptr(), ld, width, _DT_CODE[dt], ref, w, w_dt, res, ld_res,
            out.data_ptr(), ld_out)
    return out


def expert_combine_grad(dy: torch.Tensor, ys: torch.Tensor, weights: torch.Tensor, routes: ExpertRoutes,
                        dys: Optional[torch.Tensor] = None, dweights: Optional[torch.Tensor] = None,
                        stream=None) -> Tuple[torch.Tensor, torch.Tensor]:
    """Gradient of ``expert_combine`` with weights: (dys, dweights).  The
    residual's is dy itself."""
    if stream is None and routes.__class__ is ExpertRoutes:
        done = _native().combine_grad(dy, ys, weights, routes.offsets, routes.order, routes.place, dys, dweights)
        if done is not None:
            return _done(done)
    _unrecorded("expert_combine_grad", "a gradient itself", dy=dy)
    c, ref, index = _routes(routes)
    (_, width), dt = _matrix(ys, "ys")
    shape = (c.tokens * c.top, width)
    ld = _rows(ys, "ys", index, shape, dt)
    ld_dy = _rows(dy, "dy", index, (c.tokens, width), dt)
    w, w_dt = _weights(weights, index, c)
    on = _Launch(index, stream)
    if dys is None:
        dys = on.empty(shape, dt)
    ld_dys = _rows(dys, "dys", index, shape, dt)
    if dweights is None:
        dweights = on.empty(weights.shape, weights.dtype)
    _dense(dweights, "dweights", index, weights.shape, weights.dtype)
    on.call(load_library().expert_combine_grad, dy.data_ptr(), ld_dy, ys.data_ptr(), ld, width, _DT_CODE[dt], ref, w,
            w_dt, dys.data_ptr(), ld_dys, dweights.data_ptr())
    return dys, dweights


# ---------------------------------------------------------------------------
# Products over groups of rows
# ---------------------------------------------------------------------------
def _activation(name) -> int:
    if name not in ACTIVATIONS:
        raise ValueError(f"activation must be one of {sorted(ACTIVATIONS)}, got {name!r}")
    return ACTIVATIONS[name]


def _weight(w, name, index, dtype):
    """(groups, out, in, row stride, group stride) of a weight: (out, in), or
    (groups, out, in)."""
    _tensor(w, name, index, None, dtype)
    shape, strides = w.shape, w.stride()
    if len(shape) == 3:
        groups, out, inn = shape
        if strides[2] == 1 and strides[1] >= inn and (strides[0] >= out * strides[1] or groups == 1) and out > 1:
            return groups, out, inn, strides[1], strides[0] if groups > 1 else out * strides[1]
    elif len(shape) == 2:
        groups, (out, inn) = 1, shape
    else:
        raise ValueError(f"{name} must be (out, in) or (groups, out, in), got {tuple(shape)}")
    if inn > 1 and strides[-1] != 1:
        raise ValueError(f"{name}: a row's elements must be consecutive")
    ld = strides[-2] if out > 1 else max(1, inn)
    return groups, out, inn, ld, (strides[0] if groups > 1 else out * ld)


def _groups(offsets, groups, index):
    if offsets is None:
        if groups != 1:
            raise ValueError(f"{groups} groups need offsets")
        return None
    _dense(offsets, "offsets", index, (groups + 1,), torch.int32)
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
    if stream is None:
        done = _native().linear(x, w, bias, act, residual, offsets, pre, out)
        if done is not None:
            return _done(done)
    _unrecorded("linear", "its gradient is linear_grad", x=x, w=w, bias=bias, residual=residual, pre=pre, out=out)
    (rows, k), dt = _matrix(x, "x")
    index = x.get_device()
    groups, n, k_w, ld_w, group_w = _weight(w, "w", index, dt)
    if k_w != k:
        raise ValueError(f"x has {k} columns, the weight {k_w}")
    shape = (rows, n)
    ld = _rows(x, "x", index, (rows, k), dt)
    if bias is not None:
        _dense(bias, "bias", index, w.shape[:-1], dt)
    off = _groups(offsets, groups, index)
    ld_res = 0 if residual is None else _rows(residual, "residual", index, shape, dt)
    ld_pre = 0 if pre is None else _rows(pre, "pre", index, shape, dt)
    ld_out = 0 if out is None else _rows(out, "out", index, shape, dt)
    on = _Launch(index, stream)
    if out is None:
        out = on.empty(shape, dt)
        ld_out = max(1, n)
    a = LinearArgs(rows, k, n, groups, off, _DT_CODE[dt], act, x.data_ptr(), ld, w.data_ptr(), ld_w, group_w,
                   _ptr(bias), _ptr(residual), ld_res, out.data_ptr(), ld_out, _ptr(pre), ld_pre)
    on.call(load_library().linear_forward, ctypes.byref(a))
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
    if stream is None and accumulate.__class__ is bool:
        done = _native().linear_grad(dy, x, w, act, pre, offsets, dx, dw, db, accumulate, x_act, x_pre, workspace)
        if done is not None:
            if done is not True:
                _check(done)
            return dx, dw, db
    _unrecorded("linear_grad", "a gradient itself", dy=dy)
    if dx is None and dw is None and db is None:
        raise ValueError("give at least one of dx, dw and db")
    (rows, n), dt = _matrix(dy, "dy")
    index = dy.get_device()
    ld_dy = _rows(dy, "dy", index, (rows, n), dt)
    weight = w if w is not None else dw
    if weight is not None:
        groups, out, k, ld_w, group_w = _weight(weight, "w" if w is not None else "dw", index, _FLOATS)
        grouped = weight.dim() == 3
        if out != n:
            raise ValueError(f"the weight has {out} rows, dy {n} columns")
    else:
        grouped = db.dim() == 2
        groups, k = (db.shape[0] if grouped else 1), 1
    a = LinearGradArgs(rows, k, n, groups, _groups(offsets, groups, index), _DT_CODE[dt], 0, act, x_act,
                       1 if accumulate else 0, 0, dy.data_ptr(), ld_dy)
    if act:
        if pre is None:
            raise ValueError(f"the gradient through {activation} needs pre")
        a.pre_stride = _rows(pre, "pre", index, (rows, n), dt)
        a.pre = pre.data_ptr()
    if dx is not None:
        if w is None:
            raise ValueError("dx needs w")
        if w.dtype is not dt:
            raise ValueError(f"w is {w.dtype}, dy {dt}")
        a.w, a.w_stride, a.w_group_stride = w.data_ptr(), ld_w, group_w
        a.dx_stride = _rows(dx, "dx", index, (rows, k), dt)
        a.dx = dx.data_ptr()
        if x_act:
            if x_pre is None:
                raise ValueError(f"dx through {x_activation} needs x_pre")
            a.x_pre_stride = _rows(x_pre, "x_pre", index, (rows, k), dt)
            a.x_pre = x_pre.data_ptr()
    grad_dt = None
    if dw is not None:
        if x is None:
            raise ValueError("dw needs x")
        a.x_stride = _rows(x, "x", index, (rows, k), dt)
        a.x = x.data_ptr()
        _, _, _, a.dw_stride, a.dw_group_stride = _weight(dw, "dw", index, _FLOATS)
        if dw.shape != weight.shape:
            raise ValueError(f"dw has shape {tuple(dw.shape)}, expected {tuple(weight.shape)}")
        a.dw, grad_dt = dw.data_ptr(), dw.dtype
    if db is not None:
        shape = (groups, n) if grouped else (n,)
        _tensor(db, "db", index, shape, _FLOATS if grad_dt is None else grad_dt)
        _dense(db, "db", index, shape, db.dtype)
        a.db, grad_dt = db.data_ptr(), db.dtype
    a.grad_dtype = _DT_CODE[dt if grad_dt is None else grad_dt]
    lib, ref, size = load_library(), ctypes.byref(a), ctypes.c_size_t(0)
    _check_workspace(workspace, dy.device)
    on = _Launch(index, stream)
    _check(lib.linear_grad_workspace_bytes(ref, ctypes.byref(size)))
    ws, ws_bytes, _keep = on.workspace(workspace, size.value)
    on.call(lib.linear_grad, ref, ws, ws_bytes)
    return dx, dw, db


def linear_grad_workspace(rows: int, w: torch.Tensor, activation: str = "none", dw: bool = True, db: bool = False,
                          dtype: Optional[torch.dtype] = None) -> torch.Tensor:
    """A workspace for ``linear_grad`` over up to ``rows`` rows, to be used
    again and again (calls that share one must be ordered)."""
    groups, n, k, _, _ = _weight(w, "w", None, _FLOATS)
    dt = _DT_CODE[w.dtype if dtype is None else dtype]
    nbytes = ctypes.c_size_t(0)
    a = LinearGradArgs(rows=rows, in_=k, out=n, groups=groups, offsets=1, dtype=dt, activation=_activation(activation))
    a.dw, a.db = (1 if dw else None), (1 if db else None)
    _check(load_library().linear_grad_workspace_bytes(ctypes.byref(a), ctypes.byref(nbytes)))
    return torch.empty(max(nbytes.value, 256), dtype=torch.uint8, device=w.device)
