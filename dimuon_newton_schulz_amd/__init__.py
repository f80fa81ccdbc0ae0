"""Python binding of libmuon_mi355x.so (the MI355X Muon / Dimuon step, AdamW, the gradient norm and the experts' layers).

Argument marshalling only: tensors are turned into device pointers and
shapes, and every step of the method runs in the library's HIP kernels.  The
library must be built (``python -m dimuon_newton_schulz_amd.build``); there
is no fallback.

Entry points mirror the C ABI in ``include/muon_mi355x.h``:
``muon_step``, ``dimuon_step``, ``muon_workspace_bytes``,
``muon_status_string``; ``adamw_step``, ``AdamWPlan`` (AdamW for the
parameters Muon does not take, moments in 32 or 8 bits); ``grad_norm``,
``GradNormPlan`` (global gradient norm and clip coefficient, which the steps
take as ``grad_scale``); in ``experts``: ``expert_sort``, ``expert_gather``,
``expert_combine`` and its gradient, ``linear`` and ``linear_grad`` (the
experts' layers, whose weight gradients the steps read).
"""

from __future__ import annotations

import ctypes
import os
from dataclasses import dataclass
from typing import List, Optional, Sequence

import torch  # loads the HIP runtime the library then shares

LIB_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), "libmuon_mi355x.so")

MUON_F32, MUON_BF16 = 0, 1
_DT_CODE = {torch.float32: MUON_F32, torch.bfloat16: MUON_BF16}
_DT_NAME = {"f32": MUON_F32, "bf16": MUON_BF16}
MUON_CONFIG_FIELDS = 0x4D43F702   # muon_config_t.fields: grad_scale counts

STATUS_NAMES = {0: "MUON_OK", 1: "MUON_ERR_INVALID_ARG", 2: "MUON_ERR_DTYPE",
                3: "MUON_ERR_WORKSPACE", 4: "MUON_ERR_ALIAS", 5: "MUON_ERR_HIP",
                6: "MUON_ERR_UNSUPPORTED", 7: "MUON_ERR_MEMORY"}

EXPORTED_SYMBOLS = ("muon_config_default", "muon_workspace_bytes", "muon_step", "dimuon_step", "muon_step_noalloc",
                    "muon_set_launch_events", "muon_plan_create", "muon_plan_step", "muon_plan_set_lr",
                    "muon_plan_reset", "muon_plan_set_graph", "muon_plan_destroy", "muon_status_string", "muon_last_error", "muon_abi_version",
                    "adamw_config_default", "adamw_workspace_bytes", "adamw_state_elems", "adamw_step",
                    "adamw_plan_create", "adamw_plan_step", "adamw_plan_set_lr", "adamw_plan_set_step",
                    "adamw_plan_get_state", "adamw_plan_set_state", "adamw_plan_destroy",
                    "muon_grad_norm_workspace_bytes", "muon_grad_norm", "muon_grad_norm_plan_create",
                    "muon_grad_norm_plan_run", "muon_grad_norm_plan_destroy",
                    "expert_sort_workspace_bytes", "expert_sort", "expert_gather", "expert_combine",
                    "expert_combine_grad", "linear_forward", "linear_grad_workspace_bytes", "linear_grad")

LAUNCH_KINDS = {-1: "start", 0: "thin_b", 1: "momentum", 2: "condition", 3: "prescale", 4: "norm",
                5: "gram", 6: "poly", 7: "combine", 8: "postnorm", 9: "update", 10: "thin_energy",
                11: "thin_a", 12: "momentum_prescale", 13: "energy", 14: "adamw", 15: "state_get", 16: "state_set",
                17: "grad_norm", 18: "expert_sort", 19: "expert_gather", 20: "expert_combine",
                21: "expert_combine_grad", 22: "linear", 23: "linear_slope", 24: "linear_input", 25: "linear_weight",
                26: "linear_bias"}


class MuonMatrix(ctypes.Structure):
    _fields_ = [("w", ctypes.c_void_p), ("g", ctypes.c_void_p), ("mom", ctypes.c_void_p),
                ("o_out", ctypes.c_void_p), ("energy_out", ctypes.c_void_p),
                ("m", ctypes.c_int64), ("n", ctypes.c_int64),
                ("update_scale", ctypes.c_float), ("reserved0", ctypes.c_float)]


class MuonConfig(ctypes.Structure):
    _fields_ = [("lr", ctypes.c_float), ("momentum", ctypes.c_float), ("ns_steps", ctypes.c_int32),
                ("a", ctypes.c_float), ("b", ctypes.c_float), ("c", ctypes.c_float),
                ("coeff_schedule", ctypes.POINTER(ctypes.c_float)),
                ("w_dtype", ctypes.c_int32), ("g_dtype", ctypes.c_int32),
                ("mom_dtype", ctypes.c_int32), ("ns_dtype", ctypes.c_int32),
                ("dimuon_eps", ctypes.c_float), ("nesterov", ctypes.c_int32),
                ("weight_decay", ctypes.c_float), ("fields", ctypes.c_uint32),
                ("grad_scale", ctypes.c_void_p), ("reserved", ctypes.c_int32 * 1)]


class AdamWTensor(ctypes.Structure):
    _fields_ = [("w", ctypes.c_void_p), ("g", ctypes.c_void_p), ("m", ctypes.c_void_p), ("v", ctypes.c_void_p),
                ("m_scale", ctypes.c_void_p), ("v_scale", ctypes.c_void_p), ("master", ctypes.c_void_p),
                ("n", ctypes.c_int64), ("lr_scale", ctypes.c_float), ("weight_decay", ctypes.c_float)]


class AdamWCConfig(ctypes.Structure):
    _fields_ = [("beta1", ctypes.c_double), ("beta2", ctypes.c_double), ("lr", ctypes.c_float),
                ("eps", ctypes.c_float), ("seed", ctypes.c_uint64), ("grad_scale", ctypes.c_void_p),
                ("w_dtype", ctypes.c_int32), ("g_dtype", ctypes.c_int32), ("state", ctypes.c_int32),
                ("rounding", ctypes.c_int32), ("reserved", ctypes.c_int32 * 4)]


class MuonGrad(ctypes.Structure):
    _fields_ = [("g", ctypes.c_void_p), ("n", ctypes.c_int64), ("dtype", ctypes.c_int32),
                ("reserved0", ctypes.c_int32)]


class MuonError(RuntimeError):
    def __init__(self, status: int, detail: str):
        self.status = status
        super().__init__(f"{STATUS_NAMES.get(status, status)}: {detail}")


_lib = None


def load_library(path: str = LIB_PATH) -> ctypes.CDLL:
    """Load the HIP library once; raise if it has not been built."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(path):
        raise RuntimeError(f"{path} is missing: build it with "
                           "`python -m dimuon_newton_schulz_amd.build`")
    lib = ctypes.CDLL(path)
    lib.muon_config_default.argtypes = [ctypes.POINTER(MuonConfig)]
    lib.muon_config_default.restype = None
    lib.muon_workspace_bytes.argtypes = [ctypes.POINTER(MuonMatrix), ctypes.c_int64,
                                         ctypes.POINTER(MuonConfig), ctypes.POINTER(ctypes.c_size_t)]
    lib.muon_workspace_bytes.restype = ctypes.c_int
    for name in ("muon_step", "dimuon_step"):
        fn = getattr(lib, name)
        fn.argtypes = [ctypes.POINTER(MuonMatrix), ctypes.c_int64, ctypes.POINTER(MuonConfig),
                       ctypes.c_void_p, ctypes.c_size_t, ctypes.c_void_p]
        fn.restype = ctypes.c_int
    lib.muon_step_noalloc.argtypes = [ctypes.POINTER(MuonMatrix), ctypes.c_int64, ctypes.POINTER(MuonConfig),
                                      ctypes.c_int32, ctypes.c_void_p]
    lib.muon_step_noalloc.restype = ctypes.c_int
    lib.muon_set_launch_events.argtypes = [ctypes.c_void_p, ctypes.POINTER(ctypes.c_int32), ctypes.c_int32]
    lib.muon_set_launch_events.restype = ctypes.c_int32
    lib.muon_plan_create.argtypes = [ctypes.POINTER(MuonMatrix), ctypes.c_int64, ctypes.POINTER(MuonConfig),
                                     ctypes.c_int32, ctypes.c_void_p, ctypes.c_size_t, ctypes.c_void_p,
                                     ctypes.POINTER(ctypes.c_void_p)]
    lib.muon_plan_create.restype = ctypes.c_int
    lib.muon_plan_step.argtypes = [ctypes.c_void_p, ctypes.c_void_p]
    lib.muon_plan_step.restype = ctypes.c_int
    lib.muon_plan_set_lr.argtypes = [ctypes.c_void_p, ctypes.c_float]
    lib.muon_plan_set_lr.restype = ctypes.c_int
    lib.muon_plan_reset.argtypes = [ctypes.c_void_p]
    lib.muon_plan_reset.restype = ctypes.c_int
    lib.muon_plan_set_graph.argtypes = [ctypes.c_void_p, ctypes.c_int32]
    lib.muon_plan_set_graph.restype = ctypes.c_int
    lib.muon_plan_destroy.argtypes = [ctypes.c_void_p]
    lib.muon_plan_destroy.restype = None
    lib.adamw_config_default.argtypes = [ctypes.POINTER(AdamWCConfig)]
    lib.adamw_config_default.restype = None
    batch = [ctypes.POINTER(AdamWTensor), ctypes.c_int64]
    cfg_p, ws, vp = ctypes.POINTER(AdamWCConfig), [ctypes.c_void_p, ctypes.c_size_t], ctypes.c_void_p
    grads = [ctypes.POINTER(MuonGrad), ctypes.c_int64]
    norm = [*grads, ctypes.c_float, vp, vp, *ws, vp]
    for name, args in (("adamw_workspace_bytes", [*batch, cfg_p, ctypes.POINTER(ctypes.c_size_t)]),
                       ("adamw_state_elems", [*batch, ctypes.POINTER(ctypes.c_int64)]),
                       ("adamw_step", [*batch, cfg_p, ctypes.c_int64, *ws, vp]),
                       ("adamw_plan_create", [*batch, cfg_p, ctypes.c_int64, *ws, vp, ctypes.POINTER(vp)]),
                       ("adamw_plan_step", [vp, vp]),
                       ("adamw_plan_set_lr", [vp, ctypes.c_float, vp]),
                       ("adamw_plan_set_step", [vp, ctypes.c_int64, vp]),
                       ("adamw_plan_get_state", [vp, vp, vp, ctypes.c_int32, vp]),
                       ("adamw_plan_set_state", [vp, vp, vp, ctypes.c_int32, vp]),
                       ("muon_grad_norm_workspace_bytes", [*grads, ctypes.POINTER(ctypes.c_size_t)]),
                       ("muon_grad_norm", norm),
                       ("muon_grad_norm_plan_create", [*norm, ctypes.POINTER(vp)]),
                       ("muon_grad_norm_plan_run", [vp, vp])):
        fn = getattr(lib, name)
        fn.argtypes, fn.restype = args, ctypes.c_int
    for name in ("adamw_plan_destroy", "muon_grad_norm_plan_destroy"):
        getattr(lib, name).argtypes, getattr(lib, name).restype = [vp], None
    experts.bind(lib)
    lib.muon_status_string.argtypes = [ctypes.c_int]
    lib.muon_status_string.restype = ctypes.c_char_p
    lib.muon_last_error.argtypes = []
    lib.muon_last_error.restype = ctypes.c_char_p
    lib.muon_abi_version.argtypes = []
    lib.muon_abi_version.restype = ctypes.c_int32
    _lib = lib
    return lib


def muon_status_string(status: int) -> str:
    return load_library().muon_status_string(status).decode()


def _check(status: int):
    if status != 0:
        lib = load_library()
        raise MuonError(status, lib.muon_last_error().decode() or lib.muon_status_string(status).decode())


def _scalar_ptr(t: Optional[torch.Tensor]) -> Optional[int]:
    """Pointer of a grad_scale: one float32 on the device (None: no scale)."""
    if t is None:
        return None
    if t.dtype != torch.float32 or t.numel() != 1 or not t.is_cuda:
        raise ValueError(f"grad_scale must be one float32 on the GPU, got {t.dtype} {tuple(t.shape)} on {t.device}")
    return t.data_ptr()


@dataclass
class StepConfig:
    """Mirror of muon_config_t with the library's defaults."""
    lr: float = 0.02
    momentum: float = 0.95
    ns_steps: int = 5
    a: float = 3.4445
    b: float = -4.7750
    c: float = 2.0315
    coeff_schedule: Optional[Sequence[Sequence[float]]] = None
    w_dtype: str = "bf16"
    g_dtype: str = "bf16"
    mom_dtype: str = "bf16"
    ns_dtype: str = "bf16"
    dimuon_eps: float = 1e-4
    nesterov: bool = False
    weight_decay: float = 0.0
    grad_scale: Optional[torch.Tensor] = None   # one float32 on the device, e.g. grad_norm(...)[1:]

    def to_c(self):
        cfg = MuonConfig()
        cfg.lr, cfg.momentum, cfg.ns_steps = self.lr, self.momentum, self.ns_steps
        cfg.a, cfg.b, cfg.c = self.a, self.b, self.c
        keep = None
        if self.coeff_schedule is not None:
            flat = [float(v) for row in self.coeff_schedule for v in row]
            keep = (ctypes.c_float * len(flat))(*flat)
            cfg.coeff_schedule = ctypes.cast(keep, ctypes.POINTER(ctypes.c_float))
        cfg.w_dtype = _DT_NAME[self.w_dtype]
        cfg.g_dtype = _DT_NAME[self.g_dtype]
        cfg.mom_dtype = _DT_NAME[self.mom_dtype]
        cfg.ns_dtype = _DT_NAME[self.ns_dtype]
        cfg.dimuon_eps = self.dimuon_eps
        cfg.nesterov = 1 if self.nesterov else 0
        cfg.weight_decay = self.weight_decay
        cfg.fields = MUON_CONFIG_FIELDS
        cfg.grad_scale = _scalar_ptr(self.grad_scale)
        return cfg, keep


@dataclass
class Param:
    """One matrix of a batch: weight, gradient and momentum tensors."""
    w: torch.Tensor
    g: torch.Tensor
    mom: torch.Tensor
    o_out: Optional[torch.Tensor] = None
    energy_out: Optional[torch.Tensor] = None
    update_scale: float = 1.0


def _ptr(t: Optional[torch.Tensor]) -> Optional[int]:
    return None if t is None else t.data_ptr()


def _marshal(params: Sequence[Param]):
    arr = (MuonMatrix * len(params))()
    for i, p in enumerate(params):
        if p.w.dim() != 2:
            raise ValueError(f"matrix {i}: expected a 2-D weight, got {tuple(p.w.shape)}")
        for name in ("w", "g", "mom", "o_out", "energy_out"):
            t = getattr(p, name)
            if t is not None and not t.is_contiguous():
                raise ValueError(f"matrix {i}: {name} must be contiguous")
        m, n = p.w.shape
        if tuple(p.g.shape) != (m, n) or tuple(p.mom.shape) != (m, n):
            raise ValueError(f"matrix {i}: w, g and mom shapes differ")
        if p.o_out is not None and (tuple(p.o_out.shape) != (m, n) or p.o_out.dtype != torch.float32):
            raise ValueError(f"matrix {i}: o_out must be float32 {m}x{n}")
        if p.energy_out is not None and (p.energy_out.numel() != m + n or p.energy_out.dtype != torch.float32):
            raise ValueError(f"matrix {i}: energy_out must be float32 with m+n elements")
        arr[i].w, arr[i].g, arr[i].mom = _ptr(p.w), _ptr(p.g), _ptr(p.mom)
        arr[i].o_out, arr[i].energy_out = _ptr(p.o_out), _ptr(p.energy_out)
        arr[i].m, arr[i].n = m, n
        arr[i].update_scale = float(p.update_scale)
    return arr


def config_for(params: Sequence[Param], ns_dtype: str = "bf16", **kw) -> StepConfig:
    """StepConfig whose w/g/mom dtypes are those of the first matrix."""
    p = params[0]
    name = {torch.float32: "f32", torch.bfloat16: "bf16"}
    return StepConfig(w_dtype=name[p.w.dtype], g_dtype=name[p.g.dtype], mom_dtype=name[p.mom.dtype],
                      ns_dtype=ns_dtype, **kw)


def _check_dtypes(params: Sequence[Param], cfg: StepConfig):
    want = {"w": _DT_NAME[cfg.w_dtype], "g": _DT_NAME[cfg.g_dtype], "mom": _DT_NAME[cfg.mom_dtype]}
    for i, p in enumerate(params):
        for name, code in want.items():
            t = getattr(p, name)
            if _DT_CODE.get(t.dtype) != code:
                raise ValueError(f"matrix {i}: {name} is {t.dtype}, config says {getattr(cfg, name + '_dtype')}")
    _check_scale_device(params, cfg)


def _check_scale_device(params, cfg):
    if cfg.grad_scale is not None and params and cfg.grad_scale.device != params[0].w.device:
        raise ValueError(f"grad_scale is on {cfg.grad_scale.device}, the batch on {params[0].w.device}")


def muon_workspace_bytes(params: Sequence[Param], cfg: StepConfig) -> int:
    lib = load_library()
    arr = _marshal(params)
    c, _keep = cfg.to_c()
    out = ctypes.c_size_t(0)
    _check(lib.muon_workspace_bytes(arr, len(params), ctypes.byref(c), ctypes.byref(out)))
    return int(out.value)


def workspace_for(params: Sequence[Param], cfg: StepConfig, device=None) -> torch.Tensor:
    nbytes = muon_workspace_bytes(params, cfg)
    dev = device if device is not None else params[0].w.device
    return torch.empty(max(nbytes, 256), dtype=torch.uint8, device=dev)


def _check_workspace(workspace, device, any_dtype=False):
    """A caller's workspace (None: there is none): one stretch of memory on
    the batch's device, of bytes.  Muon's calls take any dtype, and of its
    size the element count."""
    if workspace is None:
        return
    if not isinstance(workspace, torch.Tensor) or not workspace.is_contiguous():
        raise ValueError("workspace must be a contiguous tensor")
    if workspace.device != device:
        raise ValueError(f"workspace is on {workspace.device}, the batch on {device}")
    if not any_dtype and workspace.dtype != torch.uint8:
        raise ValueError(f"workspace must be uint8, got {workspace.dtype}")


def _torch_stream(stream, device):
    """The launch stream as a torch stream object (None: the current stream)."""
    if stream is None:
        return torch.cuda.current_stream(device)
    if hasattr(stream, "cuda_stream"):
        return stream
    return torch.cuda.ExternalStream(int(stream), device=device)


def _step(fn_name: str, params: Sequence[Param], cfg: StepConfig, workspace: Optional[torch.Tensor],
          stream=None):
    lib = load_library()
    _check_dtypes(params, cfg)
    arr = _marshal(params)
    c, _keep = cfg.to_c()
    device = params[0].w.device
    _check_workspace(workspace, device, any_dtype=True)
    ts = _torch_stream(stream, device)
    if workspace is None:
        workspace = workspace_for(params, cfg)
        # Allocated on the current stream; if the kernels run on another one,
        # the caching allocator must not hand the block out again before they
        # finish.
        if ts != torch.cuda.current_stream(device):
            workspace.record_stream(ts)
    fn = getattr(lib, fn_name)
    with torch.cuda.device(device):
        _check(fn(arr, len(params), ctypes.byref(c), ctypes.c_void_p(workspace.data_ptr()),
                  ctypes.c_size_t(workspace.numel()), ctypes.c_void_p(ts.cuda_stream)))
    return workspace


def muon_step(params: Sequence[Param], cfg: StepConfig, workspace: Optional[torch.Tensor] = None,
              stream=None) -> torch.Tensor:
    """One Muon step over the batch (asynchronous on ``stream``).  Returns the workspace."""
    return _step("muon_step", params, cfg, workspace, stream)


def dimuon_step(params: Sequence[Param], cfg: StepConfig, workspace: Optional[torch.Tensor] = None,
                stream=None) -> torch.Tensor:
    """One Dimuon step over the batch (asynchronous on ``stream``).  Returns the workspace."""
    return _step("dimuon_step", params, cfg, workspace, stream)


NOALLOC_MAX_BYTES = 64 << 20   # MUON_NOALLOC_MAX_BYTES


def muon_step_noalloc(params: Sequence[Param], cfg: StepConfig, dimuon: bool, stream=None) -> None:
    """One Muon (dimuon False) or Dimuon step without a workspace argument:
    the library's static device scratch serves (muon_step_noalloc).  Nothing
    is allocated; calls on one GPU must be ordered (they share the scratch)."""
    lib = load_library()
    _check_dtypes(params, cfg)
    arr = _marshal(params)
    c, _keep = cfg.to_c()
    device = params[0].w.device
    ts = _torch_stream(stream, device)
    with torch.cuda.device(device):
        _check(lib.muon_step_noalloc(arr, len(params), ctypes.byref(c), 1 if dimuon else 0,
                                     ctypes.c_void_p(ts.cuda_stream)))


class LaunchTimer:
    """Per-launch HIP events for one step at a time (timing only).

    ``with LaunchTimer(capacity) as t: step(...); ...; t.durations()`` returns
    [(kind, ms)] for the launches of the last step, measured on its stream."""

    def __init__(self, capacity: int = 256):
        self.capacity = capacity
        self.events = [torch.cuda.Event(enable_timing=True) for _ in range(capacity)]
        # torch.cuda.Event creates the HIP event lazily; record once to create it.
        for e in self.events:
            e.record()
        self.handles = (ctypes.c_void_p * capacity)(*[e.cuda_event for e in self.events])
        self.kinds = (ctypes.c_int32 * capacity)()

    def __enter__(self):
        load_library().muon_set_launch_events(self.handles, self.kinds, self.capacity)
        return self

    def __exit__(self, *exc):
        load_library().muon_set_launch_events(None, None, 0)

    def durations(self, count: int):
        """(kind name, ms) of launches 1..count-1 of the last step (after synchronising)."""
        out = []
        for i in range(1, count):
            out.append((LAUNCH_KINDS[self.kinds[i]], self.events[i - 1].elapsed_time(self.events[i])))
        return out

    def recorded(self) -> int:
        lib = load_library()
        n = lib.muon_set_launch_events(self.handles, self.kinds, self.capacity)
        return n


def _own(obj):
    """Copy of a Param, AdamWParam or config for a plan: the same memory, in
    tensors that the caller's later assignments (to the object's fields, or
    to a tensor's .data) do not reach."""
    own = object.__new__(type(obj))
    own.__dict__.update((k, v.detach() if isinstance(v, torch.Tensor) else v) for k, v in obj.__dict__.items())
    return own


# The current stream's handle without a Stream object around it (0.1 instead
# of 2 us, of the 6 that a small step took), where torch has it.
_current_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _stream_handle(stream, device):
    if stream is None:
        if _current_raw_stream is not None and device.index is not None:
            return _current_raw_stream(device.index)
        stream = torch.cuda.current_stream(device)
    return stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)


class Plan:
    """A prepared batch (muon_plan_t): validated and uploaded once, then
    stepped repeatedly.  Keeps the tensors and the workspace alive, and goes on
    reading the memory it was created with: gradients must stay where they are
    (``zero_grad(set_to_none=False)``, or flat gradient buffers), since a new
    ``p.grad`` is memory that the plan does not know.  A graph that holds a
    captured step needs the plan as long as it is replayed."""

    def __init__(self, params: Sequence[Param], cfg: StepConfig, dimuon: bool,
                 workspace: Optional[torch.Tensor] = None, stream=None):
        lib = load_library()
        _check_dtypes(params, cfg)
        self.params = [_own(p) for p in params]
        self.cfg = _own(cfg)
        self.device = params[0].w.device
        _check_workspace(workspace, self.device, any_dtype=True)
        self.workspace = workspace if workspace is not None else workspace_for(params, cfg)
        arr = _marshal(params)
        c, keep = cfg.to_c()
        handle = ctypes.c_void_p(0)
        with torch.cuda.device(self.device):
            _check(lib.muon_plan_create(arr, len(params), ctypes.byref(c), 1 if dimuon else 0,
                                        ctypes.c_void_p(self.workspace.data_ptr()),
                                        ctypes.c_size_t(self.workspace.numel()),
                                        ctypes.c_void_p(_stream_handle(stream, self.device)),
                                        ctypes.byref(handle)))
        self._handle = handle
        self._lib = lib

    def step(self, stream=None):
        _check(self._lib.muon_plan_step(self._handle, ctypes.c_void_p(_stream_handle(stream, self.device))))

    def set_lr(self, lr: float):
        _check(self._lib.muon_plan_set_lr(self._handle, lr))

    def reset(self):
        """Call after writing to the momentum buffers outside the plan."""
        _check(self._lib.muon_plan_reset(self._handle))

    def set_graph(self, enable: bool = True):
        """Replay the launch sequence as a HIP graph (muon_plan_set_graph)."""
        _check(self._lib.muon_plan_set_graph(self._handle, 1 if enable else 0))

    def close(self):
        if self._handle:
            self._lib.muon_plan_destroy(self._handle)
            self._handle = ctypes.c_void_p(0)

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


ADAMW_BLOCK = 256   # elements that share a scale of the 8-bit moments
_STATE_CODE = {"f32": 0, "block8": 1}
_ROUNDING_CODE = {"nearest": 0, "stochastic": 1}


@dataclass
class AdamWConfig:
    """Mirror of adamw_config_t with the library's defaults."""
    lr: float = 1e-3
    beta1: float = 0.9
    beta2: float = 0.999
    eps: float = 1e-8
    w_dtype: str = "bf16"
    g_dtype: str = "bf16"
    state: str = "f32"                          # "f32" or "block8"
    rounding: str = "stochastic"                # of 8-bit codes: "nearest" or "stochastic"
    seed: int = 0
    grad_scale: Optional[torch.Tensor] = None   # one float32 on the device, e.g. grad_norm(...)[1:]

    def to_c(self) -> AdamWCConfig:
        c = AdamWCConfig()
        c.beta1, c.beta2, c.lr, c.eps = self.beta1, self.beta2, self.lr, self.eps
        c.seed = self.seed & 0xFFFFFFFFFFFFFFFF
        c.grad_scale = _scalar_ptr(self.grad_scale)
        c.w_dtype, c.g_dtype = _DT_NAME[self.w_dtype], _DT_NAME[self.g_dtype]
        c.state, c.rounding = _STATE_CODE[self.state], _ROUNDING_CODE[self.rounding]
        return c


@dataclass
class AdamWParam:
    """One tensor of an AdamW batch, of any shape: weight, gradient and
    moments.  32-bit moments: float32 m and v of w's size.  8-bit moments: m
    float8_e4m3fn and v uint8 of w's size, m_scale and v_scale one float32 per
    ADAMW_BLOCK elements."""
    w: torch.Tensor
    g: torch.Tensor
    m: torch.Tensor
    v: torch.Tensor
    m_scale: Optional[torch.Tensor] = None
    v_scale: Optional[torch.Tensor] = None
    master: Optional[torch.Tensor] = None   # float32 master weights (bf16 w)
    lr_scale: float = 1.0
    weight_decay: float = 0.0


def adamw_param(w: torch.Tensor, g: torch.Tensor, state: str = "f32", master: bool = False,
                lr_scale: float = 1.0, weight_decay: float = 0.0) -> AdamWParam:
    """AdamWParam with new (zero) moments and, with `master`, a float32 copy of w."""
    kw = {"lr_scale": lr_scale, "weight_decay": weight_decay,
          "master": w.detach().float() if master else None}
    if state == "f32":
        return AdamWParam(w, g, torch.zeros_like(w, dtype=torch.float32),
                          torch.zeros_like(w, dtype=torch.float32), **kw)
    if state != "block8":
        raise ValueError(f"state must be one of {sorted(_STATE_CODE)}, got {state!r}")
    codes = [torch.zeros(w.shape, dtype=torch.uint8, device=w.device) for _ in range(2)]
    scales = [torch.zeros(-(-w.numel() // ADAMW_BLOCK), device=w.device) for _ in range(2)]
    return AdamWParam(w, g, codes[0].view(torch.float8_e4m3fn), codes[1], *scales, **kw)


def adamw_config_for(params: Sequence[AdamWParam], **kw) -> AdamWConfig:
    """AdamWConfig whose dtypes and moment format are those of the first tensor."""
    p = params[0]
    name = {torch.float32: "f32", torch.bfloat16: "bf16"}
    return AdamWConfig(w_dtype=name[p.w.dtype], g_dtype=name[p.g.dtype],
                       state="f32" if p.m.dtype == torch.float32 else "block8", **kw)


def _marshal_adamw(params: Sequence[AdamWParam], cfg: AdamWConfig):
    block8 = cfg.state == "block8"
    want = {"w": _DT_NAME[cfg.w_dtype], "g": _DT_NAME[cfg.g_dtype]}
    state_dt = {"m": torch.float8_e4m3fn if block8 else torch.float32, "v": torch.uint8 if block8 else torch.float32}
    arr = (AdamWTensor * len(params))()
    for i, p in enumerate(params):
        n = p.w.numel()
        for name in ("w", "g", "m", "v", "m_scale", "v_scale", "master"):
            t = getattr(p, name)
            scale = name.endswith("_scale")
            if t is None:
                if name == "master" or (scale and not block8):
                    continue
                raise ValueError(f"tensor {i}: {name} is missing")
            if not t.is_contiguous():
                raise ValueError(f"tensor {i}: {name} must be contiguous")
            if t.device != params[0].w.device:
                raise ValueError(f"tensor {i}: {name} is on {t.device}, the batch on {params[0].w.device}")
            if t.numel() != (-(-n // ADAMW_BLOCK) if scale else n):
                raise ValueError(f"tensor {i}: {name} has {t.numel()} elements for {n} weights")
            if name in want:
                if _DT_CODE.get(t.dtype) != want[name]:
                    raise ValueError(f"tensor {i}: {name} is {t.dtype}, config says {getattr(cfg, name + '_dtype')}")
            elif t.dtype != state_dt.get(name, torch.float32):
                raise ValueError(f"tensor {i}: {name} is {t.dtype}, expected {state_dt.get(name, torch.float32)}")
            setattr(arr[i], name, t.data_ptr())
        arr[i].n, arr[i].lr_scale, arr[i].weight_decay = n, float(p.lr_scale), float(p.weight_decay)
    _check_scale_device(params, cfg)
    return arr


def _workspace_on(workspace, nbytes, device, ts):
    """The caller's workspace, or a new one that the allocator keeps until
    `ts` is done with it.  `ts` first waits for the current stream, where a new
    block may have been in use a moment ago."""
    current = torch.cuda.current_stream(device)
    if ts != current:
        ts.wait_stream(current)
    if workspace is None:
        workspace = torch.empty(max(nbytes, 256), dtype=torch.uint8, device=device)
        if ts != current:
            workspace.record_stream(ts)
    return workspace


def _gpu_device(device) -> torch.device:
    if device.type != "cuda":
        raise ValueError(f"the tensors are on {device}: they must be on the GPU")
    return device


def adamw_workspace_bytes(params: Sequence[AdamWParam], cfg: AdamWConfig) -> int:
    lib = load_library()
    arr, out = _marshal_adamw(params, cfg), ctypes.c_size_t(0)
    _check(lib.adamw_workspace_bytes(arr, len(params), ctypes.byref(cfg.to_c()), ctypes.byref(out)))
    return int(out.value)


def adamw_step(params: Sequence[AdamWParam], cfg: AdamWConfig, step: int,
               workspace: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """AdamW step number `step` (from 1 on) over the batch, asynchronous on
    ``stream``.  Returns the workspace.  Refused under stream capture."""
    lib = load_library()
    arr, c = _marshal_adamw(params, cfg), cfg.to_c()
    nbytes = ctypes.c_size_t(0)
    _check(lib.adamw_workspace_bytes(arr, len(params), ctypes.byref(c), ctypes.byref(nbytes)))
    _check_workspace(workspace, params[0].w.device)
    device = _gpu_device(params[0].w.device)
    ts = _torch_stream(stream, device)
    if workspace is None:
        workspace = _workspace_on(None, nbytes.value, device, ts)
    with torch.cuda.device(device):
        _check(lib.adamw_step(arr, len(params), ctypes.byref(c), step, workspace.data_ptr(), workspace.numel(),
                              ts.cuda_stream))
    return workspace


class AdamWPlan:
    """A prepared AdamW batch (adamw_plan_t): validated and uploaded once,
    then stepped repeatedly.  Keeps the tensors and the workspace alive, and
    goes on reading the memory it was created with (gradients must stay where
    they are, as for ``Plan``).  ``step()`` can be captured into a graph: every
    replay is the next step, and needs the plan."""

    def __init__(self, params: Sequence[AdamWParam], cfg: AdamWConfig, step: int = 0,
                 workspace: Optional[torch.Tensor] = None, stream=None):
        """`step`: the number of steps the moments have taken (0 for new ones)."""
        self._handle = ctypes.c_void_p(0)
        self._lib = lib = load_library()
        arr, c = _marshal_adamw(params, cfg), cfg.to_c()
        nbytes, elems = ctypes.c_size_t(0), ctypes.c_int64(0)
        _check(lib.adamw_workspace_bytes(arr, len(params), ctypes.byref(c), ctypes.byref(nbytes)))
        _check(lib.adamw_state_elems(arr, len(params), ctypes.byref(elems)))
        self.params, self.cfg = [_own(p) for p in params], _own(cfg)
        _check_workspace(workspace, params[0].w.device)
        self.device = _gpu_device(params[0].w.device)
        self.state_elems = elems.value
        ts = _torch_stream(stream, self.device)
        self.workspace = _workspace_on(workspace, nbytes.value, self.device, ts)
        with torch.cuda.device(self.device):
            _check(lib.adamw_plan_create(arr, len(params), ctypes.byref(c), step, self.workspace.data_ptr(),
                                         self.workspace.numel(), ts.cuda_stream, ctypes.byref(self._handle)))

    def step(self, stream=None):
        _check(self._lib.adamw_plan_step(self._handle, _stream_handle(stream, self.device)))

    def set_lr(self, lr: float, stream=None):
        _check(self._lib.adamw_plan_set_lr(self._handle, lr, _stream_handle(stream, self.device)))

    def set_step(self, step: int, stream=None):
        """Number of steps done, for resuming."""
        _check(self._lib.adamw_plan_set_step(self._handle, step, _stream_handle(stream, self.device)))

    def state_offsets(self) -> List[int]:
        """Where every tensor's values start in the buffers of get_state and set_state."""
        out, at = [], 0
        for p in self.params:
            out.append(at)
            at += -(-p.w.numel() // ADAMW_BLOCK) * ADAMW_BLOCK
        return out

    def _values(self, m, v):
        for name, t in (("m", m), ("v", v)):
            if t.dtype not in _DT_CODE or t.dtype != m.dtype:
                raise ValueError(f"{name} must be float32 or bfloat16, both of one dtype, got {t.dtype}")
            if t.numel() != self.state_elems or not t.is_contiguous() or t.device != self.device:
                raise ValueError(f"{name} must be {self.state_elems} contiguous elements on {self.device}")
        return m.data_ptr(), v.data_ptr(), _DT_CODE[m.dtype]

    def get_state(self, m: Optional[torch.Tensor] = None, v: Optional[torch.Tensor] = None,
                  dtype: torch.dtype = torch.float32, stream=None):
        """The moments as values, (m, v): flat buffers of state_elems elements
        (new ones of `dtype`, zero in the gaps, if none are given)."""
        if (m is None) != (v is None):
            raise ValueError("give both m and v, or neither")
        if m is None:
            with torch.cuda.stream(_torch_stream(stream, self.device)):
                m, v = (torch.zeros(self.state_elems, dtype=dtype, device=self.device) for _ in range(2))
        _check(self._lib.adamw_plan_get_state(self._handle, *self._values(m, v),
                                              _stream_handle(stream, self.device)))
        return m, v

    def set_state(self, m: torch.Tensor, v: torch.Tensor, stream=None):
        """Loads the moments from values laid out as get_state's."""
        _check(self._lib.adamw_plan_set_state(self._handle, *self._values(m, v),
                                              _stream_handle(stream, self.device)))

    def close(self):
        if self._handle:
            self._lib.adamw_plan_destroy(self._handle)
            self._handle = ctypes.c_void_p(0)

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


def _marshal_grads(grads: Sequence[torch.Tensor], out, tensor_norms):
    arr = (MuonGrad * len(grads))()
    for i, g in enumerate(grads):
        if g.dtype not in _DT_CODE:
            raise ValueError(f"tensor {i}: gradients are float32 or bfloat16, got {g.dtype}")
        if not g.is_contiguous():
            raise ValueError(f"tensor {i}: the gradient must be contiguous")
        if g.device != grads[0].device:
            raise ValueError(f"tensor {i} is on {g.device}, the batch on {grads[0].device}")
        arr[i].g, arr[i].n, arr[i].dtype = g.data_ptr(), g.numel(), _DT_CODE[g.dtype]
    for name, t, n in (("out", out, 2), ("tensor_norms", tensor_norms, len(grads))):
        if t is not None and (t.dtype != torch.float32 or t.numel() != n or not t.is_contiguous()
                              or t.device != grads[0].device):
            raise ValueError(f"{name} must be {n} contiguous float32 on {grads[0].device}")
    return arr


def grad_norm(grads: Sequence[torch.Tensor], max_norm: float = float("inf"), out: Optional[torch.Tensor] = None,
              tensor_norms: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None,
              stream=None) -> torch.Tensor:
    """Global gradient norm and clip coefficient: two float32 on the device,
    (N, 1 if N <= max_norm else max_norm / N).  Pass ``[1:]`` of it as
    grad_scale to the steps.  Refused under stream capture."""
    if not grads:
        raise ValueError("no gradients")
    _check_workspace(workspace, grads[0].device)
    device = _gpu_device(grads[0].device)
    ts = _torch_stream(stream, device)
    if out is None:
        with torch.cuda.stream(ts):
            out = torch.empty(2, device=device)
    lib = load_library()
    arr, nbytes = _marshal_grads(grads, out, tensor_norms), ctypes.c_size_t(0)
    _check(lib.muon_grad_norm_workspace_bytes(arr, len(grads), ctypes.byref(nbytes)))
    if workspace is None:
        workspace = _workspace_on(None, nbytes.value, device, ts)
    with torch.cuda.device(device):
        _check(lib.muon_grad_norm(arr, len(grads), max_norm, out.data_ptr(), _ptr(tensor_norms),
                                  workspace.data_ptr(), workspace.numel(), ts.cuda_stream))
    return out


class GradNormPlan:
    """A prepared global gradient norm (muon_grad_norm_plan_t): ``run()``
    launches one kernel and returns ``out``.  Keeps the tensors alive, and goes
    on reading the memory it was created with (gradients must stay where they
    are, as for ``Plan``); can be captured into a graph, which needs the plan."""

    def __init__(self, grads: Sequence[torch.Tensor], max_norm: float = float("inf"),
                 out: Optional[torch.Tensor] = None, tensor_norms: Optional[torch.Tensor] = None,
                 workspace: Optional[torch.Tensor] = None, stream=None):
        if not grads:
            raise ValueError("no gradients")
        self._handle = ctypes.c_void_p(0)
        self._lib = lib = load_library()
        _check_workspace(workspace, grads[0].device)
        self.device = _gpu_device(grads[0].device)
        self.grads, self.tensor_norms = [g.detach() for g in grads], tensor_norms
        self.out = out if out is not None else torch.zeros(2, device=self.device)
        self._written = [t.detach() for t in (self.out, tensor_norms) if t is not None]
        arr, nbytes = _marshal_grads(grads, self.out, tensor_norms), ctypes.c_size_t(0)
        _check(lib.muon_grad_norm_workspace_bytes(arr, len(grads), ctypes.byref(nbytes)))
        ts = _torch_stream(stream, self.device)
        self.workspace = _workspace_on(workspace, nbytes.value, self.device, ts)
        with torch.cuda.device(self.device):
            _check(lib.muon_grad_norm_plan_create(arr, len(grads), max_norm, self.out.data_ptr(),
                                                  _ptr(tensor_norms), self.workspace.data_ptr(),
                                                  self.workspace.numel(), ts.cuda_stream,
                                                  ctypes.byref(self._handle)))

    def run(self, stream=None) -> torch.Tensor:
        _check(self._lib.muon_grad_norm_plan_run(self._handle, _stream_handle(stream, self.device)))
        return self.out

    def close(self):
        if self._handle:
            self._lib.muon_grad_norm_plan_destroy(self._handle)
            self._handle = ctypes.c_void_p(0)

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


from . import experts  # noqa: E402 (uses what is defined above)
from .experts import (ACTIVATIONS, ExpertRoutes, expert_combine, expert_combine_grad, expert_gather,  # noqa: E402
                      expert_sort, linear, linear_grad, linear_grad_workspace)

__all__ = ["MuonMatrix", "MuonConfig", "MuonError", "StepConfig", "Param", "load_library",
           "muon_step", "dimuon_step", "muon_step_noalloc", "muon_workspace_bytes", "muon_status_string",
           "Plan", "workspace_for", "config_for", "EXPORTED_SYMBOLS", "LaunchTimer",
           "LAUNCH_KINDS", "AdamWConfig", "AdamWParam", "AdamWPlan", "adamw_param", "adamw_config_for",
           "adamw_step", "adamw_workspace_bytes", "ADAMW_BLOCK", "grad_norm", "GradNormPlan",
           "ACTIVATIONS", "ExpertRoutes", "expert_sort", "expert_gather", "expert_combine", "expert_combine_grad",
           "linear", "linear_grad", "linear_grad_workspace"]
