"""Python binding of libdq.so (include/dq.h): argument marshalling only.

Every function here has the name of the C entry point it calls.  Device
tensors are torch tensors on the handle's device (PyTorch supplies memory and
streams); host arrays are numpy.  No arithmetic of the layer happens here, and
there is no fallback: without the built library every call raises.
"""
from __future__ import annotations

import ctypes
import os
import warnings
from types import SimpleNamespace
from typing import Optional, Sequence, Tuple

import numpy as np

_HERE = os.path.dirname(os.path.abspath(__file__))
_LIB = None
_CALL = None            # the native marshalling of the small calls (csrc/binding.cpp)

DQ_F32, DQ_BF16 = 0, 1
STATUS = {0: "DQ_OK", 1: "DQ_ERR_INVALID_ARG", 2: "DQ_ERR_SHAPE", 3: "DQ_ERR_UNSUPPORTED",
          4: "DQ_ERR_OUT_OF_MEMORY", 5: "DQ_ERR_DEVICE"}

# every entry point declared in include/dq.h
EXPORTS = ("dq_last_error", "dq_status_str", "dq_lowrank_factors", "dq_prepare_weights_lowrank",
           "dq_prepare_weights", "dq_weights_destroy", "dq_weights_info", "dq_weights_export",
           "dq_qact_create", "dq_qact_create_ex", "dq_qact_destroy", "dq_qact_info", "dq_quantize_act", "dq_linear_forward",
           "dq_core_term", "dq_delta_term", "dq_linear_forward_fused", "dq_forward_form", "dq_linear", "dq_qact_export", "dq_linear_noalloc",
           "dq_prepare_weights_w6", "dq_act6_create", "dq_act6_destroy", "dq_quantize_act6", "dq_linear6_forward",
           "dq_linear6", "dq_act6_export", "dq_orbit_prepare", "dq_orbit_destroy", "dq_orbit_export",
           "dq_orbit_act_create", "dq_orbit_act_destroy", "dq_orbit_quantize_act", "dq_orbit_forward", "dq_orbit_linear",
           "dq_orbit_act_export", "dq_import_weights", "dq_rows_create", "dq_rows_destroy", "dq_linear_rows",
           "dq_linear_rows8", "dq_rmsnorm8", "dq_rope_table", "dq_norm_rope", "dq_kv_write", "dq_kv_read", "dq_attn_create",
           "dq_attn_destroy", "dq_attn_rows")
DQ_FP6_E2M3, DQ_FP6_E3M2 = 2, 3
FP6_FORMATS = {"fp6_e2m3": DQ_FP6_E2M3, "fp6_e3m2": DQ_FP6_E3M2}
NORMS = {None: 0, "head": 1, "row": 2}


class DQError(RuntimeError):
    def __init__(self, status: int, func: str, msg: str):
        super().__init__(f"{func}: {STATUS.get(status, status)}: {msg}")
        self.status = status


class Geom(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in ("T", "H", "W", "t", "h", "w")]


def library_path() -> str:
    return os.path.join(_HERE, "libdq.so")


def load():
    """Load libdq.so (raises if it has not been built), and the native
    marshalling of the small calls where torch and _dqcall.so are there; without
    it those calls take a few us more of the host."""
    global _LIB, _CALL
    if _LIB is not None:
        return _LIB
    path = library_path()
    if not os.path.exists(path):
        raise RuntimeError(f"{path} is not built; run __graft_entry__.build()")
    try:
        import torch                # (before libdq.so, which then shares the HIP runtime that torch brings)
    except ImportError:
        torch = None                # (the entry points themselves do not need it)
    lib = ctypes.CDLL(path)
    P, I32, I64, U64 = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_uint64
    PP = ctypes.POINTER(ctypes.c_void_p)
    sig = {
        "dq_last_error": ([], ctypes.c_char_p),
        "dq_status_str": ([ctypes.c_int], ctypes.c_char_p),
        "dq_lowrank_factors": ([P, ctypes.c_int, I64, I64, I32, U64, P, P], ctypes.c_int),
        "dq_prepare_weights_lowrank": ([P, ctypes.c_int, I64, I64, I32, P, P, I32, PP], ctypes.c_int),
        "dq_prepare_weights": ([P, ctypes.c_int, I64, I64, I32, U64, I32, PP], ctypes.c_int),
        "dq_weights_destroy": ([P], None),
        "dq_weights_info": ([P, P, P, P, P], ctypes.c_int),
        "dq_weights_export": ([P, P, P, P, P, P], ctypes.c_int),
        "dq_qact_create": ([P, Geom, PP], ctypes.c_int),
        "dq_qact_create_ex": ([P, Geom, I32, I32, PP], ctypes.c_int),
        "dq_qact_destroy": ([P], None),
        "dq_qact_info": ([P, P, P, P], ctypes.c_int),
        "dq_quantize_act": ([P, P, ctypes.c_int, P, P], ctypes.c_int),
        "dq_linear_forward": ([P, P, P, P], ctypes.c_int),
        "dq_core_term": ([P, P, P], ctypes.c_int),
        "dq_delta_term": ([P, P, P, P], ctypes.c_int),
        "dq_linear_forward_fused": ([P, P, P, P], ctypes.c_int),
        "dq_forward_form": ([P, P, P], ctypes.c_int),
        "dq_linear": ([P, P, ctypes.c_int, P, P, P], ctypes.c_int),
        "dq_qact_export": ([P, P, P, P, P, P, P], ctypes.c_int),
        "dq_linear_noalloc": ([P, P, ctypes.c_int, Geom, P, P], ctypes.c_int),
        "dq_prepare_weights_w6": ([P, ctypes.c_int, I64, I64, I32, P, P, I32, I32, PP], ctypes.c_int),
        "dq_act6_create": ([P, I64, PP], ctypes.c_int),
        "dq_act6_destroy": ([P], None),
        "dq_quantize_act6": ([P, P, ctypes.c_int, P, P], ctypes.c_int),
        "dq_linear6_forward": ([P, P, P, P], ctypes.c_int),
        "dq_linear6": ([P, P, ctypes.c_int, P, P, P], ctypes.c_int),
        "dq_act6_export": ([P, P, P, P, P], ctypes.c_int),
        "dq_orbit_prepare": ([P, ctypes.c_int, I64, I64, P, I32, I32, I32, PP], ctypes.c_int),
        "dq_orbit_destroy": ([P], None),
        "dq_orbit_export": ([P, P, P, P, P], ctypes.c_int),
        "dq_orbit_act_create": ([P, I64, PP], ctypes.c_int),
        "dq_orbit_act_destroy": ([P], None),
        "dq_orbit_quantize_act": ([P, P, ctypes.c_int, P, P], ctypes.c_int),
        "dq_orbit_forward": ([P, P, P, P], ctypes.c_int),
        "dq_orbit_linear": ([P, P, ctypes.c_int, P, P, P], ctypes.c_int),
        "dq_orbit_act_export": ([P, P, P, P], ctypes.c_int),
        "dq_import_weights": ([P, P, I64, I64, I32, P, P, I32, PP], ctypes.c_int),
        "dq_rows_create": ([P, I64, PP], ctypes.c_int),
        "dq_rows_destroy": ([P], None),
        "dq_linear_rows": ([P, P, ctypes.c_int, I64, I64, P, P, ctypes.c_int, I64, P], ctypes.c_int),
        "dq_linear_rows8": ([P, P, P, I64, P, P, ctypes.c_int, I64, P], ctypes.c_int),
        "dq_rmsnorm8": ([P, I64, P, I64, ctypes.c_int, P, ctypes.c_int, ctypes.c_double, I64, I64, I32, P, I64, P, P, P, I64,
                         I32, P], ctypes.c_int),
        "dq_rope_table": ([P, I32, I64, P, I32, P], ctypes.c_int),
        "dq_norm_rope": ([P, I64, ctypes.c_int, I64, I32, I32, P, P, P, I64, ctypes.c_int, I32, P], ctypes.c_int),
        "dq_kv_write": ([P, P, I64, ctypes.c_int, P, I64, P, I64, P, P, I64, I32, P, P, I64, ctypes.c_int, P, I32, P], ctypes.c_int),
        "dq_kv_read": ([P, P, I64, P, I64, P, I64, ctypes.c_int, I32, P], ctypes.c_int),
        "dq_attn_create": ([I32, PP], ctypes.c_int),
        "dq_attn_destroy": ([P], None),
        "dq_attn_rows": ([P, P, I64, P, I64, ctypes.c_int, I32, P, P, P, I64, I32, P], ctypes.c_int),
    }
    for name, (args, res) in sig.items():
        f = getattr(lib, name)
        f.argtypes = args
        f.restype = res
    _LIB = lib
    if torch is not None:
        try:
            from . import _dqcall
            _CALL = _dqcall
        except ImportError as e:
            warnings.warn(f"the small calls' native marshalling (_dqcall.so) is not there, they take a few us more: {e}; "
                          "run __graft_entry__.build()", RuntimeWarning, stacklevel=2)
    return lib


def _check(status: int, func: str):
    if status != 0:
        raise DQError(status, func, load().dq_last_error().decode())


def _ptr(a) -> ctypes.c_void_p:
    if a is None:
        return ctypes.c_void_p(None)
    if isinstance(a, np.ndarray):
        return ctypes.c_void_p(a.ctypes.data)
    return ctypes.c_void_p(a.data_ptr())


def _stream(stream) -> ctypes.c_void_p:
    if stream is None:
        import torch
        stream = torch.cuda.current_stream()
    return ctypes.c_void_p(getattr(stream, "cuda_stream", stream))


def _dtype_of(t) -> int:
    import torch
    if t.dtype == torch.bfloat16:
        return DQ_BF16
    if t.dtype == torch.float32:
        return DQ_F32
    raise TypeError(f"unsupported dtype {t.dtype}")


def _host_weight(w):
    """W^T [Co][Ci] as a contiguous CPU torch tensor; returns (tensor, dtype code)."""
    import torch
    if not isinstance(w, torch.Tensor) or w.dim() != 2:
        raise DQError(1, "weight", "the weight must be a 2-D torch tensor [Co][Ci]")
    w = w.detach().to("cpu").contiguous()
    return w, _dtype_of(w)


def _invalid(func: str, msg: str):
    raise DQError(1, func, msg)


def _device_tensor(func: str, name: str, t, shape, dtypes, device: int, align: int):
    """Checks a caller-owned device buffer before its pointer crosses the C ABI,
    which cannot see sizes: a torch tensor of one of `dtypes`, exactly `shape`,
    contiguous, on CUDA device `device`, its data `align`-byte aligned."""
    import torch
    if not isinstance(t, torch.Tensor):
        _invalid(func, f"{name} must be a torch tensor")
    if t.dtype not in dtypes:
        _invalid(func, f"{name} has dtype {t.dtype}; expected one of {[str(d) for d in dtypes]}")
    if tuple(t.shape) != tuple(shape):
        _invalid(func, f"{name} has shape {tuple(t.shape)}; expected {tuple(shape)}")
    if not t.is_contiguous():
        _invalid(func, f"{name} must be contiguous")
    if t.device.type != "cuda" or t.device.index != device:
        _invalid(func, f"{name} is on {t.device}; expected cuda:{device}")
    if t.data_ptr() % align:
        _invalid(func, f"{name} must be {align}-byte aligned")


def _check_x(func: str, w: "Weights", q: "QAct", x):
    import torch
    _device_tensor(func, "x", x, (q.N, w.Ci), (torch.bfloat16, torch.float32), w.device, 16)


def _check_y(func: str, w: "Weights", q: "QAct", y):
    import torch
    _device_tensor(func, "y", y, (q.N, w.Co), (torch.float32,), w.device, 4)


def _check_pair(func: str, w: "Weights", q: "QAct"):
    if q.weights is not w and (q.weights.Ci, q.weights.Co, q.weights.rank) != (w.Ci, w.Co, w.rank):
        _invalid(func, "the workspace was created for a different weight")


def _factor(func: str, name: str, a, shape):
    """A bf16 factor given as uint16 (or int16) bits of exactly `shape`."""
    a = np.asarray(a)
    if a.dtype not in (np.uint16, np.int16):
        _invalid(func, f"{name} must hold bf16 bits as uint16 (got {a.dtype})")
    if a.shape != tuple(shape):
        _invalid(func, f"{name} has shape {a.shape}; expected {tuple(shape)}")
    return np.ascontiguousarray(a.view(np.uint16))


class Weights:
    """Owns a dq_weights handle."""

    def __init__(self, handle: ctypes.c_void_p):
        self.handle = handle
        Ci, Co, r, dev = ctypes.c_int64(), ctypes.c_int64(), ctypes.c_int32(), ctypes.c_int32()
        _check(load().dq_weights_info(handle, ctypes.byref(Ci), ctypes.byref(Co), ctypes.byref(r), ctypes.byref(dev)),
               "dq_weights_info")
        self.Ci, self.Co, self.rank, self.device = Ci.value, Co.value, r.value, dev.value

    def __del__(self):
        if getattr(self, "handle", None) and _LIB is not None:
            _LIB.dq_weights_destroy(self.handle)
            self.handle = None


class Act6:
    """Owns a dq_act6 handle (keeps its weights alive)."""

    def __init__(self, handle: ctypes.c_void_p, weights: "Weights", N: int):
        self.handle = handle
        self.weights = weights
        self.N = N

    def __del__(self):
        if getattr(self, "handle", None) and _LIB is not None:
            _LIB.dq_act6_destroy(self.handle)
            self.handle = None


class QAct:
    """Owns a dq_qact handle (keeps its weights alive)."""

    def __init__(self, handle: ctypes.c_void_p, weights: Weights, geom: Tuple[int, ...], core_bits: int = 8):
        self.handle = handle
        self.weights = weights
        self.geom = tuple(geom)
        self.core_bits = core_bits
        N, K, nb = ctypes.c_int64(), ctypes.c_int64(), ctypes.c_int64()
        _check(load().dq_qact_info(handle, ctypes.byref(N), ctypes.byref(K), ctypes.byref(nb)), "dq_qact_info")
        self.N, self.K, self.device_bytes = N.value, K.value, nb.value

    def __del__(self):
        if getattr(self, "handle", None) and _LIB is not None:
            _LIB.dq_qact_destroy(self.handle)
            self.handle = None


def dq_lowrank_factors(w, rank: int, seed: int):
    """Host SVD factors: returns (L1 bits uint16 [Ci][rank], L2 bits uint16 [rank][Co])."""
    wt, dt = _host_weight(w)
    Co, Ci = wt.shape
    l1 = np.zeros((Ci, rank), dtype=np.uint16)
    l2 = np.zeros((rank, Co), dtype=np.uint16)
    _check(load().dq_lowrank_factors(_ptr(wt), dt, Ci, Co, rank, seed, _ptr(l1), _ptr(l2)), "dq_lowrank_factors")
    return l1, l2


def dq_prepare_weights_lowrank(w, l1: Optional[np.ndarray], l2: Optional[np.ndarray], device: int = 0) -> Weights:
    f = "dq_prepare_weights_lowrank"
    wt, dt = _host_weight(w)
    Co, Ci = wt.shape
    if (l1 is None) != (l2 is None):
        _invalid(f, "give both factors or neither")
    rank = 0 if l1 is None else np.asarray(l1).shape[-1]
    if l1 is not None and np.asarray(l1).ndim != 2:
        _invalid(f, "l1 must be 2-D [Ci][rank]")
    l1c = None if l1 is None else _factor(f, "l1", l1, (Ci, rank))
    l2c = None if l2 is None else _factor(f, "l2", l2, (rank, Co))
    h = ctypes.c_void_p()
    _check(load().dq_prepare_weights_lowrank(_ptr(wt), dt, Ci, Co, rank, _ptr(l1c), _ptr(l2c), device,
                                             ctypes.byref(h)), "dq_prepare_weights_lowrank")
    return Weights(h)


def dq_prepare_weights(w, rank: int, seed: int = 0, device: int = 0) -> Weights:
    wt, dt = _host_weight(w)
    Co, Ci = wt.shape
    h = ctypes.c_void_p()
    _check(load().dq_prepare_weights(_ptr(wt), dt, Ci, Co, rank, seed, device, ctypes.byref(h)), "dq_prepare_weights")
    return Weights(h)


def dq_weights_export(w: Weights) -> dict:
    Ci, Co, r = w.Ci, w.Co, w.rank
    cbytes = Ci // 4 * 3 if getattr(w, "fp6_format", None) else Ci // 2
    out = dict(l1=np.zeros((Ci, r), np.uint16), l2=np.zeros((r, Co), np.uint16), r=np.zeros((Co, Ci), np.float32),
               rcodes=np.zeros((Co, cbytes), np.uint8), rscales=np.zeros((Co, Ci // 32), np.uint8))
    _check(load().dq_weights_export(w.handle, _ptr(out["l1"]), _ptr(out["l2"]), _ptr(out["r"]), _ptr(out["rcodes"]),
                                    _ptr(out["rscales"])), "dq_weights_export")
    return out


def dq_qact_create(w: Weights, geom: Sequence[int], core_group: int = 32, core_bits: int = 8) -> QAct:
    """Workspace for a (T, H, W, t, h, w) geometry; core_group 64 gives the
    cores one scale per 64 channels, core_bits 4 MX-FP4 cores
    (dq_qact_create_ex)."""
    h = ctypes.c_void_p()
    if core_group == 32 and core_bits == 8:
        _check(load().dq_qact_create(w.handle, Geom(*geom), ctypes.byref(h)), "dq_qact_create")
    else:
        _check(load().dq_qact_create_ex(w.handle, Geom(*geom), core_group, core_bits, ctypes.byref(h)),
               "dq_qact_create_ex")
    return QAct(h, w, geom, core_bits)


def dq_quantize_act(w: Weights, x, q: QAct, stream=None):
    _check_pair("dq_quantize_act", w, q)
    _check_x("dq_quantize_act", w, q, x)
    _check(load().dq_quantize_act(w.handle, _ptr(x), _dtype_of(x), q.handle, _stream(stream)), "dq_quantize_act")


def dq_linear_forward(w: Weights, q: QAct, y, stream=None):
    _check_pair("dq_linear_forward", w, q)
    _check_y("dq_linear_forward", w, q, y)
    _check(load().dq_linear_forward(w.handle, q.handle, _ptr(y), _stream(stream)), "dq_linear_forward")


def dq_core_term(w: Weights, q: QAct, stream=None):
    _check_pair("dq_core_term", w, q)
    _check(load().dq_core_term(w.handle, q.handle, _stream(stream)), "dq_core_term")


def dq_delta_term(w: Weights, q: QAct, y, stream=None):
    _check_pair("dq_delta_term", w, q)
    _check_y("dq_delta_term", w, q, y)
    _check(load().dq_delta_term(w.handle, q.handle, _ptr(y), _stream(stream)), "dq_delta_term")


def dq_linear_forward_fused(w: Weights, q: QAct, y, stream=None):
    _check_pair("dq_linear_forward_fused", w, q)
    _check_y("dq_linear_forward_fused", w, q, y)
    _check(load().dq_linear_forward_fused(w.handle, q.handle, _ptr(y), _stream(stream)), "dq_linear_forward_fused")


def dq_forward_form(w: Weights, q: QAct) -> str:
    """'one kernel' or 'two kernels': the form dq_linear_forward takes for this pair."""
    _check_pair("dq_forward_form", w, q)
    flag = ctypes.c_int(0)
    _check(load().dq_forward_form(w.handle, q.handle, ctypes.byref(flag)), "dq_forward_form")
    return "one kernel" if flag.value else "two kernels"


def dq_linear(w: Weights, x, q: QAct, y, stream=None):
    _check_pair("dq_linear", w, q)
    _check_x("dq_linear", w, q, x)
    _check_y("dq_linear", w, q, y)
    _check(load().dq_linear(w.handle, _ptr(x), _dtype_of(x), q.handle, _ptr(y), _stream(stream)), "dq_linear")


def dq_qact_export(q: QAct, stream=None) -> dict:
    w = q.weights
    N, K, Ci, r = q.N, q.K, w.Ci, w.rank
    bf16 = q.core_bits == 16                      # bf16 cores: their bits, no scales
    out = dict(delta_codes=np.zeros((N, Ci // 2), np.uint8), delta_scales=np.zeros((N, Ci // 32), np.uint8),
               core_codes=np.zeros((K, Ci), np.uint16 if bf16 else np.uint8),
               core_scales=None if bf16 else np.zeros((K, Ci // 32), np.uint8),
               U=np.zeros((N, r), np.uint16))
    _check(load().dq_qact_export(q.handle, _ptr(out["delta_codes"]), _ptr(out["delta_scales"]),
                                 _ptr(out["core_codes"]), _ptr(out["core_scales"]) if not bf16 else None, _ptr(out["U"]),
                                 _stream(stream)),
           "dq_qact_export")
    return out


def dq_linear_noalloc(w: Weights, x, geom: Sequence[int], y, stream=None):
    """dq_linear without a workspace handle: the activation state lives in
    the library's fixed per-device array (calls on one GPU must not overlap)."""
    f = "dq_linear_noalloc"
    T, H, W = geom[:3]
    ws = SimpleNamespace(N=T * H * W)
    _check_x(f, w, ws, x)
    _check_y(f, w, ws, y)
    _check(load().dq_linear_noalloc(w.handle, _ptr(x), _dtype_of(x), Geom(*geom), _ptr(y), _stream(stream)), f)


# ---------------------------------------------------------------- 6-bit layers ----
def dq_prepare_weights_w6(w, l1: Optional[np.ndarray], l2: Optional[np.ndarray], fmt: str = "fp6_e2m3",
                          device: int = 0) -> Weights:
    """A 6-bit weight (Q6(R) in MX-FP6 `fmt`: "fp6_e2m3" or "fp6_e3m2")."""
    f = "dq_prepare_weights_w6"
    if fmt not in FP6_FORMATS:
        _invalid(f, f"fmt must be one of {sorted(FP6_FORMATS)}")
    wt, dt = _host_weight(w)
    Co, Ci = wt.shape
    if (l1 is None) != (l2 is None):
        _invalid(f, "give both factors or neither")
    rank = 0 if l1 is None else np.asarray(l1).shape[-1]
    if l1 is not None and np.asarray(l1).ndim != 2:
        _invalid(f, "l1 must be 2-D [Ci][rank]")
    l1c = None if l1 is None else _factor(f, "l1", l1, (Ci, rank))
    l2c = None if l2 is None else _factor(f, "l2", l2, (rank, Co))
    h = ctypes.c_void_p()
    _check(load().dq_prepare_weights_w6(_ptr(wt), dt, Ci, Co, rank, _ptr(l1c), _ptr(l2c), FP6_FORMATS[fmt], device,
                                        ctypes.byref(h)), f)
    wts = Weights(h)
    wts.fp6_format = fmt
    return wts


def dq_act6_create(w: Weights, N: int) -> Act6:
    h = ctypes.c_void_p()
    _check(load().dq_act6_create(w.handle, N, ctypes.byref(h)), "dq_act6_create")
    return Act6(h, w, N)


def dq_quantize_act6(w: Weights, x, a: Act6, stream=None):
    _check_pair("dq_quantize_act6", w, a)
    _check_x("dq_quantize_act6", w, a, x)
    _check(load().dq_quantize_act6(w.handle, _ptr(x), _dtype_of(x), a.handle, _stream(stream)), "dq_quantize_act6")


def dq_linear6_forward(w: Weights, a: Act6, y, stream=None):
    _check_pair("dq_linear6_forward", w, a)
    _check_y("dq_linear6_forward", w, a, y)
    _check(load().dq_linear6_forward(w.handle, a.handle, _ptr(y), _stream(stream)), "dq_linear6_forward")


def dq_linear6(w: Weights, x, a: Act6, y, stream=None):
    _check_pair("dq_linear6", w, a)
    _check_x("dq_linear6", w, a, x)
    _check_y("dq_linear6", w, a, y)
    _check(load().dq_linear6(w.handle, _ptr(x), _dtype_of(x), a.handle, _ptr(y), _stream(stream)), "dq_linear6")


def dq_act6_export(a: Act6, stream=None) -> dict:
    w = a.weights
    N, Ci, r = a.N, w.Ci, w.rank
    out = dict(codes=np.zeros((N, Ci // 4 * 3), np.uint8), scales=np.zeros((N, Ci // 32), np.uint8),
               U=np.zeros((N, r), np.uint16))
    _check(load().dq_act6_export(a.handle, _ptr(out["codes"]), _ptr(out["scales"]), _ptr(out["U"]), _stream(stream)),
           "dq_act6_export")
    return out


# -------------------------------------------------------- rotated-basis layers ----
class Orbit:
    """Owns a dq_orbit handle (a rotated, Lloyd-Max-coded weight)."""

    def __init__(self, handle, Ci, Co, wbits, abits, device):
        self.handle, self.Ci, self.Co, self.wbits, self.abits, self.device = handle, Ci, Co, wbits, abits, device
        self.rank = 0

    def __del__(self):
        if getattr(self, "handle", None) and _LIB is not None:
            _LIB.dq_orbit_destroy(self.handle)
            self.handle = None


class OrbitAct:
    """Owns a dq_orbit_act handle (keeps its weight alive)."""

    def __init__(self, handle, weights: Orbit, N: int):
        self.handle, self.weights, self.N = handle, weights, N

    def __del__(self):
        if getattr(self, "handle", None) and _LIB is not None:
            _LIB.dq_orbit_act_destroy(self.handle)
            self.handle = None


def dq_orbit_prepare(w, perm, wbits: int = 4, abits: int = 4, device: int = 0) -> Orbit:
    f = "dq_orbit_prepare"
    wt, dt = _host_weight(w)
    Co, Ci = wt.shape
    p = np.ascontiguousarray(np.asarray(perm), dtype=np.int32)
    if p.shape != (Ci,):
        _invalid(f, f"perm has shape {p.shape}; expected ({Ci},)")
    h = ctypes.c_void_p()
    _check(load().dq_orbit_prepare(_ptr(wt), dt, Ci, Co, _ptr(p), wbits, abits, device, ctypes.byref(h)), f)
    return Orbit(h, Ci, Co, wbits, abits, device)


def dq_orbit_export(o: Orbit) -> dict:
    out = dict(wlev=np.zeros(1 << o.wbits, np.uint16), alev=np.zeros(1 << o.abits, np.uint16),
               wcodes=np.zeros((o.Co, o.Ci // 2), np.uint8), wscale=np.zeros(o.Co, np.float32))
    _check(load().dq_orbit_export(o.handle, _ptr(out["wlev"]), _ptr(out["alev"]), _ptr(out["wcodes"]),
                                  _ptr(out["wscale"])), "dq_orbit_export")
    return out


def dq_orbit_act_create(o: Orbit, N: int) -> OrbitAct:
    h = ctypes.c_void_p()
    _check(load().dq_orbit_act_create(o.handle, N, ctypes.byref(h)), "dq_orbit_act_create")
    return OrbitAct(h, o, N)


def dq_orbit_quantize_act(o: Orbit, x, a: OrbitAct, stream=None):
    _check_pair("dq_orbit_quantize_act", o, a)
    _check_x("dq_orbit_quantize_act", o, a, x)
    _check(load().dq_orbit_quantize_act(o.handle, _ptr(x), _dtype_of(x), a.handle, _stream(stream)),
           "dq_orbit_quantize_act")


def dq_orbit_forward(o: Orbit, a: OrbitAct, y, stream=None):
    _check_pair("dq_orbit_forward", o, a)
    _check_y("dq_orbit_forward", o, a, y)
    _check(load().dq_orbit_forward(o.handle, a.handle, _ptr(y), _stream(stream)), "dq_orbit_forward")


def dq_orbit_linear(o: Orbit, x, a: OrbitAct, y, stream=None):
    _check_pair("dq_orbit_linear", o, a)
    _check_x("dq_orbit_linear", o, a, x)
    _check_y("dq_orbit_linear", o, a, y)
    _check(load().dq_orbit_linear(o.handle, _ptr(x), _dtype_of(x), a.handle, _ptr(y), _stream(stream)),
           "dq_orbit_linear")


def dq_orbit_act_export(a: OrbitAct, stream=None) -> dict:
    out = dict(codes=np.zeros((a.N, a.weights.Ci // 2), np.uint8), scale=np.zeros(a.N, np.float32))
    _check(load().dq_orbit_act_export(a.handle, _ptr(out["codes"]), _ptr(out["scale"]), _stream(stream)),
           "dq_orbit_act_export")
    return out


# ------------------------------------------------------------------- few rows ----
class Rows:
    """Owns a dq_rows handle (keeps its weights alive)."""

    def __init__(self, handle: ctypes.c_void_p, weights: Weights, max_rows: int):
        self.handle = handle
        self.weights = weights
        self.max_rows = max_rows
        self.pair = (weights.handle.value, handle.value, weights.Ci, weights.Co, weights.device)

    def __del__(self):
        if getattr(self, "handle", None) and _LIB is not None:
            _LIB.dq_rows_destroy(self.handle)
            self.handle = None


def _native():
    load()
    return _CALL


def _row_tensor(func: str, name: str, t, shape, dtypes, device: int, align: int, strided: bool = True):
    """Like _device_tensor, for a matrix whose rows may be strided (unit stride
    inside a row); returns the row stride in elements."""
    import torch
    if not isinstance(t, torch.Tensor):
        _invalid(func, f"{name} must be a torch tensor")
    if t.dtype not in dtypes:
        _invalid(func, f"{name} has dtype {t.dtype}; expected one of {[str(d) for d in dtypes]}")
    if t.shape != shape:
        _invalid(func, f"{name} has shape {tuple(t.shape)}; expected {tuple(shape)}")
    n, c = shape
    ld, one = t.stride()
    if n <= 1:
        ld = c                                          # (the stride of a single row means nothing)
    if one != 1 and c > 1 or ld < c:
        _invalid(func, f"{name} must have contiguous, non-overlapping rows")
    if not strided and ld != c:
        _invalid(func, f"{name} must be contiguous")
    if not t.is_cuda or t.get_device() != device:
        _invalid(func, f"{name} is on {t.device}; expected cuda:{device}")
    if (t.data_ptr() | (ld * t.element_size() if n > 1 else 0)) % align:
        _invalid(func, f"{name} must have {align}-byte aligned rows")
    return ld


def _stream_on(stream, device: int) -> int:
    """The given stream, or the current one of `device`."""
    if stream is None:
        import torch
        stream = torch.cuda.current_stream(device)
    return getattr(stream, "cuda_stream", stream)


def _mx8_tensors(func: str, codes, scales, n: int, c: int, device: int):
    """Row-major E4M3 codes [n][c] and E8M0 scales [n][c/32], as bytes or in torch's 8-bit float types."""
    import torch
    _row_tensor(func, "codes", codes, (n, c), (torch.float8_e4m3fn, torch.uint8), device, 8, strided=False)
    _row_tensor(func, "scales", scales, (n, c // 32), (torch.float8_e8m0fnu, torch.uint8), device, 1, strided=False)


def dq_import_weights(rcodes, rscales, l1: Optional[np.ndarray], l2: Optional[np.ndarray], device: int = 0) -> Weights:
    """A weight already coded, as dq_weights_export returns it: rcodes uint8
    [Co][Ci/2], rscales uint8 [Co][Ci/32], and the factors' bf16 bits (or
    neither)."""
    f = "dq_import_weights"
    rc, rs = np.ascontiguousarray(rcodes), np.ascontiguousarray(rscales)
    if rc.dtype != np.uint8 or rs.dtype != np.uint8 or rc.ndim != 2 or rs.ndim != 2:
        _invalid(f, "rcodes and rscales must be 2-D uint8 arrays")
    Co, Ci = rc.shape[0], rc.shape[1] * 2
    if rs.shape != (Co, Ci // 32) or Ci % 32:
        _invalid(f, f"rscales has shape {rs.shape}; expected {(Co, Ci // 32)}, Ci a multiple of 32")
    if (l1 is None) != (l2 is None):
        _invalid(f, "give both factors or neither")
    rank = 0 if l1 is None else np.asarray(l1).shape[-1]
    if l1 is not None and np.asarray(l1).ndim != 2:
        _invalid(f, "l1 must be 2-D [Ci][rank]")
    l1c = None if l1 is None else _factor(f, "l1", l1, (Ci, rank))
    l2c = None if l2 is None else _factor(f, "l2", l2, (rank, Co))
    h = ctypes.c_void_p()
    _check(load().dq_import_weights(_ptr(rc), _ptr(rs), Ci, Co, rank, _ptr(l1c), _ptr(l2c), device, ctypes.byref(h)), f)
    return Weights(h)


def dq_rows_create(w: Weights, max_rows: int) -> Rows:
    """Workspace for products of up to `max_rows` rows with `w` (or a weight of the same sizes)."""
    h = ctypes.c_void_p()
    _check(load().dq_rows_create(w.handle, max_rows, ctypes.byref(h)), "dq_rows_create")
    return Rows(h, w, max_rows)


def dq_linear_rows(w: Weights, x, a: Rows, y, stream=None):
    """y [N][Co] (fp32 or bf16) = x Q4(R) + (x L1) L2 for x [N][Ci] in bf16 or
    fp32; rows of either may be strided."""
    f = "dq_linear_rows"
    if a.weights is w and _CALL is not None:
        status = _CALL.linear_rows(a.pair, x, y, None if stream is None else getattr(stream, "cuda_stream", stream))
        if status is not None:
            return _check(status, f) if status else None
    # (not such tensors: the checks below say what is wrong)
    import torch
    _check_pair(f, w, a)
    types = (torch.bfloat16, torch.float32)
    n = x.shape[0] if isinstance(x, torch.Tensor) and x.dim() == 2 else 0
    ldx = _row_tensor(f, "x", x, (n, w.Ci), types, w.device, 16)
    ldy = _row_tensor(f, "y", y, (n, w.Co), types, w.device, 1)
    _check(load().dq_linear_rows(w.handle, x.data_ptr(), _dtype_of(x), ldx, n, a.handle, y.data_ptr(), _dtype_of(y), ldy,
                                 _stream_on(stream, w.device)), f)


def dq_linear_rows8(w: Weights, codes, scales, a: Rows, y, stream=None):
    """dq_linear_rows for rows in MX-FP8: codes [N][Ci] and scales [N][Ci/32]
    as dq_rmsnorm8 writes them."""
    f = "dq_linear_rows8"
    if a.weights is w and _CALL is not None:
        status = _CALL.linear_rows8(a.pair, codes, scales, y, None if stream is None else getattr(stream, "cuda_stream", stream))
        if status is not None:
            return _check(status, f) if status else None
    import torch
    _check_pair(f, w, a)
    n = codes.shape[0] if isinstance(codes, torch.Tensor) and codes.dim() == 2 else 0
    _mx8_tensors(f, codes, scales, n, w.Ci, w.device)
    ldy = _row_tensor(f, "y", y, (n, w.Co), (torch.bfloat16, torch.float32), w.device, 1)
    _check(load().dq_linear_rows8(w.handle, codes.data_ptr(), scales.data_ptr(), n, a.handle, y.data_ptr(), _dtype_of(y), ldy,
                                  _stream_on(stream, w.device)), f)


def dq_rmsnorm8(x, gain, eps: float, codes=None, scales=None, residual=None, h=None, y=None, group: int = 32, stream=None):
    """RMS norm of x + residual as MX-FP8 codes [N][C] and scales [N][C/32], as
    plain values y, or both; h receives x + residual (it, or y, may be x or
    residual itself).  gain [C] in bf16 or fp32, or None."""
    f = "dq_rmsnorm8"
    call = _CALL or _native()
    status = None if call is None else call.rmsnorm8(x, gain, eps, codes, scales, residual, h, y, group,
                                                     None if stream is None else getattr(stream, "cuda_stream", stream))
    if status is not None:
        return _check(status, f) if status else None
    import torch
    if not isinstance(x, torch.Tensor) or x.dim() != 2 or not x.is_cuda:
        _invalid(f, "x must be a 2-D torch tensor on a GPU")
    n, c = x.shape
    dev = x.get_device()
    types = (torch.bfloat16, torch.float32)
    ldx = _row_tensor(f, "x", x, (n, c), types, dev, 16)
    same = (x.dtype,)
    ldr, ldh, ldy = (0 if t is None else _row_tensor(f, name, t, (n, c), same, dev, 16)
                     for name, t in (("residual", residual), ("h", h), ("y", y)))
    if (codes is None) != (scales is None):
        _invalid(f, "give both codes and scales or neither")
    if codes is not None:
        _mx8_tensors(f, codes, scales, n, c, dev)
    gdt = DQ_F32
    if gain is not None:
        _device_tensor(f, "gain", gain, (c,), types, dev, 16)
        gdt = _dtype_of(gain)
    ptr = lambda t: None if t is None else t.data_ptr()
    _check(load().dq_rmsnorm8(ptr(x), ldx, ptr(residual), ldr, _dtype_of(x), ptr(gain), gdt, eps, n, c, group, ptr(h), ldh,
                              ptr(codes), ptr(scales), ptr(y), ldy, dev, _stream_on(stream, dev)), f)


# ----------------------------------------------------------------------- heads ----
class _Rope(ctypes.Structure):
    _fields_ = [("axes", ctypes.c_int32), ("interleaved", ctypes.c_int32), ("pairs", ctypes.c_int32 * 3),
                ("positions", ctypes.c_int64 * 3), ("table", ctypes.c_void_p * 3)]


class _HeadOps(ctypes.Structure):
    _fields_ = [("norm", ctypes.c_int), ("gain_dt", ctypes.c_int), ("eps", ctypes.c_double), ("rope", ctypes.c_void_p),
                ("pos", ctypes.c_void_p)]


class _KV(ctypes.Structure):
    _fields_ = [("k_codes", ctypes.c_void_p), ("k_scales", ctypes.c_void_p), ("v_codes", ctypes.c_void_p),
                ("v_scales", ctypes.c_void_p), ("pages", ctypes.c_int64), ("page_tokens", ctypes.c_int32),
                ("heads", ctypes.c_int32), ("head_dim", ctypes.c_int32), ("bits", ctypes.c_int32)]


class _Seqs(ctypes.Structure):
    _fields_ = [("seqs", ctypes.c_int64), ("first", ctypes.c_void_p), ("length", ctypes.c_void_p), ("pages", ctypes.c_void_p),
                ("pages_ld", ctypes.c_int64)]


class _AttnOps(ctypes.Structure):
    _fields_ = [("scale", ctypes.c_double), ("cap", ctypes.c_double), ("block", ctypes.c_int64), ("window", ctypes.c_int64),
                ("prefix", ctypes.c_void_p)]


def _on_gpu(func: str, name: str, t) -> int:
    import torch
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        _invalid(func, f"{name} must be a torch tensor on a GPU")
    return t.get_device()


class Rope:
    """The position axes of a rotation: for each a table [positions][pairs][2] of
    (cos, sin) in fp32 on one GPU, as dq_rope_table fills it.  Holds the tensors."""

    def __init__(self, tables, interleaved: bool = True):
        import torch
        f = "Rope"
        tables = list(tables)
        if not 1 <= len(tables) <= 3:
            _invalid(f, "a rotation has 1 to 3 axes")
        self.device = _on_gpu(f, "table", tables[0])
        for t in tables:
            if not isinstance(t, torch.Tensor) or t.dim() != 3 or t.shape[2] != 2 or 0 in t.shape:
                _invalid(f, "a table must be a tensor [positions][pairs][2]")
            _device_tensor(f, "table", t, t.shape, (torch.float32,), self.device, 8)
        self.tables, self.axes = tables, len(tables)
        self.c = _Rope(self.axes, int(bool(interleaved)))
        for i, t in enumerate(tables):
            self.c.positions[i], self.c.pairs[i], self.c.table[i] = t.shape[0], t.shape[1], t.data_ptr()
        self.address = ctypes.addressof(self.c)


class KV:
    """A paged cache: k_codes and v_codes [pages][heads][page_tokens][head_dim]
    in E4M3 (float8_e4m3fn, or uint8), or [..][head_dim / 2] in packed E2M1
    (uint8, bits=4); k_scales and v_scales [..][head_dim / 32] in E8M0.  Holds
    the tensors; fill the scales with zeros (or write every place) before they are read."""

    def __init__(self, k_codes, k_scales, v_codes, v_scales, bits: Optional[int] = None):
        import torch
        f = "KV"
        self.device = _on_gpu(f, "k_codes", k_codes)
        if k_codes.dim() != 4 or not isinstance(k_scales, torch.Tensor) or k_scales.dim() != 4:
            _invalid(f, "codes and scales must be [pages][heads][page_tokens][..]")
        pages, heads, tokens, width = k_codes.shape
        dim = 32 * k_scales.shape[3]
        held = 8 if width == dim else 4 if 2 * width == dim else 0
        if not held or bits not in (None, held):
            _invalid(f, f"{width} code bytes and {dim // 32} scales a token are neither 8 nor 4 bits" if not held else
                     f"the codes are of {held} bits, not {bits}")
        types = (torch.float8_e4m3fn, torch.uint8) if held == 8 else (torch.uint8,)
        for name, t in (("k_codes", k_codes), ("v_codes", v_codes)):
            _device_tensor(f, name, t, (pages, heads, tokens, width), types, self.device, 16)
        for name, t in (("k_scales", k_scales), ("v_scales", v_scales)):
            _device_tensor(f, name, t, (pages, heads, tokens, dim // 32), (torch.float8_e8m0fnu, torch.uint8), self.device, 4)
        self.tensors = (k_codes, k_scales, v_codes, v_scales)
        self.pages, self.heads, self.page_tokens, self.head_dim, self.bits = pages, heads, tokens, dim, held
        self.c = _KV(*(t.data_ptr() for t in self.tensors), pages, tokens, heads, dim, held)
        self.address = ctypes.addressof(self.c)


class Seqs:
    """A ragged batch: first [seqs + 1] (rows first[b] .. first[b + 1] - 1 are the
    last ones of sequence b), length [seqs] (cached tokens, those rows'
    included) and pages [seqs][n] (the cache's page of each page_tokens tokens),
    int32 on one GPU.  Holds the tensors; their values may change between calls."""

    def __init__(self, first, length, pages):
        import torch
        f = "Seqs"
        self.device = _on_gpu(f, "first", first)
        if not isinstance(pages, torch.Tensor) or pages.dim() != 2 or 0 in pages.shape:
            _invalid(f, "pages must be a tensor [seqs][pages to a sequence]")
        n = pages.shape[0]
        for name, t, shape in (("first", first, (n + 1,)), ("length", length, (n,)), ("pages", pages, tuple(pages.shape))):
            _device_tensor(f, name, t, shape, (torch.int32,), self.device, 4)
        self.tensors, self.seqs = (first, length, pages), n
        self.c = _Seqs(n, first.data_ptr(), length.data_ptr(), pages.data_ptr(), pages.shape[1])
        self.address = ctypes.addressof(self.c)


def _raw(stream):
    return None if stream is None else getattr(stream, "cuda_stream", stream)


def _head_ops(func: str, norm, gains, eps, rope, pos, n: int, dim: int, device: int, in_cache: bool):
    """The _HeadOps of a call; gains: (name, tensor or None, heads) of each part that is normed."""
    import torch
    if norm not in NORMS:
        _invalid(func, f"norm must be one of {list(NORMS)}")
    types = (torch.bfloat16, torch.float32)
    dts = set()
    for name, g, heads in gains:
        if g is None:
            continue
        if norm is None:
            _invalid(func, f"{name} without a norm")
        _device_tensor(func, name, g, (dim if norm == "head" else heads * dim,), types, device, 16)
        dts.add(_dtype_of(g))
    if len(dts) > 1:
        _invalid(func, "the gains must have one dtype")
    if rope is None:
        if pos is not None:
            _invalid(func, "pos without a rope")
    else:
        if not isinstance(rope, Rope):
            _invalid(func, "rope must be a Rope")
        if rope.device != device:
            _invalid(func, f"the rope's tables are on cuda:{rope.device}; expected cuda:{device}")
        if pos is not None:
            _device_tensor(func, "pos", pos, (n, rope.axes), (torch.int32,), device, 4)
        elif rope.axes != 1:
            _invalid(func, "a rotation by several axes needs pos")
    return _HeadOps(NORMS[norm], dts.pop() if dts else DQ_F32, float(eps), rope.address if rope else None,
                    pos.data_ptr() if pos is not None else None)


def dq_rope_table(freq, positions: int, table, stream=None):
    """Fills table [positions][pairs][2] (fp32, on a GPU) with (cos, sin) of p freq[j], angles in fp64."""
    import torch
    f = "dq_rope_table"
    fr = np.ascontiguousarray(np.asarray(freq, dtype=np.float64))
    if fr.ndim != 1:
        _invalid(f, "freq must be 1-D")
    dev = _on_gpu(f, "table", table)
    _device_tensor(f, "table", table, (positions, fr.shape[0], 2), (torch.float32,), dev, 8)
    _check(load().dq_rope_table(_ptr(fr), fr.shape[0], positions, table.data_ptr(), dev, _stream_on(stream, dev)), f)


def dq_norm_rope(x, heads: int, y, norm: Optional[str] = None, gain=None, eps: float = 1e-6, rope: Optional[Rope] = None, pos=None,
                 stream=None):
    """y [N][heads * head_dim] = the heads of x normed (norm "head" or "row", with
    gain [head_dim] or [heads * head_dim]) and rotated by their rows' positions
    pos [N][axes] (int32; None: the row's number); either in bf16 or fp32, y may
    be x itself."""
    f = "dq_norm_rope"
    call = _CALL or _native()
    if call is not None and (rope is None or isinstance(rope, Rope)):
        status = call.norm_rope(x, heads, y, NORMS.get(norm, -1), gain, eps, rope, pos, _raw(stream))
        if status is not None:
            return _check(status, f) if status else None
    import torch
    dev = _on_gpu(f, "x", x)
    if x.dim() != 2 or not isinstance(heads, int) or heads < 1 or x.shape[1] % heads:
        _invalid(f, "x must be 2-D, its width a multiple of heads")
    n, c = x.shape
    types = (torch.bfloat16, torch.float32)
    ldx, ldy = _row_tensor(f, "x", x, (n, c), types, dev, 16), _row_tensor(f, "y", y, (n, c), types, dev, 16)
    ops = _head_ops(f, norm, [("gain", gain, heads)], eps, rope, pos, n, c // heads, dev, False)
    _check(load().dq_norm_rope(x.data_ptr(), ldx, _dtype_of(x), n, heads, c // heads, None if gain is None else gain.data_ptr(),
                               ctypes.byref(ops), y.data_ptr(), ldy, _dtype_of(y), dev, _stream_on(stream, dev)), f)


def _cache_batch(func: str, kv, seqs):
    if not isinstance(kv, KV) or not isinstance(seqs, Seqs):
        _invalid(func, "kv must be a KV and seqs a Seqs")
    if seqs.device != kv.device:
        _invalid(func, f"the batch is on cuda:{seqs.device}; expected cuda:{kv.device}")
    return kv.device


def dq_kv_write(kv: KV, seqs: Seqs, k, v, q=None, y=None, norm: Optional[str] = None, gain=None, gain_q=None, eps: float = 1e-6,
                rope: Optional[Rope] = None, pos=None, stream=None):
    """Codes the N rows' keys k (normed with `gain` and rotated as in
    dq_norm_rope; pos None: by their places in their sequences) and values v into
    the cache; with queries q [N][q heads * head_dim] (normed with `gain_q`) y
    receives them in bf16 or fp32."""
    f = "dq_kv_write"
    call = _CALL or _native()
    if call is not None and isinstance(kv, KV) and isinstance(seqs, Seqs) and (rope is None or isinstance(rope, Rope)):
        status = call.kv_write(kv, seqs, k, v, q, y, NORMS.get(norm, -1), gain, gain_q, eps, rope, pos, _raw(stream))
        if status is not None:
            return _check(status, f) if status else None
    import torch
    dev = _cache_batch(f, kv, seqs)
    types = (torch.bfloat16, torch.float32)
    n = k.shape[0] if isinstance(k, torch.Tensor) and k.dim() == 2 else 0
    c = kv.heads * kv.head_dim
    ldk = _row_tensor(f, "k", k, (n, c), types, dev, 16)
    ldv = _row_tensor(f, "v", v, (n, c), (k.dtype,), dev, 16)
    if (q is None) != (y is None):
        _invalid(f, "give both q and y or neither")
    qh = ldq = ldy = ydt = 0
    if q is not None:
        cq = q.shape[1] if isinstance(q, torch.Tensor) and q.dim() == 2 else 0
        if not cq or cq % kv.head_dim:
            _invalid(f, "q must be 2-D, its width a multiple of head_dim")
        qh = cq // kv.head_dim
        ldq, ldy = _row_tensor(f, "q", q, (n, cq), (k.dtype,), dev, 16), _row_tensor(f, "y", y, (n, cq), types, dev, 16)
        ydt = _dtype_of(y)
    elif gain_q is not None:
        _invalid(f, "gain_q without q")
    ops = _head_ops(f, norm, [("gain", gain, kv.heads), ("gain_q", gain_q, qh)], eps, rope, pos, n, kv.head_dim, dev, True)
    ptr = lambda t: None if t is None else t.data_ptr()
    _check(load().dq_kv_write(kv.address, seqs.address, n, _dtype_of(k), ptr(k), ldk, ptr(v), ldv, ptr(gain), ptr(q), ldq, qh,
                              ptr(gain_q), ptr(y), ldy, ydt, ctypes.byref(ops), dev, _stream_on(stream, dev)), f)


def dq_kv_read(kv: KV, seqs: Seqs, k=None, v=None, stream=None):
    """The values of the rows' tokens: k and v [N][heads * head_dim] in bf16 or fp32, or one of them."""
    f = "dq_kv_read"
    call = _CALL or _native()
    if call is not None and isinstance(kv, KV) and isinstance(seqs, Seqs):
        status = call.kv_read(kv, seqs, k, v, _raw(stream))
        if status is not None:
            return _check(status, f) if status else None
    import torch
    dev = _cache_batch(f, kv, seqs)
    given = [t for t in (k, v) if t is not None]
    if not given:
        _invalid(f, "give k or v")
    n = given[0].shape[0] if isinstance(given[0], torch.Tensor) and given[0].dim() == 2 else 0
    ld = [0 if t is None else _row_tensor(f, name, t, (n, kv.heads * kv.head_dim),
                                          (torch.bfloat16, torch.float32) if t is given[0] else (given[0].dtype,), dev, 16)
          for name, t in (("k", k), ("v", v))]
    ptr = lambda t: None if t is None else t.data_ptr()
    _check(load().dq_kv_read(kv.address, seqs.address, n, ptr(k), ld[0], ptr(v), ld[1], _dtype_of(given[0]), dev,
                             _stream_on(stream, dev)), f)


class Attn:
    """Owns a dq_attn handle (a workspace for one stream at a time)."""

    def __init__(self, handle: ctypes.c_void_p, device: int):
        self.handle, self.device = handle, device
        self.address = handle.value

    def __del__(self):
        if getattr(self, "handle", None) and _LIB is not None:
            _LIB.dq_attn_destroy(self.handle)
            self.handle = None


def dq_attn_create(device: int = 0) -> Attn:
    """Workspace of dq_attn_rows on one GPU."""
    h = ctypes.c_void_p()
    _check(load().dq_attn_create(device, ctypes.byref(h)), "dq_attn_create")
    return Attn(h, device)


def _scale(scale):
    """The native call's scale: -1.0 for None, and None (not a number: refused there) for a -1.0 that was given."""
    return -1.0 if scale is None else None if scale == -1.0 else scale


def dq_attn_rows(kv: KV, seqs: Seqs, q, a: Attn, y, scale: Optional[float] = None, block: int = 1, window: int = 0, prefix=None,
                 cap: float = 0.0, stream=None):
    """y [N][q heads * head_dim] = softmax(scale q k) v of each row over the
    tokens of its sequence that it sees, in q's type; scale None is
    head_dim ** -0.5.  block 0: all tokens; else those up to the end of the row's
    own block of `block` tokens (1: causal), of them the last `window` (0: all),
    and the first prefix[b] (int32 [seqs], or None).  cap > 0: scores cap *
    tanh(s / cap)."""
    f = "dq_attn_rows"
    call = _CALL or _native()
    if call is not None and isinstance(kv, KV) and isinstance(seqs, Seqs) and isinstance(a, Attn):
        status = call.attn_rows(kv, seqs, q, a, y, _scale(scale), block, window, prefix, cap, _raw(stream))
        if status is not None:
            return _check(status, f) if status else None
    import torch
    dev = _cache_batch(f, kv, seqs)
    if not isinstance(a, Attn) or a.device != dev:
        _invalid(f, f"a must be a workspace of cuda:{dev}")
    types = (torch.bfloat16, torch.float32)
    n, c = q.shape if isinstance(q, torch.Tensor) and q.dim() == 2 else (0, 0)
    if not c or c % (kv.heads * kv.head_dim):
        _invalid(f, "q must be 2-D, its heads a multiple of the cache's")
    ldq = _row_tensor(f, "q", q, (n, c), types, dev, 16)
    ldy = _row_tensor(f, "y", y, (n, c), (q.dtype,), dev, 16)
    if prefix is not None:
        _device_tensor(f, "prefix", prefix, (seqs.seqs,), (torch.int32,), dev, 4)
    for name, i in (("block", block), ("window", window)):
        if not isinstance(i, int) or not 0 <= i < 2 ** 31:
            _invalid(f, f"{name} must be an integer in [0, 2^31)")
    ops = _AttnOps(kv.head_dim ** -0.5 if scale is None else float(scale), float(cap), block, window,
                   None if prefix is None else prefix.data_ptr())
    _check(load().dq_attn_rows(kv.address, seqs.address, n, q.data_ptr(), ldq, _dtype_of(q), c // kv.head_dim, ctypes.byref(ops),
                               a.handle, y.data_ptr(), ldy, dev, _stream_on(stream, dev)), f)
