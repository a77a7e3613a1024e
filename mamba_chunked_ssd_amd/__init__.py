"""mamba_chunked_ssd_amd -- the Mamba-2 chunked SSD forward pass on MI355X (gfx950).

A thin ctypes binding over ``libssd.so`` (C ABI in ``include/ssd.h``).  It only
marshals arguments: torch provides device memory and the current stream, and
every step of the forward pass runs in the library's HIP kernels.  There is no
CPU fallback: if the library is missing, importing works but any call raises.

    y = chunk_scan_fwd(x, dt, A, B, C, D, chunk_size=256)
    y, final = chunk_scan_fwd(..., initial_states=h0, return_final_states=True)

Beside it stand the operators of the layers around it: the short causal
convolution (``causal_conv_fwd``, ``_bwd``, ``_step``), the selective scan
with a decay per channel and state (``selective_scan_fwd``, ``_bwd``,
``_step``), sliding-window attention with sinks (``window_attention_fwd``,
``_bwd``, ``_step``) and the RMS norm with the residual's addition
(``rms_norm_fwd``, ``_bwd``).

The operation is the selective state-space recurrence of "Accelerating Mamba-2
with High-Performance Forward Pass Kernels in NVIDIA CUDA Tile" (section
"Mamba-2 architecture"): h_t = exp(A dt_t) h_{t-1} + dt_t B_t x_t^T,
y_t = C_t^T h_t + D x_t, for every batch and head.
"""
from __future__ import annotations

import ctypes
import os
import threading

HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(HERE, "libssd.so")

SSD_DTYPE_F32 = 0
SSD_DTYPE_BF16 = 1
SSD_DTYPE_E4M3 = 2
SSD_FLAG_KEEP_INTERMEDIATES = 1

STATUS = {
    0: "SSD_OK",
    1: "SSD_ERROR_INVALID_VALUE",
    2: "SSD_ERROR_UNSUPPORTED",
    3: "SSD_ERROR_MISALIGNED",
    4: "SSD_ERROR_WORKSPACE",
    5: "SSD_ERROR_LAUNCH",
    6: "SSD_ERROR_SCRATCH",
}
NOALLOC_SCRATCH_BYTES = 128 * 1024 * 1024

# Symbols include/ssd.h declares (checked by the CPU tests).
EXPORTS = [
    "ssd_chunk_scan_fwd_workspace_size",
    "ssd_chunk_scan_fwd_workspace_layout",
    "ssd_chunk_scan_fwd",
    "ssd_chunk_scan_fwd_profiled",
    "ssd_chunk_scan_fwd_stage_launches",
    "ssd_chunk_scan_fwd_default_plan",
    "ssd_chunk_scan_fwd_ex",
    "ssd_chunk_scan_fwd_noalloc",
    "ssd_decode_step",
    "ssd_chunk_scan_fwd_tune",
    "ssd_chunk_scan_bwd_workspace_size",
    "ssd_chunk_scan_bwd",
    "ssd_chunk_scan_bwd_profiled",
    "ssd_chunk_scan_bwd_saved",
    "ssd_causal_conv_fwd",
    "ssd_causal_conv_bwd_workspace_size",
    "ssd_causal_conv_bwd",
    "ssd_causal_conv_step",
    "ssd_selective_scan_fwd_workspace_size",
    "ssd_selective_scan_fwd",
    "ssd_selective_scan_bwd_workspace_size",
    "ssd_selective_scan_bwd",
    "ssd_selective_scan_step",
    "ssd_window_attn_fwd",
    "ssd_window_attn_bwd_workspace_size",
    "ssd_window_attn_bwd",
    "ssd_window_attn_step_workspace_size",
    "ssd_window_attn_step",
    "ssd_rms_norm_fwd",
    "ssd_rms_norm_bwd_workspace_size",
    "ssd_rms_norm_bwd",
    "ssd_status_string",
    "ssd_version",
]


class SSDError(RuntimeError):
    """A non-OK status from libssd."""

    def __init__(self, status: int, where: str):
        self.status = status
        msg = "%s: %s (%s)" % (where, STATUS.get(status, "status %d" % status), status_string(status))
        super().__init__(msg)


class Shape(ctypes.Structure):
    _fields_ = [
        ("batch", ctypes.c_int64),
        ("seqlen", ctypes.c_int64),
        ("nheads", ctypes.c_int64),
        ("headdim", ctypes.c_int64),
        ("dstate", ctypes.c_int64),
        ("ngroups", ctypes.c_int64),
        ("dtype", ctypes.c_int32),
        ("flags", ctypes.c_uint32),
        ("y_dtype", ctypes.c_int32),
        ("reserved", ctypes.c_int32),
    ]


class WorkspaceLayout(ctypes.Structure):
    _fields_ = [
        ("g2_hi", ctypes.c_size_t),
        ("g2_lo", ctypes.c_size_t),
        ("dt", ctypes.c_size_t),
        ("w", ctypes.c_size_t),
        ("s", ctypes.c_size_t),
        ("h", ctypes.c_size_t),
        ("cb", ctypes.c_size_t),
        ("total", ctypes.c_size_t),
        ("nchunks", ctypes.c_int64),
        ("padded_len", ctypes.c_int64),
    ]


class Stride(ctypes.Structure):
    """ssd_stride: elements between batch entries and between tokens ({0, 0}: dense)."""
    _fields_ = [("batch", ctypes.c_int64), ("row", ctypes.c_int64)]


SSD_ACT_NONE = 0
SSD_ACT_SILU = 1
SSD_SCAN_DT_SOFTPLUS = 1


class ConvShape(ctypes.Structure):
    _fields_ = [
        ("batch", ctypes.c_int64),
        ("seqlen", ctypes.c_int64),
        ("channels", ctypes.c_int64),
        ("width", ctypes.c_int32),
        ("activation", ctypes.c_int32),
        ("dtype", ctypes.c_int32),
        ("y_dtype", ctypes.c_int32),
        ("dx_dtype", ctypes.c_int32),
        ("reserved", ctypes.c_int32),
        ("x", Stride),
        ("dy", Stride),
    ]


class SelectiveShape(ctypes.Structure):
    _fields_ = [
        ("batch", ctypes.c_int64),
        ("seqlen", ctypes.c_int64),
        ("channels", ctypes.c_int64),
        ("dstate", ctypes.c_int64),
        ("ngroups", ctypes.c_int64),
        ("dtype", ctypes.c_int32),
        ("y_dtype", ctypes.c_int32),
        ("flags", ctypes.c_uint32),
        ("reserved", ctypes.c_int32),
        ("x", Stride),
        ("dt", Stride),
        ("B", Stride),
        ("C", Stride),
        ("z", Stride),
        ("dy", Stride),
    ]


class HeadStride(ctypes.Structure):
    """ssd_head_stride: elements between batch entries, tokens and heads ({0, 0, 0}: dense)."""
    _fields_ = [("batch", ctypes.c_int64), ("row", ctypes.c_int64), ("head", ctypes.c_int64)]


class AttnShape(ctypes.Structure):
    _fields_ = [
        ("batch", ctypes.c_int64),
        ("seqlen", ctypes.c_int64),
        ("nheads", ctypes.c_int64),
        ("nkvheads", ctypes.c_int64),
        ("headdim", ctypes.c_int64),
        ("window", ctypes.c_int64),
        ("sinks", ctypes.c_int64),
        ("scale", ctypes.c_float),
        ("dtype", ctypes.c_int32),
        ("reserved", ctypes.c_int32 * 2),
        ("q", HeadStride),
        ("k", HeadStride),
        ("v", HeadStride),
        ("y", HeadStride),
        ("dy", HeadStride),
    ]


class NormShape(ctypes.Structure):
    _fields_ = [
        ("batch", ctypes.c_int64),
        ("seqlen", ctypes.c_int64),
        ("channels", ctypes.c_int64),
        ("eps", ctypes.c_float),
        ("dtype", ctypes.c_int32),
        ("res_dtype", ctypes.c_int32),
        ("y_dtype", ctypes.c_int32),
        ("scale_block", ctypes.c_int32),
        ("reserved", ctypes.c_int32),
        ("x", Stride),
        ("residual", Stride),
        ("dy", Stride),
        ("dres", Stride),
    ]


SSD_STATE_SPLIT = 0
SSD_STATE_FUSED = 1


class Plan(ctypes.Structure):
    """ssd_plan: how the stages divide their work among thread blocks."""
    _fields_ = [
        ("state_path", ctypes.c_int32),
        ("chunk_state_heads", ctypes.c_int32),
        ("chunk_out_heads", ctypes.c_int32),
        ("fused_cols", ctypes.c_int32),
        ("reserved", ctypes.c_int32 * 4),
    ]

    def as_dict(self) -> dict:
        return {"state_path": "fused" if self.state_path == SSD_STATE_FUSED else "split",
                "chunk_state_heads": self.chunk_state_heads,
                "chunk_out_heads": self.chunk_out_heads, "fused_cols": self.fused_cols}

    def __repr__(self):
        return "Plan(%s)" % ", ".join("%s=%s" % kv for kv in self.as_dict().items())


def make_plan(state_path="split", chunk_state_heads=1, chunk_out_heads=1, fused_cols=0) -> Plan:
    sp = SSD_STATE_FUSED if state_path in ("fused", SSD_STATE_FUSED) else SSD_STATE_SPLIT
    return Plan(sp, chunk_state_heads, chunk_out_heads, fused_cols)


_lock = threading.Lock()
_lib = None


def load_library(path: str | None = None):
    """Load libssd.so (built in-tree by ``mamba_chunked_ssd_amd.build``)."""
    global _lib
    with _lock:
        if _lib is not None and path is None:
            return _lib
        p = path or LIB_PATH
        if not os.path.exists(p):
            raise RuntimeError(
                "libssd.so is not built (%s); run `python -m mamba_chunked_ssd_amd.build` "
                "or __graft_entry__.build()" % p)
        lib = ctypes.CDLL(p)
        vp, i64, sz = ctypes.c_void_p, ctypes.c_int64, ctypes.c_size_t
        sp = ctypes.POINTER(Shape)
        lib.ssd_chunk_scan_fwd_workspace_size.argtypes = [sp, i64]
        lib.ssd_chunk_scan_fwd_workspace_size.restype = sz
        lib.ssd_chunk_scan_fwd_workspace_layout.argtypes = [sp, i64, ctypes.POINTER(WorkspaceLayout)]
        lib.ssd_chunk_scan_fwd_workspace_layout.restype = ctypes.c_int
        fwd_args = [sp, vp, vp, vp, vp, vp, vp, i64, vp, vp, vp, vp, sz, vp]
        lib.ssd_chunk_scan_fwd.argtypes = fwd_args
        lib.ssd_chunk_scan_fwd.restype = ctypes.c_int
        lib.ssd_chunk_scan_fwd_profiled.argtypes = fwd_args + [ctypes.POINTER(ctypes.c_void_p)]
        lib.ssd_chunk_scan_fwd_profiled.restype = ctypes.c_int
        pp = ctypes.POINTER(Plan)
        lib.ssd_chunk_scan_fwd_stage_launches.argtypes = [sp, i64, pp, ctypes.POINTER(ctypes.c_uint32)]
        lib.ssd_chunk_scan_fwd_stage_launches.restype = ctypes.c_int
        lib.ssd_chunk_scan_fwd_default_plan.argtypes = [sp, i64, pp]
        lib.ssd_chunk_scan_fwd_default_plan.restype = ctypes.c_int
        lib.ssd_chunk_scan_fwd_ex.argtypes = fwd_args + [pp, ctypes.POINTER(ctypes.c_void_p)]
        lib.ssd_chunk_scan_fwd_ex.restype = ctypes.c_int
        lib.ssd_chunk_scan_fwd_noalloc.argtypes = [sp, vp, vp, vp, vp, vp, vp, i64, vp, vp, vp, vp]
        lib.ssd_chunk_scan_fwd_noalloc.restype = ctypes.c_int
        lib.ssd_decode_step.argtypes = [sp, vp, vp, vp, vp, vp, vp, vp, vp, vp, ctypes.POINTER(ctypes.c_void_p)]
        lib.ssd_decode_step.restype = ctypes.c_int
        lib.ssd_chunk_scan_fwd_tune.argtypes = fwd_args + [ctypes.c_int, pp, ctypes.POINTER(ctypes.c_float)]
        lib.ssd_chunk_scan_fwd_tune.restype = ctypes.c_int
        lib.ssd_chunk_scan_bwd_workspace_size.argtypes = [sp, i64]
        lib.ssd_chunk_scan_bwd_workspace_size.restype = sz
        bwd_args = [sp, vp, vp, vp, vp, vp, vp, i64, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, sz, vp]
        lib.ssd_chunk_scan_bwd.argtypes = bwd_args
        lib.ssd_chunk_scan_bwd.restype = ctypes.c_int
        lib.ssd_chunk_scan_bwd_profiled.argtypes = bwd_args + [ctypes.POINTER(ctypes.c_void_p)]
        lib.ssd_chunk_scan_bwd_profiled.restype = ctypes.c_int
        # as bwd_args, with the forward workspace and its size after d_final_states
        lib.ssd_chunk_scan_bwd_saved.argtypes = bwd_args[:11] + [vp, sz] + bwd_args[11:] + [
            ctypes.POINTER(ctypes.c_void_p)]
        lib.ssd_chunk_scan_bwd_saved.restype = ctypes.c_int
        cp, xp = ctypes.POINTER(ConvShape), ctypes.POINTER(SelectiveShape)
        lib.ssd_causal_conv_fwd.argtypes = [cp] + [vp] * 8
        lib.ssd_causal_conv_bwd_workspace_size.argtypes = [cp]
        lib.ssd_causal_conv_bwd.argtypes = [cp] + [vp] * 12 + [sz, vp]
        lib.ssd_causal_conv_step.argtypes = [cp] + [vp] * 6
        lib.ssd_selective_scan_fwd_workspace_size.argtypes = [xp]
        lib.ssd_selective_scan_fwd.argtypes = [xp] + [vp] * 13 + [sz, vp]
        lib.ssd_selective_scan_bwd_workspace_size.argtypes = [xp]
        lib.ssd_selective_scan_bwd.argtypes = [xp] + [vp] * 22 + [sz, vp]
        lib.ssd_selective_scan_step.argtypes = [xp] + [vp] * 11
        ap, np_ = ctypes.POINTER(AttnShape), ctypes.POINTER(NormShape)
        lib.ssd_window_attn_fwd.argtypes = [ap] + [vp] * 10
        lib.ssd_window_attn_bwd_workspace_size.argtypes = [ap]
        lib.ssd_window_attn_bwd.argtypes = [ap] + [vp] * 11 + [sz, vp]
        lib.ssd_window_attn_step_workspace_size.argtypes = [ap]
        lib.ssd_window_attn_step.argtypes = [ap] + [vp] * 8 + [sz, vp]
        lib.ssd_rms_norm_fwd.argtypes = [np_] + [vp] * 8
        lib.ssd_rms_norm_bwd_workspace_size.argtypes = [np_]
        lib.ssd_rms_norm_bwd.argtypes = [np_] + [vp] * 9 + [sz, vp]
        for name in ("causal_conv_bwd", "selective_scan_fwd", "selective_scan_bwd", "window_attn_bwd",
                     "window_attn_step", "rms_norm_bwd"):
            getattr(lib, "ssd_%s_workspace_size" % name).restype = sz
        for name in ("causal_conv_fwd", "causal_conv_bwd", "causal_conv_step", "selective_scan_fwd",
                     "selective_scan_bwd", "selective_scan_step", "window_attn_fwd", "window_attn_bwd",
                     "window_attn_step", "rms_norm_fwd", "rms_norm_bwd"):
            getattr(lib, "ssd_" + name).restype = ctypes.c_int
        lib.ssd_status_string.argtypes = [ctypes.c_int]
        lib.ssd_status_string.restype = ctypes.c_char_p
        lib.ssd_version.argtypes = []
        lib.ssd_version.restype = ctypes.c_int
        if path is None:
            _lib = lib
        return lib


def status_string(status: int) -> str:
    try:
        return load_library().ssd_status_string(status).decode()
    except Exception:  # pragma: no cover - library missing
        return "?"


def _dtype_code(dtype) -> int:
    if dtype in ("bf16", SSD_DTYPE_BF16):
        return SSD_DTYPE_BF16
    if dtype in ("f32", SSD_DTYPE_F32):
        return SSD_DTYPE_F32
    raise ValueError("dtype must be 'f32' or 'bf16'")


def make_shape(batch, seqlen, nheads, headdim, dstate, ngroups, dtype, keep=False,
               y_dtype="f32") -> Shape:
    return Shape(batch, seqlen, nheads, headdim, dstate, ngroups, _dtype_code(dtype),
                 SSD_FLAG_KEEP_INTERMEDIATES if keep else 0, _dtype_code(y_dtype), 0)


def workspace_size(shape: Shape, chunk_size: int) -> int:
    return int(load_library().ssd_chunk_scan_fwd_workspace_size(ctypes.byref(shape), chunk_size))


def workspace_layout(shape: Shape, chunk_size: int) -> WorkspaceLayout:
    lay = WorkspaceLayout()
    st = load_library().ssd_chunk_scan_fwd_workspace_layout(ctypes.byref(shape), chunk_size,
                                                            ctypes.byref(lay))
    if st != 0:
        raise SSDError(st, "ssd_chunk_scan_fwd_workspace_layout")
    return lay


STAGES = ("chunk_cumsum", "chunk_state", "state_pass", "chunk_out")


def default_plan(shape: Shape, chunk_size: int) -> Plan:
    """The launch plan ``ssd_chunk_scan_fwd`` uses for this problem (host only)."""
    plan = Plan()
    st = load_library().ssd_chunk_scan_fwd_default_plan(ctypes.byref(shape), chunk_size,
                                                        ctypes.byref(plan))
    if st != 0:
        raise SSDError(st, "ssd_chunk_scan_fwd_default_plan")
    return plan


def _plan_ref(plan):
    return None if plan is None else ctypes.byref(plan)


def stage_launches(shape: Shape, chunk_size: int, plan: Plan | None = None) -> tuple:
    """Names of the stages that launch a kernel of their own for this problem
    (under ``plan``; None = the default plan)."""
    mask = ctypes.c_uint32()
    st = load_library().ssd_chunk_scan_fwd_stage_launches(ctypes.byref(shape), chunk_size,
                                                          _plan_ref(plan), ctypes.byref(mask))
    if st != 0:
        raise SSDError(st, "ssd_chunk_scan_fwd_stage_launches")
    return tuple(n for i, n in enumerate(STAGES) if mask.value >> i & 1)


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _torch():
    import torch
    return torch


def _check(t, name, dtype, shape, device):
    torch = _torch()
    if not isinstance(t, torch.Tensor):
        raise TypeError("%s must be a torch.Tensor" % name)
    if t.device != device:
        raise ValueError("%s is on %s, expected %s" % (name, t.device, device))
    if t.dtype != dtype:
        raise TypeError("%s has dtype %s, expected %s" % (name, t.dtype, dtype))
    if tuple(t.shape) != tuple(shape):
        raise ValueError("%s has shape %s, expected %s" % (name, tuple(t.shape), tuple(shape)))
    if not t.is_contiguous():
        raise ValueError("%s must be contiguous" % name)


def chunk_scan_fwd(x, dt, A, B, C, D=None, chunk_size: int = 256, initial_states=None,
                   return_final_states: bool = False, *, y_dtype=None, out=None,
                   final_out=None, workspace=None, keep_intermediates: bool = False,
                   stream=None, events=None, plan: Plan | None = None):
    """Run ``ssd_chunk_scan_fwd`` on the current (or given) stream.

    x (b, L, nh, p) and dt (b, L, nh), B/C (b, L, g, n): float32 or bfloat16,
    all the same dtype; A (nh,), D (nh,) or None, initial_states
    (b, nh, p, n) or None: float32.  ``y_dtype`` (torch dtype): float32 (the
    default) or the input dtype.  Returns y, or (y, final_states).
    ``workspace`` (uint8 device tensor) may be passed to reuse an allocation;
    with ``keep_intermediates`` its layout is :func:`workspace_layout` of the
    shape with the keep flag.  ``events``: 8 raw hipEvent_t handles (ints), a
    (start, stop) pair per stage recorded by each kernel's own dispatch
    (``ssd_chunk_scan_fwd_profiled``).  ``plan``: an explicit launch plan
    (:class:`Plan`; ``ssd_chunk_scan_fwd_ex``), None for the default one.
    """
    torch = _torch()
    lib = load_library()
    if x.dim() != 4 or B.dim() != 4:
        raise ValueError("x and B must be 4-D")
    b, L, nh, p = x.shape
    g, n = B.shape[2], B.shape[3]
    if x.dtype == torch.bfloat16:
        dname = "bf16"
    elif x.dtype == torch.float32:
        dname = "f32"
    else:
        raise TypeError("x must be float32 or bfloat16")
    dev = x.device
    if dev.type != "cuda":
        raise ValueError("tensors must be on a ROCm device (got %s)" % dev)
    _check(x, "x", x.dtype, (b, L, nh, p), dev)
    _check(dt, "dt", x.dtype, (b, L, nh), dev)
    _check(A, "A", torch.float32, (nh,), dev)
    _check(B, "B", x.dtype, (b, L, g, n), dev)
    _check(C, "C", x.dtype, (b, L, g, n), dev)
    if D is not None:
        _check(D, "D", torch.float32, (nh,), dev)
    if initial_states is not None:
        _check(initial_states, "initial_states", torch.float32, (b, nh, p, n), dev)
    ytype = torch.float32 if y_dtype is None else y_dtype
    if ytype not in (torch.float32, x.dtype):
        raise TypeError("y_dtype must be float32 or the input dtype")
    shape = make_shape(b, L, nh, p, n, g, dname, keep_intermediates,
                       "bf16" if ytype == torch.bfloat16 else "f32")
    need = workspace_size(shape, chunk_size)  # 0 if invalid: the call reports why
    if workspace is None:
        workspace = torch.empty(max(need, 1), dtype=torch.uint8, device=dev)
    y = out if out is not None else torch.empty((b, L, nh, p), dtype=ytype, device=dev)
    if out is not None:
        _check(out, "out", ytype, (b, L, nh, p), dev)
    fin = None
    if return_final_states or final_out is not None:
        fin = final_out if final_out is not None else torch.empty((b, nh, p, n), dtype=torch.float32, device=dev)
        _check(fin, "final_states", torch.float32, (b, nh, p, n), dev)
    s = stream if stream is not None else torch.cuda.current_stream(dev).cuda_stream
    args = [ctypes.byref(shape), _ptr(x), _ptr(dt), _ptr(A), _ptr(B), _ptr(C), _ptr(D),
            int(chunk_size), _ptr(initial_states), _ptr(y), _ptr(fin), _ptr(workspace),
            workspace.numel() * workspace.element_size(), ctypes.c_void_p(s)]
    ev = None
    if events is not None:
        if len(events) != 8:
            raise ValueError("events: a (start, stop) pair for each of the 4 stages")
        ev = (ctypes.c_void_p * 8)(*[ctypes.c_void_p(e) for e in events])
    if plan is not None:
        st = lib.ssd_chunk_scan_fwd_ex(*args, ctypes.byref(plan), ev)
        where = "ssd_chunk_scan_fwd_ex"
    elif ev is None:
        st = lib.ssd_chunk_scan_fwd(*args)
        where = "ssd_chunk_scan_fwd"
    else:
        st = lib.ssd_chunk_scan_fwd_profiled(*args, ev)
        where = "ssd_chunk_scan_fwd_profiled"
    if st != 0:
        raise SSDError(st, where)
    if return_final_states:
        return y, fin
    return y


BWD_STAGES = ("chunk_cumsum", "chunk_state", "state_pass", "adjoint_chunk_state", "adjoint_carry",
              "score_tiles", "dx_pass", "dB_pass", "dC_pass", "w_sums", "token_finish", "reduce")


def bwd_workspace_size(shape: Shape, chunk_size: int) -> int:
    return int(load_library().ssd_chunk_scan_bwd_workspace_size(ctypes.byref(shape), chunk_size))


def chunk_scan_bwd(x, dt, A, B, C, D, dy, chunk_size: int = 256, initial_states=None,
                   d_final_states=None, *, want_dD: bool = True, want_d_initial: bool = True,
                   workspace=None, stream=None, events=None, saved_workspace=None):
    """Gradients through :func:`chunk_scan_fwd` (``ssd_chunk_scan_bwd``).

    Inputs as passed to :func:`chunk_scan_fwd`, plus ``dy`` (dL/dy, the input
    dtype), and optionally
    ``d_final_states`` (dL/dh_final, float32).  Returns a dict of float32
    tensors ``dx, ddt, dA, dB, dC`` and, when requested, ``dD`` and
    ``d_initial_states``.  ``events``: 24 raw hipEvent_t handles (a start and
    stop per stage of :data:`BWD_STAGES`).  ``saved_workspace``: the workspace
    of a :func:`chunk_scan_fwd` call on the same inputs made with
    ``keep_intermediates=True``; its chunk-start states are then read instead
    of recomputed (``ssd_chunk_scan_bwd_saved``).
    """
    torch = _torch()
    lib = load_library()
    if x.dim() != 4 or B.dim() != 4:
        raise ValueError("x and B must be 4-D")
    b, L, nh, p = x.shape
    g, n = B.shape[2], B.shape[3]
    if x.dtype == torch.bfloat16:
        dname = "bf16"
    elif x.dtype == torch.float32:
        dname = "f32"
    else:
        raise TypeError("x must be float32 or bfloat16")
    dev = x.device
    if dev.type != "cuda":
        raise ValueError("tensors must be on a ROCm device (got %s)" % dev)
    _check(x, "x", x.dtype, (b, L, nh, p), dev)
    _check(dt, "dt", x.dtype, (b, L, nh), dev)
    _check(A, "A", torch.float32, (nh,), dev)
    _check(B, "B", x.dtype, (b, L, g, n), dev)
    _check(C, "C", x.dtype, (b, L, g, n), dev)
    if D is not None:
        _check(D, "D", torch.float32, (nh,), dev)
    if initial_states is not None:
        _check(initial_states, "initial_states", torch.float32, (b, nh, p, n), dev)
    _check(dy, "dy", x.dtype, (b, L, nh, p), dev)
    if d_final_states is not None:
        _check(d_final_states, "d_final_states", torch.float32, (b, nh, p, n), dev)
    shape = make_shape(b, L, nh, p, n, g, dname)
    need = bwd_workspace_size(shape, chunk_size)
    if workspace is None:
        workspace = torch.empty(max(need, 1), dtype=torch.uint8, device=dev)
    f32 = dict(dtype=torch.float32, device=dev)
    out = {
        "dx": torch.empty((b, L, nh, p), **f32), "ddt": torch.empty((b, L, nh), **f32),
        "dA": torch.empty((nh,), **f32), "dB": torch.empty((b, L, g, n), **f32),
        "dC": torch.empty((b, L, g, n), **f32),
    }
    if want_dD:
        out["dD"] = torch.empty((nh,), **f32)
    if want_d_initial:
        out["d_initial_states"] = torch.empty((b, nh, p, n), **f32)
    s = stream if stream is not None else torch.cuda.current_stream(dev).cuda_stream
    args = [ctypes.byref(shape), _ptr(x), _ptr(dt), _ptr(A), _ptr(B), _ptr(C), _ptr(D), int(chunk_size),
            _ptr(initial_states), _ptr(dy), _ptr(d_final_states), _ptr(out["dx"]), _ptr(out["ddt"]),
            _ptr(out["dA"]), _ptr(out["dB"]), _ptr(out["dC"]), _ptr(out.get("dD")),
            _ptr(out.get("d_initial_states")), _ptr(workspace), workspace.numel() * workspace.element_size(),
            ctypes.c_void_p(s)]
    ev = None
    if events is not None:
        if len(events) != 2 * len(BWD_STAGES):
            raise ValueError("events: a (start, stop) pair for each of the %d stages" % len(BWD_STAGES))
        ev = (ctypes.c_void_p * len(events))(*[ctypes.c_void_p(e) for e in events])
    if saved_workspace is not None:
        if saved_workspace.device != dev:
            raise ValueError("saved_workspace must be on %s" % dev)
        saved = [_ptr(saved_workspace), saved_workspace.numel() * saved_workspace.element_size()]
        st = lib.ssd_chunk_scan_bwd_saved(*(args[:11] + saved + args[11:]), ev)
        where = "ssd_chunk_scan_bwd_saved"
    elif ev is None:
        st = lib.ssd_chunk_scan_bwd(*args)
        where = "ssd_chunk_scan_bwd"
    else:
        st = lib.ssd_chunk_scan_bwd_profiled(*args, ev)
        where = "ssd_chunk_scan_bwd_profiled"
    if st != 0:
        raise SSDError(st, where)
    return out


def decode_step(x, dt, A, B, C, D, state, *, y_dtype=None, out=None, stream=None, events=None):
    """One recurrent step for one new token per sequence (``ssd_decode_step``).

    x (b, nh, p) and dt (b, nh), B/C (b, g, n): float32 or bfloat16, all the
    same dtype; A (nh,), D (nh,) or None: float32; ``state`` (b, nh, p, n)
    float32 is updated in place.  Returns y (b, nh, p) (``y_dtype``: float32,
    the default, or the input dtype).  ``events``: 2 raw hipEvent_t handles
    (start, stop) recorded by the kernel's own dispatch.
    """
    torch = _torch()
    lib = load_library()
    if x.dim() != 3 or B.dim() != 3:
        raise ValueError("x must be (batch, nheads, headdim) and B (batch, ngroups, dstate)")
    b, nh, p = x.shape
    g, n = B.shape[1], B.shape[2]
    if x.dtype == torch.bfloat16:
        dname = "bf16"
    elif x.dtype == torch.float32:
        dname = "f32"
    else:
        raise TypeError("x must be float32 or bfloat16")
    dev = x.device
    _check(x, "x", x.dtype, (b, nh, p), dev)
    _check(dt, "dt", x.dtype, (b, nh), dev)
    _check(A, "A", torch.float32, (nh,), dev)
    _check(B, "B", x.dtype, (b, g, n), dev)
    _check(C, "C", x.dtype, (b, g, n), dev)
    if D is not None:
        _check(D, "D", torch.float32, (nh,), dev)
    _check(state, "state", torch.float32, (b, nh, p, n), dev)
    ytype = torch.float32 if y_dtype is None else y_dtype
    if ytype not in (torch.float32, x.dtype):
        raise TypeError("y_dtype must be float32 or the input dtype")
    y = out if out is not None else torch.empty((b, nh, p), dtype=ytype, device=dev)
    _check(y, "out", ytype, (b, nh, p), dev)
    shape = make_shape(b, 1, nh, p, n, g, dname, False, "bf16" if ytype == torch.bfloat16 else "f32")
    s = stream if stream is not None else torch.cuda.current_stream(dev).cuda_stream
    ev = None
    if events is not None:
        if len(events) != 2:
            raise ValueError("events: one (start, stop) pair")
        ev = (ctypes.c_void_p * 2)(*[ctypes.c_void_p(e) for e in events])
    st = lib.ssd_decode_step(ctypes.byref(shape), _ptr(x), _ptr(dt), _ptr(A), _ptr(B), _ptr(C), _ptr(D),
                             _ptr(state), _ptr(y), ctypes.c_void_p(s), ev)
    if st != 0:
        raise SSDError(st, "ssd_decode_step")
    return y


def tune(x, dt, A, B, C, D=None, chunk_size: int = 256, initial_states=None, *, reps: int = 5,
         y_dtype=None, out=None, final_out=None, workspace=None, stream=None):
    """Run ``ssd_chunk_scan_fwd_tune`` on these inputs: returns ``(plan, us)``,
    the fastest launch plan found and its time in microseconds.  Pass the plan
    to :func:`chunk_scan_fwd` (``plan=``) for later calls of the same shape."""
    torch = _torch()
    lib = load_library()
    b, L, nh, p = x.shape
    g, n = B.shape[2], B.shape[3]
    dname = "bf16" if x.dtype == torch.bfloat16 else "f32"
    dev = x.device
    ytype = torch.float32 if y_dtype is None else y_dtype
    shape = make_shape(b, L, nh, p, n, g, dname, False, "bf16" if ytype == torch.bfloat16 else "f32")
    for name, t, dtp, shp in (("x", x, x.dtype, (b, L, nh, p)), ("dt", dt, x.dtype, (b, L, nh)),
                              ("A", A, torch.float32, (nh,)), ("B", B, x.dtype, (b, L, g, n)),
                              ("C", C, x.dtype, (b, L, g, n))):
        _check(t, name, dtp, shp, dev)
    if D is not None:
        _check(D, "D", torch.float32, (nh,), dev)
    if initial_states is not None:
        _check(initial_states, "initial_states", torch.float32, (b, nh, p, n), dev)
    if workspace is None:
        workspace = torch.empty(max(workspace_size(shape, chunk_size), 1), dtype=torch.uint8, device=dev)
    y = out if out is not None else torch.empty((b, L, nh, p), dtype=ytype, device=dev)
    fin = final_out if final_out is not None else torch.empty((b, nh, p, n), dtype=torch.float32, device=dev)
    s = stream if stream is not None else torch.cuda.current_stream(dev).cuda_stream
    plan = Plan()
    us = ctypes.c_float()
    st = lib.ssd_chunk_scan_fwd_tune(ctypes.byref(shape), _ptr(x), _ptr(dt), _ptr(A), _ptr(B), _ptr(C), _ptr(D),
                                     int(chunk_size), _ptr(initial_states), _ptr(y), _ptr(fin), _ptr(workspace),
                                     workspace.numel() * workspace.element_size(), ctypes.c_void_p(s), int(reps),
                                     ctypes.byref(plan), ctypes.byref(us))
    if st != 0:
        raise SSDError(st, "ssd_chunk_scan_fwd_tune")
    return plan, float(us.value)


# ---------------------------------------------------------------------------
# The short causal convolution and the selective scan
# ---------------------------------------------------------------------------

_ACTIVATIONS = {None: SSD_ACT_NONE, "silu": SSD_ACT_SILU}


def _input_dtype(x, torch, name="x"):
    """ssd_dtype of an operator's first input, which its other inputs share."""
    if not isinstance(x, torch.Tensor):
        raise TypeError("%s must be a torch.Tensor" % name)
    if not x.is_cuda:
        raise ValueError("tensors must be on a ROCm device (got %s)" % x.device)
    if x.dtype == torch.bfloat16:
        return SSD_DTYPE_BF16
    if x.dtype == torch.float32:
        return SSD_DTYPE_F32
    raise TypeError("%s must be float32 or bfloat16" % name)


def _result_dtype(dtype, given, name, torch):
    if dtype is None or dtype == torch.float32:
        return torch.float32, SSD_DTYPE_F32
    if dtype != given:
        raise TypeError("%s must be float32 or the input dtype" % name)
    return dtype, SSD_DTYPE_BF16


def _dense(t, name, dtype, shape, device, tensor):
    """As :func:`_check`, which words the error; one token's calls are as fast as their checks."""
    if not (isinstance(t, tensor) and t.dtype == dtype and t.shape == shape and t.get_device() == device.index
            and t.is_contiguous()):
        _check(t, name, dtype, shape, device)


def _rows(t, name, dtype, shape, device, tensor, lead):
    """Checks an input of rows that may lie apart, one per token (``lead`` 2: batch and token) or per batch entry
    (``lead`` 1), and returns its ssd_stride, None if it is dense."""
    if isinstance(t, tensor) and t.dtype == dtype and t.shape == shape and t.get_device() == device.index:
        if t.is_contiguous():
            return None
        st = t.stride()
        width = 1
        for k in range(t.dim() - 1, lead - 1, -1):
            if shape[k] != 1 and st[k] != width:
                raise ValueError("%s: each row must be contiguous (strides %s)" % (name, st))
            width *= shape[k]
        tokens = shape[1] if lead == 2 else 1
        row = st[1] if tokens > 1 else width
        if row < width:
            raise ValueError("%s: rows of different tokens overlap (strides %s)" % (name, st))
        return Stride(st[0] if shape[0] > 1 else row * tokens, row)
    if isinstance(t, tensor) and t.dtype == dtype and t.device == device:
        raise ValueError("%s has shape %s, expected %s" % (name, tuple(t.shape), tuple(shape)))
    return _check(t, name, dtype, shape, device)


def _addr(t):
    return None if t is None else t.data_ptr()


def _rows_like(x, stride, shape, dtype, device, torch):
    """A new dense tensor of x's shape; ``empty_like`` is the cheaper call where x is dense."""
    if stride.row == 0:
        return torch.empty_like(x) if dtype == x.dtype else torch.empty_like(x, dtype=dtype)
    return torch.empty(shape, dtype=dtype, device=device)


def _call(where, device, stream, run, torch):
    """``run(stream handle)`` with ``device`` current; what it allocates
    belongs to the stream that the kernels run on."""
    index = device.index
    if index != torch.cuda.current_device():
        with torch.cuda.device(device):
            return _call(where, device, stream, run, torch)
    if stream is None:
        st, res = run(torch._C._cuda_getCurrentRawStream(index))
    else:
        given = torch.cuda.ExternalStream(stream, device=device) if stream else torch.cuda.default_stream(device)
        with torch.cuda.stream(given):
            st, res = run(stream)
    if st != 0:
        raise SSDError(st, where)
    return res


def _workspace(given, need, device, torch):
    """(address, bytes, the tensor that holds them) of the caller's workspace or a new one."""
    if given is not None:
        if given.device != device or not given.is_contiguous():
            raise ValueError("workspace must be a contiguous tensor on %s" % device)
        return given.data_ptr(), given.numel() * given.element_size(), given
    if need == 0:
        return None, 0, None
    ws = torch.empty(need, dtype=torch.uint8, device=device)
    return ws.data_ptr(), need, ws


def _conv_args(x, weight, bias, lengths, activation, lead, torch):
    tensor, f32 = torch.Tensor, torch.float32
    code = _input_dtype(x, torch)
    if not isinstance(weight, tensor):
        raise TypeError("weight must be a torch.Tensor")
    dims = x.shape
    if len(dims) != lead + 1 or weight.dim() != 2:
        raise ValueError("x must be (batch, %schannels) and weight (channels, width)" % ("seqlen, " if lead == 2 else ""))
    if activation not in _ACTIVATIONS:
        raise ValueError("activation must be None or 'silu'")
    dev, b, c, w = x.device, dims[0], dims[-1], weight.shape[1]
    L = dims[1] if lead == 2 else 1
    shape = ConvShape(b, L, c, w, _ACTIVATIONS[activation], code)
    st = _rows(x, "x", x.dtype, dims, dev, tensor, lead)
    if st is not None:
        shape.x = st
    _dense(weight, "weight", f32, (c, w), dev, tensor)
    if bias is not None:
        _dense(bias, "bias", f32, (c,), dev, tensor)
    if lengths is not None:
        _dense(lengths, "lengths", torch.int32, (b,), dev, tensor)
    return shape, dev, b, L, c, w


def causal_conv_fwd(x, weight, bias=None, initial_states=None, return_final_states: bool = False, *,
                    activation="silu", lengths=None, y_dtype=None, out=None, final_out=None, stream=None):
    """Short causal convolution over prompts (``ssd_causal_conv_fwd``):
    y_t = act(bias + sum_k weight[:, k] x_{t - width + 1 + k}), per channel.

    x (b, L, c): float32 or bfloat16, rows may lie apart (a column slice of a
    wider tensor); weight (c, width), width 2..4, and bias (c,): float32;
    ``initial_states`` (b, width - 1, c), the inputs before the first token, in
    x's dtype.  ``activation``: "silu" or None.  ``lengths``: int32 (b,) device
    tensor, tokens of each padded sequence; rows behind are 0 in y.  Returns y
    (``y_dtype``: float32, the default, or x's dtype), or (y, final_states);
    ``final_out`` may be ``initial_states`` itself.
    """
    torch = _torch()
    shape, dev, b, L, c, w = _conv_args(x, weight, bias, lengths, activation, 2, torch)
    if initial_states is not None:
        _dense(initial_states, "initial_states", x.dtype, (b, w - 1, c), dev, torch.Tensor)
    ytype, shape.y_dtype = _result_dtype(y_dtype, x.dtype, "y_dtype", torch)
    if out is not None:
        _dense(out, "out", ytype, (b, L, c), dev, torch.Tensor)
    if final_out is not None:
        _dense(final_out, "final_out", x.dtype, (b, w - 1, c), dev, torch.Tensor)

    def run(handle):
        y = out if out is not None else _rows_like(x, shape.x, (b, L, c), ytype, dev, torch)
        fin = final_out
        if fin is None and return_final_states:
            fin = torch.empty((b, max(w - 1, 0), c), dtype=x.dtype, device=dev)
        st = load_library().ssd_causal_conv_fwd(ctypes.byref(shape), x.data_ptr(), weight.data_ptr(), _addr(bias),
                                                _addr(initial_states), _addr(lengths), y.data_ptr(), _addr(fin),
                                                handle)
        return st, (y, fin) if return_final_states else y

    return _call("ssd_causal_conv_fwd", dev, stream, run, torch)


def causal_conv_bwd(x, weight, bias, dy, initial_states=None, d_final_states=None, *, activation="silu",
                    lengths=None, dx_dtype=None, want_d_initial: bool = True, workspace=None, stream=None):
    """Gradients through :func:`causal_conv_fwd` (``ssd_causal_conv_bwd``).

    Inputs as passed there, plus ``dy`` (b, L, c) (float32 or x's dtype, rows
    may lie apart) and optionally ``d_final_states`` (b, width - 1, c) float32.
    Returns a dict of ``dx`` (``dx_dtype``: float32, the default, or x's
    dtype), ``dweight``, ``dbias`` and, when requested, ``d_initial_states``
    (float32).
    """
    torch = _torch()
    lib = load_library()
    shape, dev, b, L, c, w = _conv_args(x, weight, bias, lengths, activation, 2, torch)
    if initial_states is not None:
        _dense(initial_states, "initial_states", x.dtype, (b, w - 1, c), dev, torch.Tensor)
    if d_final_states is not None:
        _dense(d_final_states, "d_final_states", torch.float32, (b, w - 1, c), dev, torch.Tensor)
    if not isinstance(dy, torch.Tensor):
        raise TypeError("dy must be a torch.Tensor")
    dytype, shape.y_dtype = _result_dtype(dy.dtype, x.dtype, "dy's dtype", torch)
    st = _rows(dy, "dy", dytype, x.shape, dev, torch.Tensor, 2)
    if st is not None:
        shape.dy = st
    dxtype, shape.dx_dtype = _result_dtype(dx_dtype, x.dtype, "dx_dtype", torch)

    def run(handle):
        f32 = dict(dtype=torch.float32, device=dev)
        res = {"dx": _rows_like(x, shape.x, (b, L, c), dxtype, dev, torch), "dweight": torch.empty_like(weight),
               "dbias": torch.empty((c,), **f32) if bias is None else torch.empty_like(bias)}
        if want_d_initial:
            res["d_initial_states"] = torch.empty((b, max(w - 1, 0), c), **f32)
        ws, size, _keep = _workspace(workspace, lib.ssd_causal_conv_bwd_workspace_size(ctypes.byref(shape)), dev, torch)
        st = lib.ssd_causal_conv_bwd(ctypes.byref(shape), x.data_ptr(), weight.data_ptr(), _addr(bias),
                                     _addr(initial_states), _addr(lengths), dy.data_ptr(), _addr(d_final_states),
                                     res["dx"].data_ptr(), res["dweight"].data_ptr(), res["dbias"].data_ptr(),
                                     _addr(res.get("d_initial_states")), ws, size, handle)
        return st, res

    return _call("ssd_causal_conv_bwd", dev, stream, run, torch)


def causal_conv_step(x, weight, bias, state, *, activation="silu", y_dtype=None, out=None, stream=None):
    """The convolution for one new token per sequence (``ssd_causal_conv_step``).

    x (b, c); ``state`` (b, width - 1, c) in x's dtype, the inputs before it,
    updated in place.  Returns y (b, c) (``y_dtype``: float32, the default, or
    x's dtype).
    """
    torch = _torch()
    shape, dev, b, _, c, w = _conv_args(x, weight, bias, None, activation, 1, torch)
    _dense(state, "state", x.dtype, (b, w - 1, c), dev, torch.Tensor)
    ytype, shape.y_dtype = _result_dtype(y_dtype, x.dtype, "y_dtype", torch)
    if out is not None:
        _dense(out, "out", ytype, (b, c), dev, torch.Tensor)

    def run(handle):
        y = out if out is not None else _rows_like(x, shape.x, (b, c), ytype, dev, torch)
        st = load_library().ssd_causal_conv_step(ctypes.byref(shape), x.data_ptr(), weight.data_ptr(), _addr(bias),
                                                 state.data_ptr(), y.data_ptr(), handle)
        return st, y

    return _call("ssd_causal_conv_step", dev, stream, run, torch)


def _scan_args(x, dt, A, B, C, D, z, dt_bias, lengths, dt_softplus, lead, torch):
    tensor, f32 = torch.Tensor, torch.float32
    code = _input_dtype(x, torch)
    if not (isinstance(A, tensor) and isinstance(B, tensor)):
        raise TypeError("A and B must be torch.Tensor")
    dims, of_b = x.shape, B.shape
    if len(dims) != lead + 1 or len(of_b) != lead + 2 or A.dim() != 2:
        raise ValueError("x must be (batch, %schannels), B (batch, %sngroups, dstate) and A (channels, dstate)"
                         % (("seqlen, ",) * 2 if lead == 2 else ("", "")))
    dev, dtype, b, c, g, n = x.device, x.dtype, dims[0], dims[-1], of_b[-2], of_b[-1]
    L = dims[1] if lead == 2 else 1
    rows = (b, L, g, n) if lead == 2 else (b, g, n)
    shape = SelectiveShape(b, L, c, n, g, code, 0, SSD_SCAN_DT_SOFTPLUS if dt_softplus else 0)
    for name, t, want in (("x", x, dims), ("dt", dt, dims), ("B", B, rows), ("C", C, rows), ("z", z, dims)):
        if t is not None or name != "z":
            st = _rows(t, name, dtype, want, dev, tensor, lead)
            if st is not None:
                setattr(shape, name, st)
    _dense(A, "A", f32, (c, n), dev, tensor)
    if D is not None:
        _dense(D, "D", f32, (c,), dev, tensor)
    if dt_bias is not None:
        _dense(dt_bias, "dt_bias", f32, (c,), dev, tensor)
    if lengths is not None:
        _dense(lengths, "lengths", torch.int32, (b,), dev, tensor)
    return shape, dev, b, L, c, g, n


def selective_scan_fwd(x, dt, A, B, C, D=None, z=None, dt_bias=None, initial_states=None,
                       return_final_states: bool = False, *, dt_softplus: bool = True, lengths=None, y_dtype=None,
                       out=None, final_out=None, workspace=None, stream=None):
    """Selective scan over prompts (``ssd_selective_scan_fwd``): per channel
    and state h_t = exp(d_t A) h_{t-1} + d_t x_t B_t with d = softplus(dt +
    dt_bias), and y_t = (C_t h_t + D x_t) silu(z_t).

    x, dt, z (b, L, c) and B, C (b, L, g, n), n <= 64: float32 or bfloat16, all
    the same dtype, rows may lie apart (column slices of wider tensors); A
    (c, n), D and dt_bias (c,), initial_states (b, c, n): float32.  z None: no
    gate.  ``lengths``: int32 (b,) device tensor, tokens of each padded
    sequence; rows behind are 0 in y.  Returns y (``y_dtype``: float32, the
    default, or x's dtype), or (y, final_states); ``final_out`` may be
    ``initial_states`` itself.
    """
    torch = _torch()
    lib = load_library()
    shape, dev, b, L, c, g, n = _scan_args(x, dt, A, B, C, D, z, dt_bias, lengths, dt_softplus, 2, torch)
    if initial_states is not None:
        _dense(initial_states, "initial_states", torch.float32, (b, c, n), dev, torch.Tensor)
    ytype, shape.y_dtype = _result_dtype(y_dtype, x.dtype, "y_dtype", torch)
    if out is not None:
        _dense(out, "out", ytype, (b, L, c), dev, torch.Tensor)
    if final_out is not None:
        _dense(final_out, "final_out", torch.float32, (b, c, n), dev, torch.Tensor)

    def run(handle):
        y = out if out is not None else _rows_like(x, shape.x, (b, L, c), ytype, dev, torch)
        fin = final_out
        if fin is None and return_final_states:
            fin = torch.empty((b, c, n), dtype=torch.float32, device=dev)
        ws, size, _keep = _workspace(workspace, lib.ssd_selective_scan_fwd_workspace_size(ctypes.byref(shape)), dev, torch)
        st = lib.ssd_selective_scan_fwd(ctypes.byref(shape), x.data_ptr(), dt.data_ptr(), A.data_ptr(), B.data_ptr(),
                                        C.data_ptr(), _addr(D), _addr(z), _addr(dt_bias), _addr(initial_states),
                                        _addr(lengths), y.data_ptr(), _addr(fin), ws, size, handle)
        return st, (y, fin) if return_final_states else y

    return _call("ssd_selective_scan_fwd", dev, stream, run, torch)


def selective_scan_bwd(x, dt, A, B, C, D, dy, z=None, dt_bias=None, initial_states=None, d_final_states=None, *,
                       dt_softplus: bool = True, lengths=None, want_d_initial: bool = True, workspace=None,
                       stream=None):
    """Gradients through :func:`selective_scan_fwd` (``ssd_selective_scan_bwd``).

    Inputs as passed there, plus ``dy`` (b, L, c) (float32 or x's dtype, rows
    may lie apart) and optionally ``d_final_states`` (b, c, n) float32.
    Returns a dict of float32 tensors ``dx, ddt, dA, dB, dC, dD, ddt_bias``,
    ``dz`` when z is given and, when requested, ``d_initial_states``.
    """
    torch = _torch()
    lib = load_library()
    shape, dev, b, L, c, g, n = _scan_args(x, dt, A, B, C, D, z, dt_bias, lengths, dt_softplus, 2, torch)
    for name, t in (("initial_states", initial_states), ("d_final_states", d_final_states)):
        if t is not None:
            _dense(t, name, torch.float32, (b, c, n), dev, torch.Tensor)
    if not isinstance(dy, torch.Tensor):
        raise TypeError("dy must be a torch.Tensor")
    dytype, shape.y_dtype = _result_dtype(dy.dtype, x.dtype, "dy's dtype", torch)
    st = _rows(dy, "dy", dytype, x.shape, dev, torch.Tensor, 2)
    if st is not None:
        shape.dy = st

    def run(handle):
        def new(*dims):
            return torch.empty(dims, dtype=torch.float32, device=dev)

        like = torch.empty_like
        res = {"dx": new(b, L, c), "dB": new(b, L, g, n), "dA": like(A), "dD": new(c)}
        res["ddt"], res["dC"], res["ddt_bias"] = like(res["dx"]), like(res["dB"]), like(res["dD"])
        if z is not None:
            res["dz"] = like(res["dx"])
        if want_d_initial:
            res["d_initial_states"] = new(b, c, n)
        ws, size, _keep = _workspace(workspace, lib.ssd_selective_scan_bwd_workspace_size(ctypes.byref(shape)), dev, torch)
        st = lib.ssd_selective_scan_bwd(
            ctypes.byref(shape), x.data_ptr(), dt.data_ptr(), A.data_ptr(), B.data_ptr(), C.data_ptr(), _addr(D),
            _addr(z), _addr(dt_bias), _addr(initial_states), _addr(lengths), dy.data_ptr(), _addr(d_final_states),
            res["dx"].data_ptr(), res["ddt"].data_ptr(), res["dA"].data_ptr(), res["dB"].data_ptr(),
            res["dC"].data_ptr(), res["dD"].data_ptr(), _addr(res.get("dz")), res["ddt_bias"].data_ptr(),
            _addr(res.get("d_initial_states")), ws, size, handle)
        return st, res

    return _call("ssd_selective_scan_bwd", dev, stream, run, torch)


def selective_scan_step(x, dt, A, B, C, D, state, z=None, dt_bias=None, *, dt_softplus: bool = True, y_dtype=None,
                        out=None, stream=None):
    """The scan for one new token per sequence (``ssd_selective_scan_step``).

    x, dt, z (b, c) and B, C (b, g, n); ``state`` (b, c, n) float32 is updated
    in place.  Returns y (b, c) (``y_dtype``: float32, the default, or x's
    dtype).
    """
    torch = _torch()
    shape, dev, b, _, c, g, n = _scan_args(x, dt, A, B, C, D, z, dt_bias, None, dt_softplus, 1, torch)
    _dense(state, "state", torch.float32, (b, c, n), dev, torch.Tensor)
    ytype, shape.y_dtype = _result_dtype(y_dtype, x.dtype, "y_dtype", torch)
    if out is not None:
        _dense(out, "out", ytype, (b, c), dev, torch.Tensor)

    def run(handle):
        y = out if out is not None else _rows_like(x, shape.x, (b, c), ytype, dev, torch)
        st = load_library().ssd_selective_scan_step(
            ctypes.byref(shape), x.data_ptr(), dt.data_ptr(), A.data_ptr(), B.data_ptr(), C.data_ptr(), _addr(D),
            _addr(z), _addr(dt_bias), state.data_ptr(), y.data_ptr(), handle)
        return st, y

    return _call("ssd_selective_scan_step", dev, stream, run, torch)


# ---------------------------------------------------------------------------
# Sliding-window attention with sinks, and the RMS norm with the residual's addition
# ---------------------------------------------------------------------------

def _heads(t, name, dtype, shape, device, tensor, lead):
    """Checks an input of heads that may lie apart, (batch, seqlen, heads, headdim) or without seqlen (``lead`` 1), and
    returns its ssd_head_stride, None if it is dense."""
    if isinstance(t, tensor) and t.dtype == dtype and t.shape == shape and t.get_device() == device.index:
        if t.is_contiguous():
            return None
        st = t.stride()
        if st[-1] != 1 and shape[-1] != 1:
            raise ValueError("%s: each head must be contiguous (strides %s)" % (name, st))
        row = st[1] if lead == 2 and shape[1] > 1 else shape[-1]
        if row < shape[-1]:
            raise ValueError("%s: rows of different tokens overlap (strides %s)" % (name, st))
        return HeadStride(st[0] if shape[0] > 1 else 0, row, st[-2] if shape[-2] > 1 else shape[-1])
    if isinstance(t, tensor) and t.dtype == dtype and t.device == device:
        raise ValueError("%s has shape %s, expected %s" % (name, tuple(t.shape), tuple(shape)))
    return _check(t, name, dtype, shape, device)


def _attn_args(q, k, v, window, sinks, scale, lead, torch):
    tensor = torch.Tensor
    code = _input_dtype(q, torch, "q")
    if not isinstance(k, tensor):
        raise TypeError("k must be a torch.Tensor")
    dims, of_k = q.shape, k.shape
    if len(dims) != lead + 2 or len(of_k) != lead + 2:
        raise ValueError("q must be (batch, %snheads, headdim) and k (batch, %snkvheads, headdim)"
                         % (("seqlen, ",) * 2 if lead == 2 else ("", "")))
    for name, n in (("window", window), ("sinks", sinks)):
        if n is not None and not -1 << 63 <= n < 1 << 63:  # (ctypes would drop the bits above)
            raise ValueError("%s must fit 64 bits" % name)
    dev, dtype, b, h, d, kv = q.device, q.dtype, dims[0], dims[-2], dims[-1], of_k[-2]
    L = dims[1] if lead == 2 else 1
    shape = AttnShape(b, L, h, kv, d, max(L, 1) if window is None else window, sinks, d ** -0.5 if scale is None else scale,
                      code)
    kdims = dims[:lead] + (kv, d)
    for name, t, want in (("q", q, dims), ("k", k, kdims), ("v", v, kdims)):
        st = _heads(t, name, dtype, want, dev, tensor, lead)
        if st is not None:
            setattr(shape, name, st)
    return shape, dev, dtype, b, L, h, kv, d


def _cache(k_cache, v_cache, dtype, shape, dev, torch):
    for name, t in (("k_cache", k_cache), ("v_cache", v_cache)):
        _dense(t, name, dtype, (shape.batch, shape.nkvheads, shape.sinks + shape.window, shape.headdim), dev,
               torch.Tensor)


def window_attention_fwd(q, k, v, window=None, sinks: int = 0, *, scale=None, lengths=None, positions=None,
                         k_cache=None, v_cache=None, return_lse: bool = False, out=None, stream=None):
    """Causal attention over prompts in which a token sees the last ``window``
    tokens, itself among them, and the sequence's first ``sinks``
    (``ssd_window_attn_fwd``).

    q (b, L, h, d) and k, v (b, L, kv, d), h a multiple of kv, d 32, 64 or 128:
    float32 or bfloat16, all the same dtype, heads may lie apart (column slices
    of a wider projection, heads outside tokens).  ``window`` None: every earlier token of the call.
    ``scale``: d ** -0.5 if None.  ``lengths``: int32 (b,) device tensor, tokens
    of each padded sequence; rows behind are 0.  ``k_cache`` and ``v_cache``
    (b, kv, sinks + window, d) are brought up to date; with ``positions``, int32
    (b,), the tokens each sequence has behind it, the tokens in them are read
    too.  Returns y (b, L, h, d) in q's dtype, or (y, lse) with lse (b, h, L)
    float32, which :func:`window_attention_bwd` takes.
    """
    torch = _torch()
    shape, dev, dtype, b, L, h, kv, d = _attn_args(q, k, v, window, sinks, scale, 2, torch)
    if lengths is not None:
        _dense(lengths, "lengths", torch.int32, (b,), dev, torch.Tensor)
    if positions is not None:
        _dense(positions, "positions", torch.int32, (b,), dev, torch.Tensor)
    if k_cache is not None or v_cache is not None or positions is not None:
        if window is None:
            raise ValueError("a cache needs a window")
        _cache(k_cache, v_cache, dtype, shape, dev, torch)
    if out is not None:
        _dense(out, "out", dtype, (b, L, h, d), dev, torch.Tensor)

    def run(handle):
        y = out if out is not None else _rows_like(q, shape.q, (b, L, h, d), dtype, dev, torch)
        lse = torch.empty((b, h, L), dtype=torch.float32, device=dev) if return_lse else None
        st = load_library().ssd_window_attn_fwd(ctypes.byref(shape), q.data_ptr(), k.data_ptr(), v.data_ptr(),
                                                _addr(positions), _addr(lengths), _addr(k_cache), _addr(v_cache),
                                                y.data_ptr(), _addr(lse), handle)
        return st, (y, lse) if return_lse else y

    return _call("ssd_window_attn_fwd", dev, stream, run, torch)


def window_attention_bwd(q, k, v, y, lse, dy, window=None, sinks: int = 0, *, scale=None, lengths=None, workspace=None,
                         stream=None):
    """Gradients through :func:`window_attention_fwd` without positions (``ssd_window_attn_bwd``).

    Inputs as passed there, ``y`` and ``lse`` as it returned them, and ``dy``
    (b, L, h, d) in q's dtype, heads may lie apart.  Returns a dict of ``dq``,
    ``dk`` and ``dv`` in q's dtype.
    """
    torch = _torch()
    lib = load_library()
    shape, dev, dtype, b, L, h, kv, d = _attn_args(q, k, v, window, sinks, scale, 2, torch)
    _dense(lse, "lse", torch.float32, (b, h, L), dev, torch.Tensor)
    for name, t in (("y", y), ("dy", dy)):
        st = _heads(t, name, dtype, q.shape, dev, torch.Tensor, 2)
        if st is not None:
            setattr(shape, name, st)
    if lengths is not None:
        _dense(lengths, "lengths", torch.int32, (b,), dev, torch.Tensor)

    def run(handle):
        res = {"dq": _rows_like(q, shape.q, (b, L, h, d), dtype, dev, torch),
               "dk": _rows_like(k, shape.k, (b, L, kv, d), dtype, dev, torch)}
        res["dv"] = torch.empty_like(res["dk"])
        ws, size, _keep = _workspace(workspace, lib.ssd_window_attn_bwd_workspace_size(ctypes.byref(shape)), dev, torch)
        st = lib.ssd_window_attn_bwd(ctypes.byref(shape), q.data_ptr(), k.data_ptr(), v.data_ptr(), y.data_ptr(),
                                     lse.data_ptr(), dy.data_ptr(), _addr(lengths), res["dq"].data_ptr(),
                                     res["dk"].data_ptr(), res["dv"].data_ptr(), ws, size, handle)
        return st, res

    return _call("ssd_window_attn_bwd", dev, stream, run, torch)


def window_attention_step(q, k, v, k_cache, v_cache, positions, window, sinks: int = 0, *, scale=None, out=None,
                          workspace=None, stream=None):
    """The attention for one new token per sequence (``ssd_window_attn_step``).

    q (b, h, d), k and v (b, kv, d); ``k_cache`` and ``v_cache`` (b, kv, sinks +
    window, d) take the new token's and are read whole.  ``positions``: int32
    (b,) device tensor, the new token's own (the tokens before it); negative
    for an empty place of the batch, whose row is 0.  It is not changed: the
    layers of a model share it.  Returns y (b, h, d) in q's dtype.
    """
    torch = _torch()
    lib = load_library()
    if window is None:
        raise ValueError("a cache needs a window")
    shape, dev, dtype, b, _, h, kv, d = _attn_args(q, k, v, window, sinks, scale, 1, torch)
    _dense(positions, "positions", torch.int32, (b,), dev, torch.Tensor)
    _cache(k_cache, v_cache, dtype, shape, dev, torch)
    if out is not None:
        _dense(out, "out", dtype, (b, h, d), dev, torch.Tensor)

    def run(handle):
        y = out if out is not None else _rows_like(q, shape.q, (b, h, d), dtype, dev, torch)
        ws, size, _keep = _workspace(workspace, lib.ssd_window_attn_step_workspace_size(ctypes.byref(shape)), dev, torch)
        st = lib.ssd_window_attn_step(ctypes.byref(shape), q.data_ptr(), k.data_ptr(), v.data_ptr(),
                                      positions.data_ptr(), k_cache.data_ptr(), v_cache.data_ptr(), y.data_ptr(), ws,
                                      size, handle)
        return st, y

    return _call("ssd_window_attn_step", dev, stream, run, torch)


def _stored(t, name, torch):
    if not isinstance(t, torch.Tensor):
        raise TypeError("%s must be a torch.Tensor" % name)
    if t.dtype == torch.bfloat16:
        return SSD_DTYPE_BF16
    if t.dtype == torch.float32:
        return SSD_DTYPE_F32
    raise TypeError("%s must be float32 or bfloat16" % name)


def _norm_args(x, name, weight, eps, lengths, torch):
    code = _input_dtype(x, torch, name)
    dims, dev = x.shape, x.device
    if len(dims) == 3:
        shape = NormShape(dims[0], dims[1], dims[2], eps, code, code, code)
    elif len(dims) == 2:
        shape = NormShape(1, dims[0], dims[1], eps, code, code, code)
    else:
        raise ValueError("%s must be (tokens, channels) or (batch, seqlen, channels)" % name)
    if weight is not None:
        _dense(weight, "weight", torch.float32, (dims[-1],), dev, torch.Tensor)
    if lengths is not None:
        if len(dims) == 2:
            raise ValueError("lengths belong to (batch, seqlen, channels)")
        _dense(lengths, "lengths", torch.int32, (dims[0],), dev, torch.Tensor)
    return shape, dev, dims


def _norm_rows(t, name, dtype, shape, device, torch):
    """:func:`_rows` of tokens in one or two dimensions."""
    if isinstance(t, torch.Tensor) and t.dtype == dtype and t.shape == shape and t.get_device() == device.index \
            and t.is_contiguous():
        return None
    if len(shape) == 2 and isinstance(t, torch.Tensor) and t.dim() == 2:
        return _rows(t[None], name, dtype, (1, *shape), device, torch.Tensor, 2)
    return _rows(t, name, dtype, shape, device, torch.Tensor, 2)


def rms_norm_fwd(x, weight=None, residual=None, *, eps: float = 1e-5, lengths=None, y_dtype=None, scale_block: int = 0,
                 return_residual: bool = False, residual_dtype=None, out=None, scales_out=None, residual_out=None,
                 stream=None):
    """Root-mean-square norm over the last dimension of x + residual
    (``ssd_rms_norm_fwd``): u = x + residual, y = u (mean(u^2) + eps)^-1/2 weight.

    x and ``residual`` (b, L, c) or (tokens, c): float32 or bfloat16 each, rows may
    lie apart; weight (c,) float32, None: 1.  ``y_dtype``: float32, the default,
    x's dtype, or torch.float8_e4m3fn with a float32 scale for each row
    (``scale_block`` 0) or each 32, 64 or 128 columns of it, y being code times
    scale.  ``lengths``: int32 (b,) device tensor, tokens of each padded
    sequence; rows behind are 0.  Returns y, followed by the scales (b, L,
    blocks) of an 8-bit y and, if asked for, u in the residual's dtype
    (``residual_dtype``, float32 if None, where there is no residual);
    ``residual_out`` may be ``residual`` itself.
    """
    torch = _torch()
    shape, dev, dims = _norm_args(x, "x", weight, eps, lengths, torch)
    st = _norm_rows(x, "x", x.dtype, dims, dev, torch)
    if st is not None:
        shape.x = st
    rtype = torch.float32 if residual_dtype is None else residual_dtype
    if residual is not None:
        shape.res_dtype, rtype = _stored(residual, "residual", torch), residual.dtype
        st = _norm_rows(residual, "residual", rtype, dims, dev, torch)
        if st is not None:
            shape.residual = st
    elif rtype not in (torch.float32, torch.bfloat16):
        raise TypeError("residual_dtype must be float32 or bfloat16")
    else:
        shape.res_dtype = SSD_DTYPE_F32 if rtype == torch.float32 else SSD_DTYPE_BF16
    codes = y_dtype == torch.float8_e4m3fn
    if codes:
        ytype, shape.y_dtype, shape.scale_block = y_dtype, SSD_DTYPE_E4M3, scale_block
        if scale_block not in (0, 32, 64, 128):
            raise ValueError("scale_block must be 0 (the row), 32, 64 or 128")
        sdims = dims[:-1] + (-(-dims[-1] // scale_block) if scale_block else 1,)
        if scales_out is not None:
            _dense(scales_out, "scales_out", torch.float32, sdims, dev, torch.Tensor)
    else:
        ytype, shape.y_dtype = _result_dtype(y_dtype, x.dtype, "y_dtype", torch)
        if scale_block != 0 or scales_out is not None:
            raise ValueError("scales belong to an 8-bit y")
    if out is not None:
        _dense(out, "out", ytype, dims, dev, torch.Tensor)
    if residual_out is not None:
        _dense(residual_out, "residual_out", rtype, dims, dev, torch.Tensor)

    def run(handle):
        y = out if out is not None else _rows_like(x, shape.x, dims, ytype, dev, torch)
        scales, u = scales_out, residual_out
        if codes and scales is None:
            scales = torch.empty(sdims, dtype=torch.float32, device=dev)
        if u is None and return_residual:
            u = torch.empty(dims, dtype=rtype, device=dev) if residual is None else \
                _rows_like(residual, shape.residual, dims, rtype, dev, torch)
        st = load_library().ssd_rms_norm_fwd(ctypes.byref(shape), x.data_ptr(), _addr(residual), _addr(weight),
                                             _addr(lengths), y.data_ptr(), _addr(scales), _addr(u), handle)
        got = (y,) + ((scales,) if codes else ()) + ((u,) if return_residual else ())
        return st, got if len(got) > 1 else y

    return _call("ssd_rms_norm_fwd", dev, stream, run, torch)


def rms_norm_bwd(dy, u, weight=None, d_residual=None, *, eps: float = 1e-5, lengths=None, dx_dtype=None,
                 want_dresidual: bool = False, want_dweight: bool = True, workspace=None, stream=None):
    """Gradients through :func:`rms_norm_fwd` (``ssd_rms_norm_bwd``).

    ``dy`` and ``u`` (b, L, c) or (tokens, c), u being x + residual as the forward
    pass returns it (or x): float32 or bfloat16 each, rows may lie apart;
    ``d_residual`` in u's dtype, what reaches u by way of the residual stream.
    Returns a dict of ``dx`` (``dx_dtype``: float32, the default, or bfloat16)
    and, when requested, ``dresidual``, the same gradient in u's dtype, and
    ``dweight`` (float32).
    """
    torch = _torch()
    lib = load_library()
    shape, dev, dims = _norm_args(u, "u", weight, eps, lengths, torch)
    shape.y_dtype = _stored(dy, "dy", torch)
    for name, t, dtype, field in (("u", u, u.dtype, "residual"), ("dy", dy, dy.dtype, "dy"),
                                  ("d_residual", d_residual, u.dtype, "dres")):
        if t is not None:
            st = _norm_rows(t, name, dtype, dims, dev, torch)
            if st is not None:
                setattr(shape, field, st)
    xtype = torch.float32 if dx_dtype is None else dx_dtype
    if xtype not in (torch.float32, torch.bfloat16):
        raise TypeError("dx_dtype must be float32 or bfloat16")
    shape.dtype = SSD_DTYPE_F32 if xtype == torch.float32 else SSD_DTYPE_BF16

    def run(handle):
        res = {"dx": _rows_like(u, shape.residual, dims, xtype, dev, torch)}
        if want_dresidual:
            res["dresidual"] = _rows_like(u, shape.residual, dims, u.dtype, dev, torch)
        if want_dweight:
            res["dweight"] = torch.empty((dims[-1],), dtype=torch.float32, device=dev) if weight is None else \
                torch.empty_like(weight)
        ws, size, _keep = _workspace(workspace, lib.ssd_rms_norm_bwd_workspace_size(ctypes.byref(shape)), dev, torch)
        st = lib.ssd_rms_norm_bwd(ctypes.byref(shape), dy.data_ptr(), u.data_ptr(), _addr(weight), _addr(d_residual),
                                  _addr(lengths), res["dx"].data_ptr(), _addr(res.get("dresidual")),
                                  _addr(res.get("dweight")), ws, size, handle)
        return st, res

    return _call("ssd_rms_norm_bwd", dev, stream, run, torch)
