"""Python binding of the C ABI in include/caat.h (argument marshalling only).

Every step of the path runs in the CUDA kernels of libcaat.so; this module only turns torch
tensors into pointers, sizes and a stream, calls the library and turns error codes into
exceptions.  There is no fallback: if libcaat.so is missing or fails to load, every call
raises.
"""
from __future__ import annotations

import array
import ctypes
import importlib.util
import os
import struct
import sys
from typing import Optional

import numpy as np

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libcaat.so")

CAAT_OK = 0
CAAT_ERR_INVALID_ARG = 1
CAAT_ERR_UNSUPPORTED = 2
CAAT_ERR_CUDA = 3
CAAT_ERR_TIMEOUT = 4
CAAT_ERR_WORKSPACE = 5

CAAT_VARIANT_ROWPAR = 0
CAAT_VARIANT_MLP = 1
CAAT_VARIANT_ROWPAR_HOST = 2
CAAT_VARIANT_ROWPAR_BWD = 4
CAAT_BWD_FLAG_TRANSPOSED_OPERANDS = 0x1

CAAT_FLAG_FORCE_GEMM_PATH = 0x1
CAAT_FLAG_FORCE_DECODE_PATH = 0x2
CAAT_FLAG_SINGLE_CTA = 0x4
CAAT_FLAG_FUSED_NORM = 0x8
CAAT_FLAG_ORDER_ROWBLOCK = 0x10
CAAT_FLAG_OVERLAP_NORM = 0x20
CAAT_FLAG_ORDER_GROUPED = 0x40
CAAT_FLAG_W_PERMUTED = 0x80
CAAT_FLAG_TEST_STALL = 0x100
CAAT_FLAG_NORM_BESIDE_GEMM = 0x200

CAAT_NOALLOC_SCRATCH_BYTES = 1048576

CAAT_ROPE_SCALING_NONE = 0
CAAT_ROPE_SCALING_LINEAR = 1
CAAT_ROPE_SCALING_NTK = 2
CAAT_ROPE_SCALING_YARN = 3
CAAT_ROPE_FLAG_INTERLEAVED = 0x1
CAAT_ROPE_FLAG_BACKWARD = 0x2
CAAT_VARIANT_ATTN = 0
CAAT_VARIANT_ATTN_BWD = 1
CAAT_VARIANT_ATTN_DECODE = 2

# Every symbol include/caat.h declares (checked by the ABI tests).
EXPORTS = [
    "caat_rowpar_forward", "caat_rowpar_forward_ex", "caat_rowpar_forward_host",
    "caat_rowpar_forward_noalloc", "caat_mlp_forward", "caat_mlp_forward_ex",
    "caat_workspace_size", "caat_sync_mask", "caat_get_device_status", "caat_timing_create",
    "caat_timing_destroy", "caat_timing_reset", "caat_timing_read", "caat_status_string",
    "caat_version", "caat_permute_weights", "caat_speedup_model", "caat_rowpar_backward",
    "caat_plan_create", "caat_plan_execute", "caat_plan_destroy", "caat_rowpar_tp_local",
    "caat_rowpar_tp_finish", "caat_rowpar_tp_local_push", "caat_rowpar_tp_reduce", "caat_rowpar_tp_finish_wait",
    "caat_rope_frequencies", "caat_rope", "caat_attn_forward", "caat_attn_backward", "caat_attn_decode",
    "caat_attn_workspace_size",
]

CAAT_TP_MAX_WORLD = 8


class CaatError(RuntimeError):
    def __init__(self, code: int, what: str):
        self.code = code
        super().__init__(f"{what}: {status_string(code)} ({code})")


class RowparArgs(ctypes.Structure):
    _fields_ = [
        ("X", ctypes.c_void_p), ("W", ctypes.c_void_p), ("residual", ctypes.c_void_p),
        ("gamma", ctypes.c_void_p), ("sync_idx", ctypes.c_void_p), ("out", ctypes.c_void_p),
        ("h_out", ctypes.c_void_p), ("workspace", ctypes.c_void_p), ("ws_bytes", ctypes.c_size_t),
        ("stream", ctypes.c_void_p), ("timing", ctypes.c_void_p),
        ("T", ctypes.c_int64), ("K", ctypes.c_int64), ("H", ctypes.c_int64),
        ("p", ctypes.c_double), ("eps", ctypes.c_float), ("private_scale", ctypes.c_float),
        ("P", ctypes.c_int32), ("flags", ctypes.c_uint32),
    ]


class BwdArgs(ctypes.Structure):
    _fields_ = [
        ("X", ctypes.c_void_p), ("W", ctypes.c_void_p), ("h", ctypes.c_void_p), ("gamma", ctypes.c_void_p),
        ("dout", ctypes.c_void_p), ("sync_idx", ctypes.c_void_p), ("dX", ctypes.c_void_p),
        ("dW", ctypes.c_void_p), ("dR", ctypes.c_void_p), ("dgamma", ctypes.c_void_p),
        ("workspace", ctypes.c_void_p), ("ws_bytes", ctypes.c_size_t), ("stream", ctypes.c_void_p),
        ("timing", ctypes.c_void_p), ("T", ctypes.c_int64), ("K", ctypes.c_int64), ("H", ctypes.c_int64),
        ("p", ctypes.c_double), ("eps", ctypes.c_float), ("private_scale", ctypes.c_float),
        ("P", ctypes.c_int32), ("flags", ctypes.c_uint32),
    ]


class TpArgs(ctypes.Structure):
    _fields_ = [
        ("X", ctypes.c_void_p), ("W", ctypes.c_void_p), ("residual", ctypes.c_void_p),
        ("gamma", ctypes.c_void_p), ("zs", ctypes.c_void_p), ("h", ctypes.c_void_p), ("out", ctypes.c_void_p),
        ("workspace", ctypes.c_void_p), ("ws_bytes", ctypes.c_size_t), ("stream", ctypes.c_void_p),
        ("timing", ctypes.c_void_p), ("T", ctypes.c_int64), ("K_r", ctypes.c_int64), ("H", ctypes.c_int64),
        ("p", ctypes.c_double), ("eps", ctypes.c_float), ("private_scale", ctypes.c_float),
        ("flags", ctypes.c_uint32),
    ]


class TpPeers(ctypes.Structure):
    _fields_ = [
        ("world", ctypes.c_int32), ("rank", ctypes.c_int32), ("epoch", ctypes.c_uint32),
        ("recv", ctypes.c_void_p * CAAT_TP_MAX_WORLD), ("gather", ctypes.c_void_p * CAAT_TP_MAX_WORLD),
        ("flags", ctypes.c_void_p * CAAT_TP_MAX_WORLD),
    ]


class MlpArgs(ctypes.Structure):
    _fields_ = [
        ("X", ctypes.c_void_p), ("A", ctypes.c_void_p), ("W2", ctypes.c_void_p),
        ("residual", ctypes.c_void_p), ("gamma", ctypes.c_void_p), ("sync_idx", ctypes.c_void_p),
        ("out", ctypes.c_void_p), ("h_out", ctypes.c_void_p), ("workspace", ctypes.c_void_p),
        ("ws_bytes", ctypes.c_size_t), ("stream", ctypes.c_void_p), ("timing", ctypes.c_void_p),
        ("T", ctypes.c_int64), ("H", ctypes.c_int64), ("F", ctypes.c_int64),
        ("p", ctypes.c_double), ("eps", ctypes.c_float), ("private_scale", ctypes.c_float),
        ("P", ctypes.c_int32), ("flags", ctypes.c_uint32),
    ]


class RopeArgs(ctypes.Structure):
    _fields_ = [
        ("q", ctypes.c_void_p), ("k", ctypes.c_void_p), ("v", ctypes.c_void_p), ("q_out", ctypes.c_void_p),
        ("k_out", ctypes.c_void_p), ("v_out", ctypes.c_void_p), ("positions", ctypes.c_void_p),
        ("slots", ctypes.c_void_p), ("inv_freq", ctypes.c_void_p), ("stream", ctypes.c_void_p),
        ("timing", ctypes.c_void_p), ("T", ctypes.c_int64), ("cache_rows", ctypes.c_int64),
        ("q_stride_rank", ctypes.c_int64), ("q_stride_token", ctypes.c_int64), ("k_stride_rank", ctypes.c_int64),
        ("k_stride_token", ctypes.c_int64), ("v_stride_rank", ctypes.c_int64), ("v_stride_token", ctypes.c_int64),
        ("P", ctypes.c_int32), ("heads_q", ctypes.c_int32), ("heads_k", ctypes.c_int32), ("dh", ctypes.c_int32),
        ("rot", ctypes.c_int32), ("mscale", ctypes.c_float), ("flags", ctypes.c_uint32),
    ]


_ATTN_TAIL = [
    ("cu_q", ctypes.c_void_p), ("cu_k", ctypes.c_void_p), ("workspace", ctypes.c_void_p),
    ("ws_bytes", ctypes.c_size_t), ("stream", ctypes.c_void_p), ("timing", ctypes.c_void_p),
    ("Tq", ctypes.c_int64), ("Tk", ctypes.c_int64), ("q_stride_rank", ctypes.c_int64),
    ("q_stride_token", ctypes.c_int64), ("k_stride_rank", ctypes.c_int64), ("k_stride_token", ctypes.c_int64),
    ("v_stride_rank", ctypes.c_int64), ("v_stride_token", ctypes.c_int64), ("n_seq", ctypes.c_int32),
    ("P", ctypes.c_int32), ("heads_q", ctypes.c_int32), ("heads_k", ctypes.c_int32), ("dh", ctypes.c_int32),
    ("scale", ctypes.c_float), ("flags", ctypes.c_uint32),
]


class AttnArgs(ctypes.Structure):
    _fields_ = [("q", ctypes.c_void_p), ("k", ctypes.c_void_p), ("v", ctypes.c_void_p), ("out", ctypes.c_void_p),
                ("lse", ctypes.c_void_p)] + _ATTN_TAIL


class AttnBwdArgs(ctypes.Structure):
    _fields_ = [("q", ctypes.c_void_p), ("k", ctypes.c_void_p), ("v", ctypes.c_void_p), ("out", ctypes.c_void_p),
                ("lse", ctypes.c_void_p), ("dout", ctypes.c_void_p), ("dq", ctypes.c_void_p), ("dk", ctypes.c_void_p),
                ("dv", ctypes.c_void_p)] + _ATTN_TAIL


class AttnDecodeArgs(ctypes.Structure):
    _fields_ = [
        ("q", ctypes.c_void_p), ("k_cache", ctypes.c_void_p), ("v_cache", ctypes.c_void_p), ("lens", ctypes.c_void_p),
        ("out", ctypes.c_void_p), ("workspace", ctypes.c_void_p), ("ws_bytes", ctypes.c_size_t),
        ("stream", ctypes.c_void_p), ("timing", ctypes.c_void_p), ("B", ctypes.c_int64), ("capacity", ctypes.c_int64),
        ("q_stride_rank", ctypes.c_int64), ("q_stride_token", ctypes.c_int64), ("P", ctypes.c_int32),
        ("heads_q", ctypes.c_int32), ("heads_k", ctypes.c_int32), ("dh", ctypes.c_int32), ("scale", ctypes.c_float),
        ("flags", ctypes.c_uint32),
    ]


# The attention block's calls are short enough for the marshalling to show: ordinary ones go through
# the compiled marshalling, the others have their arguments packed in one go (native layout, the same as the structures above) and passed as bytes.
_PACK_ROPE = struct.Struct("@11P8q5ifI0P")
_PACK_ATTN = struct.Struct("@5P2PPN2P8q5ifI0P")
_PACK_ATTN_BWD = struct.Struct("@9P2PPN2P8q5ifI0P")
_PACK_ATTN_DECODE = struct.Struct("@6PN2P4q4ifI0P")
_PACKED = {"caat_rope": (_PACK_ROPE, RopeArgs), "caat_attn_forward": (_PACK_ATTN, AttnArgs),
           "caat_attn_backward": (_PACK_ATTN_BWD, AttnBwdArgs), "caat_attn_decode": (_PACK_ATTN_DECODE, AttnDecodeArgs)}

_SIZE_MAX = ctypes.c_size_t(-1).value
_lib = None
_marshal = None  # the compiled marshalling of the attention block's calls, bound to the library
_marshal_sought = False


def _bind_marshal(L):
    """Loads the compiled marshalling and gives it the library's functions.  Built for another PyTorch or
    interpreter, or not at all, it is left out: the calls are then marshalled here, which takes the host 5 us
    longer."""
    global _marshal, _marshal_sought
    import torch
    from . import build
    _marshal, _marshal_sought = None, True
    name = __package__ + "._marshal"
    spec = importlib.util.spec_from_file_location(name, build.marshal_path(torch.__version__))
    try:
        m = importlib.util.module_from_spec(spec)
        spec.loader.exec_module(m)
    except ImportError:
        return
    m.bind(*(ctypes.cast(f, ctypes.c_void_p).value for f in (
        L.caat_rope, L.caat_attn_forward, L.caat_attn_backward, L.caat_attn_decode, L.caat_attn_workspace_size)))
    _marshal = m


def _fast():
    """The compiled marshalling (or None), after the library has been loaded."""
    L = lib()
    if not _marshal_sought:
        _bind_marshal(L)
    return _marshal


def lib() -> ctypes.CDLL:
    """Loads libcaat.so (raises if it is missing: there is no fallback path)."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(LIB_PATH):
        raise RuntimeError(f"libcaat.so not built ({LIB_PATH}); run `python -m partial_activation_sync_caat_b200.build`")
    L = ctypes.CDLL(LIB_PATH)
    i64, i32, u32, dbl, vp, sz = (ctypes.c_int64, ctypes.c_int32, ctypes.c_uint32, ctypes.c_double,
                                  ctypes.c_void_p, ctypes.c_size_t)
    L.caat_rowpar_forward.argtypes = [vp, vp, vp, vp, vp, ctypes.c_int, dbl, vp, i64, i64, i64, vp, sz, vp]
    L.caat_rowpar_forward.restype = ctypes.c_int
    L.caat_rowpar_forward_ex.argtypes = [ctypes.POINTER(RowparArgs)]
    L.caat_rowpar_forward_ex.restype = ctypes.c_int
    L.caat_rowpar_forward_host.argtypes = [ctypes.POINTER(RowparArgs)]
    L.caat_rowpar_forward_host.restype = ctypes.c_int
    L.caat_rowpar_forward_noalloc.argtypes = [ctypes.POINTER(RowparArgs)]
    L.caat_rowpar_forward_noalloc.restype = ctypes.c_int
    L.caat_mlp_forward.argtypes = [vp, vp, vp, vp, vp, vp, ctypes.c_int, dbl, vp, i64, i64, i64, vp, sz, vp]
    L.caat_mlp_forward.restype = ctypes.c_int
    L.caat_mlp_forward_ex.argtypes = [ctypes.POINTER(MlpArgs)]
    L.caat_mlp_forward_ex.restype = ctypes.c_int
    L.caat_workspace_size.argtypes = [i64, i64, i64, ctypes.c_int, ctypes.c_int]
    L.caat_workspace_size.restype = sz
    L.caat_sync_mask.argtypes = [i64, dbl, vp, vp, ctypes.POINTER(i64)]
    L.caat_plan_create.restype = ctypes.c_int
    L.caat_plan_create.argtypes = [ctypes.POINTER(RowparArgs), ctypes.POINTER(vp)]
    L.caat_plan_execute.restype = ctypes.c_int
    L.caat_plan_execute.argtypes = [vp, vp]
    L.caat_plan_destroy.restype = ctypes.c_int
    L.caat_plan_destroy.argtypes = [vp]
    L.caat_rowpar_tp_local.argtypes = [ctypes.POINTER(TpArgs)]
    L.caat_rowpar_tp_local.restype = ctypes.c_int
    L.caat_rowpar_tp_finish.argtypes = [ctypes.POINTER(TpArgs)]
    for name in ("caat_rowpar_tp_local_push", "caat_rowpar_tp_reduce", "caat_rowpar_tp_finish_wait"):
        getattr(L, name).argtypes = [ctypes.POINTER(TpArgs), ctypes.POINTER(TpPeers)]
        getattr(L, name).restype = ctypes.c_int
    L.caat_rowpar_tp_finish.restype = ctypes.c_int
    L.caat_rowpar_backward.restype = ctypes.c_int
    L.caat_rowpar_backward.argtypes = [ctypes.POINTER(BwdArgs)]
    L.caat_speedup_model.restype = ctypes.c_int
    L.caat_speedup_model.argtypes = [dbl, dbl, dbl, dbl, dbl, ctypes.POINTER(dbl), ctypes.POINTER(dbl)]
    L.caat_rope_frequencies.argtypes = [ctypes.c_int, dbl, ctypes.c_int, dbl, dbl, vp, ctypes.POINTER(ctypes.c_float)]
    L.caat_rope_frequencies.restype = ctypes.c_int
    for name, args in (("caat_rope", RopeArgs), ("caat_attn_forward", AttnArgs), ("caat_attn_backward", AttnBwdArgs),
                       ("caat_attn_decode", AttnDecodeArgs)):
        getattr(L, name).argtypes = [ctypes.POINTER(args)]
        getattr(L, name).restype = ctypes.c_int
    for name, (packed, args) in _PACKED.items():
        assert packed.size == ctypes.sizeof(args), name
        fast = L[name]  # a function object of its own
        fast.argtypes, fast.restype = [ctypes.c_char_p], ctypes.c_int
        setattr(L, "packed_" + name, fast)
    L.caat_attn_workspace_size.argtypes = [i64, i64] + [ctypes.c_int] * 6
    L.caat_attn_workspace_size.restype = sz
    L.caat_permute_weights.restype = ctypes.c_int
    L.caat_permute_weights.argtypes = [vp, vp, vp, dbl, ctypes.c_int, i64, i64, vp]
    L.caat_sync_mask.restype = ctypes.c_int
    L.caat_get_device_status.argtypes = [vp, ctypes.POINTER(i32)]
    L.caat_get_device_status.restype = ctypes.c_int
    L.caat_timing_create.argtypes = [ctypes.c_int, ctypes.POINTER(vp)]
    L.caat_timing_create.restype = ctypes.c_int
    L.caat_timing_destroy.argtypes = [vp]
    L.caat_timing_destroy.restype = ctypes.c_int
    L.caat_timing_reset.argtypes = [vp]
    L.caat_timing_reset.restype = ctypes.c_int
    L.caat_timing_read.argtypes = [vp, ctypes.POINTER(ctypes.c_float), ctypes.c_int, ctypes.c_int,
                                   ctypes.POINTER(ctypes.c_int), ctypes.POINTER(ctypes.c_int)]
    L.caat_timing_read.restype = ctypes.c_int
    L.caat_status_string.argtypes = [ctypes.c_int]
    L.caat_status_string.restype = ctypes.c_char_p
    L.caat_version.argtypes = []
    L.caat_version.restype = ctypes.c_char_p
    _lib = L
    if sys.modules.get("torch") is not None:  # else with the first call that needs it: host-only ones do not
        _bind_marshal(L)
    return L


def status_string(code: int) -> str:
    return lib().caat_status_string(int(code)).decode()


def version() -> str:
    return lib().caat_version().decode()


def _check(code: int, what: str):
    if code != CAAT_OK:
        raise CaatError(code, what)


# ---------------------------------------------------------------------------------------
# marshalling helpers
# ---------------------------------------------------------------------------------------

def _ptr(t) -> Optional[int]:
    if t is None:
        return None
    import torch
    if not isinstance(t, torch.Tensor):
        raise TypeError("expected a torch.Tensor")
    if not t.is_contiguous():
        raise ValueError("tensors must be contiguous")
    return t.data_ptr()


def _bf16_dev(t, name):
    import torch
    if t.dtype != torch.bfloat16:
        raise TypeError(f"{name} must be bfloat16")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    return _ptr(t)


def _stream_ptr(stream) -> Optional[int]:
    import torch
    if stream is None:
        stream = torch.cuda.current_stream()
    return stream.cuda_stream or None


def _sync_idx_host(sync_idx):
    if sync_idx is None:
        return None, None
    arr = np.ascontiguousarray(np.asarray(sync_idx, dtype=np.int32))
    return arr, arr.ctypes.data


# ---------------------------------------------------------------------------------------
# host-only bookkeeping
# ---------------------------------------------------------------------------------------

def caat_sync_mask(H: int, p: float, sync_idx=None):
    """(mask uint8[H], n_s) as computed by the library on the host (no GPU needed)."""
    mask = np.zeros(int(H), dtype=np.uint8)
    ns = ctypes.c_int64(0)
    arr, ptr = _sync_idx_host(sync_idx)
    code = lib().caat_sync_mask(int(H), float(p), ptr, mask.ctypes.data, ctypes.byref(ns))
    _check(code, "caat_sync_mask")
    return mask, int(ns.value)


def caat_speedup_model(h: float, s: float, r: float, p: float, C: float):
    """(speedup, p_star) of the paper's model (App. C Eq. 34-35); host only."""
    sp, ps = ctypes.c_double(0.0), ctypes.c_double(0.0)
    _check(lib().caat_speedup_model(float(h), float(s), float(r), float(p), float(C), ctypes.byref(sp),
                                    ctypes.byref(ps)), "caat_speedup_model")
    return sp.value, ps.value


def caat_permute_weights(W, W_out, sync_idx, P: int, p: float, stream=None):
    """W_out[m, i] = W[m, perm(i)]: the shared channels first, then the private ones (both
    ascending).  W, W_out: device bf16 [P, H, K/P], not overlapping.  Asynchronous."""
    P_, H, Kp = W.shape
    if P_ != P or tuple(W_out.shape) != tuple(W.shape):
        raise CaatError(CAAT_ERR_INVALID_ARG, "caat_permute_weights: shapes")
    arr, ptr = _sync_idx_host(sync_idx)
    code = lib().caat_permute_weights(_ptr(W), _ptr(W_out), ptr, float(p), int(P), int(H), int(Kp * P),
                                      _stream_ptr(stream))
    _check(code, "caat_permute_weights")


def caat_workspace_size(T: int, K: int, H: int, P: int, variant: int = CAAT_VARIANT_ROWPAR) -> int:
    n = lib().caat_workspace_size(int(T), int(K), int(H), int(P), int(variant))
    if n == ctypes.c_size_t(-1).value:
        raise CaatError(CAAT_ERR_INVALID_ARG, "caat_workspace_size")
    return int(n)


def alloc_workspace(nbytes: int, device=None, stream=None):
    """A device buffer for the workspace (allocated by torch, owned by the caller) of calls on `stream`
    (None: the current one).  It comes from that stream's pool: one from another stream's may have just been
    freed by work that is still queued there, and may be handed out again while the calls run."""
    import torch
    n = max(256, (int(nbytes) + 255) // 256 * 256)
    if stream is None:
        return torch.empty(n, dtype=torch.uint8, device="cuda" if device is None else device)
    with torch.cuda.stream(stream):
        return torch.empty(n, dtype=torch.uint8, device="cuda" if device is None else device)


# ---------------------------------------------------------------------------------------
# forward calls
# ---------------------------------------------------------------------------------------

def caat_rowpar_forward(X, W, residual, gamma, sync_idx, P: int, p: float, out, *, workspace=None,
                        h_out=None, eps: float = 1e-5, private_scale: float = 1.0, flags: int = 0,
                        stream=None, timing=None):
    """Queues the partially synchronized row-parallel layer + residual + RMSNorm.

    X [P,T,K/P], W [P,H,K/P], residual [P,T,H], gamma [H], out [P,T,H] (bf16 CUDA tensors);
    sync_idx: None (first floor(H p) channels) or a host int list of floor(H p) channels.
    """
    P = int(P)
    T = int(X.shape[1])
    K = int(X.shape[2]) * P
    H = int(W.shape[1])
    if workspace is None:
        workspace = alloc_workspace(caat_workspace_size(T, K, H, P, CAAT_VARIANT_ROWPAR), X.device, stream)
    arr, idx_ptr = _sync_idx_host(sync_idx)
    a = RowparArgs()
    a.X = _bf16_dev(X, "X")
    a.W = _bf16_dev(W, "W")
    a.residual = _bf16_dev(residual, "residual")
    a.gamma = _bf16_dev(gamma, "gamma")
    a.sync_idx = idx_ptr
    a.out = _bf16_dev(out, "out")
    a.h_out = _bf16_dev(h_out, "h_out") if h_out is not None else None
    a.workspace = _ptr(workspace)
    a.ws_bytes = workspace.numel() * workspace.element_size()
    a.stream = _stream_ptr(stream)
    a.timing = timing.handle if timing is not None else None
    a.T, a.K, a.H = T, K, H
    a.p = float(p)
    a.eps = float(eps)
    a.private_scale = float(private_scale)
    a.P = P
    a.flags = int(flags)
    _check(lib().caat_rowpar_forward_ex(ctypes.byref(a)), "caat_rowpar_forward")
    return out


class Plan:
    """A caat_plan: the row-parallel call with its buffers bound once; execute() only queues
    the kernels.  The tensors given at creation must outlive the plan (they are kept here)."""

    def __init__(self, X, W, residual, gamma, sync_idx, P: int, p: float, out, *, workspace=None, h_out=None,
                 eps: float = 1e-5, private_scale: float = 1.0, flags: int = 0):
        P = int(P)
        T, K, H = int(X.shape[1]), int(X.shape[2]) * P, int(W.shape[1])
        if workspace is None:
            workspace = alloc_workspace(caat_workspace_size(T, K, H, P, CAAT_VARIANT_ROWPAR), X.device)
        self._keep = (X, W, residual, gamma, out, h_out, workspace)
        arr, idx_ptr = _sync_idx_host(sync_idx)
        a = RowparArgs()
        a.X, a.W = _bf16_dev(X, "X"), _bf16_dev(W, "W")
        a.residual, a.gamma = _bf16_dev(residual, "residual"), _bf16_dev(gamma, "gamma")
        a.sync_idx = idx_ptr
        a.out = _bf16_dev(out, "out")
        a.h_out = _bf16_dev(h_out, "h_out") if h_out is not None else None
        a.workspace = _ptr(workspace)
        a.ws_bytes = workspace.numel() * workspace.element_size()
        a.stream = None
        a.timing = None
        a.T, a.K, a.H = T, K, H
        a.p, a.eps, a.private_scale, a.P, a.flags = float(p), float(eps), float(private_scale), P, int(flags)
        h = ctypes.c_void_p(None)
        _check(lib().caat_plan_create(ctypes.byref(a), ctypes.byref(h)), "caat_plan_create")
        self.handle = h.value

    def execute(self, stream=None):
        _check(lib().caat_plan_execute(self.handle, _stream_ptr(stream)), "caat_plan_execute")

    def close(self):
        if self.handle:
            lib().caat_plan_destroy(self.handle)
            self.handle = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


def _f32_dev(t, name):
    import torch
    if t.dtype != torch.float32:
        raise TypeError(f"{name} must be float32")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    return _ptr(t)


def _tp_args(T, K_r, H, p, eps, private_scale, stream, timing):
    a = TpArgs()
    a.T, a.K_r, a.H = int(T), int(K_r), int(H)
    a.p = float(p)
    a.eps = float(eps)
    a.private_scale = float(private_scale)
    a.stream = _stream_ptr(stream)
    a.timing = timing.handle if timing is not None else None
    a.flags = 0
    return a


def caat_rowpar_tp_local(X, W, residual, p: float, zs, h, *, workspace=None, private_scale: float = 1.0,
                         stream=None, timing=None):
    """Local step of one rank of the layer over real devices: X [T,K_r], W [H,K_r], residual
    [T,H] (bf16, this rank's); writes zs [T, floor(H p)] (fp32, this rank's partial of the shared
    channels) and the private channels of h [T,H] (bf16)."""
    T, K_r = int(X.shape[0]), int(X.shape[1])
    H = int(W.shape[0])
    if workspace is None:
        workspace = alloc_workspace(256, X.device, stream)
    a = _tp_args(T, K_r, H, p, 1e-5, private_scale, stream, timing)
    a.X = _bf16_dev(X, "X")
    a.W = _bf16_dev(W, "W")
    a.residual = _bf16_dev(residual, "residual")
    a.zs = _f32_dev(zs, "zs") if zs is not None and zs.numel() else None
    a.h = _bf16_dev(h, "h")
    a.workspace = _ptr(workspace)
    a.ws_bytes = workspace.numel() * workspace.element_size()
    _check(lib().caat_rowpar_tp_local(ctypes.byref(a)), "caat_rowpar_tp_local")
    return zs, h


def caat_rowpar_tp_finish(zs, residual, h, gamma, p: float, out, *, eps: float = 1e-5, stream=None, timing=None):
    """Finishing step after the exchange: zs [T, floor(H p)] holds the sum over the ranks;
    writes the shared channels of h [T,H] and out [T,H] = RMSNorm(h) * gamma."""
    T, H = int(h.shape[0]), int(h.shape[1])
    a = _tp_args(T, 0, H, p, eps, 1.0, stream, timing)
    a.residual = _bf16_dev(residual, "residual")
    a.gamma = _bf16_dev(gamma, "gamma")
    a.zs = _f32_dev(zs, "zs") if zs is not None and zs.numel() else None
    a.h = _bf16_dev(h, "h")
    a.out = _bf16_dev(out, "out")
    _check(lib().caat_rowpar_tp_finish(ctypes.byref(a)), "caat_rowpar_tp_finish")
    return out


def tp_peers(world: int, rank: int, epoch: int, recv, gather, flags) -> TpPeers:
    """Descriptor of the peer-memory exchange for one rank and call: recv[q], gather[q], flags[q]
    are rank q's buffers (CUDA tensors, or device addresses as ints, valid in this process):
    recv [world, T, n_s / world] fp32, gather [T, n_s] fp32, flags [2, world] int32 zeroed once."""
    world = int(world)
    if not 1 <= world <= CAAT_TP_MAX_WORLD:
        raise ValueError(f"world must be 1..{CAAT_TP_MAX_WORLD}")
    pe = TpPeers()
    pe.world, pe.rank, pe.epoch = world, int(rank), int(epoch)

    def addr(x):
        return int(x) if isinstance(x, int) else _ptr(x)
    for q in range(world):
        pe.recv[q] = addr(recv[q])
        pe.gather[q] = addr(gather[q])
        pe.flags[q] = addr(flags[q])
    return pe


def caat_rowpar_tp_local_push(X, W, residual, p: float, h, peers: TpPeers, *, workspace=None,
                              private_scale: float = 1.0, stream=None, timing=None):
    """Local step of the peer-memory exchange: as caat_rowpar_tp_local, with this rank's fp32
    partials of the shared channels stored into their owners' receive buffers (peers.recv)."""
    T, K_r = int(X.shape[0]), int(X.shape[1])
    H = int(W.shape[0])
    if workspace is None:
        workspace = alloc_workspace(256, X.device, stream)
    a = _tp_args(T, K_r, H, p, 1e-5, private_scale, stream, timing)
    a.X = _bf16_dev(X, "X")
    a.W = _bf16_dev(W, "W")
    a.residual = _bf16_dev(residual, "residual")
    a.h = _bf16_dev(h, "h")
    a.workspace = _ptr(workspace)
    a.ws_bytes = workspace.numel() * workspace.element_size()
    _check(lib().caat_rowpar_tp_local_push(ctypes.byref(a), ctypes.byref(peers)), "caat_rowpar_tp_local_push")
    return h


def caat_rowpar_tp_reduce(T: int, H: int, p: float, peers: TpPeers, *, workspace, stream=None, timing=None):
    """Owner step of the peer-memory exchange: sums this rank's slice of the shared channels over
    the ranks and writes it into every rank's gather buffer.  workspace: >= 256 bytes, device."""
    a = _tp_args(T, 0, H, p, 1e-5, 1.0, stream, timing)
    a.workspace = _ptr(workspace)
    a.ws_bytes = workspace.numel() * workspace.element_size()
    _check(lib().caat_rowpar_tp_reduce(ctypes.byref(a), ctypes.byref(peers)), "caat_rowpar_tp_reduce")


def caat_rowpar_tp_finish_wait(residual, h, gamma, p: float, out, peers: TpPeers, *, eps: float = 1e-5, stream=None,
                               timing=None):
    """Finishing step of the peer-memory exchange: waits for every owner's slice, then as
    caat_rowpar_tp_finish with zs = this rank's gather buffer."""
    T, H = int(h.shape[0]), int(h.shape[1])
    a = _tp_args(T, 0, H, p, eps, 1.0, stream, timing)
    a.residual = _bf16_dev(residual, "residual")
    a.gamma = _bf16_dev(gamma, "gamma")
    a.h = _bf16_dev(h, "h")
    a.out = _bf16_dev(out, "out")
    _check(lib().caat_rowpar_tp_finish_wait(ctypes.byref(a), ctypes.byref(peers)), "caat_rowpar_tp_finish_wait")
    return out


def caat_rowpar_backward(X, W, h, gamma, dout, sync_idx, P: int, p: float, dX, dW, dgamma, *, dR=None,
                         workspace=None, eps: float = 1e-5, private_scale: float = 1.0, stream=None, timing=None,
                         flags: int = 0):
    """Queues the backward of the layer: dX [P,T,K/P], dW [P,H,K/P] (bf16), dgamma [H] (fp32)
    and optionally dR [P,T,H] (bf16), from the forward's inputs, its pre-norm stream h and
    dout = dL/d(out).  flags: 0, or CAAT_BWD_FLAG_TRANSPOSED_OPERANDS (test hook: the gradient
    GEMMs on transposed K-major copies, bit-identical to the default MN-major reads)."""
    P = int(P)
    T = int(X.shape[1])
    K = int(X.shape[2]) * P
    H = int(W.shape[1])
    if workspace is None:
        workspace = alloc_workspace(caat_workspace_size(T, K, H, P, CAAT_VARIANT_ROWPAR_BWD), X.device, stream)
    arr, idx_ptr = _sync_idx_host(sync_idx)
    a = BwdArgs()
    a.X, a.W, a.h = _bf16_dev(X, "X"), _bf16_dev(W, "W"), _bf16_dev(h, "h")
    a.gamma, a.dout = _bf16_dev(gamma, "gamma"), _bf16_dev(dout, "dout")
    a.sync_idx = idx_ptr
    a.dX, a.dW = _bf16_dev(dX, "dX"), _bf16_dev(dW, "dW")
    a.dR = _bf16_dev(dR, "dR") if dR is not None else None
    if dgamma.dtype.__str__() != "torch.float32" or not dgamma.is_cuda:
        raise TypeError("dgamma must be a float32 CUDA tensor")
    a.dgamma = _ptr(dgamma)
    a.workspace = _ptr(workspace)
    a.ws_bytes = workspace.numel() * workspace.element_size()
    a.stream = _stream_ptr(stream)
    a.timing = timing.handle if timing is not None else None
    a.T, a.K, a.H = T, K, H
    a.p = float(p)
    a.eps = float(eps)
    a.private_scale = float(private_scale)
    a.P = P
    a.flags = int(flags)
    _check(lib().caat_rowpar_backward(ctypes.byref(a)), "caat_rowpar_backward")


# ---------------------------------------------------------------------------------------
# the attention block: rotary positions, causal attention, decoding
# ---------------------------------------------------------------------------------------

_ROPE_SCALINGS = {"none": CAAT_ROPE_SCALING_NONE, "linear": CAAT_ROPE_SCALING_LINEAR, "ntk": CAAT_ROPE_SCALING_NTK,
                  "yarn": CAAT_ROPE_SCALING_YARN}


def caat_rope_frequencies(rot: int, theta: float = 10000.0, scaling: str = "none", factor: float = 1.0,
                          trained_length: float = 4096.0):
    """(frequencies float64[rot / 2], mscale): the rotation per position of each pair, scaled for
    contexts longer than the trained one ("none", "linear", "ntk", "yarn"), and the factor on the
    rotated vectors.  Host only."""
    if scaling not in _ROPE_SCALINGS:
        raise ValueError(f"scaling must be one of {sorted(_ROPE_SCALINGS)}")
    f = np.zeros(max(int(rot), 2) // 2, dtype=np.float64)
    m = ctypes.c_float(1.0)
    _check(lib().caat_rope_frequencies(int(rot), float(theta), _ROPE_SCALINGS[scaling], float(factor),
                                       float(trained_length), f.ctypes.data, ctypes.byref(m)), "caat_rope_frequencies")
    return f, float(m.value)


def _current(t, name):
    """Index of the tensor's device, which has to be the current one: the library queues there."""
    import torch
    dev = t.get_device()
    if dev < 0:
        raise ValueError(f"{name} must be a CUDA tensor")
    if dev != torch._C._cuda_getDevice():
        raise ValueError(f"{name} is on cuda:{dev}, but the current device is cuda:{torch.cuda.current_device()}")
    return dev


def _raw_stream(stream, dev):
    if stream is None:
        import torch
        return torch._C._cuda_getCurrentRawStream(dev)
    if stream.device_index != dev:
        raise ValueError(f"the stream is on cuda:{stream.device_index}, the tensors on cuda:{dev}")
    return stream.cuda_stream


def _like(t, name, dtype, shape, dev):
    """Address of a contiguous tensor after checks of its type, shape and device."""
    if t.dtype is dtype and t.shape == shape and t.get_device() == dev and t.is_contiguous():
        return t.data_ptr()
    _refuse(t, name, dtype, shape, dev)
    raise ValueError(f"{name} must be contiguous")


def _refuse(t, name, dtype, shape, dev):
    if t.dtype is not dtype:
        raise TypeError(f"{name} must be {dtype}")
    if t.get_device() != dev:
        raise ValueError(f"{name} is on {t.device}, not on device {dev}")
    if t.shape != shape:
        raise ValueError(f"{name} must have the shape {tuple(shape)}, not {tuple(t.shape)}")


def _heads4(t, name, dtype, dev, shape=None):
    """Address and (rank, token) strides of a [P, T, heads, dh] tensor whose heads lie side by side
    within a token (a contiguous tensor, strides 0, or a slice of a fused projection)."""
    if t.dim() != 4:
        raise ValueError(f"{name} must be [P, T, heads, dh]")
    if t.dtype is not dtype or t.get_device() != dev or (shape is not None and t.shape != shape):
        _refuse(t, name, dtype, t.shape if shape is None else shape, dev)
    if t.is_contiguous():
        return t.data_ptr(), 0, 0
    P, T, heads, dh = t.shape
    s = t.stride()
    if (dh > 1 and s[3] != 1) or (heads > 1 and s[2] != dh):
        raise ValueError(f"{name}: the heads of a token must be contiguous and side by side")
    # a dimension of one element has no stride of its own
    token = s[1] if T > 1 else heads * dh
    if token < heads * dh:  # (0, 0) would mean contiguous
        raise ValueError(f"{name}: the tokens must not share memory")
    return t.data_ptr(), s[0] if P > 1 else max(s[0], token * T), token


def _workspace(workspace, nbytes, dev, stream):
    """(tensor or None, address, bytes) of a call's workspace; one allocated here belongs to the call's stream."""
    if workspace is None:
        if nbytes == 0:
            return None, None, 0
        workspace = alloc_workspace(nbytes, dev, stream)
        return workspace, workspace.data_ptr(), nbytes
    if workspace.get_device() != dev:
        raise ValueError(f"workspace is on {workspace.device}, not on device {dev}")
    return workspace, _ptr(workspace), workspace.numel() * workspace.element_size()


def _offsets(cu, name):
    """(what keeps them, address, count) of host int32 offsets from a sequence, an array or a CPU tensor."""
    if isinstance(cu, (list, tuple)):
        try:
            arr = array.array("i", cu)
        except OverflowError:
            raise CaatError(CAAT_ERR_INVALID_ARG, name) from None
        except TypeError:
            raise ValueError(f"{name} must be a one-dimensional host array of integers") from None
        ptr, n = arr.buffer_info()
    else:
        arr = np.asarray(cu)
        if arr.ndim != 1 or arr.dtype.kind not in "iu":
            raise ValueError(f"{name} must be a one-dimensional host array of integers")
        if arr.dtype != np.int32 and arr.size and (arr.min() < 0 or arr.max() > 2**31 - 1):
            raise CaatError(CAAT_ERR_INVALID_ARG, name)
        arr = np.ascontiguousarray(arr, dtype=np.int32)
        ptr, n = arr.__array_interface__["data"][0], arr.size
    if n < 1:
        raise ValueError(f"{name} must hold at least one offset")
    return arr, ptr, n


def caat_attn_workspace_size(Tq: int, Tk: int, n_seq: int, P: int, heads_q: int, heads_k: int, dh: int,
                             variant: int = CAAT_VARIANT_ATTN) -> int:
    n = lib().caat_attn_workspace_size(int(Tq), int(Tk), int(n_seq), int(P), int(heads_q), int(heads_k), int(dh),
                                       int(variant))
    if n == _SIZE_MAX:
        raise CaatError(CAAT_ERR_INVALID_ARG, "caat_attn_workspace_size")
    return int(n)


def _rope_out(o, x, name, dtype, dev):
    """Address of a rotation's output: contiguous, or the input itself."""
    if o is x:
        return x.data_ptr()
    if o.data_ptr() == x.data_ptr() and o.numel():
        if o.stride() != x.stride() or o.shape != x.shape or o.dtype is not dtype:
            raise ValueError(f"{name} in place must have its input's type, shape and strides")
        return o.data_ptr()
    return _like(o, name, dtype, x.shape, dev)


def _rope(q, k, v, positions, slots, inv_freq, q_out, k_out, v_out, interleaved, backward, mscale, stream, timing):
    import torch
    first = q if q is not None else k
    if first is None:
        raise ValueError("caat_rope: q and k are both None")
    dev = _current(first, "q" if q is not None else "k")
    bf = torch.bfloat16
    if first.dim() != 4:
        raise ValueError("q and k must be [P, T, heads, dh]")
    P, T, heads, dh = first.shape
    hq = hk = rows = 0
    q_ptr = k_ptr = v_ptr = qo = ko = vo = slot = 0
    qr = qt = kr = kt = vr = vt = 0
    if q is not None:
        hq = heads
        q_ptr, qr, qt = _heads4(q, "q", bf, dev)
        qo = _rope_out(q_out, q, "q_out", bf, dev)
    if k is not None:
        hk = k.shape[2] if k.dim() == 4 else 0
        k_ptr, kr, kt = _heads4(k, "k", bf, dev, (P, T, hk, dh))
        if slots is None:
            ko = _rope_out(k_out, k, "k_out", bf, dev)
        else:
            v_ptr, vr, vt = _heads4(v, "v", bf, dev, (P, T, hk, dh))
            rows = k_out.numel() // max(P * hk * dh, 1)
            slab = k_out.shape
            cache = slab if len(slab) == 5 and slab[0] == P and slab[3:] == (hk, dh) else (P, rows, hk, dh)
            ko = _like(k_out, "k_cache", bf, cache, dev)
            vo = _like(v_out, "v_cache", bf, cache, dev)
            slot = _like(slots, "slots", torch.int64, (T,), dev)
    pos = 0 if positions is None else _like(positions, "positions", torch.int32, (T,), dev)
    freq = inv_freq
    if type(freq) is not np.ndarray or freq.dtype != np.float64 or not freq.flags.c_contiguous:
        freq = np.ascontiguousarray(freq, dtype=np.float64)
    if freq.ndim != 1:
        raise ValueError("inv_freq must be one-dimensional")
    code = (_lib or lib()).packed_caat_rope(_PACK_ROPE.pack(
        q_ptr, k_ptr, v_ptr, qo, ko, vo, pos, slot, freq.__array_interface__["data"][0], _raw_stream(stream, dev),
        0 if timing is None else timing.handle, T, rows, qr, qt, kr, kt, vr, vt, P, hq, hk, dh, 2 * freq.size, mscale,
        (CAAT_ROPE_FLAG_INTERLEAVED if interleaved else 0) | (CAAT_ROPE_FLAG_BACKWARD if backward else 0)))
    if code:
        _check(code, "caat_rope")


def caat_rope(q, k, positions, inv_freq, *, q_out, k_out, interleaved: bool = False, backward: bool = False,
              mscale: float = 1.0, stream=None, timing=None):
    """Queues the rotation of q [P,T,heads_q,dh] and k [P,T,heads_k,dh] (bf16; either may be None, and
    may be a slice of a fused projection) by their positions (CUDA int32 [T], or None: 0..T-1).

    inv_freq: host float64 [rot / 2] (caat_rope_frequencies); the first rot elements of a head turn.
    q_out, k_out: contiguous, or q and k themselves (in place).  backward: by the negative angle, the
    gradient of the same call."""
    fast = _marshal or _fast()
    code = None
    if fast and stream is None and timing is None:
        code = fast.rope(q, k, None, positions, None, inv_freq, q_out, k_out, None, interleaved, backward, mscale)
    if code is None:
        _rope(q, k, None, positions, None, inv_freq, q_out, k_out, None, interleaved, backward, mscale, stream, timing)
    elif code:
        _check(code, "caat_rope")
    return q_out, k_out


def caat_rope_append(q, k, v, positions, slots, inv_freq, k_cache, v_cache, *, q_out=None, interleaved: bool = False,
                     backward: bool = False, mscale: float = 1.0, stream=None, timing=None):
    """As caat_rope, with the rotated k and v of token t written to row slots[t] (CUDA int64 [T]; -1:
    not written) of the caches [P,rows,heads_k,dh] (or [P,B,capacity,heads_k,dh], row = b * capacity +
    position).  Slots outside the cache are skipped and reported by caat_get_device_status."""
    if k is None or v is None or slots is None:
        raise ValueError("caat_rope_append needs k, v and slots")
    fast = _marshal or _fast()
    code = None
    if fast and stream is None and timing is None:
        code = fast.rope(q, k, v, positions, slots, inv_freq, q_out, k_cache, v_cache, interleaved, backward, mscale)
    if code is None:
        _rope(q, k, v, positions, slots, inv_freq, q_out, k_cache, v_cache, interleaved, backward, mscale, stream, timing)
    elif code:
        _check(code, "caat_rope")
    return q_out


def _attn_qkv(q, k, v, cu_q, cu_k):
    """Checks of what the forward and the backward share: (device, what must outlive the call,
    addresses of q, k and v, addresses and count of the offsets, strides)."""
    import torch
    dev = _current(q, "q")
    bf = torch.bfloat16
    q_ptr, qr, qt = _heads4(q, "q", bf, dev)
    k_ptr, kr, kt = _heads4(k, "k", bf, dev)
    v_ptr, vr, vt = _heads4(v, "v", bf, dev, k.shape)
    if k.shape[0] != q.shape[0] or k.shape[3] != q.shape[3]:
        raise ValueError("q, k and v must have the same ranks and head size")
    cq, cq_ptr, n = _offsets(cu_q, "cu_q")
    ck, ck_ptr = None, 0
    if cu_k is not None:
        ck, ck_ptr, nk = _offsets(cu_k, "cu_k")
        if nk != n:
            raise ValueError("cu_q and cu_k must have the same length")
    return dev, (cq, ck), (q_ptr, k_ptr, v_ptr), (cq_ptr, ck_ptr), n - 1, (qr, qt, kr, kt, vr, vt)


def caat_attn_forward(q, k, v, cu_q, out, *, cu_k=None, lse=None, scale: Optional[float] = None, workspace=None,
                      stream=None, timing=None):
    """Queues causal attention over packed sequences on every rank.

    q [P,Tq,heads_q,dh], k, v [P,Tk,heads_k,dh] (bf16, contiguous or slices of a fused projection);
    cu_q, cu_k: host offsets [n_seq + 1] of the sequences' queries and keys (cu_k None: cu_q; the last
    query sees the last key); out [P,Tq,heads_q*dh] bf16, the X of caat_rowpar_forward; lse
    [P,heads_q,Tq] fp32, needed by the backward.  scale None: dh ** -0.5."""
    fast = _marshal or _fast()
    if fast and stream is None and timing is None:
        code = fast.attn_forward(q, k, v, cu_q, cu_k, out, lse, scale, workspace)
        if code is not None:
            if code:
                _check(code, "caat_attn_forward")
            return out
    import torch
    dev, keep, qkv, cu, n, strides = _attn_qkv(q, k, v, cu_q, cu_k)
    P, Tq, hq, dh = q.shape
    Tk, hk = k.shape[1:3]
    L = _lib or lib()
    out_ptr = _like(out, "out", torch.bfloat16, (P, Tq, hq * dh), dev)
    lse_ptr = 0 if lse is None else _like(lse, "lse", torch.float32, (P, hq, Tq), dev)
    tail = (_raw_stream(stream, dev), 0 if timing is None else timing.handle, Tq, Tk, *strides, n, P, hq, hk, dh,
            dh ** -0.5 if scale is None else scale, 0)
    ws, ws_ptr, ws_bytes = (None, 0, 0) if workspace is None else _workspace(workspace, 0, dev, stream)
    code = L.packed_caat_attn_forward(_PACK_ATTN.pack(*qkv, out_ptr, lse_ptr, *cu, ws_ptr, ws_bytes, *tail))
    if code == CAAT_ERR_WORKSPACE and workspace is None:  # only long work lists need one
        need = L.caat_attn_workspace_size(Tq, Tk, n, P, hq, hk, dh, CAAT_VARIANT_ATTN)
        ws, ws_ptr, ws_bytes = _workspace(None, need, dev, stream)
        code = L.packed_caat_attn_forward(_PACK_ATTN.pack(*qkv, out_ptr, lse_ptr, *cu, ws_ptr, ws_bytes, *tail))
    if code:
        _check(code, "caat_attn_forward")
    del keep, ws
    return out


def caat_attn_backward(q, k, v, out, lse, dout, cu_q, dq, dk, dv, *, cu_k=None, scale: Optional[float] = None,
                       workspace=None, stream=None, timing=None):
    """Queues the gradients of caat_attn_forward: dq [P,Tq,heads_q,dh], dk, dv [P,Tk,heads_k,dh] (bf16,
    contiguous) from the forward's inputs, its out and lse, and dout [P,Tq,heads_q*dh]."""
    fast = _marshal or _fast()
    if fast and stream is None and timing is None:
        code = fast.attn_backward(q, k, v, cu_q, cu_k, out, lse, dout, dq, dk, dv, scale, workspace)
        if code is not None:
            if code:
                _check(code, "caat_attn_backward")
            return dq, dk, dv
    import torch
    dev, keep, qkv, cu, n, strides = _attn_qkv(q, k, v, cu_q, cu_k)
    bf = torch.bfloat16
    P, Tq, hq, dh = q.shape
    Tk, hk = k.shape[1:3]
    L = _lib or lib()
    need = 0
    if workspace is None:
        need = L.caat_attn_workspace_size(Tq, Tk, n, P, hq, hk, dh, CAAT_VARIANT_ATTN_BWD)
        if need == _SIZE_MAX:
            need = 0  # sizes the call itself refuses
    ws, ws_ptr, ws_bytes = _workspace(workspace, need, dev, stream)
    rows = (P, Tq, hq * dh)
    code = L.packed_caat_attn_backward(_PACK_ATTN_BWD.pack(
        *qkv, _like(out, "out", bf, rows, dev), _like(lse, "lse", torch.float32, (P, hq, Tq), dev),
        _like(dout, "dout", bf, rows, dev), _like(dq, "dq", bf, q.shape, dev), _like(dk, "dk", bf, k.shape, dev),
        _like(dv, "dv", bf, k.shape, dev), *cu, ws_ptr, ws_bytes, _raw_stream(stream, dev),
        0 if timing is None else timing.handle, Tq, Tk, *strides, n, P, hq, hk, dh, dh ** -0.5 if scale is None else scale,
        0))
    if code:
        _check(code, "caat_attn_backward")
    del keep, ws
    return dq, dk, dv


def caat_attn_decode(q, k_cache, v_cache, lens, out, *, scale: Optional[float] = None, workspace=None, stream=None,
                     timing=None):
    """Queues attention of one new token per sequence over its cache on every rank.

    q [P,B,heads_q,dh], caches [P,B,capacity,heads_k,dh] (bf16), lens CUDA int32 [B] (keys of each
    sequence, the new token's included), out [P,B,heads_q*dh]: the X of caat_rowpar_forward."""
    fast = _marshal or _fast()
    if fast and stream is None and timing is None:
        code = fast.attn_decode(q, k_cache, v_cache, lens, out, scale, workspace)
        if code is not None:
            if code:
                _check(code, "caat_attn_decode")
            return out
    import torch
    bf = torch.bfloat16
    dev = _current(q, "q")
    q_ptr, qr, qt = _heads4(q, "q", bf, dev)
    P, B, hq, dh = q.shape
    cache = k_cache.shape
    if len(cache) != 5 or cache[0] != P or cache[1] != B or cache[4] != dh:
        raise ValueError(f"k_cache must be [{P}, {B}, capacity, heads_k, {dh}], not {tuple(cache)}")
    cap, hk = cache[2], cache[3]
    L = _lib or lib()
    head = (q_ptr, _like(k_cache, "k_cache", bf, cache, dev), _like(v_cache, "v_cache", bf, cache, dev),
            _like(lens, "lens", torch.int32, (B,), dev), _like(out, "out", bf, (P, B, hq * dh), dev))
    tail = (_raw_stream(stream, dev), 0 if timing is None else timing.handle, B, cap, qr, qt, P, hq, hk, dh,
            dh ** -0.5 if scale is None else scale, 0)
    ws, ws_ptr, ws_bytes = (None, 0, 0) if workspace is None else _workspace(workspace, 0, dev, stream)
    code = L.packed_caat_attn_decode(_PACK_ATTN_DECODE.pack(*head, ws_ptr, ws_bytes, *tail))
    if code == CAAT_ERR_WORKSPACE and workspace is None:  # where no cluster takes a sequence's heads
        need = L.caat_attn_workspace_size(B, cap, 0, P, hq, hk, dh, CAAT_VARIANT_ATTN_DECODE)
        ws, ws_ptr, ws_bytes = _workspace(None, need, dev, stream)
        code = L.packed_caat_attn_decode(_PACK_ATTN_DECODE.pack(*head, ws_ptr, ws_bytes, *tail))
    if code:
        _check(code, "caat_attn_decode")
    del ws
    return out


def caat_rowpar_forward_host(X, W, residual, gamma, sync_idx, P: int, p: float, out, workspace, *,
                             h_out=None, eps: float = 1e-5, private_scale: float = 1.0, flags: int = 0,
                             stream=None, timing=None):
    """The layer on HOST tensors (pinned CPU bf16 tensors): the library copies the inputs into
    `workspace` (a device buffer of caat_workspace_size(..., CAAT_VARIANT_ROWPAR_HOST) bytes),
    runs the kernels and copies out (and h_out) back, all queued on `stream`."""
    import torch
    P = int(P)
    T = int(X.shape[1])
    K = int(X.shape[2]) * P
    H = int(W.shape[1])
    for name, t in (("X", X), ("W", W), ("residual", residual), ("gamma", gamma), ("out", out)):
        if t.dtype != torch.bfloat16 or t.is_cuda:
            raise ValueError(f"{name} must be a bfloat16 CPU tensor")
    arr, idx_ptr = _sync_idx_host(sync_idx)
    a = RowparArgs()
    a.X, a.W, a.residual, a.gamma, a.out = _ptr(X), _ptr(W), _ptr(residual), _ptr(gamma), _ptr(out)
    a.h_out = _ptr(h_out) if h_out is not None else None
    a.sync_idx = idx_ptr
    a.workspace = _ptr(workspace)
    a.ws_bytes = workspace.numel() * workspace.element_size()
    a.stream = _stream_ptr(stream)
    a.timing = timing.handle if timing is not None else None
    a.T, a.K, a.H = T, K, H
    a.p = float(p)
    a.eps = float(eps)
    a.private_scale = float(private_scale)
    a.P = P
    a.flags = int(flags)
    _check(lib().caat_rowpar_forward_host(ctypes.byref(a)), "caat_rowpar_forward_host")
    return out


def caat_rowpar_forward_noalloc(X, W, residual, gamma, sync_idx, P: int, p: float, out, *, h_out=None,
                                eps: float = 1e-5, private_scale: float = 1.0, flags: int = 0,
                                stream=None, timing=None):
    """The layer without any device allocation, for callers that cannot allocate device memory:
    the library's built-in scratch array (CAAT_NOALLOC_SCRATCH_BYTES per GPU) replaces the
    workspace.  Calls that overlap on the GPU share that array and race; serialize them."""
    P = int(P)
    T = int(X.shape[1])
    K = int(X.shape[2]) * P
    H = int(W.shape[1])
    arr, idx_ptr = _sync_idx_host(sync_idx)
    a = RowparArgs()
    a.X = _bf16_dev(X, "X")
    a.W = _bf16_dev(W, "W")
    a.residual = _bf16_dev(residual, "residual")
    a.gamma = _bf16_dev(gamma, "gamma")
    a.sync_idx = idx_ptr
    a.out = _bf16_dev(out, "out")
    a.h_out = _bf16_dev(h_out, "h_out") if h_out is not None else None
    a.workspace = None
    a.ws_bytes = 0
    a.stream = _stream_ptr(stream)
    a.timing = timing.handle if timing is not None else None
    a.T, a.K, a.H = T, K, H
    a.p = float(p)
    a.eps = float(eps)
    a.private_scale = float(private_scale)
    a.P = P
    a.flags = int(flags)
    _check(lib().caat_rowpar_forward_noalloc(ctypes.byref(a)), "caat_rowpar_forward_noalloc")
    return out


def caat_mlp_forward(X, A, W2, residual, gamma, sync_idx, P: int, p: float, out, *, workspace=None,
                     h_out=None, eps: float = 1e-5, private_scale: float = 1.0, flags: int = 0,
                     stream=None, timing=None):
    """Queues the MLP block: FC1 + SwiGLU, partially synced FC2, residual, RMSNorm.

    X [P,T,H], A [P,2F/P,H], W2 [P,H,F/P], residual [P,T,H], gamma [H], out [P,T,H].
    """
    P = int(P)
    T = int(X.shape[1])
    H = int(X.shape[2])
    F = int(W2.shape[2]) * P
    if workspace is None:
        workspace = alloc_workspace(caat_workspace_size(T, F, H, P, CAAT_VARIANT_MLP), X.device, stream)
    arr, idx_ptr = _sync_idx_host(sync_idx)
    a = MlpArgs()
    a.X = _bf16_dev(X, "X")
    a.A = _bf16_dev(A, "A")
    a.W2 = _bf16_dev(W2, "W2")
    a.residual = _bf16_dev(residual, "residual")
    a.gamma = _bf16_dev(gamma, "gamma")
    a.sync_idx = idx_ptr
    a.out = _bf16_dev(out, "out")
    a.h_out = _bf16_dev(h_out, "h_out") if h_out is not None else None
    a.workspace = _ptr(workspace)
    a.ws_bytes = workspace.numel() * workspace.element_size()
    a.stream = _stream_ptr(stream)
    a.timing = timing.handle if timing is not None else None
    a.T, a.H, a.F = T, H, F
    a.p = float(p)
    a.eps = float(eps)
    a.private_scale = float(private_scale)
    a.P = P
    a.flags = int(flags)
    _check(lib().caat_mlp_forward_ex(ctypes.byref(a)), "caat_mlp_forward")
    return out


def caat_get_device_status(stream=None) -> int:
    """Synchronizes the stream and returns (and clears) the device status word."""
    v = ctypes.c_int32(0)
    lib().caat_get_device_status(_stream_ptr(stream), ctypes.byref(v))
    return int(v.value)


class Timing:
    """Per-kernel CUDA-event recorder of the library (caat_timing_*)."""

    MAX_KERNELS = 8

    def __init__(self, capacity: int = 256):
        h = ctypes.c_void_p()
        _check(lib().caat_timing_create(int(capacity), ctypes.byref(h)), "caat_timing_create")
        self.handle = h.value
        self.capacity = capacity

    def reset(self):
        _check(lib().caat_timing_reset(self.handle), "caat_timing_reset")

    def read(self):
        """List of per-call lists of kernel durations in ms."""
        buf = (ctypes.c_float * (self.capacity * self.MAX_KERNELS))()
        nr, nk = ctypes.c_int(0), ctypes.c_int(0)
        _check(lib().caat_timing_read(self.handle, buf, self.capacity, self.MAX_KERNELS,
                                      ctypes.byref(nr), ctypes.byref(nk)), "caat_timing_read")
        return [[buf[r * self.MAX_KERNELS + k] for k in range(nk.value)] for r in range(nr.value)]

    def close(self):
        if self.handle:
            lib().caat_timing_destroy(self.handle)
            self.handle = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass
