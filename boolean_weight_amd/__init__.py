"""Python binding of the MBOK C ABI (include/mbok.h): argument marshalling only.

Every step of the layer runs in the HIP library libmbok.so built in this
directory; this module turns torch tensors into device pointers and sizes,
checks that the buffers are large enough and on the GPU (the C ABI receives
plain pointers and cannot check sizes), and raises MbokError on a nonzero
status.  There is no CPU fallback: without the built library every call
raises.
"""
from __future__ import annotations

import contextlib
import ctypes
import functools
import os
import threading
import warnings

import torch

__all__ = [
    "MBOK_F32", "MBOK_F16", "MBOK_BF16", "MBOK_GROUP", "MBOK_MAX_K", "MBOK_MAX_T",
    "MbokError", "mbok_desc", "library_path", "load_library",
    "mbok_desc_init", "mbok_packed_bytes", "mbok_alpha_bytes", "mbok_residual_binarize",
    "mbok_refit", "MBOK_MAX_REFIT_ROUNDS", "mbok_residual_energy", "mbok_allocate_kernels",
    "mbok_pack", "mbok_gemv", "mbok_gemv_workspace_bytes", "mbok_gemm", "mbok_gemm_precise",
    "mbok_status_str",
    "mbok_gemvt", "mbok_gemvt_workspace_bytes", "mbok_gemvt_noalloc", "mbok_gemvt_scratch_bytes",
    "mbok_svid_workspace_bytes", "mbok_svid_decompose", "mbok_svid_pack",
    "mbok_svid_gemv_workspace_bytes", "mbok_svid_gemv", "MBOK_MAX_SVID_ITERS",
    "mbok_gemmt", "mbok_gemmt_precise", "mbok_gemmt_workspace_bytes", "mbok_scale_grad",
    "mbok_scale_grad_workspace_bytes", "MBOK_ACT_SILU", "MBOK_ACT_GELU", "mbok_gated_stack",
    "mbok_gated_pack", "mbok_gated", "mbok_gated_precise", "mbok_gated_backward",
    "mbok_gated_backward_precise", "mbok_distill_desc",
    "mbok_distill_desc_init", "mbok_distill", "mbok_distill_backward", "MBOK_MAX_TOP",
    "MBOK_MAX_VOCAB", "MBOK_MAX_DISTILL_ROWS", "MBOK_DISTILL_STATS",
    "MBOK_ACT_NONE", "mbok_linear", "mbok_linear_precise", "mbok_linear_backward",
    "mbok_linear_backward_precise", "mbok_linear_backward_workspace_bytes",
    "mbok_logp_desc", "mbok_logp_desc_init", "mbok_logp", "mbok_logp_backward",
    "MBOK_LOGP_STATS", "mbok_policy_desc", "mbok_policy_desc_init", "mbok_policy",
    "mbok_preference_desc", "mbok_preference_desc_init", "mbok_preference", "MBOK_MAX_PAIRS",
    "MBOK_E4M3", "MBOK_ADAMW_BLOCK", "MBOK_MAX_ADAMW_TENSORS", "mbok_adamw_plan",
    "mbok_adamw_plan_init", "mbok_adamw",
    "mbok_version", "workspace_for",
    "alpha_torch_dtype", "quantize_and_pack", "allocate_for_budget",
]

MBOK_F32, MBOK_F16, MBOK_BF16, MBOK_E4M3 = 0, 1, 2, 3
MBOK_GROUP = 128
MBOK_ROW_BLOCK = 64
MBOK_MAX_K = 4
MBOK_MAX_T = 65536
MBOK_LAYOUT_L64 = 1
MBOK_MAX_REFIT_ROUNDS = 64
MBOK_MAX_SVID_ITERS = 1000
MBOK_ACT_SILU, MBOK_ACT_GELU, MBOK_ACT_NONE = 0, 1, 2
MBOK_MAX_TOP = 1024
MBOK_MAX_VOCAB = 1 << 19
MBOK_MAX_DISTILL_ROWS = 1 << 23
MBOK_DISTILL_STATS = 8
MBOK_LOGP_STATS = 4
MBOK_MAX_PAIRS = 1 << 23
MBOK_ADAMW_BLOCK = 256
MBOK_MAX_ADAMW_TENSORS = 65536

_HERE = os.path.dirname(os.path.abspath(__file__))
_LIB = None


class MbokError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        super().__init__(f"{where}: {mbok_status_str(status)} ({status})")


class mbok_desc(ctypes.Structure):
    _fields_ = [("m", ctypes.c_int32), ("n", ctypes.c_int32), ("K", ctypes.c_int32),
                ("group", ctypes.c_int32), ("alpha_dtype", ctypes.c_int32),
                ("layout", ctypes.c_int32)]

    def __repr__(self):
        return (f"mbok_desc(m={self.m}, n={self.n}, K={self.K}, group={self.group}, "
                f"alpha_dtype={self.alpha_dtype}, layout={self.layout})")


class mbok_distill_desc(ctypes.Structure):
    _fields_ = [("vocab", ctypes.c_int32), ("top", ctypes.c_int32),
                ("temperature", ctypes.c_float)]

    def __repr__(self):
        return (f"mbok_distill_desc(vocab={self.vocab}, top={self.top}, "
                f"temperature={self.temperature})")


class mbok_logp_desc(ctypes.Structure):
    _fields_ = [("vocab", ctypes.c_int32), ("temperature", ctypes.c_float)]

    def __repr__(self):
        return f"mbok_logp_desc(vocab={self.vocab}, temperature={self.temperature})"


class mbok_policy_desc(ctypes.Structure):
    _fields_ = [("vocab", ctypes.c_int32), ("temperature", ctypes.c_float),
                ("clip_low", ctypes.c_float), ("clip_high", ctypes.c_float),
                ("kl", ctypes.c_float)]

    def __repr__(self):
        return (f"mbok_policy_desc(vocab={self.vocab}, temperature={self.temperature}, "
                f"clip_low={self.clip_low}, clip_high={self.clip_high}, kl={self.kl})")


class mbok_preference_desc(ctypes.Structure):
    _fields_ = [("beta", ctypes.c_float), ("smoothing", ctypes.c_float),
                ("margin", ctypes.c_float), ("mean", ctypes.c_int32), ("vocab", ctypes.c_int32)]
    vocab_left_out = False  # see mbok_preference_desc_init

    def __repr__(self):
        return (f"mbok_preference_desc(beta={self.beta}, smoothing={self.smoothing}, "
                f"margin={self.margin}, mean={self.mean}, vocab={self.vocab})")


class _AdamwTensor(ctypes.Structure):
    _fields_ = [(n, ctypes.c_void_p) for n in ("param", "grad", "m", "v", "m_scale", "v_scale",
                                               "out", "layer")] + \
        [("count", ctypes.c_int64), ("weight_decay", ctypes.c_double),
         ("grad_dtype", ctypes.c_int32), ("state_dtype", ctypes.c_int32),
         ("out_dtype", ctypes.c_int32)]


class _AdamwPlan(ctypes.Structure):
    _fields_ = [("table_bytes", ctypes.c_int64), ("tensors", ctypes.c_int32),
                ("parts", ctypes.c_int32), ("lds_bytes", ctypes.c_int32)]


class _AdamwStep(ctypes.Structure):
    _fields_ = [("lr", ctypes.c_double), ("beta1", ctypes.c_double), ("beta2", ctypes.c_double),
                ("eps", ctypes.c_double), ("step", ctypes.c_int64),
                ("grad_scale", ctypes.c_float), ("seed", ctypes.c_uint32)]


def library_path() -> str:
    return os.environ.get("MBOK_LIBRARY", os.path.join(_HERE, "libmbok.so"))


def load_library() -> ctypes.CDLL:
    """Load libmbok.so (once).  Raises RuntimeError if it has not been built."""
    global _LIB
    if _LIB is not None:
        return _LIB
    path = library_path()
    if not os.path.exists(path):
        raise RuntimeError(f"MBOK HIP library not built: {path} is missing "
                           "(run `python -m boolean_weight_amd.build`)")
    lib = ctypes.CDLL(path)
    P, I32, I64, SZ = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_size_t
    D = ctypes.POINTER(mbok_desc)
    DD, F = ctypes.POINTER(mbok_distill_desc), ctypes.c_float
    DL, DP = ctypes.POINTER(mbok_logp_desc), ctypes.POINTER(mbok_policy_desc)
    DR, AT = ctypes.POINTER(mbok_preference_desc), ctypes.POINTER(_AdamwTensor)
    AP, AS = ctypes.POINTER(_AdamwPlan), ctypes.POINTER(_AdamwStep)
    linear = [D, P, P, I32, I64, I64, P, I32, I32, P, I64, P, I32, I64, P, I64, P]
    linear_backward = [D, P, P, I64, P, I64, I64, I32, P, I64, P, I32, P, I64, P, P]
    sigs = {
        "mbok_desc_init": (ctypes.c_int, [D, I32, I32, I32, I32]),
        "mbok_packed_bytes": (SZ, [D]),
        "mbok_alpha_bytes": (SZ, [D]),
        "mbok_residual_binarize": (ctypes.c_int, [D, P, I64, P, P, P, P]),
        "mbok_refit": (ctypes.c_int, [D, P, I64, P, P, I32, P]),
        "mbok_residual_energy": (ctypes.c_int, [D, P, I64, P, P, P]),
        "mbok_allocate_kernels": (ctypes.c_int, [I32, P, P, I32, I64, P]),
        "mbok_pack": (ctypes.c_int, [D, P, P, P, P]),
        "mbok_gemv_workspace_bytes": (SZ, [D]),
        "mbok_gemv": (ctypes.c_int, [D, P, P, I32, P, P, P]),
        "mbok_gemm": (ctypes.c_int, [D, P, P, I32, I64, I64, P, I64, P]),
        "mbok_gemm_precise": (ctypes.c_int, [D, P, P, I32, I64, I64, P, I64, P]),
        "mbok_gemvt_workspace_bytes": (SZ, [D]),
        "mbok_gemvt": (ctypes.c_int, [D, P, P, I32, P, P, P]),
        "mbok_gemvt_scratch_bytes": (SZ, []),
        "mbok_gemvt_noalloc": (ctypes.c_int, [D, P, P, I32, P, P]),
        "mbok_svid_workspace_bytes": (SZ, [D]),
        "mbok_svid_decompose": (ctypes.c_int, [D, P, I64, P, P, P, I32, P, P]),
        "mbok_svid_pack": (ctypes.c_int, [D, P, P, P, P]),
        "mbok_svid_gemv_workspace_bytes": (SZ, [D]),
        "mbok_svid_gemv": (ctypes.c_int, [D, P, P, P, I32, P, P, P]),
        "mbok_gemmt": (ctypes.c_int, [D, P, P, I64, I64, P, I64, P, P]),
        "mbok_gemmt_precise": (ctypes.c_int, [D, P, P, I64, I64, P, I64, P, P]),
        "mbok_gemmt_workspace_bytes": (SZ, [D, I64]),
        "mbok_scale_grad": (ctypes.c_int, [D, P, P, I64, I64, P, I64, P, I32, P, P]),
        "mbok_scale_grad_workspace_bytes": (SZ, [D, I64]),
        "mbok_gated_stack": (ctypes.c_int, [D, D]),
        "mbok_gated_pack": (ctypes.c_int, [D, P, P, P, P, P, P]),
        "mbok_gated": (ctypes.c_int, [D, P, P, I32, I64, I64, I32, P, I64, P, I64, P]),
        "mbok_gated_precise": (ctypes.c_int, [D, P, P, I32, I64, I64, I32, P, I64, P, I64, P]),
        "mbok_gated_backward": (ctypes.c_int, [D, P, P, I64, P, I64, I64, I32, P, I64, P, I64, P,
                                               P]),
        "mbok_gated_backward_precise": (ctypes.c_int, [D, P, P, I64, P, I64, I64, I32, P, I64, P,
                                                       I64, P, P]),
        "mbok_distill_desc_init": (ctypes.c_int, [DD, I32, I32, F]),
        "mbok_distill": (ctypes.c_int, [DD, P, I32, I64, I64, P, I32, P, I64, P, P, P, P, P, I32,
                                        I64, P]),
        "mbok_distill_backward": (ctypes.c_int, [DD, P, I32, I64, I64, P, I32, P, I64, P, P, P, P,
                                                 P, I32, I64, P]),
        "mbok_linear": (ctypes.c_int, linear),
        "mbok_linear_precise": (ctypes.c_int, linear),
        "mbok_linear_backward": (ctypes.c_int, linear_backward),
        "mbok_linear_backward_precise": (ctypes.c_int, linear_backward),
        "mbok_linear_backward_workspace_bytes": (SZ, [D, I64]),
        "mbok_logp_desc_init": (ctypes.c_int, [DL, I32, F]),
        "mbok_logp": (ctypes.c_int, [DL, P, I32, I64, I64, P, P, P, P]),
        "mbok_logp_backward": (ctypes.c_int, [DL, P, I32, I64, I64, P, P, P, P, I32, I64, P]),
        "mbok_policy_desc_init": (ctypes.c_int, [DP, I32, F, F, F, F]),
        "mbok_policy": (ctypes.c_int, [DP, P, I32, I64, I64, P, P, P, P, P, P, P, P, P, P, I32,
                                       I64, P]),
        "mbok_preference_desc_init": (ctypes.c_int, [DR, F, F, F, I32, I32]),
        "mbok_preference": (ctypes.c_int, [DR, P, I64, P, P, P, I64, P, P, P, P]),
        "mbok_adamw_table_bytes": (SZ, [AT, I32]),
        "mbok_adamw_plan_init": (ctypes.c_int, [AP, AT, I32, P]),
        "mbok_adamw": (ctypes.c_int, [AP, P, AS, P, P]),
        "mbok_status_str": (ctypes.c_char_p, [ctypes.c_int]),
        "mbok_version": (ctypes.c_char_p, []),
    }
    for name, (res, args) in sigs.items():
        fn = getattr(lib, name)
        fn.restype = res
        fn.argtypes = args
    _LIB = lib
    return lib


# ------------------------------------------------------------------ helpers

def _stream(stream) -> int:
    if stream is None:
        return torch.cuda.current_stream().cuda_stream
    if isinstance(stream, torch.cuda.Stream):
        return stream.cuda_stream
    return int(stream)


def _dev(t: torch.Tensor, name: str) -> torch.Tensor:
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if not t.is_cuda:
        raise ValueError(f"{name} must be on the GPU (the library takes device pointers)")
    return t


def _nbytes_from(t: torch.Tensor) -> int:
    """Bytes addressable from t.data_ptr() to the end of its storage."""
    st = t.untyped_storage()
    return st.nbytes() - (t.data_ptr() - st.data_ptr())


def _check(status: int, where: str):
    if status != 0:
        raise MbokError(status, where)


def alpha_torch_dtype(alpha_dtype: int) -> torch.dtype:
    return {MBOK_F32: torch.float32, MBOK_F16: torch.float16}[alpha_dtype]


def _x_dtype(t: torch.Tensor) -> int:
    if t.dtype == torch.bfloat16:
        return MBOK_BF16
    if t.dtype == torch.float32:
        return MBOK_F32
    raise ValueError(f"activations must be bfloat16 or float32, got {t.dtype}")


# ---------------------------------------------------------------- the C ABI

def mbok_status_str(status: int) -> str:
    return load_library().mbok_status_str(int(status)).decode()


def mbok_version() -> str:
    return load_library().mbok_version().decode()


def mbok_desc_init(m: int, n: int, K: int, alpha_dtype: int = MBOK_F16) -> mbok_desc:
    d = mbok_desc()
    _check(load_library().mbok_desc_init(ctypes.byref(d), m, n, K, alpha_dtype), "mbok_desc_init")
    return d


def mbok_packed_bytes(d: mbok_desc) -> int:
    return int(load_library().mbok_packed_bytes(ctypes.byref(d)))


def mbok_alpha_bytes(d: mbok_desc) -> int:
    return int(load_library().mbok_alpha_bytes(ctypes.byref(d)))


def mbok_residual_binarize(d: mbok_desc, W: torch.Tensor, signs: torch.Tensor,
                           alpha: torch.Tensor, flag: torch.Tensor | None = None,
                           stream=None) -> None:
    """W fp32 [m, ldw] -> signs int8 [K, m, n] and alpha [K, m, n/128]."""
    _dev(W, "W"), _dev(signs, "signs"), _dev(alpha, "alpha")
    if W.dtype != torch.float32 or W.dim() != 2 or W.shape[0] != d.m or W.shape[1] < d.n:
        raise ValueError("W must be float32 [m, >= n]")
    if W.stride(1) != 1:
        raise ValueError("W rows must be contiguous")
    ldw = W.stride(0)
    if _nbytes_from(W) < ((d.m - 1) * ldw + d.n) * 4:
        raise ValueError("W buffer too small")
    if signs.dtype != torch.int8 or _nbytes_from(signs) < d.K * d.m * d.n:
        raise ValueError("signs must be int8 with K*m*n elements")
    if alpha.dtype != alpha_torch_dtype(d.alpha_dtype) or _nbytes_from(alpha) < mbok_alpha_bytes(d):
        raise ValueError("alpha has the wrong dtype or size")
    fptr = None
    if flag is not None:
        _dev(flag, "flag")
        if flag.dtype != torch.int32 or flag.numel() < 1:
            raise ValueError("flag must be int32 with >= 1 element")
        fptr = flag.data_ptr()
    _check(load_library().mbok_residual_binarize(
        ctypes.byref(d), W.data_ptr(), ldw, signs.data_ptr(), alpha.data_ptr(), fptr,
        _stream(stream)), "mbok_residual_binarize")


def mbok_refit(d: mbok_desc, W: torch.Tensor, signs: torch.Tensor, alpha: torch.Tensor,
               rounds: int = 2, stream=None) -> None:
    """Alternating least-squares refit of signs int8 [K, m, n] and alpha
    [K, m, n/128] (both updated in place) for W fp32 [m, ldw]."""
    _dev(W, "W"), _dev(signs, "signs"), _dev(alpha, "alpha")
    if W.dtype != torch.float32 or W.dim() != 2 or W.shape[0] != d.m or W.shape[1] < d.n:
        raise ValueError("W must be float32 [m, >= n]")
    if W.stride(1) != 1:
        raise ValueError("W rows must be contiguous")
    ldw = W.stride(0)
    if _nbytes_from(W) < ((d.m - 1) * ldw + d.n) * 4:
        raise ValueError("W buffer too small")
    if signs.dtype != torch.int8 or not signs.is_contiguous() or \
            _nbytes_from(signs) < d.K * d.m * d.n:
        raise ValueError("signs must be contiguous int8 with K*m*n elements")
    if alpha.dtype != alpha_torch_dtype(d.alpha_dtype) or not alpha.is_contiguous() \
            or _nbytes_from(alpha) < mbok_alpha_bytes(d):
        raise ValueError("alpha has the wrong dtype or size")
    _check(load_library().mbok_refit(ctypes.byref(d), W.data_ptr(), ldw, signs.data_ptr(),
                                     alpha.data_ptr(), int(rounds), _stream(stream)),
           "mbok_refit")


def mbok_residual_energy(d: mbok_desc, W: torch.Tensor, row_energy: torch.Tensor,
                         layer_energy: torch.Tensor, stream=None) -> None:
    """Residual energies of the greedy chain after 0..K kernels: row_energy
    float64 [K+1, m] and layer_energy float64 [K+1] (both overwritten)."""
    _dev(W, "W"), _dev(row_energy, "row_energy"), _dev(layer_energy, "layer_energy")
    if W.dtype != torch.float32 or W.dim() != 2 or W.shape[0] != d.m or W.shape[1] < d.n:
        raise ValueError("W must be float32 [m, >= n]")
    if W.stride(1) != 1:
        raise ValueError("W rows must be contiguous")
    ldw = W.stride(0)
    if _nbytes_from(W) < ((d.m - 1) * ldw + d.n) * 4:
        raise ValueError("W buffer too small")
    for t, cnt, nm in ((row_energy, (d.K + 1) * d.m, "row_energy"),
                       (layer_energy, d.K + 1, "layer_energy")):
        if t.dtype != torch.float64 or not t.is_contiguous() or t.numel() < cnt:
            raise ValueError(f"{nm} must be contiguous float64 with {cnt} elements")
    _check(load_library().mbok_residual_energy(ctypes.byref(d), W.data_ptr(), ldw,
                                               row_energy.data_ptr(), layer_energy.data_ptr(),
                                               _stream(stream)), "mbok_residual_energy")


def mbok_allocate_kernels(sizes, errors, budget: int) -> list:
    """Kernels per weight under a total bit budget (host only).  sizes: L
    entry counts; errors: L rows of kmax residual energies (K = 1..kmax)."""
    import numpy as np

    sz = np.ascontiguousarray(np.asarray(sizes, dtype=np.int64).reshape(-1))
    er = np.ascontiguousarray(np.asarray(errors, dtype=np.float64))
    if er.ndim != 2 or er.shape[0] != sz.shape[0]:
        raise ValueError("errors must be [L, kmax] with one row per size")
    out = np.zeros(sz.shape[0], dtype=np.int32)
    _check(load_library().mbok_allocate_kernels(
        int(sz.shape[0]), sz.ctypes.data, er.ctypes.data, int(er.shape[1]), int(budget),
        out.ctypes.data), "mbok_allocate_kernels")
    return out.tolist()


def mbok_pack(d: mbok_desc, signs: torch.Tensor, alpha: torch.Tensor, packed: torch.Tensor,
              stream=None) -> None:
    """signs int8 [K, m, n] + alpha [K, m, n/128] -> packed uint8 [mbok_packed_bytes]."""
    _dev(signs, "signs"), _dev(alpha, "alpha"), _dev(packed, "packed")
    if signs.dtype != torch.int8 or not signs.is_contiguous() or signs.numel() < d.K * d.m * d.n:
        raise ValueError("signs must be contiguous int8 with K*m*n elements")
    if alpha.dtype != alpha_torch_dtype(d.alpha_dtype) or not alpha.is_contiguous() \
            or _nbytes_from(alpha) < mbok_alpha_bytes(d):
        raise ValueError("alpha has the wrong dtype or size")
    if _nbytes_from(packed) < mbok_packed_bytes(d):
        raise ValueError("packed buffer too small")
    _check(load_library().mbok_pack(ctypes.byref(d), signs.data_ptr(), alpha.data_ptr(),
                                    packed.data_ptr(), _stream(stream)), "mbok_pack")


def mbok_gemv_workspace_bytes(d: mbok_desc) -> int:
    return int(load_library().mbok_gemv_workspace_bytes(ctypes.byref(d)))


_WORKSPACES: dict = {}
_WORKSPACE_LOCKS: dict = {}


def _torch_stream(device: torch.device, stream) -> torch.cuda.Stream:
    """The torch stream of a call's `stream` argument (a handle of 0 is the
    default stream; an ExternalStream of it would be one of torch's own)."""
    if stream is None:
        return torch.cuda.current_stream(device)
    if isinstance(stream, torch.cuda.Stream):
        return stream
    handle = int(stream)
    if handle == 0:
        return torch.cuda.default_stream(device)
    return torch.cuda.ExternalStream(handle, device=device)


def workspace_for(nbytes: int, device=None, stream=None) -> torch.Tensor | None:
    """A workspace of at least nbytes, kept per (device, stream) so that calls
    which may overlap never share one.

    The tensor is allocated with the target stream current, so torch's caching
    allocator ties its memory to that stream: when a larger request replaces
    it, the old block is reused only in that stream's order, after the work
    already enqueued there that reads it.  While that stream is captured
    into a graph the tensor is a new one of the graph's pool and is not kept:
    the graph holds its memory, which a kept one's replacement would free.

    The calls below that keep a workspace by themselves enqueue all their
    kernels before another thread's call on the same stream may use it; two
    threads that pass one tensor to calls on one stream have to see to that."""
    if nbytes == 0:
        return None
    dev = torch.device(device) if device is not None else torch.device("cuda", torch.cuda.current_device())
    target = _torch_stream(dev, stream)
    with torch.cuda.stream(target):
        if torch.cuda.is_current_stream_capturing():
            return torch.empty(nbytes, dtype=torch.uint8, device=dev)
        key = (dev.index, target.cuda_stream)
        ws = _WORKSPACES.get(key)
        if ws is None or ws.numel() < nbytes:
            ws = torch.empty(max(nbytes, 1 << 20), dtype=torch.uint8, device=dev)
            _WORKSPACES[key] = ws
    return ws


class _Kept:
    """The kept workspace of a device and stream (its tensor, None for 0 bytes),
    for the `with` block's thread alone: a call's kernels, of which the first
    writes the workspace and the last reads it, are enqueued without another
    thread's between them (the library's calls run without the interpreter's
    lock)."""
    __slots__ = ("nbytes", "device", "stream", "lock")

    def __init__(self, nbytes: int, device: torch.device, stream):
        self.nbytes, self.device, self.stream = nbytes, device, stream

    def __enter__(self) -> torch.Tensor | None:
        index, stream = self.device.index, self.stream
        handle = _raw_stream(index) if stream is None else _stream(stream)
        key = (index, handle)
        lock = _WORKSPACE_LOCKS.get(key)
        if lock is None:
            lock = _WORKSPACE_LOCKS.setdefault(key, threading.RLock())
        self.lock = lock
        lock.acquire()
        ws = _WORKSPACES.get(key)
        if ws is not None and ws.numel() >= self.nbytes:
            return ws
        try:
            return workspace_for(self.nbytes, self.device, stream)
        except BaseException:
            lock.release()
            raise

    def __exit__(self, *_):
        self.lock.release()


_NO_WORKSPACE = contextlib.nullcontext()


def _own_or_kept(need: int, device: torch.device, stream):
    """The kept workspace, see _Kept; under graph capture one of the call's own,
    from the graph's pool, so that no later call's growth frees it and no two
    graphs share it."""
    # the launch stream current, unless it is
    here = stream is None and device.index == _current_device()
    with _NO_WORKSPACE if here else torch.cuda.stream(_torch_stream(device, stream)):
        if torch.cuda.is_current_stream_capturing():
            return contextlib.nullcontext(torch.empty(need, dtype=torch.uint8, device=device))
    return _Kept(need, device, stream)


def _given_or_kept(need: int, workspace, device: torch.device, stream):
    """Context of mbok_gemv's and mbok_gemvt's workspace tensor, or None."""
    if workspace is None or workspace is False or need == 0:
        return _NO_WORKSPACE
    if workspace is True:
        return _own_or_kept(need, device, stream)
    _dev(workspace, "workspace")
    if _nbytes_from(workspace) < need:
        raise ValueError("workspace too small")
    return contextlib.nullcontext(workspace)


def mbok_gemv(d: mbok_desc, packed: torch.Tensor, x: torch.Tensor, y: torch.Tensor,
              workspace: torch.Tensor | None | bool = True, stream=None) -> None:
    """y[m] (fp32, overwritten) = W_hat x for x bf16 / fp32 [n].

    workspace: True (default) uses a workspace kept for this device and
    stream (under graph capture one of the graph's own); a tensor is used as
    given; None/False runs without one."""
    _dev(packed, "packed"), _dev(x, "x"), _dev(y, "y")
    if _nbytes_from(packed) < mbok_packed_bytes(d):
        raise ValueError("packed buffer too small")
    xd = _x_dtype(x)
    if x.numel() < d.n or not x.is_contiguous():
        raise ValueError("x must be contiguous with n elements")
    if y.dtype != torch.float32 or y.numel() < d.m or not y.is_contiguous():
        raise ValueError("y must be contiguous float32 with m elements")
    need = mbok_gemv_workspace_bytes(d)
    with _given_or_kept(need, workspace, y.device, stream) as ws:
        _check(load_library().mbok_gemv(ctypes.byref(d), packed.data_ptr(), x.data_ptr(), xd,
                                        y.data_ptr(), None if ws is None else ws.data_ptr(),
                                        _stream(stream)), "mbok_gemv")


def mbok_gemvt_workspace_bytes(d: mbok_desc) -> int:
    return int(load_library().mbok_gemvt_workspace_bytes(ctypes.byref(d)))


def mbok_gemvt(d: mbok_desc, packed: torch.Tensor, g: torch.Tensor, dx: torch.Tensor,
               workspace: torch.Tensor | None | bool = True, stream=None) -> None:
    """dx[n] (fp32, overwritten) = W_hat^T g for g bf16 / fp32 [m].

    workspace: True (default) uses a workspace kept for this device and
    stream (under graph capture one of the graph's own); a tensor is used as
    given; None/False runs without one."""
    _dev(packed, "packed"), _dev(g, "g"), _dev(dx, "dx")
    if _nbytes_from(packed) < mbok_packed_bytes(d):
        raise ValueError("packed buffer too small")
    gd = _x_dtype(g)
    if g.numel() < d.m or not g.is_contiguous():
        raise ValueError("g must be contiguous with m elements")
    if dx.dtype != torch.float32 or dx.numel() < d.n or not dx.is_contiguous():
        raise ValueError("dx must be contiguous float32 with n elements")
    need = mbok_gemvt_workspace_bytes(d)
    with _given_or_kept(need, workspace, dx.device, stream) as ws:
        _check(load_library().mbok_gemvt(ctypes.byref(d), packed.data_ptr(), g.data_ptr(), gd,
                                         dx.data_ptr(), None if ws is None else ws.data_ptr(),
                                         _stream(stream)), "mbok_gemvt")


def mbok_gemvt_scratch_bytes() -> int:
    return int(load_library().mbok_gemvt_scratch_bytes())


def mbok_gemvt_noalloc(d: mbok_desc, packed: torch.Tensor, g: torch.Tensor, dx: torch.Tensor,
                       stream=None) -> None:
    """mbok_gemvt with the library's static scratch instead of a workspace
    (for callers that cannot allocate device memory).  Calls that overlap in
    time on one GPU share that scratch and race."""
    _dev(packed, "packed"), _dev(g, "g"), _dev(dx, "dx")
    if _nbytes_from(packed) < mbok_packed_bytes(d):
        raise ValueError("packed buffer too small")
    gd = _x_dtype(g)
    if g.numel() < d.m or not g.is_contiguous():
        raise ValueError("g must be contiguous with m elements")
    if dx.dtype != torch.float32 or dx.numel() < d.n or not dx.is_contiguous():
        raise ValueError("dx must be contiguous float32 with n elements")
    _check(load_library().mbok_gemvt_noalloc(ctypes.byref(d), packed.data_ptr(), g.data_ptr(),
                                             gd, dx.data_ptr(), _stream(stream)),
           "mbok_gemvt_noalloc")


def mbok_svid_workspace_bytes(d: mbok_desc) -> int:
    return int(load_library().mbok_svid_workspace_bytes(ctypes.byref(d)))


def mbok_svid_gemv_workspace_bytes(d: mbok_desc) -> int:
    return int(load_library().mbok_svid_gemv_workspace_bytes(ctypes.byref(d)))


def mbok_svid_decompose(d: mbok_desc, W: torch.Tensor, signs: torch.Tensor, s_out: torch.Tensor,
                        s_in: torch.Tensor, iters: int = 32, workspace: torch.Tensor | None = None,
                        stream=None) -> None:
    """Successive SVID of W fp32 [m, ldw] into signs int8 [K, m, n], s_out
    [K, m] and s_in [K, n] (scale dtype).  A workspace is allocated when none
    is given."""
    _dev(W, "W"), _dev(signs, "signs"), _dev(s_out, "s_out"), _dev(s_in, "s_in")
    if W.dtype != torch.float32 or W.dim() != 2 or W.shape[0] != d.m or W.shape[1] < d.n:
        raise ValueError("W must be float32 [m, >= n]")
    if W.stride(1) != 1:
        raise ValueError("W rows must be contiguous")
    ldw = W.stride(0)
    if _nbytes_from(W) < ((d.m - 1) * ldw + d.n) * 4:
        raise ValueError("W buffer too small")
    at = alpha_torch_dtype(d.alpha_dtype)
    if signs.dtype != torch.int8 or not signs.is_contiguous() or signs.numel() < d.K * d.m * d.n:
        raise ValueError("signs must be contiguous int8 with K*m*n elements")
    for t, cnt, nm in ((s_out, d.K * d.m, "s_out"), (s_in, d.K * d.n, "s_in")):
        if t.dtype != at or not t.is_contiguous() or t.numel() < cnt:
            raise ValueError(f"{nm} must be contiguous {at} with {cnt} elements")
    need = mbok_svid_workspace_bytes(d)
    if workspace is None:
        workspace = torch.empty(need, dtype=torch.uint8, device=W.device)
    _dev(workspace, "workspace")
    if _nbytes_from(workspace) < need:
        raise ValueError("workspace too small")
    _check(load_library().mbok_svid_decompose(
        ctypes.byref(d), W.data_ptr(), ldw, signs.data_ptr(), s_out.data_ptr(), s_in.data_ptr(),
        int(iters), workspace.data_ptr(), _stream(stream)), "mbok_svid_decompose")


def mbok_svid_pack(d: mbok_desc, signs: torch.Tensor, s_out: torch.Tensor, packed: torch.Tensor,
                   stream=None) -> None:
    """signs int8 [K, m, n] + s_out [K, m] -> packed uint8 [mbok_packed_bytes]."""
    _dev(signs, "signs"), _dev(s_out, "s_out"), _dev(packed, "packed")
    if signs.dtype != torch.int8 or not signs.is_contiguous() or signs.numel() < d.K * d.m * d.n:
        raise ValueError("signs must be contiguous int8 with K*m*n elements")
    if s_out.dtype != alpha_torch_dtype(d.alpha_dtype) or not s_out.is_contiguous() or \
            s_out.numel() < d.K * d.m:
        raise ValueError("s_out has the wrong dtype or size")
    if _nbytes_from(packed) < mbok_packed_bytes(d):
        raise ValueError("packed buffer too small")
    _check(load_library().mbok_svid_pack(ctypes.byref(d), signs.data_ptr(), s_out.data_ptr(),
                                         packed.data_ptr(), _stream(stream)), "mbok_svid_pack")


def mbok_svid_gemv(d: mbok_desc, packed: torch.Tensor, s_in: torch.Tensor, x: torch.Tensor,
                   y: torch.Tensor, stream=None) -> None:
    """y[m] (fp32, overwritten) = sum_k s_out^k (.) (B_k (s_in^k (.) x)) for x bf16 / fp32 [n]."""
    _dev(packed, "packed"), _dev(s_in, "s_in"), _dev(x, "x"), _dev(y, "y")
    if _nbytes_from(packed) < mbok_packed_bytes(d):
        raise ValueError("packed buffer too small")
    if s_in.dtype != alpha_torch_dtype(d.alpha_dtype) or not s_in.is_contiguous() or \
            s_in.numel() < d.K * d.n:
        raise ValueError("s_in has the wrong dtype or size")
    xd = _x_dtype(x)
    if x.numel() < d.n or not x.is_contiguous():
        raise ValueError("x must be contiguous with n elements")
    if y.dtype != torch.float32 or y.numel() < d.m or not y.is_contiguous():
        raise ValueError("y must be contiguous float32 with m elements")
    _check(load_library().mbok_svid_gemv(ctypes.byref(d), packed.data_ptr(), s_in.data_ptr(),
                                         x.data_ptr(), xd, y.data_ptr(), None, _stream(stream)),
           "mbok_svid_gemv")


def mbok_gemm(d: mbok_desc, packed: torch.Tensor, X: torch.Tensor, Y: torch.Tensor,
              stream=None) -> None:
    """Y[T, m] (fp32, overwritten) = X W_hat^T for X bf16 [T, n] (row stride ldx)."""
    _gemm_call("mbok_gemm", d, packed, X, Y, stream)


def mbok_gemm_precise(d: mbok_desc, packed: torch.Tensor, X: torch.Tensor, Y: torch.Tensor,
                      stream=None) -> None:
    """mbok_gemm with each prefill weight carried as two bf16 terms (hi + lo)."""
    _gemm_call("mbok_gemm_precise", d, packed, X, Y, stream)


def _gemm_call(name: str, d: mbok_desc, packed: torch.Tensor, X: torch.Tensor, Y: torch.Tensor,
               stream) -> None:
    _dev(packed, "packed"), _dev(X, "X"), _dev(Y, "Y")
    if _nbytes_from(packed) < mbok_packed_bytes(d):
        raise ValueError("packed buffer too small")
    xd = _x_dtype(X)
    if X.dim() != 2 or X.shape[1] < d.n or X.stride(1) != 1:
        raise ValueError("X must be 2-D [T, >= n] with contiguous rows")
    if Y.dtype != torch.float32 or Y.dim() != 2 or Y.shape[0] != X.shape[0] or \
            Y.shape[1] < d.m or Y.stride(1) != 1:
        raise ValueError("Y must be float32 [T, >= m] with contiguous rows")
    T = X.shape[0]
    ldx, ldy = X.stride(0), Y.stride(0)
    if T > 0:
        if _nbytes_from(X) < ((T - 1) * ldx + d.n) * X.element_size():
            raise ValueError("X buffer too small")
        if _nbytes_from(Y) < ((T - 1) * ldy + d.m) * 4:
            raise ValueError("Y buffer too small")
    fn = getattr(load_library(), name)
    _check(fn(ctypes.byref(d), packed.data_ptr(), X.data_ptr(), xd, T, ldx, Y.data_ptr(), ldy,
              _stream(stream)), name)


# ------------------------------------- fine-tuning and the gated feed-forward block

_FLOATS = {torch.float32: MBOK_F32, torch.float16: MBOK_F16, torch.bfloat16: MBOK_BF16}
# These calls take a few microseconds on the GPU at their smallest, so what
# Python adds to a launch counts: the raw stream handle and current device
# come from the C functions behind torch.cuda.current_stream() and
# current_device() (together 1.3 us less per call), tensors are asked for each
# attribute once, and layer sizes are remembered by shape.  A torch without GPU
# support has neither function; the host-only calls work there.
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream",
                      lambda dev: torch.cuda.current_stream(dev).cuda_stream)
_current_device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)


@functools.lru_cache(maxsize=4096)
def _packed_bytes(m: int, n: int, K: int, alpha_dtype: int) -> int:
    return mbok_packed_bytes(mbok_desc_init(m, n, K, alpha_dtype))


@functools.lru_cache(maxsize=4096)
def _slices_bytes(name: str, m: int, n: int, K: int, alpha_dtype: int, T: int) -> int:
    d = mbok_desc_init(m, n, K, alpha_dtype)
    return int(getattr(load_library(), name)(ctypes.byref(d), T))


def _launch(fn, name: str, dev: int, stream, *args) -> None:
    """fn(*args, stream) with the tensors' device current."""
    if dev == _current_device():
        status = fn(*args, _raw_stream(dev) if stream is None else _stream(stream))
    else:
        with torch.cuda.device(dev):
            status = fn(*args, _raw_stream(dev) if stream is None else _stream(stream))
    if status:
        raise MbokError(status, name)


def _first(t: torch.Tensor, name: str) -> int:
    """The device of a call's first tensor; the others have to be on it."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    dev = t.get_device()
    if dev < 0:
        raise ValueError(f"{name} must be on the GPU (the library takes device pointers)")
    return dev


def _elsewhere(t, name: str):
    _dev(t, name)
    raise ValueError(f"{name} is on another device than the other tensors")


def _matrix(t: torch.Tensor, name: str, dev: int, rows: int, cols: int, dtype) -> int:
    """Row stride of a [rows, >= cols] matrix with contiguous rows."""
    if not isinstance(t, torch.Tensor) or t.get_device() != dev:
        _elsewhere(t, name)
    if t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
    shape = t.shape
    if len(shape) != 2 or shape[0] != rows or shape[1] < cols:
        raise ValueError(f"{name} must be [{rows}, >= {cols}], got {tuple(shape)}")
    ld, step = t.stride()
    if step != 1 and shape[1] > 1:
        raise ValueError(f"{name} rows must be contiguous")
    if rows == 1:
        # the stride of a single row is arbitrary and never used; one value per
        # operand, so that views of one row are the same matrix to the library
        return (cols + 7) // 8 * 8
    if ld < cols:
        raise ValueError(f"{name} rows must not overlap")
    return ld


def _vector(t: torch.Tensor, name: str, dev: int, count: int, dtype) -> int:
    if not isinstance(t, torch.Tensor) or t.get_device() != dev:
        _elsewhere(t, name)
    if t.dtype != dtype or not t.is_contiguous() or t.numel() < count:
        raise ValueError(f"{name} must be contiguous {dtype} with {count} elements")
    return t.data_ptr()


def _packed(packed: torch.Tensor, dev: int, m: int, n: int, K: int, alpha_dtype: int) -> int:
    if not isinstance(packed, torch.Tensor) or packed.get_device() != dev:
        _elsewhere(packed, "packed")
    if not packed.is_contiguous() or \
            packed.numel() * packed.itemsize < _packed_bytes(m, n, K, alpha_dtype):
        raise ValueError("packed must be contiguous and hold the layer")
    return packed.data_ptr()


def _slices(name: str, m: int, n: int, K: int, alpha_dtype: int, T: int, workspace, dev: int,
            stream):
    """Context of the workspace tensor of a call that may split its sum, or None."""
    if workspace is None or workspace is False:
        return _NO_WORKSPACE
    need = _slices_bytes(name, m, n, K, alpha_dtype, T)
    if need == 0:
        return _NO_WORKSPACE
    if workspace is not True:
        ws = workspace
        if not isinstance(ws, torch.Tensor) or ws.get_device() != dev:
            _elsewhere(ws, "workspace")
        if not ws.is_contiguous() or ws.numel() * ws.itemsize < need:
            raise ValueError("workspace must be contiguous and large enough")
        return contextlib.nullcontext(ws)
    return _own_or_kept(need, torch.device("cuda", dev), stream)


def mbok_gemmt_workspace_bytes(d: mbok_desc, T: int) -> int:
    return int(load_library().mbok_gemmt_workspace_bytes(ctypes.byref(d), T))


def mbok_scale_grad_workspace_bytes(d: mbok_desc, T: int) -> int:
    return int(load_library().mbok_scale_grad_workspace_bytes(ctypes.byref(d), T))


def mbok_gemmt(d: mbok_desc, packed: torch.Tensor, dY: torch.Tensor, dX: torch.Tensor,
               workspace: torch.Tensor | None | bool = True, stream=None) -> None:
    """dX[T, n] (bf16, overwritten) = dY W_hat for dY bf16 [T, m] (row strides
    lddx, lddy).

    workspace: True (default) uses a workspace kept for this device and
    stream (under graph capture one of the graph's own); a tensor is used as
    given; None/False runs without one."""
    _gemmt_call("mbok_gemmt", d, packed, dY, dX, workspace, stream)


def mbok_gemmt_precise(d: mbok_desc, packed: torch.Tensor, dY: torch.Tensor, dX: torch.Tensor,
                       workspace: torch.Tensor | None | bool = True, stream=None) -> None:
    """mbok_gemmt with each weight carried as two bf16 terms (twice the matrix
    work)."""
    _gemmt_call("mbok_gemmt_precise", d, packed, dY, dX, workspace, stream)


def _gemmt_call(name: str, d: mbok_desc, packed, dY, dX, workspace, stream) -> None:
    dev = _first(dY, "dY")
    m, n, K, at = d.m, d.n, d.K, d.alpha_dtype
    T = dY.shape[0]
    lddy = _matrix(dY, "dY", dev, T, m, torch.bfloat16)
    lddx = _matrix(dX, "dX", dev, T, n, torch.bfloat16)
    pp = _packed(packed, dev, m, n, K, at)
    with _slices("mbok_gemmt_workspace_bytes", m, n, K, at, T, workspace, dev, stream) as ws:
        _launch(getattr(load_library(), name), name, dev, stream, ctypes.byref(d), pp,
                dY.data_ptr(), T, lddy, dX.data_ptr(), lddx, None if ws is None else ws.data_ptr())


def mbok_scale_grad(d: mbok_desc, packed: torch.Tensor, dY: torch.Tensor, X: torch.Tensor,
                    dalpha: torch.Tensor, accumulate: bool = False,
                    workspace: torch.Tensor | None | bool = True, stream=None) -> None:
    """dalpha fp32 [K, m, n/128] = (or, accumulate, +=) sum over each group's
    columns of B_k (.) (dY^T X), for dY bf16 [T, m] and X bf16 [T, n].

    workspace: as for mbok_gemmt."""
    dev = _first(dY, "dY")
    m, n, K, at = d.m, d.n, d.K, d.alpha_dtype
    T = dY.shape[0]
    lddy = _matrix(dY, "dY", dev, T, m, torch.bfloat16)
    ldx = _matrix(X, "X", dev, T, n, torch.bfloat16)
    out = _vector(dalpha, "dalpha", dev, K * m * (n // MBOK_GROUP), torch.float32)
    pp = _packed(packed, dev, m, n, K, at)
    with _slices("mbok_scale_grad_workspace_bytes", m, n, K, at, T, workspace, dev, stream) as ws:
        _launch(load_library().mbok_scale_grad, "mbok_scale_grad", dev, stream, ctypes.byref(d),
                pp, dY.data_ptr(), T, lddy, X.data_ptr(), ldx, out, int(bool(accumulate)),
                None if ws is None else ws.data_ptr())


def mbok_gated_stack(d: mbok_desc) -> mbok_desc:
    """The descriptor of the stacked layer (8 gate rows, 8 up rows per 16-row
    tile) of two projections of shape d: 16 ceil(m / 8) rows."""
    out = mbok_desc()
    _check(load_library().mbok_gated_stack(ctypes.byref(d), ctypes.byref(out)),
           "mbok_gated_stack")
    return out


def mbok_gated_pack(d: mbok_desc, signs_gate: torch.Tensor, alpha_gate: torch.Tensor,
                    signs_up: torch.Tensor, alpha_up: torch.Tensor, packed: torch.Tensor,
                    stream=None) -> None:
    """signs int8 [K, m, n] + alpha [K, m, n/128] of both projections -> packed
    uint8 [mbok_packed_bytes(mbok_gated_stack(d))]."""
    dev = _first(packed, "packed")
    m, n, K = d.m, d.n, d.K
    ns, na, at = K * m * n, K * m * (n // MBOK_GROUP), alpha_torch_dtype(d.alpha_dtype)
    ptrs = [_vector(signs_gate, "signs_gate", dev, ns, torch.int8),
            _vector(alpha_gate, "alpha_gate", dev, na, at),
            _vector(signs_up, "signs_up", dev, ns, torch.int8),
            _vector(alpha_up, "alpha_up", dev, na, at)]
    pp = _packed(packed, dev, 16 * ((m + 7) // 8), n, K, d.alpha_dtype)
    _launch(load_library().mbok_gated_pack, "mbok_gated_pack", dev, stream, ctypes.byref(d),
            *ptrs, pp)


def mbok_gated(d: mbok_desc, packed: torch.Tensor, X: torch.Tensor, H: torch.Tensor,
               pre: torch.Tensor | None = None, act: int = MBOK_ACT_SILU, stream=None) -> None:
    """H[T, m] (bf16, overwritten) = act(X Wg^T) (.) (X Wu^T) for X bf16 [T, n];
    d describes one projection, packed is mbok_gated_pack's buffer.  pre bf16
    [T, 16 ceil(m / 8)] receives the pre-activations in the stacked order."""
    _gated_call("mbok_gated", d, packed, X, H, pre, act, stream)


def mbok_gated_precise(d: mbok_desc, packed: torch.Tensor, X: torch.Tensor, H: torch.Tensor,
                       pre: torch.Tensor | None = None, act: int = MBOK_ACT_SILU,
                       stream=None) -> None:
    """mbok_gated with each weight carried as two bf16 terms for T > 16 (twice
    the matrix work)."""
    _gated_call("mbok_gated_precise", d, packed, X, H, pre, act, stream)


def _gated_call(name: str, d: mbok_desc, packed, X, H, pre, act, stream) -> None:
    dev = _first(X, "X")
    m, n = d.m, d.n
    T, m2 = X.shape[0], 16 * ((m + 7) // 8)
    ldx = _matrix(X, "X", dev, T, n, torch.bfloat16)
    ldh = _matrix(H, "H", dev, T, m, torch.bfloat16)
    pre_ptr, ldpre = None, 0
    if pre is not None:
        ldpre = _matrix(pre, "pre", dev, T, m2, torch.bfloat16)
        pre_ptr = pre.data_ptr()
    _launch(getattr(load_library(), name), name, dev, stream, ctypes.byref(d),
            _packed(packed, dev, m2, n, d.K, d.alpha_dtype), X.data_ptr(), MBOK_BF16, T, ldx, act,
            H.data_ptr(), ldh, pre_ptr, ldpre)


def mbok_gated_backward(d: mbok_desc, packed: torch.Tensor, pre: torch.Tensor, dH: torch.Tensor,
                        dpre: torch.Tensor, dX: torch.Tensor | None = None,
                        act: int = MBOK_ACT_SILU,
                        workspace: torch.Tensor | None | bool = True, stream=None) -> None:
    """Gradients of the gated block: dpre bf16 [T, 16 ceil(m / 8)] (stacked
    order; may be pre itself) and, unless None, dX bf16 [T, n], from pre as
    mbok_gated wrote it and dH bf16 [T, m].

    workspace: as for mbok_gemmt."""
    _gated_backward_call("mbok_gated_backward", d, packed, pre, dH, dpre, dX, act, workspace,
                         stream)


def mbok_gated_backward_precise(d: mbok_desc, packed: torch.Tensor, pre: torch.Tensor,
                                dH: torch.Tensor, dpre: torch.Tensor,
                                dX: torch.Tensor | None = None, act: int = MBOK_ACT_SILU,
                                workspace: torch.Tensor | None | bool = True,
                                stream=None) -> None:
    """mbok_gated_backward with dX as mbok_gemmt_precise computes it."""
    _gated_backward_call("mbok_gated_backward_precise", d, packed, pre, dH, dpre, dX, act,
                         workspace, stream)


def _gated_backward_call(name: str, d: mbok_desc, packed, pre, dH, dpre, dX, act, workspace,
                         stream) -> None:
    dev = _first(dH, "dH")
    m, n, K, at = d.m, d.n, d.K, d.alpha_dtype
    T, m2 = dH.shape[0], 16 * ((m + 7) // 8)
    lddh = _matrix(dH, "dH", dev, T, m, torch.bfloat16)
    ldpre = _matrix(pre, "pre", dev, T, m2, torch.bfloat16)
    lddpre = _matrix(dpre, "dpre", dev, T, m2, torch.bfloat16)
    pp = _packed(packed, dev, m2, n, K, at)
    dx_ptr, lddx, held = None, 0, _NO_WORKSPACE
    if dX is not None:
        lddx = _matrix(dX, "dX", dev, T, n, torch.bfloat16)
        dx_ptr = dX.data_ptr()
        held = _slices("mbok_gemmt_workspace_bytes", m2, n, K, at, T, workspace, dev, stream)
    with held as ws:
        _launch(getattr(load_library(), name), name, dev, stream, ctypes.byref(d), pp,
                pre.data_ptr(), ldpre, dH.data_ptr(), lddh, T, act, dpre.data_ptr(), lddpre,
                dx_ptr, lddx, None if ws is None else ws.data_ptr())


def mbok_distill_desc_init(vocab: int, top: int, temperature: float = 1.0) -> mbok_distill_desc:
    d = mbok_distill_desc()
    _check(load_library().mbok_distill_desc_init(ctypes.byref(d), vocab, top, temperature),
           "mbok_distill_desc_init")
    return d


def _distill_args(d, dev, Z, t_logits, t_index, t_lse, weight):
    """(T, vocabulary, the arguments both distillation calls begin with), checked."""
    vocab, top, T = d.vocab, d.top, Z.shape[0]
    dz, dt = Z.dtype, t_logits.dtype
    zt, tt = _FLOATS.get(dz), _FLOATS.get(dt)
    if zt is None or tt is None:
        raise ValueError("Z and t_logits must be float32, float16 or bfloat16")
    ldz = _matrix(Z, "Z", dev, T, vocab, dz)
    ldt = _matrix(t_index, "t_index", dev, T, top, torch.int32)
    if _matrix(t_logits, "t_logits", dev, T, top, dt) != ldt and T > 1:
        raise ValueError("t_logits and t_index must have the same row stride")
    return T, vocab, (
        ctypes.byref(d), Z.data_ptr(), zt, T, ldz, t_logits.data_ptr(), tt, t_index.data_ptr(),
        ldt, None if t_lse is None else _vector(t_lse, "t_lse", dev, T, torch.float32),
        None if weight is None else _vector(weight, "weight", dev, T, torch.float32))


def _distill_grad(dZ, dev, T, vocab, z_dtype):
    if not isinstance(dZ, torch.Tensor):
        raise TypeError("dZ must be a torch.Tensor")
    dt = dZ.dtype
    if dt != z_dtype and dt != torch.bfloat16:
        raise ValueError("dZ must have the dtype of Z or bfloat16")
    ld = _matrix(dZ, "dZ", dev, T, vocab, dt)
    return dZ.data_ptr(), _FLOATS[dt], ld


def mbok_distill(d: mbok_distill_desc, Z: torch.Tensor, t_logits: torch.Tensor,
                 t_index: torch.Tensor, loss: torch.Tensor, stats: torch.Tensor | None = None,
                 dZ: torch.Tensor | None = None, t_lse: torch.Tensor | None = None,
                 weight: torch.Tensor | None = None, stream=None) -> None:
    """loss[T] (fp32, overwritten) = weight tau^2 KL(teacher || softmax(Z / tau))
    over the teacher's listed logits t_logits [T, top] at the tokens t_index
    (int32; negative: no entry), renormalised, or with t_lse [T] as the
    teacher's own probabilities with the rest as one class.  stats fp32 [T,
    MBOK_DISTILL_STATS] is what mbok_distill_backward takes; dZ (dtype of Z or
    bf16; may be Z) receives the gradient of sum(loss) in the same pass."""
    dev = _first(Z, "Z")
    _first(t_logits, "t_logits")
    T, vocab, args = _distill_args(d, dev, Z, t_logits, t_index, t_lse, weight)
    grad = (None, args[2], 0) if dZ is None else _distill_grad(dZ, dev, T, vocab, Z.dtype)
    _launch(load_library().mbok_distill, "mbok_distill", dev, stream, *args,
            _vector(loss, "loss", dev, T, torch.float32),
            None if stats is None else _vector(stats, "stats", dev, T * MBOK_DISTILL_STATS,
                                               torch.float32), *grad)


def mbok_distill_backward(d: mbok_distill_desc, Z: torch.Tensor, t_logits: torch.Tensor,
                          t_index: torch.Tensor, stats: torch.Tensor, dloss: torch.Tensor,
                          dZ: torch.Tensor, t_lse: torch.Tensor | None = None,
                          weight: torch.Tensor | None = None, stream=None) -> None:
    """dZ (dtype of Z or bf16; may be Z) = dloss[t] * d loss[t] / d Z[t, :] after
    mbok_distill with stats on the same inputs; dloss fp32 [T]."""
    dev = _first(Z, "Z")
    _first(t_logits, "t_logits")
    T, vocab, args = _distill_args(d, dev, Z, t_logits, t_index, t_lse, weight)
    _launch(load_library().mbok_distill_backward, "mbok_distill_backward", dev, stream, *args,
            _vector(stats, "stats", dev, T * MBOK_DISTILL_STATS, torch.float32),
            _vector(dloss, "dloss", dev, T, torch.float32),
            *_distill_grad(dZ, dev, T, vocab, Z.dtype))


# ------------------------------------------------------- the layer with its epilogue

def mbok_linear(d: mbok_desc, packed: torch.Tensor, X: torch.Tensor, Y: torch.Tensor,
                bias: torch.Tensor | None = None, act: int = MBOK_ACT_NONE,
                residual: torch.Tensor | None = None, pre: torch.Tensor | None = None,
                stream=None) -> None:
    """Y[T, m] (bf16 or fp32, overwritten) = residual + act(X W_hat^T + bias) for X
    bf16 [T, n]; bias [m] fp32, fp16 or bf16; residual of Y's dtype, and may be Y.
    pre bf16 [T, m] receives the pre-activations for mbok_linear_backward."""
    _linear_call("mbok_linear", d, packed, X, Y, bias, act, residual, pre, stream)


def mbok_linear_precise(d: mbok_desc, packed: torch.Tensor, X: torch.Tensor, Y: torch.Tensor,
                        bias: torch.Tensor | None = None, act: int = MBOK_ACT_NONE,
                        residual: torch.Tensor | None = None, pre: torch.Tensor | None = None,
                        stream=None) -> None:
    """mbok_linear with each weight carried as two bf16 terms for T > 16 (twice the
    matrix work)."""
    _linear_call("mbok_linear_precise", d, packed, X, Y, bias, act, residual, pre, stream)


def _linear_call(name: str, d: mbok_desc, packed, X, Y, bias, act, residual, pre, stream) -> None:
    dev = _first(X, "X")
    m, n = d.m, d.n
    T = X.shape[0]
    ldx = _matrix(X, "X", dev, T, n, torch.bfloat16)
    if not isinstance(Y, torch.Tensor):
        raise TypeError("Y must be a torch.Tensor")
    yt = Y.dtype
    if yt != torch.bfloat16 and yt != torch.float32:
        raise ValueError(f"Y must be bfloat16 or float32, got {yt}")
    ldy = _matrix(Y, "Y", dev, T, m, yt)
    b_ptr, bt, r_ptr, ldr, p_ptr, ldpre = None, MBOK_F32, None, 0, None, 0
    if bias is not None:
        if not isinstance(bias, torch.Tensor):
            raise TypeError("bias must be a torch.Tensor")
        bt = _FLOATS.get(bias.dtype)
        if bt is None:
            raise ValueError(f"bias must be float32, float16 or bfloat16, got {bias.dtype}")
        b_ptr = _vector(bias, "bias", dev, m, bias.dtype)
    if residual is not None:
        ldr = _matrix(residual, "residual", dev, T, m, yt)
        r_ptr = residual.data_ptr()
    if pre is not None:
        ldpre = _matrix(pre, "pre", dev, T, m, torch.bfloat16)
        p_ptr = pre.data_ptr()
    _launch(getattr(load_library(), name), name, dev, stream, ctypes.byref(d),
            _packed(packed, dev, m, n, d.K, d.alpha_dtype), X.data_ptr(), MBOK_BF16, T, ldx,
            b_ptr, bt, act, r_ptr, ldr, Y.data_ptr(), _FLOATS[yt], ldy, p_ptr, ldpre)


def mbok_linear_backward_workspace_bytes(d: mbok_desc, T: int) -> int:
    return int(load_library().mbok_linear_backward_workspace_bytes(ctypes.byref(d), T))


def mbok_linear_backward(d: mbok_desc, packed: torch.Tensor, dY: torch.Tensor,
                         pre: torch.Tensor | None = None, dpre: torch.Tensor | None = None,
                         dbias: torch.Tensor | None = None, dX: torch.Tensor | None = None,
                         act: int = MBOK_ACT_NONE, accumulate: bool = False,
                         workspace: torch.Tensor | None | bool = True, stream=None) -> None:
    """Gradients of mbok_linear from dY bf16 [T, m]: dpre bf16 [T, m] (with an
    activation; from pre, and may be pre or dY), dbias fp32 [m] (accumulate: added
    to) and dX bf16 [T, n], each where asked for.  The residual's is dY.

    workspace: as for mbok_gemmt."""
    _linear_backward_call("mbok_linear_backward", d, packed, dY, pre, dpre, dbias, dX, act,
                          accumulate, workspace, stream)


def mbok_linear_backward_precise(d: mbok_desc, packed: torch.Tensor, dY: torch.Tensor,
                                 pre: torch.Tensor | None = None,
                                 dpre: torch.Tensor | None = None,
                                 dbias: torch.Tensor | None = None,
                                 dX: torch.Tensor | None = None, act: int = MBOK_ACT_NONE,
                                 accumulate: bool = False,
                                 workspace: torch.Tensor | None | bool = True,
                                 stream=None) -> None:
    """mbok_linear_backward with dX as mbok_gemmt_precise computes it (of the same bf16
    dpre)."""
    _linear_backward_call("mbok_linear_backward_precise", d, packed, dY, pre, dpre, dbias, dX,
                          act, accumulate, workspace, stream)


def _linear_backward_call(name: str, d: mbok_desc, packed, dY, pre, dpre, dbias, dX, act,
                          accumulate, workspace, stream) -> None:
    dev = _first(dY, "dY")
    m, n, K, at = d.m, d.n, d.K, d.alpha_dtype
    T = dY.shape[0]
    lddy = _matrix(dY, "dY", dev, T, m, torch.bfloat16)
    ptrs, lds = [None, None, None], [0, 0, 0]
    for i, (t, what, cols) in enumerate(((pre, "pre", m), (dpre, "dpre", m), (dX, "dX", n))):
        if t is not None:
            lds[i] = _matrix(t, what, dev, T, cols, torch.bfloat16)
            ptrs[i] = t.data_ptr()
    b_ptr = None if dbias is None else _vector(dbias, "dbias", dev, m, torch.float32)
    with _slices("mbok_linear_backward_workspace_bytes", m, n, K, at, T, workspace, dev,
                 stream) as ws:
        _launch(getattr(load_library(), name), name, dev, stream, ctypes.byref(d),
                _packed(packed, dev, m, n, K, at), ptrs[0], lds[0], dY.data_ptr(), lddy, T, act,
                ptrs[1], lds[1], b_ptr, int(bool(accumulate)), ptrs[2], lds[2],
                None if ws is None else ws.data_ptr())


# -------------------------------------- log-probabilities, policy and preference losses

def mbok_logp_desc_init(vocab: int, temperature: float = 1.0) -> mbok_logp_desc:
    d = mbok_logp_desc()
    _check(load_library().mbok_logp_desc_init(ctypes.byref(d), vocab, temperature),
           "mbok_logp_desc_init")
    return d


def _rows(Z, label, vocab):
    """(device, rows, the arguments the calls on rows of logits begin with), checked."""
    dev = _first(Z, "Z")
    T, zt = Z.shape[0], _FLOATS.get(Z.dtype)
    if zt is None:
        raise ValueError("Z must be float32, float16 or bfloat16")
    ldz = _matrix(Z, "Z", dev, T, vocab, Z.dtype)
    return dev, T, (Z.data_ptr(), zt, T, ldz, _vector(label, "label", dev, T, torch.int32))


def _optional(t, name: str, dev: int, count: int):
    return None if t is None else _vector(t, name, dev, count, torch.float32)


def mbok_logp(d: mbok_logp_desc, Z: torch.Tensor, label: torch.Tensor, logp: torch.Tensor,
              stats: torch.Tensor | None = None, stream=None) -> None:
    """logp[T] (fp32, overwritten): log-probability of each row's token label[T]
    (int32; negative: none, logp 0) under softmax(Z / tau).  stats fp32 [T,
    MBOK_LOGP_STATS] is what mbok_logp_backward takes."""
    dev, T, args = _rows(Z, label, d.vocab)
    _launch(load_library().mbok_logp, "mbok_logp", dev, stream, ctypes.byref(d), *args,
            _vector(logp, "logp", dev, T, torch.float32),
            _optional(stats, "stats", dev, T * MBOK_LOGP_STATS))


def mbok_logp_backward(d: mbok_logp_desc, Z: torch.Tensor, label: torch.Tensor,
                       stats: torch.Tensor, dlogp: torch.Tensor, dZ: torch.Tensor,
                       stream=None) -> None:
    """dZ (dtype of Z or bf16; may be Z) = the gradient of sum(dlogp * logp) after
    mbok_logp or mbok_policy with stats on the same inputs; dlogp fp32 [T]."""
    vocab = d.vocab
    dev, T, args = _rows(Z, label, vocab)
    _launch(load_library().mbok_logp_backward, "mbok_logp_backward", dev, stream,
            ctypes.byref(d), *args, _vector(stats, "stats", dev, T * MBOK_LOGP_STATS,
                                            torch.float32),
            _vector(dlogp, "dlogp", dev, T, torch.float32),
            *_distill_grad(dZ, dev, T, vocab, Z.dtype))


def mbok_policy_desc_init(vocab: int, temperature: float = 1.0, clip_low: float = 0.2,
                          clip_high: float = 0.2, kl: float = 0.0) -> mbok_policy_desc:
    d = mbok_policy_desc()
    _check(load_library().mbok_policy_desc_init(ctypes.byref(d), vocab, temperature, clip_low,
                                                clip_high, kl), "mbok_policy_desc_init")
    return d


def mbok_policy(d: mbok_policy_desc, Z: torch.Tensor, label: torch.Tensor,
                advantage: torch.Tensor, loss: torch.Tensor,
                old_logp: torch.Tensor | None = None, ref_logp: torch.Tensor | None = None,
                weight: torch.Tensor | None = None, logp: torch.Tensor | None = None,
                stats: torch.Tensor | None = None, dlogp: torch.Tensor | None = None,
                dZ: torch.Tensor | None = None, stream=None) -> None:
    """loss[T] (fp32, overwritten): clipped policy loss with a KL term of each
    row's token, from advantage [T], the log-probabilities old_logp [T] it was
    sampled with (None: the present ones), a reference model's ref_logp [T] (None: no
    KL term) and weight [T].  dZ (dtype of Z or bf16; may be Z) receives the gradient
    of sum(loss) in the same pass; logp, stats and dlogp are as for mbok_logp and
    mbok_logp_backward."""
    vocab = d.vocab
    dev, T, args = _rows(Z, label, vocab)
    grad = (None, args[1], 0) if dZ is None else _distill_grad(dZ, dev, T, vocab, Z.dtype)
    _launch(load_library().mbok_policy, "mbok_policy", dev, stream, ctypes.byref(d), *args,
            _vector(advantage, "advantage", dev, T, torch.float32),
            _optional(old_logp, "old_logp", dev, T), _optional(ref_logp, "ref_logp", dev, T),
            _optional(weight, "weight", dev, T), _vector(loss, "loss", dev, T, torch.float32),
            _optional(logp, "logp", dev, T), _optional(stats, "stats", dev, T * MBOK_LOGP_STATS),
            _optional(dlogp, "dlogp", dev, T), *grad)


def mbok_preference_desc_init(beta: float, smoothing: float = 0.0, margin: float = 0.0,
                              mean: bool = False,
                              vocab: int | None = None) -> mbok_preference_desc:
    """vocab: the logits' V, as mbok_logp's descriptor has it.  Left out, every label of
    0 to MBOK_MAX_VOCAB - 1 counts as a token, a padding id of V or more too, whose row
    mbok_logp gives no log-probability: mbok_preference warns if it is given labels then."""
    d = mbok_preference_desc()
    _check(load_library().mbok_preference_desc_init(
        ctypes.byref(d), beta, smoothing, margin, int(bool(mean)),
        MBOK_MAX_VOCAB if vocab is None else vocab), "mbok_preference_desc_init")
    d.vocab_left_out = vocab is None
    return d


def mbok_preference(d: mbok_preference_desc, offsets: torch.Tensor, logp: torch.Tensor,
                    loss: torch.Tensor, ref_logp: torch.Tensor | None = None,
                    label: torch.Tensor | None = None, weight: torch.Tensor | None = None,
                    dlogp: torch.Tensor | None = None, stream=None) -> None:
    """loss[pairs] (fp32, overwritten) of paired log ratios: sequences 2p (chosen)
    and 2p + 1 (rejected) are rows offsets[s] .. offsets[s + 1] - 1 (int32 [2 pairs +
    1]) of logp [T], less the reference model's ref_logp [T]; rows without a token
    (label negative, or the descriptor's vocab or more) do not count.  dlogp [T] receives the gradient for mbok_logp_backward."""
    dev = _first(logp, "logp")
    T = logp.numel()
    if not isinstance(offsets, torch.Tensor):
        raise TypeError("offsets must be a torch.Tensor")
    if offsets.dim() != 1 or offsets.numel() < 3 or offsets.numel() % 2 == 0:
        raise ValueError("offsets must be [2 pairs + 1]")
    pairs = offsets.numel() // 2
    if label is not None and d.vocab_left_out:
        d.vocab_left_out = False  # once
        warnings.warn("mbok_preference: the descriptor has no vocabulary, so labels of V or more "
                      "count as tokens; pass vocab to mbok_preference_desc_init", stacklevel=2)
    _launch(load_library().mbok_preference, "mbok_preference", dev, stream, ctypes.byref(d),
            _vector(offsets, "offsets", dev, 2 * pairs + 1, torch.int32), pairs,
            _vector(logp, "logp", dev, T, torch.float32),
            _optional(ref_logp, "ref_logp", dev, T),
            None if label is None else _vector(label, "label", dev, T, torch.int32), T,
            _optional(weight, "weight", dev, pairs),
            _vector(loss, "loss", dev, pairs, torch.float32), _optional(dlogp, "dlogp", dev, T))


# ------------------------------------------------------------------ the optimizer step

class mbok_adamw_plan:
    """The tensors of an optimizer step (mbok_adamw_plan_init): the library's plan,
    its table on the device, and the tensors, which it keeps alive.

    The plan may be dropped while a step that it was given to still runs on one of
    torch's streams: the table's memory is not given away before.  On a stream that is
    not torch's (which may end first), or that the call was given as a handle, the step
    has to have run by then."""

    def __init__(self, plan, table: torch.Tensor, tensors: list):
        self._plan, self.table, self.tensors = plan, table, tensors
        self._args = (ctypes.byref(plan), table.data_ptr())
        self.device = table.get_device()
        self._streams = set()  # handles that the table's memory waits for

    def _read_on(self, handle: int, stream) -> None:
        """The table is read on a stream other, perhaps, than the one it is tied to."""
        s = _torch_stream(torch.device("cuda", self.device), stream)
        # a stream of another owner has its handle for an id
        if handle == 0 or s.stream_id != handle:
            self.table.record_stream(s)
            self._streams.add(handle)

    def __repr__(self):
        return f"mbok_adamw_plan({self._plan.tensors} tensors, {self._plan.parts} parts)"


_ADAMW_KEYS = {"param", "grad", "m", "v", "m_scale", "v_scale", "out", "layer", "weight_decay"}


def _adamw_tensor(i: int, t: dict, dev: int) -> _AdamwTensor:
    unknown = set(t) - _ADAMW_KEYS
    missing = {"param", "grad", "m", "v"} - set(t)
    if unknown or missing:
        raise ValueError(f"tensor {i}: unknown {sorted(unknown)}, missing {sorted(missing)}")

    def flat(name, dtype, count):
        x = t[name]
        if isinstance(x, torch.Tensor) and x.numel() != count:
            raise ValueError(f"tensor {i}: {name} must have {count} elements, got {x.numel()}")
        return _vector(x, f"tensor {i}: {name}", dev, count, dtype)

    if not isinstance(t["grad"], torch.Tensor) or not isinstance(t["m"], torch.Tensor):
        raise TypeError(f"tensor {i}: grad and m must be torch.Tensors")
    count = t["param"].numel()
    a = _AdamwTensor()
    a.count, a.weight_decay = count, float(t.get("weight_decay", 0.0))
    a.param = flat("param", torch.float32, count)
    gt = _FLOATS.get(t["grad"].dtype)
    if gt is None:
        raise ValueError(f"tensor {i}: grad must be float32, float16 or bfloat16")
    a.grad, a.grad_dtype = flat("grad", t["grad"].dtype, count), gt
    eight = t["m"].dtype == torch.float8_e4m3fn
    st = torch.float8_e4m3fn if eight else torch.float32
    a.m, a.v = flat("m", st, count), flat("v", st, count)
    a.state_dtype = MBOK_E4M3 if eight else MBOK_F32
    scales = [t.get(k) is not None for k in ("m_scale", "v_scale")]
    if scales != [eight, eight]:
        raise ValueError(f"tensor {i}: 8-bit states, and they alone, have m_scale and v_scale")
    if eight:
        blocks = (count + MBOK_ADAMW_BLOCK - 1) // MBOK_ADAMW_BLOCK
        a.m_scale = flat("m_scale", torch.float32, blocks)
        a.v_scale = flat("v_scale", torch.float32, blocks)
    layer, out = t.get("layer"), t.get("out")
    if layer is not None:
        if out is None:
            raise ValueError(f"tensor {i}: a layer's scales need its packed buffer as out")
        a.layer = ctypes.addressof(layer)
        a.out = _packed(out, dev, layer.m, layer.n, layer.K, layer.alpha_dtype)
    elif out is not None:
        if not isinstance(out, torch.Tensor):
            raise TypeError(f"tensor {i}: out must be a torch.Tensor")
        ot = _FLOATS.get(out.dtype)
        if ot is None:
            raise ValueError(f"tensor {i}: out must be float32, float16 or bfloat16")
        a.out, a.out_dtype = flat("out", out.dtype, count), ot
    return a


def mbok_adamw_plan_init(tensors) -> mbok_adamw_plan:
    """The plan of a step over many tensors.  Each is a dict of contiguous tensors:
    param (fp32), grad (fp32, fp16 or bf16), m and v (both fp32, or both
    float8_e4m3fn with fp32 m_scale and v_scale of one value per MBOK_ADAMW_BLOCK;
    8-bit v holds the second moment's root), optionally out (a copy in fp32, fp16 or
    bf16; with layer, a mbok_desc, the layer's packed buffer, whose scales the step
    writes from param [K, m, n/128]) and weight_decay.  The plan holds their
    addresses: gradients are expected in the same tensors at every step, and a graph
    that captured a step needs the plan as long as it is replayed (after eager steps it
    may be dropped, see mbok_adamw_plan)."""
    tensors = [dict(t) for t in tensors]
    if not tensors:
        raise ValueError("a plan needs at least one tensor")
    if "param" not in tensors[0]:
        raise ValueError("tensor 0: missing ['param']")
    dev = _first(tensors[0]["param"], "tensor 0: param")
    for i, t in enumerate(tensors):
        if not isinstance(t.get("param"), torch.Tensor):
            raise TypeError(f"tensor {i}: param must be a torch.Tensor")
    items = (_AdamwTensor * len(tensors))(*(_adamw_tensor(i, t, dev)
                                            for i, t in enumerate(tensors)))
    lib, plan = load_library(), _AdamwPlan()
    host = torch.zeros(max(16, lib.mbok_adamw_table_bytes(items, len(tensors))),
                       dtype=torch.uint8)
    _check(lib.mbok_adamw_plan_init(ctypes.byref(plan), items, len(tensors), host.data_ptr()),
           "mbok_adamw_plan_init")
    return mbok_adamw_plan(plan, host.to(torch.device("cuda", dev)), tensors)


def mbok_adamw(plan: mbok_adamw_plan, lr: float, step: int, beta1: float = 0.9,
               beta2: float = 0.999, eps: float = 1e-8, grad_scale: float = 1.0, seed: int = 0,
               live: torch.Tensor | None = None, stream=None) -> None:
    """One AdamW step on every tensor of the plan, in one launch; step counts from
    1.  Gradients are multiplied by grad_scale.  live fp32 [4] on the device (lr,
    grad_scale, step, skip) is read in place of those arguments when the step runs,
    for steps captured into a graph; a step below 1 there is skipped."""
    if not isinstance(plan, mbok_adamw_plan):
        raise TypeError("plan must be mbok_adamw_plan_init's")
    dev = plan.device
    ptr = None if live is None else _vector(live, "live", dev, 4, torch.float32)
    s = _AdamwStep(lr, beta1, beta2, eps, step, grad_scale, seed & 0xffffffff)
    handle = _raw_stream(dev) if stream is None else _stream(stream)
    if handle not in plan._streams and (handle == 0 or not isinstance(stream, int)):
        plan._read_on(handle, stream)
    _launch(load_library().mbok_adamw, "mbok_adamw", dev, handle, *plan._args, ctypes.byref(s),
            ptr)


# ---------------------------------------------------------------- conveniences

def quantize_and_pack(W: torch.Tensor, K: int, alpha_dtype: int = MBOK_F16, stream=None):
    """Greedy residual binarization of a device fp32 W, then packing.

    Returns (desc, packed, signs, alpha); every step runs in the library."""
    m, n = W.shape
    d = mbok_desc_init(m, n, K, alpha_dtype)
    signs = torch.empty((K, m, n), dtype=torch.int8, device=W.device)
    alpha = torch.empty((K, m, n // MBOK_GROUP), dtype=alpha_torch_dtype(alpha_dtype),
                        device=W.device)
    flag = torch.zeros(1, dtype=torch.int32, device=W.device)
    mbok_residual_binarize(d, W, signs, alpha, flag, stream)
    packed = torch.empty(mbok_packed_bytes(d), dtype=torch.uint8, device=W.device)
    mbok_pack(d, signs, alpha, packed, stream)
    if int(flag.item()) != 0:
        raise ValueError("W holds NaN or Inf")
    return d, packed, signs, alpha


def allocate_for_budget(weights, avg_kernels: float, kmax: int = MBOK_MAX_K,
                        alpha_dtype: int = MBOK_F16, stream=None):
    """Kernels per weight for a set of device fp32 weights under an average
    budget of `avg_kernels` kernels per entry: the residual energies of each
    weight's greedy chain (mbok_residual_energy, K = 1..kmax) feed
    mbok_allocate_kernels with budget floor(avg_kernels * total entries).
    Returns (K list, layer energies [L][kmax + 1] as nested lists)."""
    errors, sizes, energies = [], [], []
    for W in weights:
        m, n = W.shape
        d = mbok_desc_init(m, n, kmax, alpha_dtype)
        rows = torch.empty((kmax + 1, m), dtype=torch.float64, device=W.device)
        layer = torch.empty(kmax + 1, dtype=torch.float64, device=W.device)
        mbok_residual_energy(d, W, rows, layer, stream)
        e = layer.cpu().tolist()
        energies.append(e)
        errors.append(e[1:])
        sizes.append(m * n)
    budget = int(avg_kernels * sum(sizes))
    return mbok_allocate_kernels(sizes, errors, budget), energies
