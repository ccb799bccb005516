"""Thin ctypes binding of libkda.so (the C ABI in ``include/kda.h``).

The functions carry the C entry points' names and do argument marshalling
only: shapes are read off the tensors, outputs and the workspace are
allocated with PyTorch when the caller does not pass them, and the call goes
to the library on the current CUDA stream.  Every step of the computation runs
in the library's CUDA kernels; there is no Python or CPU fallback, and a
missing or unloadable library raises.
"""
from __future__ import annotations

import ctypes
import functools
import os

from . import build as _build

KDA_OK = 0
KDA_ERR_ARG = -1
KDA_ERR_SHAPE = -2
KDA_ERR_DTYPE = -3
KDA_ERR_ALIGN = -4
KDA_ERR_UNSUPPORTED = -5
KDA_ERR_CUDA = -6
KDA_ERR_TIMEOUT = -7
KDA_ERR_WORKSPACE = -8

KDA_F32 = 0
KDA_BF16 = 1

IMPLS = {"auto": 0, "simt": 1, "tc": 2}
# KDA_DECAY_*: log_alpha [T, H, d_k] per key channel (KDA), [T, H] per head
# (Gated DeltaNet), or none (DeltaNet, log_alpha may be None)
DECAY_MODES = {"channel": 0, "head": 1, "none": 2}


class kda_options(ctypes.Structure):
    """Mirror of ``struct kda_options`` (field order and types as in kda.h)."""
    _fields_ = [
        ("chunk", ctypes.c_int),
        ("l2norm_qk", ctypes.c_int),
        ("beta_is_logit", ctypes.c_int),
        ("g_min", ctypes.c_float),
        ("q_scale", ctypes.c_float),
        ("eps_l2", ctypes.c_float),
        ("eps_norm", ctypes.c_float),
        ("gate", ctypes.c_void_p),
        ("norm_weight", ctypes.c_void_p),
        ("workspace", ctypes.c_void_p),
        ("workspace_bytes", ctypes.c_size_t),
        ("max_seqlen", ctypes.c_int),
        ("impl", ctypes.c_int),
        ("debug_timeout", ctypes.c_int),
        ("timeout_spins", ctypes.c_longlong),
        ("phase_events", ctypes.c_void_p),
        ("decay_mode", ctypes.c_int),
        ("snapshot_every", ctypes.c_int),
        ("snapshots", ctypes.c_void_p),
        ("decay_from_logit", ctypes.c_int),
        ("decay_scale", ctypes.c_void_p),
        ("decay_bias", ctypes.c_void_p),
        ("conv_weight", ctypes.c_void_p),
        ("conv_state", ctypes.c_void_p),
    ]


class kda_gdr_options(ctypes.Structure):
    """Mirror of ``struct kda_gdr_options`` (field order and types as in kda.h)."""
    _fields_ = [
        ("l2norm_qk", ctypes.c_int),
        ("beta_is_logit", ctypes.c_int),
        ("decay_from_logit", ctypes.c_int),
        ("decay_scale", ctypes.c_void_p),
        ("decay_bias", ctypes.c_void_p),
        ("q_scale", ctypes.c_float),
        ("eps_l2", ctypes.c_float),
        ("ldq", ctypes.c_longlong),
        ("ldk", ctypes.c_longlong),
        ("ldv", ctypes.c_longlong),
        ("slots", ctypes.c_void_p),
        ("n_slots", ctypes.c_int),
        ("snapshots", ctypes.c_void_p),
        ("max_seqlen", ctypes.c_int),
        ("impl", ctypes.c_int),
        ("workspace", ctypes.c_void_p),
        ("workspace_bytes", ctypes.c_size_t),
    ]


class kda_glr_options(ctypes.Structure):
    """Mirror of ``struct kda_glr_options`` (field order and types as in kda.h)."""
    _fields_ = [
        ("decay_from", ctypes.c_int),
        ("decay_scale", ctypes.c_void_p),
        ("decay_bias", ctypes.c_void_p),
        ("input_scale", ctypes.c_int),
        ("input_gate", ctypes.c_void_p),
        ("ldx", ctypes.c_longlong),
        ("ldla", ctypes.c_longlong),
        ("ldg", ctypes.c_longlong),
        ("slots", ctypes.c_void_p),
        ("n_slots", ctypes.c_int),
        ("checkpoints", ctypes.c_void_p),
        ("max_seqlen", ctypes.c_int),
        ("workspace", ctypes.c_void_p),
        ("workspace_bytes", ctypes.c_size_t),
    ]


class KdaError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        super().__init__(f"{where}: {kda_status_string(status)} ({status})")


_LIB = None
EXPORTS = ("kda_options_init", "kda_prefill", "kda_prefill_noalloc",
           "kda_prefill_workspace_size", "kda_prefill_path",
           "kda_decode_step", "kda_gated_rmsnorm", "kda_get_last_error", "kda_status_string",
           "kda_abi_version", "kda_gdr_options_init", "kda_gdr_prefill",
           "kda_gdr_prefill_workspace_size", "kda_gdr_prefill_path", "kda_gdr_decode_step",
           "kda_linear", "kda_rmsnorm", "kda_quantize_i8", "kda_linear_i8",
           "kda_linear_i8_workspace_size", "kda_glr_options_init", "kda_glr_scan", "kda_glr_step",
           "kda_glr_scan_backward", "kda_glr_backward_workspace_size")
PATH_NAMES = {1: "simt", 2: "tc"}


def lib_path() -> str:
    return _build.LIB


def load(path: str | None = None):
    """Load libkda.so (building it first if it is missing or stale)."""
    global _LIB
    if _LIB is not None and path is None:
        return _LIB
    if path is None:
        path = _build.build()
    lib = ctypes.CDLL(path)
    vp, ci, cf = ctypes.c_void_p, ctypes.c_int, ctypes.c_float
    po = ctypes.POINTER(kda_options)
    lib.kda_options_init.argtypes = [po]
    lib.kda_options_init.restype = None
    lib.kda_prefill.argtypes = [vp, vp, vp, vp, vp, vp, vp, ci, vp, vp, ci, ci, ci, ci, ci, po, vp]
    lib.kda_prefill.restype = ci
    lib.kda_prefill_workspace_size.argtypes = [ci, ci, ci, ci, ci, po]
    lib.kda_prefill_workspace_size.restype = ctypes.c_size_t
    pi = ctypes.POINTER(ctypes.c_int)
    lib.kda_prefill_path.argtypes = [ci, ci, ci, ci, ci, ci, po, pi, pi]
    lib.kda_prefill_path.restype = ci
    lib.kda_decode_step.argtypes = [vp, vp, vp, vp, vp, vp, vp, ci, ci, ci, ci, ci, po, vp]
    lib.kda_decode_step.restype = ci
    lib.kda_gated_rmsnorm.argtypes = [vp, vp, vp, vp, ci, ci, ci, cf, ci, vp]
    lib.kda_gated_rmsnorm.restype = ci
    lib.kda_get_last_error.argtypes = [vp]
    lib.kda_get_last_error.restype = ci
    lib.kda_status_string.argtypes = [ci]
    lib.kda_status_string.restype = ctypes.c_char_p
    lib.kda_abi_version.restype = ci
    lib.kda_prefill_noalloc.argtypes = lib.kda_prefill.argtypes
    lib.kda_prefill_noalloc.restype = ci
    pg, cl = ctypes.POINTER(kda_gdr_options), ctypes.c_longlong
    lib.kda_gdr_options_init.argtypes = [pg]
    lib.kda_gdr_options_init.restype = None
    lib.kda_gdr_prefill.argtypes = [vp, vp, vp, vp, vp, vp, vp, ci, vp, vp, ci, ci, ci, ci, ci,
                                    ci, pg, vp]
    lib.kda_gdr_prefill.restype = ci
    lib.kda_gdr_prefill_workspace_size.argtypes = [ci, ci, ci, ci, ci, ci, ci, pg]
    lib.kda_gdr_prefill_workspace_size.restype = ctypes.c_size_t
    lib.kda_gdr_prefill_path.argtypes = [ci, ci, ci, ci, ci, ci, ci, pg]
    lib.kda_gdr_prefill_path.restype = ci
    lib.kda_gdr_decode_step.argtypes = [vp, vp, vp, vp, vp, vp, vp, ci, ci, ci, ci, ci, ci, ci,
                                        pg, vp]
    lib.kda_gdr_decode_step.restype = ci
    lib.kda_linear.argtypes = [vp, cl, vp, cl, vp, vp, cl, vp, cl, ci, ci, ci, ci, ci, vp]
    lib.kda_linear.restype = ci
    lib.kda_rmsnorm.argtypes = [vp, cl, vp, cl, vp, vp, cl, vp, cl, vp, cl, vp, ci, ci, cf, ci, vp]
    lib.kda_rmsnorm.restype = ci
    lib.kda_quantize_i8.argtypes = [vp, cl, vp, cl, vp, ci, ci, ci, vp]
    lib.kda_quantize_i8.restype = ci
    cz = ctypes.c_size_t
    lib.kda_linear_i8.argtypes = [vp, cl, vp, vp, cl, vp, vp, vp, cl, vp, cl, ci, ci, ci, ci, ci,
                                  vp, cz, vp]
    lib.kda_linear_i8.restype = ci
    lib.kda_linear_i8_workspace_size.argtypes = [ci, ci, ci]
    lib.kda_linear_i8_workspace_size.restype = cz
    pl = ctypes.POINTER(kda_glr_options)
    lib.kda_glr_options_init.argtypes = [pl]
    lib.kda_glr_options_init.restype = None
    lib.kda_glr_scan.argtypes = [vp, vp, vp, vp, ci, vp, vp, ci, ci, ci, pl, vp]
    lib.kda_glr_scan.restype = ci
    lib.kda_glr_step.argtypes = [vp, vp, vp, vp, ci, ci, ci, ci, pl, vp]
    lib.kda_glr_step.restype = ci
    lib.kda_glr_scan_backward.argtypes = [vp, vp, vp, vp, vp, ci, vp, vp, vp, vp, vp, vp, ci, ci,
                                          ci, pl, vp]
    lib.kda_glr_scan_backward.restype = ci
    lib.kda_glr_backward_workspace_size.argtypes = [ci, ci, ci, ci, pl]
    lib.kda_glr_backward_workspace_size.restype = cz
    if path == _build.LIB or _LIB is None:
        _LIB = lib
    return lib


def kda_status_string(status: int) -> str:
    return load().kda_status_string(int(status)).decode()


def kda_abi_version() -> int:
    return load().kda_abi_version()


def kda_options_init(**overrides) -> kda_options:
    """Default options (C kda_options_init), then keyword overrides."""
    opt = kda_options()
    load().kda_options_init(ctypes.byref(opt))
    for key, val in overrides.items():
        if key == "impl" and isinstance(val, str):
            val = IMPLS[val]
        if key == "decay_mode" and isinstance(val, str):
            val = DECAY_MODES[val]
        setattr(opt, key, val)
    return opt


# ---------------------------------------------------------------- marshalling
def _ptr(x) -> int | None:
    if x is None:
        return None
    if isinstance(x, int):
        return x
    return x.data_ptr()


def _dtype_code(t) -> int:
    import torch
    if t.dtype == torch.bfloat16:
        return KDA_BF16
    if t.dtype == torch.float32:
        return KDA_F32
    raise TypeError(f"unsupported dtype {t.dtype}: use bfloat16 or float32")


def _stream(stream) -> int | None:
    import torch
    if stream is None:
        return torch.cuda.current_stream().cuda_stream
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


def _check_cuda(*ts):
    for t in ts:
        if t is None:
            continue
        if not t.is_cuda:
            raise ValueError("libkda takes CUDA tensors (device memory)")
        if not t.is_contiguous():
            raise ValueError("libkda takes contiguous tensors")


def _opts(gate, norm_weight, chunk, l2norm_qk, beta_is_logit, g_min, q_scale, eps_l2,
          eps_norm, workspace, workspace_bytes, max_seqlen, impl, debug_timeout,
          timeout_spins, decay_mode="channel", decay_from_logit=False, decay_scale=None,
          decay_bias=None, conv_weight=None, conv_state=None) -> kda_options:
    _check_cuda(decay_scale, decay_bias, conv_weight, conv_state)
    return kda_options_init(
        decay_mode=decay_mode,
        chunk=int(chunk), l2norm_qk=int(bool(l2norm_qk)), beta_is_logit=int(bool(beta_is_logit)),
        g_min=float(g_min), q_scale=float(q_scale), eps_l2=float(eps_l2),
        eps_norm=float(eps_norm), gate=_ptr(gate), norm_weight=_ptr(norm_weight),
        workspace=_ptr(workspace), workspace_bytes=int(workspace_bytes),
        max_seqlen=int(max_seqlen), impl=impl, debug_timeout=int(bool(debug_timeout)),
        timeout_spins=int(timeout_spins), decay_from_logit=int(bool(decay_from_logit)),
        decay_scale=_ptr(decay_scale), decay_bias=_ptr(decay_bias),
        conv_weight=_ptr(conv_weight), conv_state=_ptr(conv_state))


def kda_prefill_workspace_size(T_total: int, N: int, H: int, d_k: int, d_v: int,
                               opt: kda_options | None = None) -> int:
    o = opt if opt is not None else kda_options_init()
    return int(load().kda_prefill_workspace_size(T_total, N, H, d_k, d_v, ctypes.byref(o)))


def kda_prefill_path(T_total: int, N: int, H: int, d_k: int, d_v: int, dtype: int = KDA_BF16,
                     opt: kda_options | None = None) -> tuple[str, int, int]:
    """(path name, kernels per call, chunk) that kda_prefill uses for these sizes."""
    o = opt if opt is not None else kda_options_init()
    launches, chunk = ctypes.c_int(0), ctypes.c_int(0)
    rc = load().kda_prefill_path(T_total, N, H, d_k, d_v, dtype, ctypes.byref(o),
                                 ctypes.byref(launches), ctypes.byref(chunk))
    if rc < 0:
        raise KdaError(rc, "kda_prefill_path")
    return PATH_NAMES[rc], launches.value, chunk.value


def kda_prefill(q, k, v, log_alpha, beta, S0=None, cu_seqlens=None, N: int | None = None,
                o=None, S_T=None, *, gate=None, norm_weight=None, chunk: int = 0,
                l2norm_qk: bool = True, beta_is_logit: bool = False, g_min: float = -5.0,
                q_scale: float = 1.0, eps_l2: float = 1e-6, eps_norm: float = 1e-6,
                workspace=None, max_seqlen: int = 0, impl="auto", debug_timeout: bool = False,
                timeout_spins: int = 0, phase_events=None, decay_mode="channel",
                snapshot_every: int = 0, snapshots=None, decay_from_logit: bool = False,
                decay_scale=None, decay_bias=None, conv_weight=None, conv_state=None,
                stream=None):
    """Chunked prefill (C ``kda_prefill``).

    q, k, log_alpha [T, H, d_k]; v [T, H, d_v]; beta [T, H]; S0 [N, H, d_k, d_v]
    fp32 or None; cu_seqlens [N+1] int32 (device) or None.  Returns (o, S_T);
    o holds y = RMSNorm(o) * w * sigmoid(gate) when ``gate`` is given.
    ``decay_mode`` "head" takes log_alpha [T, H]; "none" ignores it (None is fine).
    With ``snapshot_every`` (a multiple of 64) it returns (o, S_T, snapshots),
    snapshots [N, L // snapshot_every, H, d_k, d_v] fp32 with L = max_seqlen
    (T // N without cu_seqlens, T with them): slot m holds the state after
    (m + 1) * snapshot_every tokens of the sequence (zeros, or the given
    buffer's contents, past its length).
    The prologue from raw projections: ``decay_from_logit`` takes log_alpha as
    decay logits z and forms g_min * sigmoid(A_h (z + b)) with ``decay_scale``
    A [H] and ``decay_bias`` b [H, d_k] (fp32, None = ones / zeros);
    ``conv_weight`` [3, H, d, 4] fp32 runs q, k, v through the width-4 causal
    short convolution + Swish first, ``conv_state`` [N, 3, 3, H, d] (dtype of
    q) holding the raw rows before each sequence (None = zeros).
    """
    import torch
    _check_cuda(q, k, v, log_alpha, beta, S0, cu_seqlens, gate, norm_weight, o, S_T)
    T, H, d_k = q.shape
    d_v = v.shape[2]
    if cu_seqlens is not None:
        N = cu_seqlens.numel() - 1
    N = N or 1
    dt = _dtype_code(q)
    if o is None:
        o = torch.empty((T, H, d_v), dtype=q.dtype, device=q.device)
    if S_T is None:
        S_T = torch.empty((N, H, d_k, d_v), dtype=torch.float32, device=q.device)
    impl_code = IMPLS[impl] if isinstance(impl, str) else int(impl)
    opt = _opts(gate, norm_weight, chunk, l2norm_qk, beta_is_logit, g_min, q_scale, eps_l2,
                eps_norm, None, 0, max_seqlen, impl_code, debug_timeout, timeout_spins,
                decay_mode, decay_from_logit, decay_scale, decay_bias, conv_weight, conv_state)
    if phase_events is not None:  # list of torch.cuda.Event, (launches + 1) of them
        if any(not e.cuda_event for e in phase_events):
            raise ValueError("phase_events: record each event once first (torch creates "
                             "the CUDA event lazily)")
        ev_arr = (ctypes.c_void_p * len(phase_events))(*[e.cuda_event for e in phase_events])
        opt.phase_events = ctypes.cast(ev_arr, ctypes.c_void_p)
    if snapshot_every:
        L = max_seqlen if max_seqlen > 0 else (T if cu_seqlens is not None else T // N)
        if snapshots is None:
            snapshots = torch.zeros((N, L // snapshot_every, H, d_k, d_v), dtype=torch.float32,
                                    device=q.device)
        _check_cuda(snapshots)
        opt.snapshot_every = int(snapshot_every)
        opt.snapshots = _ptr(snapshots)
    need = kda_prefill_workspace_size(T, N, H, d_k, d_v, opt)
    if need > 0:
        if workspace is None:
            workspace = torch.empty(need, dtype=torch.uint8, device=q.device)
        opt.workspace = _ptr(workspace)
        opt.workspace_bytes = workspace.numel() * workspace.element_size()
    rc = load().kda_prefill(_ptr(q), _ptr(k), _ptr(v), _ptr(log_alpha), _ptr(beta), _ptr(S0),
                            _ptr(cu_seqlens), N, _ptr(o), _ptr(S_T), T, H, d_k, d_v, dt,
                            ctypes.byref(opt), _stream(stream))
    if rc != KDA_OK:
        raise KdaError(rc, "kda_prefill")
    if snapshot_every:
        return o, S_T, snapshots
    return o, S_T


_DECODE_OPTS: dict = {}


def kda_decode_step(q, k, v, log_alpha, beta, S, o=None, *, gate=None, norm_weight=None,
                    l2norm_qk: bool = True, beta_is_logit: bool = False, g_min: float = -5.0,
                    q_scale: float = 1.0, eps_l2: float = 1e-6, eps_norm: float = 1e-6,
                    decay_mode="channel", decay_from_logit: bool = False, decay_scale=None,
                    decay_bias=None, conv_weight=None, conv_state=None, stream=None):
    """One decode step (C ``kda_decode_step``); S [N, H, d_k, d_v] is updated in place.
    Returns o [N, H, d_v].  log_alpha is [N, H] with decay_mode "head".  With
    ``conv_weight``, ``conv_state`` [N, 3, 3, H, d] (the raw q, k, v rows of the
    3 previous tokens) is read and moved on by this token in place."""
    import torch
    _check_cuda(q, k, v, log_alpha, beta, S, o, gate, norm_weight)
    N, H, d_k = q.shape
    d_v = v.shape[2]
    if o is None:
        o = torch.empty((N, H, d_v), dtype=q.dtype, device=q.device)
    # a decode loop calls this once per token: the options struct is built once
    # per distinct setting
    key = (_ptr(gate), _ptr(norm_weight), bool(l2norm_qk), bool(beta_is_logit), float(g_min),
           float(q_scale), float(eps_l2), float(eps_norm), decay_mode, bool(decay_from_logit),
           _ptr(decay_scale), _ptr(decay_bias), _ptr(conv_weight), _ptr(conv_state))
    opt = _DECODE_OPTS.get(key)
    if opt is None:
        opt = _opts(gate, norm_weight, 0, l2norm_qk, beta_is_logit, g_min, q_scale, eps_l2,
                    eps_norm, None, 0, 0, 0, False, 0, decay_mode, decay_from_logit,
                    decay_scale, decay_bias, conv_weight, conv_state)
        if len(_DECODE_OPTS) > 64:
            _DECODE_OPTS.clear()
        _DECODE_OPTS[key] = opt
    rc = load().kda_decode_step(_ptr(q), _ptr(k), _ptr(v), _ptr(log_alpha), _ptr(beta),
                                _ptr(S), _ptr(o), N, H, d_k, d_v, _dtype_code(q),
                                ctypes.byref(opt), _stream(stream))
    if rc != KDA_OK:
        raise KdaError(rc, "kda_decode_step")
    return o


def kda_gated_rmsnorm(o, gate, w=None, y=None, *, eps: float = 1e-6, stream=None):
    """y = o / sqrt(mean(o^2) + eps) * w * sigmoid(gate) per (row, head)
    (C ``kda_gated_rmsnorm``); o, gate [rows, H, d_v]."""
    import torch
    _check_cuda(o, gate, w, y)
    rows, H, d_v = o.shape
    if y is None:
        y = torch.empty_like(o)
    rc = load().kda_gated_rmsnorm(_ptr(o), _ptr(gate), _ptr(w), _ptr(y), rows, H, d_v,
                                  float(eps), _dtype_code(o), _stream(stream))
    if rc != KDA_OK:
        raise KdaError(rc, "kda_gated_rmsnorm")
    return y


def kda_get_last_error(stream=None) -> int:
    """Synchronise the stream and return (and clear) the device status word."""
    return int(load().kda_get_last_error(_stream(stream)))


NOALLOC_SCRATCH_BYTES = 64 << 20


def kda_prefill_noalloc(q, k, v, log_alpha, beta, S0=None, cu_seqlens=None, N: int | None = None,
                        o=None, S_T=None, *, gate=None, norm_weight=None, l2norm_qk: bool = True,
                        beta_is_logit: bool = False, g_min: float = -5.0, q_scale: float = 1.0,
                        eps_l2: float = 1e-6, eps_norm: float = 1e-6, max_seqlen: int = 0,
                        decay_mode="channel", stream=None):
    """Prefill with the library's built-in scratch (C ``kda_prefill_noalloc``).

    For callers that must not allocate device memory: the library allocates
    nothing for this call (pass ``o`` and ``S_T`` to allocate nothing here
    either).  Same arguments and results as :func:`kda_prefill`; sizes whose
    scratch exceeds 64 MiB raise KdaError(KDA_ERR_WORKSPACE)."""
    import torch
    _check_cuda(q, k, v, log_alpha, beta, S0, cu_seqlens, gate, norm_weight, o, S_T)
    T, H, d_k = q.shape
    d_v = v.shape[2]
    if cu_seqlens is not None:
        N = cu_seqlens.numel() - 1
    N = N or 1
    if o is None:
        o = torch.empty((T, H, d_v), dtype=q.dtype, device=q.device)
    if S_T is None:
        S_T = torch.empty((N, H, d_k, d_v), dtype=torch.float32, device=q.device)
    opt = _opts(gate, norm_weight, 64, l2norm_qk, beta_is_logit, g_min, q_scale, eps_l2,
                eps_norm, None, 0, max_seqlen, IMPLS["tc"], False, 0, decay_mode)
    rc = load().kda_prefill_noalloc(_ptr(q), _ptr(k), _ptr(v), _ptr(log_alpha), _ptr(beta),
                                    _ptr(S0), _ptr(cu_seqlens), N, _ptr(o), _ptr(S_T), T, H, d_k,
                                    d_v, _dtype_code(q), ctypes.byref(opt), _stream(stream))
    if rc != KDA_OK:
        raise KdaError(rc, "kda_prefill_noalloc")
    return o, S_T


# ------------------------------------------------- the gated delta rule
def kda_gdr_options_init(**overrides) -> kda_gdr_options:
    """Default options (C kda_gdr_options_init), then keyword overrides."""
    opt = kda_gdr_options()
    load().kda_gdr_options_init(ctypes.byref(opt))
    for key, val in overrides.items():
        if key == "impl" and isinstance(val, str):
            val = IMPLS[val]
        setattr(opt, key, val)
    return opt


class _Host:
    """What every call needs, looked up once: a call's own work on the host is a few
    microseconds, as long as the smallest kernels run."""

    def __init__(self):
        import torch
        lib = load()
        self.linear, self.step, self.prefill = (lib.kda_linear, lib.kda_gdr_decode_step,
                                                lib.kda_gdr_prefill)
        self.rmsnorm, self.quantize_i8 = lib.kda_rmsnorm, lib.kda_quantize_i8
        self.linear_i8, self.linear_i8_size = lib.kda_linear_i8, lib.kda_linear_i8_workspace_size
        self.glr_scan, self.glr_step = lib.kda_glr_scan, lib.kda_glr_step
        self.glr_backward, self.glr_backward_size = (lib.kda_glr_scan_backward,
                                                     lib.kda_glr_backward_workspace_size)
        self.codes = {torch.bfloat16: KDA_BF16, torch.float32: KDA_F32}
        self.f32, self.i32, self.u8, self.i8 = (torch.float32, torch.int32, torch.uint8,
                                                torch.int8)
        self.bf16 = torch.bfloat16
        self.empty, self.empty_like = torch.empty, torch.empty_like
        self.current_device = torch._C._cuda_getDevice
        # (device) -> address of the current stream
        self.current_stream = torch._C._cuda_getCurrentRawStream


_HOST = None


def _host() -> _Host:
    global _HOST
    if _HOST is None:
        _HOST = _Host()
    return _HOST


def _code(host, dtype) -> int:
    code = host.codes.get(dtype)
    if code is None:
        raise TypeError(f"unsupported dtype {dtype}: use bfloat16 or float32")
    return code


def _one_device(host, first, *ts) -> int:
    """The device of `first`, which has to be everyone's and the current one: the
    launch goes to a stream of the current device."""
    dev = first.get_device()
    if dev < 0:
        raise ValueError("libkda takes CUDA tensors (device memory)")
    for t in ts:
        if t is not None and t.get_device() != dev:
            raise ValueError("libkda takes tensors on one device")
    if dev != host.current_device():
        raise ValueError("the tensors are not on the current CUDA device: wrap the call in "
                         "torch.cuda.device(tensor.device)")
    return dev


def _on_stream(call):
    """`call` with ``stream`` (a torch stream or its address, None = the current one) as the
    current stream: what it allocates then belongs to the stream that the kernels run on,
    so that the allocator hands none of it out before they are done."""
    @functools.wraps(call)
    def on_stream(*args, stream=None, **kw):
        if stream is None:
            return call(*args, **kw)
        import torch
        if isinstance(stream, int):
            stream = torch.cuda.ExternalStream(stream) if stream else torch.cuda.default_stream()
        if stream.device.index != torch.cuda.current_device():
            raise ValueError("the stream is not one of the current CUDA device")
        with torch.cuda.stream(stream):
            return call(*args, **kw)
    return on_stream


def _token_stride(x, name: str) -> int:
    """Elements between the rows of successive tokens of x [..., H, d]: heads and
    channels are dense, tokens evenly spaced (so that x may be a slice of a wider
    projection); 0 for dense rows."""
    if x.is_contiguous():
        return 0
    *rows, H, d = x.shape
    st = x.stride()
    if (d > 1 and st[-1] != 1) or (H > 1 and st[-2] != d):
        raise ValueError(f"{name}: each token's heads and channels have to be contiguous")
    if len(rows) == 2 and rows[0] > 1 and rows[1] > 1 and st[0] != rows[1] * st[1]:
        raise ValueError(f"{name}: tokens have to be evenly spaced")
    if max(rows, default=1) < 2:
        return 0
    ld = st[0] if len(rows) == 1 or rows[1] < 2 else st[1]
    if ld < H * d:  # a broadcast token, or tokens that overlap
        raise ValueError(f"{name}: tokens have to lie apart")
    return ld


def _sizes(where: str, *sizes):
    """Sizes as the library takes them, in 32 bits: a larger one would reach it cut off.  (Calls look at
    all of them at once, by their high bits, before they come here: 0.1 us and not 0.5.)"""
    if max(sizes) > 0x7fffffff:
        raise KdaError(KDA_ERR_SHAPE, where)


def _expect(x, name, shape, dtype):
    """x as the library reads it: this shape and type, contiguous."""
    if x.shape != shape:
        raise ValueError(f"{name}: shape {tuple(x.shape)}, expected {shape}")
    if x.dtype != dtype:
        raise TypeError(f"{name}: {x.dtype}, expected {dtype}")
    if not x.is_contiguous():
        raise ValueError(f"{name}: libkda takes contiguous tensors")


def _gdr_call(host, q, k, v, log_alpha, beta, S0, S_T, slots, o, decay_scale, decay_bias, N,
              l2norm_qk, beta_is_logit, decay_from_logit, q_scale, eps_l2):
    """Checks what the two entry points share; returns (o, options, sizes)."""
    shape, values, dtype = q.shape, v.shape, q.dtype
    if k.shape != shape or values[:-2] != shape[:-2]:
        raise ValueError("q and k [..., H_k, d_k] and v [..., H_v, d_v] of the same tokens")
    if k.dtype != dtype or v.dtype != dtype:
        raise TypeError("q, k and v of one dtype")
    Hk, dk = shape[-2:]
    Hv, dv = values[-2:]
    per_head = values[:-1]
    _expect(log_alpha, "log_alpha", per_head, host.f32)
    _expect(beta, "beta", per_head, dtype)
    if o is None:
        o = (host.empty_like(v) if v.is_contiguous()
             else host.empty(values, dtype=dtype, device=q.device))
    else:
        _expect(o, "o", values, dtype)
    n_slots, at = N, None
    if slots is not None:
        _expect(slots, "slots", (N,), host.i32)
        n_slots, at = S_T.shape[0], slots.data_ptr()
    states = (n_slots, Hv, dk, dv)
    _expect(S_T, "state", states, host.f32)
    if S0 is not None and S0 is not S_T:
        _expect(S0, "S0", states, host.f32)
    A = b = None
    if decay_scale is not None:
        _expect(decay_scale, "decay_scale", (Hv,), host.f32)
        A = decay_scale.data_ptr()
    if decay_bias is not None:
        _expect(decay_bias, "decay_bias", (Hv,), host.f32)
        b = decay_bias.data_ptr()
    opt = kda_gdr_options(
        1 if l2norm_qk else 0, 1 if beta_is_logit else 0, 1 if decay_from_logit else 0, A, b,
        q_scale, eps_l2, _token_stride(q, "q"), _token_stride(k, "k"), _token_stride(v, "v"), at,
        n_slots)
    return o, opt, (Hk, Hv, dk, dv)


def kda_gdr_prefill_workspace_size(T_total: int, N: int, H_k: int, H_v: int, d_k: int, d_v: int,
                                   dtype: int = KDA_BF16,
                                   opt: kda_gdr_options | None = None) -> int:
    o = opt if opt is not None else kda_gdr_options_init()
    return int(load().kda_gdr_prefill_workspace_size(T_total, N, H_k, H_v, d_k, d_v, dtype,
                                                     ctypes.byref(o)))


def kda_gdr_prefill_path(T_total: int, N: int, H_k: int, H_v: int, d_k: int, d_v: int,
                         dtype: int = KDA_BF16, opt: kda_gdr_options | None = None) -> str:
    """The implementation kda_gdr_prefill uses for these sizes: "simt" or "tc"."""
    o = opt if opt is not None else kda_gdr_options_init()
    rc = load().kda_gdr_prefill_path(T_total, N, H_k, H_v, d_k, d_v, dtype, ctypes.byref(o))
    if rc < 0:
        raise KdaError(rc, "kda_gdr_prefill_path")
    return PATH_NAMES[rc]


@_on_stream
def kda_gdr_prefill(q, k, v, log_alpha, beta, S0=None, cu_seqlens=None, N: int | None = None,
                    o=None, S_T=None, *, slots=None, l2norm_qk: bool = True,
                    beta_is_logit: bool = False, decay_from_logit: bool = False, decay_scale=None,
                    decay_bias=None, q_scale: float = 1.0, eps_l2: float = 1e-6,
                    max_seqlen: int = 0, impl="auto", workspace=None):
    """The gated delta rule over packed sequences (C ``kda_gdr_prefill``).

    q, k [T, H_k, d_k]; v [T, H_v, d_v]; each token's heads contiguous, tokens any
    even distance apart (slices of one projection).  log_alpha [T, H_v] fp32;
    beta [T, H_v]; S0 [N, H_v, d_k, d_v] fp32 or None (zeros); cu_seqlens [N+1]
    int32 on the device, or None for N sequences of T / N tokens.  ``max_seqlen``:
    the longest sequence, 0 = T (T / N without cu_seqlens); short ones are taken
    token by token, without a workspace.  Returns (o, S_T).  With ``slots`` [N] int32, S0 and S_T are pools
    [n_slots, H_v, d_k, d_v] and sequence n's state is matrix slots[n]; S_T has
    to be given (it may be S0).  ``decay_from_logit``: log_alpha holds logits z,
    the log decay is -A softplus(z + b) with decay_scale A [H_v] and decay_bias
    b [H_v] (fp32, None = ones / zeros).  ``stream``: the stream to run on, None =
    the current one."""
    host = _host()
    dev = _one_device(host, q, k, v, log_alpha, beta, S0, cu_seqlens, o, S_T, slots, decay_scale,
                      decay_bias, workspace)
    if q.dim() != 3 or v.dim() != 3:
        raise ValueError("q, k [T, H_k, d_k] and v [T, H_v, d_v]")
    T = q.shape[0]
    if cu_seqlens is not None:
        N = cu_seqlens.numel() - 1
        _expect(cu_seqlens, "cu_seqlens", (N + 1,), host.i32)
    elif N is None:
        N = 1
    if S_T is None:
        if slots is not None:
            raise ValueError("with slots, S_T is the pool that the states are written to")
        S_T = host.empty((max(N, 0), v.shape[1], q.shape[2], v.shape[2]), dtype=host.f32,
                         device=q.device)
    o, opt, sizes = _gdr_call(host, q, k, v, log_alpha, beta, S0, S_T, slots, o, decay_scale,
                              decay_bias, N, l2norm_qk, beta_is_logit, decay_from_logit, q_scale,
                              eps_l2)
    dt = _code(host, q.dtype)
    if max_seqlen == 0 and cu_seqlens is None and N > 0:
        max_seqlen = T // N  # every length is known
    opt.max_seqlen = max_seqlen
    opt.impl = IMPLS[impl] if isinstance(impl, str) else int(impl)
    if workspace is not None and not workspace.is_contiguous():
        raise ValueError("workspace: libkda takes contiguous tensors")
    need = load().kda_gdr_prefill_workspace_size(T, N, *sizes, dt, opt)
    if need > 0:
        if workspace is None:
            workspace = host.empty(need, dtype=host.u8, device=q.device)
        opt.workspace = workspace.data_ptr()
        opt.workspace_bytes = workspace.numel() * workspace.element_size()
    rc = host.prefill(q.data_ptr(), k.data_ptr(), v.data_ptr(), log_alpha.data_ptr(),
                      beta.data_ptr(), _ptr(S0), _ptr(cu_seqlens), N, o.data_ptr(),
                      S_T.data_ptr(), T, *sizes, dt, opt, host.current_stream(dev))
    if rc != KDA_OK:
        raise KdaError(rc, "kda_gdr_prefill")
    return o, S_T


@_on_stream
def kda_gdr_decode_step(q, k, v, log_alpha, beta, S, o=None, *, slots=None, snapshots=None,
                        l2norm_qk: bool = True, beta_is_logit: bool = False,
                        decay_from_logit: bool = False, decay_scale=None, decay_bias=None,
                        q_scale: float = 1.0, eps_l2: float = 1e-6):
    """L recurrent tokens for each of N sequences (C ``kda_gdr_decode_step``).

    q, k [N, L, H_k, d_k]; v [N, L, H_v, d_v]; log_alpha, beta [N, L, H_v]; or all
    without L for one token.  S [N, H_v, d_k, d_v] fp32 (a pool
    [n_slots, H_v, d_k, d_v] with ``slots`` [N] int32) is updated in place.
    Returns o [N, (L,) H_v, d_v].  ``snapshots``: True or a tensor
    [N, L, H_v, d_k, d_v] fp32 for the state after each token; then returns
    (o, snapshots).  ``stream`` as in kda_gdr_prefill."""
    host = _host()
    dev = _one_device(host, q, k, v, log_alpha, beta, S, o, slots, decay_scale, decay_bias)
    if q.dim() not in (3, 4) or v.dim() != q.dim():
        raise ValueError("q, k and v [N, H, d] or [N, L, H, d]")
    N, L = q.shape[0], q.shape[1] if q.dim() == 4 else 1
    o, opt, sizes = _gdr_call(host, q, k, v, log_alpha, beta, None, S, slots, o, decay_scale,
                              decay_bias, N, l2norm_qk, beta_is_logit, decay_from_logit, q_scale,
                              eps_l2)
    if snapshots is False:
        snapshots = None
    if snapshots is not None:
        shape = (N, L, *sizes[1:])
        if snapshots is True:
            snapshots = host.empty(shape, dtype=host.f32, device=q.device)
        else:
            _one_device(host, q, snapshots)
            _expect(snapshots, "snapshots", shape, host.f32)
        opt.snapshots = snapshots.data_ptr()
    rc = host.step(q.data_ptr(), k.data_ptr(), v.data_ptr(), log_alpha.data_ptr(),
                   beta.data_ptr(), S.data_ptr(), o.data_ptr(), N, L, *sizes,
                   _code(host, q.dtype), opt, host.current_stream(dev))
    if rc != KDA_OK:
        raise KdaError(rc, "kda_gdr_decode_step")
    return o if snapshots is None else (o, snapshots)


# ------------------------------------------------- projections
# KDA_ACT_*
ACTS = {"none": 0, "relu": 1, "silu": 2, "gelu": 3, "gelu_tanh": 4, "sigmoid": 5}


def _rows(x, name: str, rows: int, width: int) -> int:
    """Elements between the rows of x [rows, width], columns dense; 0 for dense rows."""
    if x.shape != (rows, width):
        raise ValueError(f"{name}: shape {tuple(x.shape)}, expected {(rows, width)}")
    if x.is_contiguous():
        return 0
    if width > 1 and x.stride(1) != 1:
        raise ValueError(f"{name}: each row has to be contiguous")
    if rows < 2:
        return 0
    if x.stride(0) < width:  # a broadcast row, or rows that overlap
        raise ValueError(f"{name}: rows have to lie apart")
    return x.stride(0)


@_on_stream
def kda_linear(x, w, bias=None, residual=None, y=None, *, act="none"):
    """y = act(x w^T + bias) + residual (C ``kda_linear``).

    x [M, K], w [N, K], bias [N] or None, residual [M, N] or None, all of one
    dtype; rows contiguous, any distance apart.  ``act``: a key of ``ACTS``.
    y [M, N] may be the residual itself.  ``stream`` as in kda_gdr_prefill."""
    host = _host()
    dev = _one_device(host, x, w, bias, residual, y)
    if x.dim() != 2 or w.dim() != 2:
        raise ValueError("x [M, K] and w [N, K]")
    M, (N, K), dtype = x.shape[0], w.shape, x.dtype
    if (M | N | K) >> 31:
        _sizes("kda_linear", M, N, K)
    code = _code(host, dtype)
    ldx, ldw, ldr, ldy, b, r = _rows(x, "x", M, K), _rows(w, "w", N, K), 0, 0, None, None
    if w.dtype != dtype:
        raise TypeError("x, w, bias, residual and y of one dtype")
    if bias is not None:
        _expect(bias, "bias", (N,), dtype)
        b = bias.data_ptr()
    if residual is not None:
        ldr, r = _rows(residual, "residual", M, N), residual.data_ptr()
        if residual.dtype != dtype:
            raise TypeError("x, w, bias, residual and y of one dtype")
    if y is None:
        y = host.empty((M, N), dtype=dtype, device=x.device)
    else:
        ldy = _rows(y, "y", M, N)
        if y.dtype != dtype:
            raise TypeError("x, w, bias, residual and y of one dtype")
    rc = host.linear(x.data_ptr(), ldx, w.data_ptr(), ldw, b, r, ldr, y.data_ptr(), ldy, M, N, K,
                     ACTS[act], code, host.current_stream(dev))
    if rc != KDA_OK:
        raise KdaError(rc, "kda_linear")
    return y


def _workspace(host, workspace, need, device):
    """(address, bytes, the tensor that holds them) of a workspace of `need` bytes at least, allocated if not given."""
    if need == 0:
        return None, 0, None
    if workspace is None:
        workspace = host.empty(need, dtype=host.u8, device=device)
    elif not workspace.is_contiguous():
        raise ValueError("workspace: libkda takes contiguous tensors")
    return workspace.data_ptr(), workspace.numel() * workspace.element_size(), workspace


@_on_stream
def kda_linear_i8(x, x_scale, w, w_scale, bias=None, residual=None, y=None, *, act="none",
                  dtype=None, workspace=None):
    """y = act(x_scale_m w_scale_n (x w^T) + bias) + residual (C ``kda_linear_i8``).

    x [M, K], w [N, K] int8, rows contiguous, any distance apart; x_scale [M], w_scale
    [N] fp32; bias [N], residual [M, N] of ``dtype`` (None: y's, the residual's or the
    bias's, else bfloat16) or None.  ``act``: a key of ``ACTS``.  y [M, N] may be the residual
    itself.  The integer sum is exact up to K = 1024, and up to 2^24 for any K; the header says what
    it loses beyond.  ``stream`` as in kda_gdr_prefill."""
    host = _host()
    dev = _one_device(host, x, x_scale, w, w_scale, bias, residual, y, workspace)
    if x.dim() != 2 or w.dim() != 2:
        raise ValueError("x [M, K] and w [N, K]")
    if x.dtype != host.i8 or w.dtype != host.i8:
        raise TypeError("x and w: int8")
    M, (N, K) = x.shape[0], w.shape
    if (M | N | K) >> 31:
        _sizes("kda_linear_i8", M, N, K)
    if dtype is None:
        dtype = next((t.dtype for t in (y, residual, bias) if t is not None), host.bf16)
    code = _code(host, dtype)
    ldx, ldw, ldr, ldy, b, r = _rows(x, "x", M, K), _rows(w, "w", N, K), 0, 0, None, None
    _expect(x_scale, "x_scale", (M,), host.f32)
    _expect(w_scale, "w_scale", (N,), host.f32)
    if bias is not None:
        _expect(bias, "bias", (N,), dtype)
        b = bias.data_ptr()
    if residual is not None:
        ldr, r = _rows(residual, "residual", M, N), residual.data_ptr()
        if residual.dtype != dtype:
            raise TypeError("bias, residual and y of one dtype")
    if y is None:
        y = host.empty((M, N), dtype=dtype, device=x.device)
    else:
        ldy = _rows(y, "y", M, N)
        if y.dtype != dtype:
            raise TypeError("bias, residual and y of one dtype")
    args = (x.data_ptr(), ldx, x_scale.data_ptr(), w.data_ptr(), ldw, w_scale.data_ptr(), b, r, ldr,
            y.data_ptr(), ldy, M, N, K, ACTS[act], code)
    at, size, _ = _workspace(host, workspace, 0 if workspace is None else 1, x.device)
    rc = host.linear_i8(*args, at, size, host.current_stream(dev))
    if rc == KDA_ERR_WORKSPACE and workspace is None:  # only some products need one
        at, size, workspace = _workspace(host, None, host.linear_i8_size(M, N, K), x.device)
        rc = host.linear_i8(*args, at, size, host.current_stream(dev))
    if rc != KDA_OK:
        raise KdaError(rc, "kda_linear_i8")
    return y


# ------------------------------------------------- the norm before a layer
def _like(host, x):
    """A new dense tensor of x's shape and type."""
    return (host.empty_like(x) if x.is_contiguous()
            else host.empty(x.shape, dtype=x.dtype, device=x.device))


def _norm(x, w, residual, total, y, q, scale, eps, i8):
    host = _host()
    dev = _one_device(host, x, w, residual, total, y, q, scale)
    if x.dim() != 2:
        raise ValueError("x [M, D]")
    (M, D), dtype = x.shape, x.dtype
    if (M | D) >> 31:
        _sizes("kda_rmsnorm", M, D)
    code = _code(host, dtype)
    ldx, ldr, lds, ldy, ldq = _rows(x, "x", M, D), 0, 0, 0, 0
    at = dict.fromkeys(("w", "residual", "sum", "y", "q", "scale"))
    if w is not None:
        _expect(w, "w", (D,), host.f32)
        at["w"] = w.data_ptr()
    if residual is None:
        if total is not None:
            raise ValueError("total: the sum with a residual, and there is none")
    else:
        ldr, at["residual"] = _rows(residual, "residual", M, D), residual.data_ptr()
        if total is None:
            total = _like(host, residual)
        lds, at["sum"] = _rows(total, "total", M, D), total.data_ptr()
        if residual.dtype != dtype or total.dtype != dtype:
            raise TypeError("x, residual, total and y of one dtype")
    if y is None and not i8:
        y = _like(host, x)
    if y is not None:
        ldy, at["y"] = _rows(y, "y", M, D), y.data_ptr()
        if y.dtype != dtype:
            raise TypeError("x, residual, total and y of one dtype")
    if i8:
        if q is None:
            q = host.empty((M, D), dtype=host.i8, device=x.device)
        if scale is None:
            scale = host.empty((M,), dtype=host.f32, device=x.device)
        _expect(scale, "scale", (M,), host.f32)
        ldq, at["q"], at["scale"] = _rows(q, "q", M, D), q.data_ptr(), scale.data_ptr()
        if q.dtype != host.i8:
            raise TypeError("q: int8")
    rc = host.rmsnorm(x.data_ptr(), ldx, at["residual"], ldr, at["w"], at["sum"], lds, at["y"],
                      ldy, at["q"], ldq, at["scale"], M, D, eps, code, host.current_stream(dev))
    if rc != KDA_OK:
        raise KdaError(rc, "kda_rmsnorm")
    return y, q, scale, total


@_on_stream
def kda_rmsnorm(x, w=None, residual=None, y=None, *, total=None, eps: float = 1e-6):
    """s = x + residual; y = s / sqrt(mean(s^2) + eps) * w per row (C ``kda_rmsnorm``).

    x, residual [M, D] of one dtype, rows contiguous, any distance apart; w [D] fp32 or None
    (ones).  Returns y, or with a residual (y, s); ``total``: where s goes, which may be x or the
    residual itself.  ``stream`` as in kda_gdr_prefill."""
    y, _, _, total = _norm(x, w, residual, total, y, None, None, eps, False)
    return y if residual is None else (y, total)


@_on_stream
def kda_rmsnorm_i8(x, w=None, residual=None, q=None, scale=None, *, total=None, y=None,
                   eps: float = 1e-6):
    """kda_rmsnorm with its output in 8-bit integers: q [M, D] int8 and scale [M] fp32, the
    values scale * q (C ``kda_rmsnorm``).  Returns (q, scale), or with a residual
    (q, scale, s); ``y``: where the output goes in the data type too."""
    _, q, scale, total = _norm(x, w, residual, total, y, q, scale, eps, True)
    return (q, scale) if residual is None else (q, scale, total)


@_on_stream
def kda_quantize_i8(x, q=None, scale=None):
    """x [M, D] in 8-bit integers with a scale per row (C ``kda_quantize_i8``): (q, scale)."""
    host = _host()
    dev = _one_device(host, x, q, scale)
    if x.dim() != 2:
        raise ValueError("x [M, D]")
    M, D = x.shape
    if (M | D) >> 31:
        _sizes("kda_quantize_i8", M, D)
    code = _code(host, x.dtype)
    if q is None:
        q = host.empty((M, D), dtype=host.i8, device=x.device)
    if scale is None:
        scale = host.empty((M,), dtype=host.f32, device=x.device)
    _expect(scale, "scale", (M,), host.f32)
    if q.dtype != host.i8:
        raise TypeError("q: int8")
    rc = host.quantize_i8(x.data_ptr(), _rows(x, "x", M, D), q.data_ptr(), _rows(q, "q", M, D),
                          scale.data_ptr(), M, D, code, host.current_stream(dev))
    if rc != KDA_OK:
        raise KdaError(rc, "kda_quantize_i8")
    return q, scale


# ------------------------------------------------- the gated linear recurrence
DECAY_FROM = {"log": 0, "softplus": 1, "sigmoid": 2}                # KDA_GLR_*
INPUT_SCALES = {"none": 0, "complement": 1, "normalized": 2}        # KDA_GLR_INPUT_*
GLR_TILE = 64


def kda_glr_options_init(**overrides) -> kda_glr_options:
    """Default options (C kda_glr_options_init), then keyword overrides."""
    opt = kda_glr_options()
    load().kda_glr_options_init(ctypes.byref(opt))
    for key, val in overrides.items():
        setattr(opt, key, val)
    return opt


def _tokens(x, name: str, shape, dtype) -> int:
    """Elements between the rows of successive tokens of x [..., D], channels dense, tokens
    evenly spaced; 0 for dense rows."""
    if x.shape != shape:
        raise ValueError(f"{name}: shape {tuple(x.shape)}, expected {tuple(shape)}")
    if x.dtype != dtype:
        raise TypeError(f"{name}: {x.dtype}, expected {dtype}")
    return 0 if x.is_contiguous() else _token_stride(x.unsqueeze(-2), name)


def _glr_options(host, x, log_alpha, decay_from, decay_scale, decay_bias, input_scale, input_gate,
                 slots, pool, N):
    """Options of a call on tokens x [..., D] (log_alpha and the gate alike); checks them."""
    shape, dtype, D = x.shape, x.dtype, x.shape[-1]
    ldx, ldla = _tokens(x, "x", shape, dtype), _tokens(log_alpha, "log_alpha", shape, dtype)
    ldg, gate, A, b, at, n_slots = 0, None, None, None, None, N
    if input_gate is not None:
        ldg, gate = _tokens(input_gate, "input_gate", shape, dtype), input_gate.data_ptr()
    if decay_scale is not None:
        _expect(decay_scale, "decay_scale", (D,), host.f32)
        A = decay_scale.data_ptr()
    if decay_bias is not None:
        _expect(decay_bias, "decay_bias", (D,), host.f32)
        b = decay_bias.data_ptr()
    if slots is not None:
        _expect(slots, "slots", (N,), host.i32)
        at, n_slots = slots.data_ptr(), pool.shape[0]
    return n_slots, kda_glr_options(DECAY_FROM[decay_from], A, b, INPUT_SCALES[input_scale], gate,
                                    ldx, ldla, ldg, at, min(n_slots, 0x7fffffff))


def _sequences(host, T, cu_seqlens, N, max_seqlen):
    """(N, the longest sequence as far as it is known)"""
    if cu_seqlens is not None:
        N = cu_seqlens.numel() - 1
        _expect(cu_seqlens, "cu_seqlens", (N + 1,), host.i32)
    elif N is None:
        N = 1
    if max_seqlen == 0 and cu_seqlens is None and N > 0:
        max_seqlen = T // N
    return N, max_seqlen


@_on_stream
def kda_glr_scan(x, log_alpha, h0=None, cu_seqlens=None, N: int | None = None, y=None, h_T=None, *,
                 slots=None, decay_from="log", decay_scale=None, decay_bias=None,
                 input_scale="none", input_gate=None, checkpoints=None, max_seqlen: int = 0):
    """The gated linear recurrence over packed sequences (C ``kda_glr_scan``).

    h_t = a_t h_{t-1} + c_t sigmoid(i_t) x_t per channel, a = e^g; x, log_alpha and input_gate
    (i, or None) [T, D] of one dtype, channels contiguous, tokens any even distance apart.
    ``decay_from``: "log" (g = min(log_alpha, 0)), "softplus" or "sigmoid" (g = -A f(log_alpha + b)
    with decay_scale A >= 0 and decay_bias b [D] fp32, None = ones / zeros).  ``input_scale``: "none"
    (c = 1), "complement" (1 - a) or "normalized" (sqrt(1 - a^2)).  h0 [N, D] fp32 or None
    (zeros); cu_seqlens, N, max_seqlen, slots (h0 and h_T are pools [n_slots, D] then) and
    stream as in kda_gdr_prefill.  Returns (y, h_T); with ``checkpoints`` (True, or a tensor
    [T // 64 + N, D] fp32) (y, h_T, checkpoints), which kda_glr_scan_backward takes.  Like every
    call here it records nothing for autograd: the gradient is that call's, made by the caller."""
    host = _host()
    if checkpoints is False:
        checkpoints = None
    dev = _one_device(host, x, log_alpha, h0, cu_seqlens, y, h_T, slots, decay_scale, decay_bias,
                      input_gate, None if checkpoints is True else checkpoints)
    if x.dim() != 2:
        raise ValueError("x [T, D]")
    (T, D), dtype = x.shape, x.dtype
    code = _code(host, dtype)
    N, max_seqlen = _sequences(host, T, cu_seqlens, N, max_seqlen)
    if (T | D | N | max_seqlen) >> 31:
        _sizes("kda_glr_scan", T, D, N, max_seqlen)
    if h_T is None:
        if slots is not None:
            raise ValueError("with slots, h_T is the pool that the states are written to")
        h_T = host.empty((max(N, 0), D), dtype=host.f32, device=x.device)
    n_slots, opt = _glr_options(host, x, log_alpha, decay_from, decay_scale, decay_bias,
                                input_scale, input_gate, slots, h_T, N)
    _expect(h_T, "h_T", (n_slots, D), host.f32)
    if h0 is not None and h0 is not h_T:
        _expect(h0, "h0", (n_slots, D), host.f32)
    if y is None:
        y = _like(host, x)
    else:
        _expect(y, "y", (T, D), dtype)
    if checkpoints is not None:
        rows = (T // GLR_TILE + N, D)
        if checkpoints is True:
            checkpoints = host.empty(rows, dtype=host.f32, device=x.device)
        else:
            _expect(checkpoints, "checkpoints", rows, host.f32)
        opt.checkpoints = checkpoints.data_ptr()
    opt.max_seqlen = max_seqlen
    rc = host.glr_scan(x.data_ptr(), log_alpha.data_ptr(), _ptr(h0), _ptr(cu_seqlens), N,
                       y.data_ptr(), h_T.data_ptr(), T, D, code, opt, host.current_stream(dev))
    if rc != KDA_OK:
        raise KdaError(rc, "kda_glr_scan")
    return (y, h_T) if checkpoints is None else (y, h_T, checkpoints)


@_on_stream
def kda_glr_step(x, log_alpha, h, y=None, *, slots=None, decay_from="log", decay_scale=None,
                 decay_bias=None, input_scale="none", input_gate=None):
    """L tokens for each of N sequences, states in place (C ``kda_glr_step``): x, log_alpha and
    input_gate [N, L, D], or without L for one token; h [N, D] fp32 (a pool [n_slots, D] with
    ``slots`` [N] int32).  The rest as in kda_glr_scan.  Returns y."""
    host = _host()
    dev = _one_device(host, x, log_alpha, h, y, slots, decay_scale, decay_bias, input_gate)
    if x.dim() not in (2, 3):
        raise ValueError("x [N, D] or [N, L, D]")
    N, D = x.shape[0], x.shape[-1]
    L = x.shape[1] if x.dim() == 3 else 1
    if (N | L | D) >> 31:
        _sizes("kda_glr_step", N, L, D)
    n_slots, opt = _glr_options(host, x, log_alpha, decay_from, decay_scale, decay_bias,
                                input_scale, input_gate, slots, h, N)
    _expect(h, "h", (n_slots, D), host.f32)
    if y is None:
        y = _like(host, x)
    else:
        _expect(y, "y", x.shape, x.dtype)
    rc = host.glr_step(x.data_ptr(), log_alpha.data_ptr(), h.data_ptr(), y.data_ptr(), N, L, D,
                       _code(host, x.dtype), opt, host.current_stream(dev))
    if rc != KDA_OK:
        raise KdaError(rc, "kda_glr_step")
    return y


@_on_stream
def kda_glr_scan_backward(dy, dh_T, x, log_alpha, checkpoints, cu_seqlens=None,
                          N: int | None = None, *, decay_from="log", decay_scale=None,
                          decay_bias=None, input_scale="none", input_gate=None,
                          max_seqlen: int = 0, workspace=None):
    """The gradient of kda_glr_scan (C ``kda_glr_scan_backward``): dy [T, D] and dh_T [N, D] fp32
    are those of its outputs (either may be None: zeros), the rest is what it was given and the
    checkpoints that it returned.  Returns (dx, dlog_alpha, dinput_gate, dh0, ddecay_scale,
    ddecay_bias), None for what the call had not (the last two come with logits, whether or not
    the parameters were given); rows behind the last sequence are not written."""
    host = _host()
    dev = _one_device(host, x, dy, dh_T, log_alpha, checkpoints, cu_seqlens, decay_scale,
                      decay_bias, input_gate, workspace)
    if x.dim() != 2:
        raise ValueError("x [T, D]")
    (T, D), dtype, device = x.shape, x.dtype, x.device
    code = _code(host, dtype)
    N, max_seqlen = _sequences(host, T, cu_seqlens, N, max_seqlen)
    if (T | D | N | max_seqlen) >> 31:
        _sizes("kda_glr_scan_backward", T, D, N, max_seqlen)
    _, opt = _glr_options(host, x, log_alpha, decay_from, decay_scale, decay_bias, input_scale,
                          input_gate, None, None, N)
    if dy is not None:
        _expect(dy, "dy", (T, D), dtype)
    if dh_T is not None:
        _expect(dh_T, "dh_T", (N, D), host.f32)
    _expect(checkpoints, "checkpoints", (T // GLR_TILE + N, D), host.f32)
    opt.checkpoints = checkpoints.data_ptr()
    opt.max_seqlen = max_seqlen
    dx, dla = _like(host, x), _like(host, x)
    dgate = _like(host, x) if input_gate is not None else None
    dh0 = host.empty((N, D), dtype=host.f32, device=device)
    dA = db = None
    if decay_from != "log":
        dA, db = (host.empty(D, dtype=host.f32, device=device) for _ in range(2))
        opt.workspace, opt.workspace_bytes, workspace = _workspace(
            host, workspace, host.glr_backward_size(T, N, D, code, opt), device)
    rc = host.glr_backward(_ptr(dy), _ptr(dh_T), x.data_ptr(), log_alpha.data_ptr(),
                           _ptr(cu_seqlens), N, dx.data_ptr(), dla.data_ptr(), _ptr(dgate),
                           dh0.data_ptr(), _ptr(dA), _ptr(db), T, D, code, opt,
                           host.current_stream(dev))
    if rc != KDA_OK:
        raise KdaError(rc, "kda_glr_scan_backward")
    return dx, dla, dgate, dh0, dA, db
