"""Python binding of libosdn (the C ABI in include/osdn.h): argument marshalling only.

Every function here takes CUDA tensors, checks their dtype/shape/contiguity, allocates the
outputs the caller did not pass (``torch.empty`` on the inputs' device), and calls the
C entry point of the same name on the current CUDA stream.  All arithmetic runs in the
library's kernels.  There is no fallback: if ``libosdn.so`` is missing, importing this module
raises, and a non-OK status raises :class:`OsdnError`.
"""
from __future__ import annotations

import ctypes
import functools
import os
import re
from typing import Optional

import torch

_PKG = os.path.dirname(os.path.abspath(__file__))
# OSDN_LIBRARY selects another build of the library (the debug-bounds build, libosdn_debug.so)
LIB_PATH = os.environ.get("OSDN_LIBRARY") or os.path.join(_PKG, "libosdn.so")
HEADER = os.path.join(os.path.dirname(_PKG), "include", "osdn.h")

OSDN_OK = 0
OSDN_ERR_INVALID_ARG = 1
OSDN_ERR_UNSUPPORTED = 2
OSDN_ERR_ALIGNMENT = 3
OSDN_ERR_CUDA = 4
OSDN_ERR_DEVICE_TIMEOUT = 5
OSDN_ERR_DEVICE_BOUNDS = 6
OSDN_BF16 = 0
OSDN_F32 = 1

_vp = ctypes.c_void_p
_i32 = ctypes.c_int32
_f32 = ctypes.c_float


class OsdnError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        super().__init__(f"{where}: {status_string(status)} (status {status})")


def _load() -> ctypes.CDLL:
    if not os.path.exists(LIB_PATH):
        raise ImportError(
            f"{LIB_PATH} is missing: build it with `python -m delta_rule_recurrent_osdn_b200.build`"
            " (there is no non-CUDA implementation)")
    lib = ctypes.CDLL(LIB_PATH)
    lib.osdn_abi_version.argtypes = []
    lib.osdn_abi_version.restype = _i32
    lib.osdn_status_string.argtypes = [ctypes.c_int]
    lib.osdn_status_string.restype = ctypes.c_char_p
    lib.osdn_precond_scan.argtypes = [_vp, _vp, _vp, _f32, _vp, _vp, _vp, _vp, _vp, _i32, _i32,
                                      _i32, _i32, _i32, ctypes.c_int, _vp]
    lib.osdn_precond_scan.restype = ctypes.c_int
    lib.osdn_chunk_fwd.argtypes = [_vp, _vp, _vp, _vp, _vp, _vp, _i32, _f32, _vp, _vp, _vp, _vp,
                                   _i32, _i32, _i32, _i32, _i32, _i32, _i32, ctypes.c_int, _vp]
    lib.osdn_chunk_fwd.restype = ctypes.c_int
    lib.osdn_fwd_workspace_bytes.argtypes = [_i32, _i32, _i32, _i32, ctypes.c_int]
    lib.osdn_fwd_workspace_bytes.restype = ctypes.c_size_t
    lib.osdn_fwd.argtypes = [_vp, _vp, _vp, _vp, _vp, _vp, _i32, _f32, _vp, _vp, _f32, _vp, _vp,
                             _vp, _vp, _vp, _vp, _i32, _i32, _i32, _i32, _i32, _i32, _i32,
                             ctypes.c_int, _vp, ctypes.c_size_t, _vp]
    lib.osdn_fwd.restype = ctypes.c_int
    lib.osdn_step.argtypes = [_vp, _vp, _vp, _vp, _vp, _vp, _i32, _f32, _f32, _vp, _vp, _vp, _vp,
                              _vp, _i32, _i32, _i32, _i32, ctypes.c_int, _vp]
    lib.osdn_step.restype = ctypes.c_int
    lib.osdn_bwd_workspace_bytes.argtypes = [_i32, _i32, _i32, _i32, _i32, _i32, ctypes.c_int]
    lib.osdn_bwd_workspace_bytes.restype = ctypes.c_size_t
    lib.osdn_bwd.argtypes = [_vp, _vp, _vp, _vp, _vp, _f32, _vp, _vp, _f32, _vp, _vp, _vp, _vp,
                             _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _i32, _i32, _i32, _i32, _i32,
                             _i32, ctypes.c_int, _vp, ctypes.c_size_t, _vp]
    lib.osdn_bwd.restype = ctypes.c_int
    lib.osdn_rho_geomean.argtypes = [_vp, _vp, _i32, _i32, _i32, _i32, _vp, _vp]
    lib.osdn_rho_geomean.restype = ctypes.c_int
    lib.osdn_get_device_status.argtypes = [_vp]
    lib.osdn_get_device_status.restype = ctypes.c_int
    lib.osdn_debug_watchdog_selftest.argtypes = [ctypes.c_int64, _vp]
    lib.osdn_debug_watchdog_selftest.restype = ctypes.c_int
    _declare_layer_operators(lib)
    return lib


def _declare_layer_operators(lib):
    """Argument types of the convolution, the scan and the norm: p a pointer, i an int32, l an
    int64, f a float, z a size_t, e an enum."""
    types = {"p": _vp, "i": _i32, "l": ctypes.c_int64, "f": _f32, "z": ctypes.c_size_t,
             "e": ctypes.c_int}
    for name, sig in (
            ("osdn_conv_fwd", "ppppipppiiiiiep"),
            ("osdn_conv_step", "ppppipiiiep"),
            ("osdn_conv_bwd", "ppppipeppppppiiiiiepzp"),
            ("osdn_ssm_fwd", "pppppppipppp" + "iiiiiii" + "epzp"),
            ("osdn_ssm_step", "pppppppippiiiiiep"),
            ("osdn_ssm_bwd", "pppppppi" + "ppp" + "pppppppp" + "p" + "iiiiiii" + "epzp"),
            ("osdn_norm_fwd", "pppppiiffppliep"),
            ("osdn_norm_bwd", "pppppiiff" + "ppppppp" + "liepzp")):
        fn = getattr(lib, name)
        fn.argtypes = [types[c] for c in sig]
        fn.restype = ctypes.c_int
    for name, sig in (("osdn_conv_bwd_workspace_bytes", "iiii"),
                      ("osdn_ssm_fwd_workspace_bytes", "iiiiiie"),
                      ("osdn_ssm_bwd_workspace_bytes", "iiiiiie"),
                      ("osdn_norm_bwd_workspace_bytes", "li")):
        fn = getattr(lib, name)
        fn.argtypes = [types[c] for c in sig]
        fn.restype = ctypes.c_size_t


LIB = _load()


def header_symbols() -> list:
    """Names of the functions include/osdn.h declares."""
    text = open(HEADER).read()
    return sorted(set(re.findall(r"^OSDN_API\s+[\w\s\*]*?(osdn_\w+)\s*\(", text, re.M)))


def status_string(status: int) -> str:
    return LIB.osdn_status_string(int(status)).decode()


def _check(status: int, where: str):
    if status != OSDN_OK:
        raise OsdnError(status, where)


def _p(t: Optional[torch.Tensor]):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(stream) -> ctypes.c_void_p:
    if stream is None:
        stream = torch.cuda.current_stream()
    return ctypes.c_void_p(stream.cuda_stream)


def _io(t: torch.Tensor) -> int:
    if t.dtype == torch.bfloat16:
        return OSDN_BF16
    if t.dtype == torch.float32:
        return OSDN_F32
    raise TypeError(f"io tensors must be bfloat16 or float32, got {t.dtype}")


def _req(t, name, dtype=None, shape=None):
    if t is None:
        return
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if dtype is not None and t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if shape is not None and tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")


def _seqs(cu_seqlens, B):
    if cu_seqlens is None:
        return 0, B
    _req(cu_seqlens, "cu_seqlens", torch.int32)
    n = cu_seqlens.numel() - 1
    return n, n


def osdn_precond_scan(k, beta, r=None, eta: float = 0.0, d0=None, cu_seqlens=None,
                      k_tilde=None, dT=None, return_dT: bool = True, rho=None, stream=None):
    """Phase 1: returns ``(k_tilde, dT)`` (``dT`` is None when ``return_dT`` is False).  Given a
    float32 tensor ``rho`` of shape [B, T, H], also writes the per-token residual-contraction
    ratio (1 - beta_t <d_t, k_t^2>)^2 there."""
    B, T, H, Dk = k.shape
    io = _io(k)
    num_seqs, N = _seqs(cu_seqlens, B)
    _req(k, "k")
    _req(beta, "beta", torch.float32, (B, T, H))
    _req(r, "r", torch.float32, (B, T, H))
    _req(d0, "d0", torch.float32, (N, H, Dk))
    if k_tilde is None:
        k_tilde = torch.empty_like(k)
    _req(k_tilde, "k_tilde", k.dtype, k.shape)
    if dT is None and return_dT:
        dT = torch.empty((N, H, Dk), dtype=torch.float32, device=k.device)
    _req(dT, "dT", torch.float32, (N, H, Dk))
    _req(rho, "rho", torch.float32, (B, T, H))
    _check(LIB.osdn_precond_scan(_p(k), _p(beta), _p(r), float(eta), _p(d0), _p(k_tilde), _p(dT),
                                 _p(rho), _p(cu_seqlens), num_seqs, B, T, H, Dk, io,
                                 _stream(stream)),
           "osdn_precond_scan")
    return k_tilde, dT


def _alpha(alpha, B, T, H, Dk):
    """(pointer, per_channel flag) of a gated backbone's decay: [B, T, H] or [B, T, H, Dk]."""
    if alpha is None:
        return None, 0
    per_channel = alpha.dim() == 4
    _req(alpha, "alpha", torch.float32, (B, T, H, Dk) if per_channel else (B, T, H))
    return _p(alpha), int(per_channel)


def osdn_chunk_fwd(q, k, k_tilde, v, beta, scale: float = 1.0, S0=None, chunk: int = 64,
                   cu_seqlens=None, o=None, ST=None, return_ST: bool = True, stream=None,
                   alpha=None):
    """Phase 2: returns ``(o, ST)`` (``ST`` is None when ``return_ST`` is False).  ``alpha``: the
    decay of a gated backbone, [B, T, H] (Gated DeltaNet) or [B, T, H, Dk] (Kimi Delta Attention)
    float32, or None."""
    B, T, H, Dk = q.shape
    Dv = v.shape[-1]
    io = _io(q)
    num_seqs, N = _seqs(cu_seqlens, B)
    for name, t in (("q", q), ("k", k), ("k_tilde", k_tilde)):
        _req(t, name, q.dtype, (B, T, H, Dk))
    _req(v, "v", q.dtype, (B, T, H, Dv))
    _req(beta, "beta", torch.float32, (B, T, H))
    _req(S0, "S0", torch.float32, (N, H, Dv, Dk))
    if o is None:
        o = torch.empty_like(v)
    _req(o, "o", q.dtype, (B, T, H, Dv))
    if ST is None and return_ST:
        ST = torch.empty((N, H, Dv, Dk), dtype=torch.float32, device=q.device)
    _req(ST, "ST", torch.float32, (N, H, Dv, Dk))
    a_ptr, apc = _alpha(alpha, B, T, H, Dk)
    _check(LIB.osdn_chunk_fwd(_p(q), _p(k), _p(k_tilde), _p(v), _p(beta), a_ptr, apc,
                              float(scale), _p(S0),
                              _p(o), _p(ST), _p(cu_seqlens), num_seqs, B, T, H, Dk, Dv,
                              int(chunk), io, _stream(stream)),
           "osdn_chunk_fwd")
    return o, ST


def osdn_fwd_workspace_bytes(B: int, T: int, H: int, Dk: int, dtype=torch.bfloat16) -> int:
    io = OSDN_BF16 if dtype == torch.bfloat16 else OSDN_F32
    return int(LIB.osdn_fwd_workspace_bytes(B, T, H, Dk, io))


def osdn_fwd(q, k, v, beta, r=None, eta: float = 0.0, d0=None, S0=None, scale: float = 1.0,
             chunk: int = 64, cu_seqlens=None, o=None, ST=None, dT=None, k_tilde=None,
             workspace=None, return_states: bool = True, rho=None, stream=None, alpha=None):
    """Both phases: returns ``(o, ST, dT)`` (states None when ``return_states`` is False).
    ``alpha``: the decay of a gated backbone, as for :func:`osdn_chunk_fwd`.

    The call needs a device workspace of ``osdn_fwd_workspace_bytes`` bytes (for bf16 it holds
    the residual of k~'s rounding, and k~ itself when ``k_tilde`` is not given); when
    ``workspace`` is None it is allocated with torch (device memory plumbing).
    """
    B, T, H, Dk = q.shape
    Dv = v.shape[-1]
    io = _io(q)
    num_seqs, N = _seqs(cu_seqlens, B)
    for name, t in (("q", q), ("k", k)):
        _req(t, name, q.dtype, (B, T, H, Dk))
    _req(v, "v", q.dtype, (B, T, H, Dv))
    _req(beta, "beta", torch.float32, (B, T, H))
    _req(r, "r", torch.float32, (B, T, H))
    _req(d0, "d0", torch.float32, (N, H, Dk))
    _req(S0, "S0", torch.float32, (N, H, Dv, Dk))
    _req(k_tilde, "k_tilde", q.dtype, (B, T, H, Dk))
    if o is None:
        o = torch.empty_like(v)
    _req(o, "o", q.dtype, (B, T, H, Dv))
    if return_states:
        if ST is None:
            ST = torch.empty((N, H, Dv, Dk), dtype=torch.float32, device=q.device)
        if dT is None:
            dT = torch.empty((N, H, Dk), dtype=torch.float32, device=q.device)
    _req(ST, "ST", torch.float32, (N, H, Dv, Dk))
    _req(dT, "dT", torch.float32, (N, H, Dk))
    _req(rho, "rho", torch.float32, (B, T, H))
    ws_bytes = 0
    need = int(LIB.osdn_fwd_workspace_bytes(B, T, H, Dk, io))
    if workspace is None and need > 0:
        workspace = torch.empty(need, dtype=torch.uint8, device=q.device)
    if workspace is not None:
        _req(workspace, "workspace")
        ws_bytes = workspace.numel() * workspace.element_size()
    a_ptr, apc = _alpha(alpha, B, T, H, Dk)
    _check(LIB.osdn_fwd(_p(q), _p(k), _p(v), _p(beta), _p(r), a_ptr, apc, float(eta), _p(d0),
                        _p(S0),
                        float(scale), _p(o), _p(ST), _p(dT), _p(rho), _p(k_tilde), _p(cu_seqlens),
                        num_seqs, B, T, H, Dk, Dv, int(chunk), io, _p(workspace), ws_bytes,
                        _stream(stream)),
           "osdn_fwd")
    return o, ST, dT


def osdn_step(q, k, v, beta, S, d, r=None, eta: float = 0.0, scale: float = 1.0, o=None,
              k_tilde=None, rho=None, stream=None, alpha=None):
    """One recurrent step per (sequence, head) (the decode path).  q, k: [N, H, Dk]; v: [N, H, Dv];
    beta, r: [N, H] float32; S: [N, H, Dv, Dk] and d: [N, H, Dk] float32, updated in place;
    alpha: the decay of a gated backbone, [N, H] (Gated DeltaNet) or [N, H, Dk] (Kimi Delta
    Attention) float32, or None.  Returns o [N, H, Dv] (and writes k_tilde [N, H, Dk] when given)."""
    N, H, Dk = q.shape
    Dv = v.shape[-1]
    io = _io(q)
    _req(q, "q")
    _req(k, "k", q.dtype, (N, H, Dk))
    _req(v, "v", q.dtype, (N, H, Dv))
    _req(beta, "beta", torch.float32, (N, H))
    _req(r, "r", torch.float32, (N, H))
    _req(S, "S", torch.float32, (N, H, Dv, Dk))
    _req(d, "d", torch.float32, (N, H, Dk))
    if o is None:
        o = torch.empty_like(v)
    _req(o, "o", q.dtype, (N, H, Dv))
    _req(k_tilde, "k_tilde", q.dtype, (N, H, Dk))
    _req(rho, "rho", torch.float32, (N, H))
    per_channel = alpha is not None and alpha.dim() == 3
    _req(alpha, "alpha", torch.float32, (N, H, Dk) if per_channel else (N, H))
    _check(LIB.osdn_step(_p(q), _p(k), _p(v), _p(beta), _p(r), _p(alpha), int(per_channel),
                         float(eta), float(scale), _p(S), _p(d), _p(o), _p(k_tilde), _p(rho), N, H,
                         Dk, Dv, io, _stream(stream)),
           "osdn_step")
    return o


def osdn_bwd(q, k, v, beta, dO, r=None, eta: float = 0.0, d0=None, S0=None, scale: float = 1.0,
             dST=None, ddT=None, cu_seqlens=None, workspace=None, stream=None):
    """Gradients of L (given dL/do = dO, and optionally dL/dS_T, dL/dd_T) with respect to every
    input of :func:`osdn_fwd`.  Returns a dict of float32 tensors dq, dk, dv, dbeta, dr (None
    without r), deta (one element), dS0, dd0.  A workspace of ``osdn_bwd_workspace_bytes``
    bytes is allocated with torch when none is given (device memory plumbing)."""
    B, T, H, Dk = q.shape
    Dv = v.shape[-1]
    io = _io(q)
    num_seqs, N = _seqs(cu_seqlens, B)
    for name, t in (("q", q), ("k", k)):
        _req(t, name, q.dtype, (B, T, H, Dk))
    _req(v, "v", q.dtype, (B, T, H, Dv))
    _req(dO, "dO", q.dtype, (B, T, H, Dv))
    _req(beta, "beta", torch.float32, (B, T, H))
    _req(r, "r", torch.float32, (B, T, H))
    _req(d0, "d0", torch.float32, (N, H, Dk))
    _req(S0, "S0", torch.float32, (N, H, Dv, Dk))
    _req(dST, "dST", torch.float32, (N, H, Dv, Dk))
    _req(ddT, "ddT", torch.float32, (N, H, Dk))
    f32 = dict(dtype=torch.float32, device=q.device)
    g = {"dq": torch.empty((B, T, H, Dk), **f32), "dk": torch.empty((B, T, H, Dk), **f32),
         "dv": torch.empty((B, T, H, Dv), **f32), "dbeta": torch.empty((B, T, H), **f32),
         "dr": None if r is None else torch.empty((B, T, H), **f32),
         "deta": torch.empty((1,), **f32), "dS0": torch.empty((N, H, Dv, Dk), **f32),
         "dd0": torch.empty((N, H, Dk), **f32)}
    need = int(LIB.osdn_bwd_workspace_bytes(num_seqs, B, T, H, Dk, Dv, io))
    if workspace is None:
        workspace = torch.empty(max(need, 1), dtype=torch.uint8, device=q.device)
    _req(workspace, "workspace")
    _check(LIB.osdn_bwd(_p(q), _p(k), _p(v), _p(beta), _p(r), float(eta), _p(d0), _p(S0),
                        float(scale), _p(dO), _p(dST), _p(ddT), _p(g["dq"]), _p(g["dk"]),
                        _p(g["dv"]), _p(g["dbeta"]), _p(g["dr"]), _p(g["deta"]), _p(g["dS0"]),
                        _p(g["dd0"]), _p(cu_seqlens), num_seqs, B, T, H, Dk, Dv, io,
                        _p(workspace), workspace.numel(), _stream(stream)),
           "osdn_bwd")
    return g


def osdn_rho_geomean(rho, cu_seqlens=None, q_geo=None, stream=None):
    """q_geo [N, H] float32: exp(mean_t log rho_t) per (sequence, head), from a residual-ratio
    tensor rho [B, T, H] (the ``rho`` output of the scan or the forward pass)."""
    B, T, H = rho.shape
    _req(rho, "rho", torch.float32)
    num_seqs, N = _seqs(cu_seqlens, B)
    if q_geo is None:
        q_geo = torch.empty((N, H), dtype=torch.float32, device=rho.device)
    _req(q_geo, "q_geo", torch.float32, (N, H))
    _check(LIB.osdn_rho_geomean(_p(rho), _p(cu_seqlens), num_seqs, B, T, H, _p(q_geo),
                                _stream(stream)), "osdn_rho_geomean")
    return q_geo


# ------------------------------------------------------------------------------------------
# Layer operators around the mixer: the short causal convolution, the selective scan, the norm.

# A call launches on the current stream of its tensors' device, and a decoder makes thousands of
# them a second: the checks below look at each tensor once, and pointers go to ctypes as integers.
_current_device = torch.cuda.current_device
_raw_stream = torch._C._cuda_getCurrentRawStream


def _placed(fn):
    """Runs an entry point with its first tensor's device current and, when `stream` is given, that
    stream: outputs and workspace are then allocated for the stream that the call launches on."""
    first = fn.__code__.co_varnames[0]

    @functools.wraps(fn)
    def call(*args, stream=None, **kw):
        t = args[0] if args else kw[first]
        if not t.is_cuda:
            raise ValueError("tensors must be CUDA tensors")
        if stream is None and t.device.index == _current_device():
            return fn(*args, **kw)
        if stream is not None and stream.device != t.device:
            raise ValueError(f"stream is on {stream.device}, the tensors on {t.device}")
        with torch.cuda.device(t.device), torch.cuda.stream(stream):
            return fn(*args, **kw)
    return call


def _refuse(t, name, dtype, shape, device):
    _req(t, name, dtype, shape)
    raise ValueError(f"{name} is on {t.device}, expected {device}")


def _ptr(t, name, dtype, shape, device):
    """Address of a tensor (None for None) after checking its type, shape, device and layout."""
    if t is None:
        return None
    if t.dtype is not dtype or t.shape != shape or t.device != device or not t.is_contiguous():
        _refuse(t, name, dtype, shape, device)
    return t.data_ptr()


def _out(t, name, dtype, shape, device):
    """The caller's output tensor, checked, or a new one."""
    if t is None:
        return torch.empty(shape, dtype=dtype, device=device)
    _ptr(t, name, dtype, shape, device)
    return t


def _fits(where, *sizes):
    """The C entry points take sizes as int32, and ctypes would pass the lower half of a larger one."""
    if max(sizes) > 0x7FFFFFFF:
        raise OsdnError(OSDN_ERR_UNSUPPORTED, where)


def _packed(cu_seqlens, B, device):
    """(address, num_seqs, N) of packed offsets, or (None, 0, B)."""
    if cu_seqlens is None:
        return None, 0, B
    n = cu_seqlens.numel() - 1
    return _ptr(cu_seqlens, "cu_seqlens", torch.int32, (n + 1,), device), n, n


def _scratch(t, need, device):
    """(tensor, address, bytes) of the caller's workspace or of a new one."""
    if t is None:
        if need == 0:
            return None, None, 0
        t = torch.empty(need, dtype=torch.uint8, device=device)
    else:
        _req(t, "workspace")
        if t.device != device:
            raise ValueError(f"workspace is on {t.device}, expected {device}")
    return t, t.data_ptr(), t.numel() * t.element_size()


def _addr(t):
    return None if t is None else t.data_ptr()


def _silu_flag(activation):
    if activation not in (None, "silu"):
        raise ValueError(f"activation must be 'silu' or None, got {activation!r}")
    return int(activation == "silu")


def _conv_dims(x, weight, lead):
    """(C, W) of a convolution's input [lead sizes, ...channels] and filters [C, W]."""
    if x.dim() < lead + 1:
        raise ValueError(f"x has shape {tuple(x.shape)}, expected {lead} leading sizes and channels")
    if weight.dim() != 2:
        raise ValueError(f"weight has shape {tuple(weight.shape)}, expected [C, W]")
    C = x.shape[lead]
    for n in x.shape[lead + 1:]:
        C *= n
    return C, weight.shape[1]


@_placed
def osdn_conv_fwd(x, weight, bias=None, state0=None, activation: Optional[str] = "silu",
                  cu_seqlens=None, y=None, stateT=None, return_state: bool = True):
    """Short causal convolution over each channel's last W tokens: returns ``(y, stateT)``
    (``stateT`` None when ``return_state`` is False).  x: [B, T, C], or [B, T, H, D] with
    C = H * D (q, k or v as the mixer takes them); weight: [C, W] float32, W in 2..4; bias: [C]
    float32; state0, stateT: [N, W - 1, C] in x's dtype, the last inputs, oldest first;
    activation: "silu" or None; stream: where to launch (default: the current stream)."""
    C, W = _conv_dims(x, weight, 2)
    io, dev, dt = _io(x), x.device, x.dtype
    B, T = x.shape[0], x.shape[1]
    cu, num_seqs, N = _packed(cu_seqlens, B, dev)
    _fits("osdn_conv_fwd", B, T, C, W, N)
    y = torch.empty_like(x) if y is None else _out(y, "y", dt, x.shape, dev)
    if stateT is not None or return_state:
        stateT = _out(stateT, "stateT", dt, (N, W - 1, C), dev)
    _check(LIB.osdn_conv_fwd(_ptr(x, "x", dt, x.shape, dev),
                             _ptr(weight, "weight", torch.float32, (C, W), dev),
                             _ptr(bias, "bias", torch.float32, (C,), dev),
                             _ptr(state0, "state0", dt, (N, W - 1, C), dev),
                             _silu_flag(activation), y.data_ptr(), _addr(stateT), cu, num_seqs, B, T,
                             C, W, io, _raw_stream(dev.index)), "osdn_conv_fwd")
    return y, stateT


@_placed
def osdn_conv_step(x, weight, state, bias=None, activation: Optional[str] = "silu", y=None):
    """One token per sequence of :func:`osdn_conv_fwd`: x [N, C] (or [N, H, D]); state
    [N, W - 1, C] in x's dtype, moved on by one token in place.  Returns y of x's shape."""
    C, W = _conv_dims(x, weight, 1)
    io, dev, dt, N = _io(x), x.device, x.dtype, x.shape[0]
    _fits("osdn_conv_step", N, C, W)
    if state is None:
        raise ValueError("state is required")
    y = torch.empty_like(x) if y is None else _out(y, "y", dt, x.shape, dev)
    _check(LIB.osdn_conv_step(_ptr(x, "x", dt, x.shape, dev),
                              _ptr(weight, "weight", torch.float32, (C, W), dev),
                              _ptr(bias, "bias", torch.float32, (C,), dev),
                              _ptr(state, "state", dt, (N, W - 1, C), dev), _silu_flag(activation),
                              y.data_ptr(), N, C, W, io, _raw_stream(dev.index)), "osdn_conv_step")
    return y


@_placed
def osdn_conv_bwd(x, weight, dy, bias=None, state0=None, dstateT=None,
                  activation: Optional[str] = "silu", cu_seqlens=None, workspace=None):
    """Gradients of :func:`osdn_conv_fwd` given dy (x's shape; x's dtype or float32, as
    :func:`osdn_bwd` returns for q, k and v) and optionally dstateT [N, W - 1, C] float32.
    Returns a dict: dx in x's dtype; dweight, dbias (None without bias) and dstate0 (None without
    state0) in float32."""
    C, W = _conv_dims(x, weight, 2)
    io, dev, dt = _io(x), x.device, x.dtype
    B, T = x.shape[0], x.shape[1]
    f32 = torch.float32
    if dy.dtype not in (dt, f32):
        raise TypeError(f"dy must be {dt} or torch.float32, got {dy.dtype}")
    cu, num_seqs, N = _packed(cu_seqlens, B, dev)
    _fits("osdn_conv_bwd", B, T, C, W, N)
    g = {"dx": torch.empty_like(x), "dweight": torch.empty((C, W), dtype=f32, device=dev),
         "dbias": None if bias is None else torch.empty((C,), dtype=f32, device=dev),
         "dstate0": None if state0 is None else torch.empty((N, W - 1, C), dtype=f32, device=dev)}
    ws, ws_ptr, ws_bytes = _scratch(workspace, LIB.osdn_conv_bwd_workspace_bytes(B, T, C, W), dev)
    _check(LIB.osdn_conv_bwd(_ptr(x, "x", dt, x.shape, dev), _ptr(weight, "weight", f32, (C, W), dev),
                             _ptr(bias, "bias", f32, (C,), dev),
                             _ptr(state0, "state0", dt, (N, W - 1, C), dev), _silu_flag(activation),
                             _ptr(dy, "dy", dy.dtype, x.shape, dev), _io(dy),
                             _ptr(dstateT, "dstateT", f32, (N, W - 1, C), dev), g["dx"].data_ptr(),
                             g["dweight"].data_ptr(), _addr(g["dbias"]), _addr(g["dstate0"]), cu,
                             num_seqs, B, T, C, W, io, ws_ptr, ws_bytes, _raw_stream(dev.index)),
           "osdn_conv_bwd")
    return g


def _ssm_args(x, dt, A, b, c, D, dt_bias, lead, dev):
    """Addresses of the scan's common inputs after their checks, and (H, G, Dk, Dv)."""
    H, Dv = x.shape[-2:]
    G, Dk = b.shape[-2:]
    f32, io = torch.float32, x.dtype
    return (_ptr(x, "x", io, (*lead, H, Dv), dev), _ptr(dt, "dt", f32, (*lead, H), dev),
            _ptr(A, "A", f32, (H,), dev), _ptr(b, "b", io, (*lead, G, Dk), dev),
            _ptr(c, "c", io, (*lead, G, Dk), dev), _ptr(D, "D", f32, (H,), dev),
            _ptr(dt_bias, "dt_bias", f32, (H,), dev)), H, G, Dk, Dv


def osdn_ssm_fwd_workspace_bytes(B: int, T: int, H: int, Dk: int, Dv: int, dtype=torch.bfloat16,
                                 num_seqs: int = 0) -> int:
    io = OSDN_BF16 if dtype == torch.bfloat16 else OSDN_F32
    _fits("osdn_ssm_fwd_workspace_bytes", num_seqs, B, T, H, Dk, Dv)
    return int(LIB.osdn_ssm_fwd_workspace_bytes(num_seqs, B, T, H, Dk, Dv, io))


@_placed
def osdn_ssm_fwd(x, dt, A, b, c, D=None, dt_bias=None, softplus: bool = True, S0=None,
                 cu_seqlens=None, y=None, ST=None, workspace=None, return_ST: bool = True):
    """Selective state-space scan: S_t = exp(step_t A) S_{t-1} + step_t x_t b_t^T and
    y_t = S_t c_t + D x_t with step = softplus(dt + dt_bias) (softplus False: dt + dt_bias).
    x: [B, T, H, Dv]; b, c: [B, T, G, Dk], shared by H / G heads each; dt: [B, T, H] float32;
    A, D, dt_bias: [H] float32; S0, ST: [N, H, Dv, Dk] float32, the mixer's state layout.
    Returns ``(y, ST)`` (``ST`` None when ``return_ST`` is False)."""
    io, dev = _io(x), x.device
    B, T = x.shape[0], x.shape[1]
    args, H, G, Dk, Dv = _ssm_args(x, dt, A, b, c, D, dt_bias, (B, T), dev)
    cu, num_seqs, N = _packed(cu_seqlens, B, dev)
    _fits("osdn_ssm_fwd", B, T, H, G, Dk, Dv, N)
    y = torch.empty_like(x) if y is None else _out(y, "y", x.dtype, x.shape, dev)
    if ST is not None or return_ST:
        ST = _out(ST, "ST", torch.float32, (N, H, Dv, Dk), dev)
    ws, ws_ptr, ws_bytes = _scratch(
        workspace, LIB.osdn_ssm_fwd_workspace_bytes(num_seqs, B, T, H, Dk, Dv, io), dev)
    _check(LIB.osdn_ssm_fwd(*args, int(softplus),
                            _ptr(S0, "S0", torch.float32, (N, H, Dv, Dk), dev), y.data_ptr(), _addr(ST),
                            cu, num_seqs, B, T, H, G, Dk, Dv, io, ws_ptr, ws_bytes,
                            _raw_stream(dev.index)), "osdn_ssm_fwd")
    return y, ST


@_placed
def osdn_ssm_step(x, dt, A, b, c, S, D=None, dt_bias=None, softplus: bool = True, y=None):
    """One token per sequence of :func:`osdn_ssm_fwd` (the decode path): x [N, H, Dv]; b, c
    [N, G, Dk]; dt [N, H] float32; S [N, H, Dv, Dk] float32, updated in place.  Returns y."""
    io, dev, N = _io(x), x.device, x.shape[0]
    args, H, G, Dk, Dv = _ssm_args(x, dt, A, b, c, D, dt_bias, (N,), dev)
    _fits("osdn_ssm_step", N, H, G, Dk, Dv)
    if S is None:
        raise ValueError("S is required")
    y = torch.empty_like(x) if y is None else _out(y, "y", x.dtype, x.shape, dev)
    _check(LIB.osdn_ssm_step(*args, int(softplus), _ptr(S, "S", torch.float32, (N, H, Dv, Dk), dev),
                             y.data_ptr(), N, H, G, Dk, Dv, io, _raw_stream(dev.index)),
           "osdn_ssm_step")
    return y


@_placed
def osdn_ssm_bwd(x, dt, A, b, c, dy, D=None, dt_bias=None, softplus: bool = True, S0=None,
                 dST=None, cu_seqlens=None, workspace=None):
    """Gradients of :func:`osdn_ssm_fwd` given dy (x's shape and dtype) and optionally dST.
    Returns a dict: dx, db, dc in x's dtype; ddt, dA, dD, ddt_bias and dS0 in float32 (the last
    three None where their input is)."""
    io, dev, f32 = _io(x), x.device, torch.float32
    B, T = x.shape[0], x.shape[1]
    args, H, G, Dk, Dv = _ssm_args(x, dt, A, b, c, D, dt_bias, (B, T), dev)
    cu, num_seqs, N = _packed(cu_seqlens, B, dev)
    _fits("osdn_ssm_bwd", B, T, H, G, Dk, Dv, N)

    def like(t):
        return None if t is None else torch.empty_like(t)

    g = {"dx": like(x), "ddt": like(dt), "dA": like(A), "db": like(b), "dc": like(c),
         "dD": like(D), "ddt_bias": like(dt_bias), "dS0": like(S0)}
    ws, ws_ptr, ws_bytes = _scratch(
        workspace, LIB.osdn_ssm_bwd_workspace_bytes(num_seqs, B, T, H, Dk, Dv, io), dev)
    _check(LIB.osdn_ssm_bwd(*args, int(softplus), _ptr(S0, "S0", f32, (N, H, Dv, Dk), dev),
                            _ptr(dy, "dy", x.dtype, x.shape, dev),
                            _ptr(dST, "dST", f32, (N, H, Dv, Dk), dev),
                            *(_addr(g[k]) for k in ("dx", "ddt", "dA", "db", "dc", "dD", "ddt_bias",
                                                    "dS0")),
                            cu, num_seqs, B, T, H, G, Dk, Dv, io, ws_ptr, ws_bytes,
                            _raw_stream(dev.index)), "osdn_ssm_bwd")
    return g


def _gate_act(gate_act):
    if gate_act not in ("silu", "sigmoid"):
        raise ValueError(f"gate_act must be 'silu' or 'sigmoid', got {gate_act!r}")
    return int(gate_act == "sigmoid")


def _norm_args(f, x, gate, w_post, w_next, dev):
    """Addresses of the norm's common inputs after their checks, and (R, D)."""
    D, dt, shape = f.shape[-1], f.dtype, f.shape
    return (_ptr(f, "f", dt, shape, dev), _ptr(x, "x", dt, shape, dev),
            _ptr(gate, "gate", dt, shape, dev), _ptr(w_post, "w_post", torch.float32, (D,), dev),
            _ptr(w_next, "w_next", torch.float32, (D,), dev)), (f.numel() // D if D else 0), D


@_placed
def osdn_norm_fwd(f, x=None, gate=None, w_post=None, w_next=None, gate_act: str = "silu",
                  gate_first: bool = False, scale: float = 1.0, eps: float = 1e-5, x_out=None,
                  h=None, return_x_out: bool = True):
    """Block norm over the last dimension of f: u = rmsnorm(f) * w_post * act(gate) (gate_first:
    rmsnorm(f * act(gate)) * w_post), x_out = x + scale * u, h = rmsnorm(x_out) * w_next.  Every
    part is optional: w_post, gate, x (no residual), w_next (h is None then).  x, gate: f's shape
    and dtype; w_post, w_next: [D] float32.  Returns ``(x_out, h)``; ``return_x_out`` False (with
    w_next) skips x_out."""
    io, dev = _io(f), f.device
    args, R, D = _norm_args(f, x, gate, w_post, w_next, dev)
    _fits("osdn_norm_fwd", D)
    if x_out is not None or return_x_out or w_next is None:
        x_out = torch.empty_like(f) if x_out is None else _out(x_out, "x_out", f.dtype, f.shape, dev)
    if w_next is not None:
        h = torch.empty_like(f) if h is None else _out(h, "h", f.dtype, f.shape, dev)
    elif h is not None:
        raise ValueError("h needs w_next")
    _check(LIB.osdn_norm_fwd(*args, _gate_act(gate_act), int(gate_first), scale, eps, _addr(x_out),
                             _addr(h), R, D, io, _raw_stream(dev.index)), "osdn_norm_fwd")
    return x_out, h


@_placed
def osdn_norm_bwd(f, dx_out=None, dh=None, x=None, gate=None, w_post=None, w_next=None,
                  gate_act: str = "silu", gate_first: bool = False, scale: float = 1.0,
                  eps: float = 1e-5, workspace=None):
    """Gradients of :func:`osdn_norm_fwd` from its inputs, given dx_out (or None for 0) and dh
    (exactly when w_next is given).  Returns a dict: df, dx, dgate in f's dtype, dw_post, dw_next
    in float32; None where the input is."""
    io, dev = _io(f), f.device
    args, R, D = _norm_args(f, x, gate, w_post, w_next, dev)
    _fits("osdn_norm_bwd", D)
    if (dh is None) != (w_next is None):
        raise ValueError("dh is given exactly when w_next is")
    if dh is None and dx_out is None:
        raise ValueError("dx_out or dh is required")

    def like(t):
        return None if t is None else torch.empty_like(t)

    g = {"df": like(f), "dx": like(x), "dgate": like(gate), "dw_post": like(w_post),
         "dw_next": like(w_next)}
    ws, ws_ptr, ws_bytes = _scratch(workspace, LIB.osdn_norm_bwd_workspace_bytes(R, D), dev)
    _check(LIB.osdn_norm_bwd(*args, _gate_act(gate_act), int(gate_first), scale, eps,
                             _ptr(dx_out, "dx_out", f.dtype, f.shape, dev),
                             _ptr(dh, "dh", f.dtype, f.shape, dev),
                             *(_addr(g[k]) for k in ("df", "dx", "dgate", "dw_post", "dw_next")),
                             R, D, io, ws_ptr, ws_bytes, _raw_stream(dev.index)), "osdn_norm_bwd")
    return g


def osdn_get_device_status(stream=None) -> int:
    """Synchronize the stream and return (and clear) the device status word."""
    return int(LIB.osdn_get_device_status(_stream(stream)))


def osdn_debug_watchdog_selftest(spin_limit: int, stream=None):
    _check(LIB.osdn_debug_watchdog_selftest(int(spin_limit), _stream(stream)),
           "osdn_debug_watchdog_selftest")
