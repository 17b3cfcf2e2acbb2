"""Python binding of libosdn (the C ABI in include/osdn.h): argument marshalling only.

Every function here takes CUDA tensors, checks their dtype/shape/contiguity, allocates the
outputs the caller did not pass (``torch.empty`` on the inputs' device), and calls the
C entry point of the same name on the current CUDA stream.  All arithmetic runs in the
library's kernels.  There is no fallback: if ``libosdn.so`` is missing, importing this module
raises, and a non-OK status raises :class:`OsdnError`.
"""
from __future__ import annotations

import ctypes
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

class _On:
    """Makes a tensor's device current, and `stream` (default: that device's current stream) the
    stream that the call launches on and that its outputs and workspace are allocated for."""

    def __init__(self, t, stream):
        if not t.is_cuda:
            raise ValueError("tensors must be CUDA tensors")
        self.device = t.device
        self.stream = stream
        self.inner = []
        if t.device.index != torch.cuda.current_device():
            self.inner.append(torch.cuda.device(t.device))
        if stream is not None:
            if stream.device != t.device:
                raise ValueError(f"stream is on {stream.device}, the tensors on {t.device}")
            self.inner.append(torch.cuda.stream(stream))

    def __enter__(self):
        for c in self.inner:
            c.__enter__()
        s = self.stream if self.stream is not None else torch.cuda.current_stream()
        self.handle = ctypes.c_void_p(s.cuda_stream)
        return self

    def __exit__(self, *exc):
        for c in reversed(self.inner):
            c.__exit__(*exc)

    def need(self, t, name, dtype=None, shape=None):
        if t is not None:
            _req(t, name, dtype, shape)
            if t.device != self.device:
                raise ValueError(f"{name} is on {t.device}, expected {self.device}")

    def out(self, t, name, dtype, shape):
        """The caller's output tensor, checked, or a new one."""
        if t is None:
            return torch.empty(shape, dtype=dtype, device=self.device)
        self.need(t, name, dtype, shape)
        return t

    def workspace(self, t, need):
        """(tensor, bytes) of the caller's workspace or of a new one; (None, 0) for no bytes."""
        if t is None:
            if need == 0:
                return None, 0
            t = torch.empty(need, dtype=torch.uint8, device=self.device)
        self.need(t, "workspace")
        return t, t.numel() * t.element_size()


def _silu_flag(activation):
    if activation not in (None, "silu"):
        raise ValueError(f"activation must be 'silu' or None, got {activation!r}")
    return int(activation == "silu")


def _conv_dims(x, weight, lead):
    """(leading sizes, C, W) of a convolution's input [*lead, ...channels] and filters [C, W]."""
    if x.dim() < lead + 1:
        raise ValueError(f"x has shape {tuple(x.shape)}, expected {lead} leading sizes and channels")
    if weight.dim() != 2:
        raise ValueError(f"weight has shape {tuple(weight.shape)}, expected [C, W]")
    head, tail = x.shape[:lead], x.shape[lead:]
    return head, tail.numel(), weight.shape[1]


def osdn_conv_fwd(x, weight, bias=None, state0=None, activation: Optional[str] = "silu",
                  cu_seqlens=None, y=None, stateT=None, return_state: bool = True, stream=None):
    """Short causal convolution over each channel's last W tokens: returns ``(y, stateT)``
    (``stateT`` None when ``return_state`` is False).  x: [B, T, C], or [B, T, H, D] with
    C = H * D (q, k or v as the mixer takes them); weight: [C, W] float32, W in 2..4; bias: [C]
    float32; state0, stateT: [N, W - 1, C] in x's dtype, the last inputs, oldest first;
    activation: "silu" or None."""
    with _On(x, stream) as on:
        (B, T), C, W = _conv_dims(x, weight, 2)
        io = _io(x)
        on.need(x, "x")
        on.need(weight, "weight", torch.float32, (C, W))
        on.need(bias, "bias", torch.float32, (C,))
        on.need(cu_seqlens, "cu_seqlens", torch.int32)
        num_seqs, N = _seqs(cu_seqlens, B)
        on.need(state0, "state0", x.dtype, (N, W - 1, C))
        y = on.out(y, "y", x.dtype, x.shape)
        if stateT is not None or return_state:
            stateT = on.out(stateT, "stateT", x.dtype, (N, W - 1, C))
        _check(LIB.osdn_conv_fwd(_p(x), _p(weight), _p(bias), _p(state0), _silu_flag(activation),
                                 _p(y), _p(stateT), _p(cu_seqlens), num_seqs, B, T, C, W, io,
                                 on.handle), "osdn_conv_fwd")
    return y, stateT


def osdn_conv_step(x, weight, state, bias=None, activation: Optional[str] = "silu", y=None,
                   stream=None):
    """One token per sequence of :func:`osdn_conv_fwd`: x [N, C] (or [N, H, D]); state
    [N, W - 1, C] in x's dtype, moved on by one token in place.  Returns y of x's shape."""
    with _On(x, stream) as on:
        (N,), C, W = _conv_dims(x, weight, 1)
        io = _io(x)
        on.need(x, "x")
        on.need(weight, "weight", torch.float32, (C, W))
        on.need(bias, "bias", torch.float32, (C,))
        if state is None:
            raise ValueError("state is required")
        on.need(state, "state", x.dtype, (N, W - 1, C))
        y = on.out(y, "y", x.dtype, x.shape)
        _check(LIB.osdn_conv_step(_p(x), _p(weight), _p(bias), _p(state), _silu_flag(activation),
                                  _p(y), N, C, W, io, on.handle), "osdn_conv_step")
    return y


def osdn_conv_bwd(x, weight, dy, bias=None, state0=None, dstateT=None,
                  activation: Optional[str] = "silu", cu_seqlens=None, workspace=None,
                  stream=None):
    """Gradients of :func:`osdn_conv_fwd` given dy (x's shape; x's dtype or float32, as
    :func:`osdn_bwd` returns for q, k and v) and optionally dstateT [N, W - 1, C] float32.
    Returns a dict: dx in x's dtype; dweight, dbias (None without bias) and dstate0 (None without
    state0) in float32."""
    with _On(x, stream) as on:
        (B, T), C, W = _conv_dims(x, weight, 2)
        io = _io(x)
        on.need(x, "x")
        on.need(weight, "weight", torch.float32, (C, W))
        on.need(bias, "bias", torch.float32, (C,))
        on.need(dy, "dy", None, x.shape)
        if dy.dtype not in (x.dtype, torch.float32):
            raise TypeError(f"dy must be {x.dtype} or torch.float32, got {dy.dtype}")
        on.need(cu_seqlens, "cu_seqlens", torch.int32)
        num_seqs, N = _seqs(cu_seqlens, B)
        on.need(state0, "state0", x.dtype, (N, W - 1, C))
        on.need(dstateT, "dstateT", torch.float32, (N, W - 1, C))
        f32 = dict(dtype=torch.float32, device=x.device)
        g = {"dx": torch.empty_like(x), "dweight": torch.empty((C, W), **f32),
             "dbias": None if bias is None else torch.empty((C,), **f32),
             "dstate0": None if state0 is None else torch.empty((N, W - 1, C), **f32)}
        ws, ws_bytes = on.workspace(workspace, LIB.osdn_conv_bwd_workspace_bytes(B, T, C, W))
        _check(LIB.osdn_conv_bwd(_p(x), _p(weight), _p(bias), _p(state0), _silu_flag(activation),
                                 _p(dy), _io(dy), _p(dstateT), _p(g["dx"]), _p(g["dweight"]),
                                 _p(g["dbias"]), _p(g["dstate0"]), _p(cu_seqlens), num_seqs, B, T,
                                 C, W, io, _p(ws), ws_bytes, on.handle), "osdn_conv_bwd")
    return g


def _ssm_check(on, x, dt, A, b, c, D, dt_bias, lead):
    """Checks the scan's common inputs; returns (H, G, Dk, Dv)."""
    H, Dv = x.shape[-2:]
    G, Dk = b.shape[-2:]
    on.need(x, "x", None, (*lead, H, Dv))
    on.need(b, "b", x.dtype, (*lead, G, Dk))
    on.need(c, "c", x.dtype, (*lead, G, Dk))
    on.need(dt, "dt", torch.float32, (*lead, H))
    for name, t in (("A", A), ("D", D), ("dt_bias", dt_bias)):
        on.need(t, name, torch.float32, (H,))
    return H, G, Dk, Dv


def osdn_ssm_fwd_workspace_bytes(B: int, T: int, H: int, Dk: int, Dv: int, dtype=torch.bfloat16,
                                 num_seqs: int = 0) -> int:
    io = OSDN_BF16 if dtype == torch.bfloat16 else OSDN_F32
    return int(LIB.osdn_ssm_fwd_workspace_bytes(num_seqs, B, T, H, Dk, Dv, io))


def osdn_ssm_fwd(x, dt, A, b, c, D=None, dt_bias=None, softplus: bool = True, S0=None,
                 cu_seqlens=None, y=None, ST=None, workspace=None, return_ST: bool = True,
                 stream=None):
    """Selective state-space scan: S_t = exp(step_t A) S_{t-1} + step_t x_t b_t^T and
    y_t = S_t c_t + D x_t with step = softplus(dt + dt_bias) (softplus False: dt + dt_bias).
    x: [B, T, H, Dv]; b, c: [B, T, G, Dk], shared by H / G heads each; dt: [B, T, H] float32;
    A, D, dt_bias: [H] float32; S0, ST: [N, H, Dv, Dk] float32, the mixer's state layout.
    Returns ``(y, ST)`` (``ST`` None when ``return_ST`` is False)."""
    with _On(x, stream) as on:
        B, T = x.shape[:2]
        H, G, Dk, Dv = _ssm_check(on, x, dt, A, b, c, D, dt_bias, (B, T))
        io = _io(x)
        on.need(cu_seqlens, "cu_seqlens", torch.int32)
        num_seqs, N = _seqs(cu_seqlens, B)
        on.need(S0, "S0", torch.float32, (N, H, Dv, Dk))
        y = on.out(y, "y", x.dtype, x.shape)
        if ST is not None or return_ST:
            ST = on.out(ST, "ST", torch.float32, (N, H, Dv, Dk))
        ws, ws_bytes = on.workspace(
            workspace, LIB.osdn_ssm_fwd_workspace_bytes(num_seqs, B, T, H, Dk, Dv, io))
        _check(LIB.osdn_ssm_fwd(_p(x), _p(dt), _p(A), _p(b), _p(c), _p(D), _p(dt_bias),
                                int(softplus), _p(S0), _p(y), _p(ST), _p(cu_seqlens), num_seqs, B,
                                T, H, G, Dk, Dv, io, _p(ws), ws_bytes, on.handle), "osdn_ssm_fwd")
    return y, ST


def osdn_ssm_step(x, dt, A, b, c, S, D=None, dt_bias=None, softplus: bool = True, y=None,
                  stream=None):
    """One token per sequence of :func:`osdn_ssm_fwd` (the decode path): x [N, H, Dv]; b, c
    [N, G, Dk]; dt [N, H] float32; S [N, H, Dv, Dk] float32, updated in place.  Returns y."""
    with _On(x, stream) as on:
        N = x.shape[0]
        H, G, Dk, Dv = _ssm_check(on, x, dt, A, b, c, D, dt_bias, (N,))
        io = _io(x)
        if S is None:
            raise ValueError("S is required")
        on.need(S, "S", torch.float32, (N, H, Dv, Dk))
        y = on.out(y, "y", x.dtype, x.shape)
        _check(LIB.osdn_ssm_step(_p(x), _p(dt), _p(A), _p(b), _p(c), _p(D), _p(dt_bias),
                                 int(softplus), _p(S), _p(y), N, H, G, Dk, Dv, io, on.handle),
               "osdn_ssm_step")
    return y


def osdn_ssm_bwd(x, dt, A, b, c, dy, D=None, dt_bias=None, softplus: bool = True, S0=None,
                 dST=None, cu_seqlens=None, workspace=None, stream=None):
    """Gradients of :func:`osdn_ssm_fwd` given dy (x's shape and dtype) and optionally dST.
    Returns a dict: dx, db, dc in x's dtype; ddt, dA, dD, ddt_bias and dS0 in float32 (the last
    three None where their input is)."""
    with _On(x, stream) as on:
        B, T = x.shape[:2]
        H, G, Dk, Dv = _ssm_check(on, x, dt, A, b, c, D, dt_bias, (B, T))
        io = _io(x)
        on.need(dy, "dy", x.dtype, x.shape)
        on.need(cu_seqlens, "cu_seqlens", torch.int32)
        num_seqs, N = _seqs(cu_seqlens, B)
        on.need(S0, "S0", torch.float32, (N, H, Dv, Dk))
        on.need(dST, "dST", torch.float32, (N, H, Dv, Dk))

        def like(t):
            return None if t is None else torch.empty_like(t)

        g = {"dx": like(x), "ddt": like(dt), "dA": like(A), "db": like(b), "dc": like(c),
             "dD": like(D), "ddt_bias": like(dt_bias), "dS0": like(S0)}
        ws, ws_bytes = on.workspace(
            workspace, LIB.osdn_ssm_bwd_workspace_bytes(num_seqs, B, T, H, Dk, Dv, io))
        _check(LIB.osdn_ssm_bwd(_p(x), _p(dt), _p(A), _p(b), _p(c), _p(D), _p(dt_bias),
                                int(softplus), _p(S0), _p(dy), _p(dST), _p(g["dx"]), _p(g["ddt"]),
                                _p(g["dA"]), _p(g["db"]), _p(g["dc"]), _p(g["dD"]),
                                _p(g["ddt_bias"]), _p(g["dS0"]), _p(cu_seqlens), num_seqs, B, T, H,
                                G, Dk, Dv, io, _p(ws), ws_bytes, on.handle), "osdn_ssm_bwd")
    return g


def _gate_act(gate_act):
    if gate_act not in ("silu", "sigmoid"):
        raise ValueError(f"gate_act must be 'silu' or 'sigmoid', got {gate_act!r}")
    return int(gate_act == "sigmoid")


def _norm_check(on, f, x, gate, w_post, w_next):
    """Checks the norm's common inputs; returns (R, D)."""
    D = f.shape[-1]
    on.need(f, "f")
    for name, t in (("x", x), ("gate", gate)):
        on.need(t, name, f.dtype, f.shape)
    for name, t in (("w_post", w_post), ("w_next", w_next)):
        on.need(t, name, torch.float32, (D,))
    return (f.numel() // D if D else 0), D


def osdn_norm_fwd(f, x=None, gate=None, w_post=None, w_next=None, gate_act: str = "silu",
                  gate_first: bool = False, scale: float = 1.0, eps: float = 1e-5, x_out=None,
                  h=None, return_x_out: bool = True, stream=None):
    """Block norm over the last dimension of f: u = rmsnorm(f) * w_post * act(gate) (gate_first:
    rmsnorm(f * act(gate)) * w_post), x_out = x + scale * u, h = rmsnorm(x_out) * w_next.  Every
    part is optional: w_post, gate, x (no residual), w_next (h is None then).  x, gate: f's shape
    and dtype; w_post, w_next: [D] float32.  Returns ``(x_out, h)``; ``return_x_out`` False (with
    w_next) skips x_out."""
    with _On(f, stream) as on:
        R, D = _norm_check(on, f, x, gate, w_post, w_next)
        io = _io(f)
        if x_out is not None or return_x_out or w_next is None:
            x_out = on.out(x_out, "x_out", f.dtype, f.shape)
        if w_next is not None:
            h = on.out(h, "h", f.dtype, f.shape)
        elif h is not None:
            raise ValueError("h needs w_next")
        _check(LIB.osdn_norm_fwd(_p(f), _p(x), _p(gate), _p(w_post), _p(w_next),
                                 _gate_act(gate_act), int(gate_first), float(scale), float(eps),
                                 _p(x_out), _p(h), R, D, io, on.handle), "osdn_norm_fwd")
    return x_out, h


def osdn_norm_bwd(f, dx_out=None, dh=None, x=None, gate=None, w_post=None, w_next=None,
                  gate_act: str = "silu", gate_first: bool = False, scale: float = 1.0,
                  eps: float = 1e-5, workspace=None, stream=None):
    """Gradients of :func:`osdn_norm_fwd` from its inputs, given dx_out (or None for 0) and dh
    (exactly when w_next is given).  Returns a dict: df, dx, dgate in f's dtype, dw_post, dw_next
    in float32; None where the input is."""
    with _On(f, stream) as on:
        R, D = _norm_check(on, f, x, gate, w_post, w_next)
        io = _io(f)
        for name, t in (("dx_out", dx_out), ("dh", dh)):
            on.need(t, name, f.dtype, f.shape)
        if (dh is None) != (w_next is None):
            raise ValueError("dh is given exactly when w_next is")
        if dh is None and dx_out is None:
            raise ValueError("dx_out or dh is required")

        def like(t):
            return None if t is None else torch.empty_like(t)

        g = {"df": like(f), "dx": like(x), "dgate": like(gate), "dw_post": like(w_post),
             "dw_next": like(w_next)}
        ws, ws_bytes = on.workspace(workspace, LIB.osdn_norm_bwd_workspace_bytes(R, D))
        _check(LIB.osdn_norm_bwd(_p(f), _p(x), _p(gate), _p(w_post), _p(w_next),
                                 _gate_act(gate_act), int(gate_first), float(scale), float(eps),
                                 _p(dx_out), _p(dh), _p(g["df"]), _p(g["dx"]), _p(g["dgate"]),
                                 _p(g["dw_post"]), _p(g["dw_next"]), R, D, io, _p(ws), ws_bytes,
                                 on.handle), "osdn_norm_bwd")
    return g


def osdn_get_device_status(stream=None) -> int:
    """Synchronize the stream and return (and clear) the device status word."""
    return int(LIB.osdn_get_device_status(_stream(stream)))


def osdn_debug_watchdog_selftest(spin_limit: int, stream=None):
    _check(LIB.osdn_debug_watchdog_selftest(int(spin_limit), _stream(stream)),
           "osdn_debug_watchdog_selftest")
