"""Binding of a hybrid's training and residual operators of libgdn.so (the C ABI
in include/gdn_hybrid.h): argument marshalling only, by the extension module
that attn.py loads; what it refuses raises ValueError, and where there is no
memory for outputs that it allocates, torch.OutOfMemoryError.

Tensors of a call are on one device, which need not be the current one; work
goes to that device's current stream, or to the one given.
"""
from __future__ import annotations

import contextlib
import ctypes

import torch
from torch._C import _cuda_getCurrentRawStream

from .attn import GdnAttnPrefillDesc, _native
from .gdn import _DT, GDN_OK, GdnError, lib

HYBRID_ABI_VERSION = 1
_i64, _i32, _f32, _vp = ctypes.c_int64, ctypes.c_int32, ctypes.c_float, ctypes.c_void_p


class GdnAttnBwdDesc(ctypes.Structure):
    _fields_ = [("N", _i64), ("total_T", _i64), ("ld_q", _i64), ("ld_k", _i64), ("ld_v", _i64),
                ("ld_dq", _i64), ("ld_dk", _i64), ("ld_dv", _i64), ("window", _i64),
                ("H_q", _i32), ("H_k", _i32), ("d", _i32), ("io_dtype", _i32), ("grad_dtype", _i32),
                ("scale", _f32)]


class GdnQkBwdDesc(ctypes.Structure):
    _fields_ = [("rows", _i64), ("ld_q", _i64), ("ld_k", _i64), ("ld_dq", _i64), ("ld_dk", _i64),
                ("H_q", _i32), ("H_k", _i32), ("d", _i32), ("rope_dim", _i32), ("rope_mode", _i32),
                ("io_dtype", _i32), ("grad_dtype", _i32), ("rope_scale", _f32), ("eps", _f32)]


class GdnAddNormDesc(ctypes.Structure):
    _fields_ = [("rows", _i64), ("ld_x", _i64), ("C", _i32), ("io_dtype", _i32),
                ("res_dtype", _i32), ("group", _i32), ("eps", _f32)]


class GdnAddNormBwdDesc(ctypes.Structure):
    _fields_ = [("rows", _i64), ("ld_dx", _i64), ("C", _i32), ("io_dtype", _i32),
                ("res_dtype", _i32), ("eps", _f32)]


# Entry points: pointers behind the descriptor, with a workspace's bytes before the last `behind` of them.
_CALLS = {"gdn_attn_prefill_save": (GdnAttnPrefillDesc, 6, None), "gdn_attn_backward": (GdnAttnBwdDesc, 11, 3),
          "gdn_qk_norm_rope_backward": (GdnQkBwdDesc, 13, 4), "gdn_add_norm": (GdnAddNormDesc, 6, None),
          "gdn_add_norm_backward": (GdnAddNormBwdDesc, 8, 3)}

# Addresses of the C functions that the calls below run.
_fn = {}


def _use(lib) -> None:
    """Declares the entry points of a loaded library and runs them from now on."""
    for name, (desc, n, behind) in _CALLS.items():
        f = getattr(lib, name)
        args = [_vp] * n if behind is None else [_vp] * (n - behind) + [ctypes.c_size_t] + [_vp] * behind
        f.argtypes = [ctypes.POINTER(desc)] + args + [_vp]
        f.restype = ctypes.c_int
        _fn[name] = ctypes.cast(f, _vp).value
        if behind is not None:
            size = getattr(lib, name + "_workspace_size")
            size.argtypes, size.restype = [ctypes.POINTER(desc)], ctypes.c_size_t
            _fn[name + "_workspace_size"] = ctypes.cast(size, _vp).value
    lib.gdn_hybrid_abi_version.argtypes = []
    lib.gdn_hybrid_abi_version.restype = ctypes.c_int
    if lib.gdn_hybrid_abi_version() != HYBRID_ABI_VERSION:
        raise ImportError("libgdn.so hybrid ABI version mismatch")


_use(lib)


def hybrid_abi_version() -> int:
    return lib.gdn_hybrid_abi_version()


def _done(r, name):
    """The outputs of a call that answers (status, outputs ...)."""
    if r[0] != GDN_OK:
        raise GdnError(r[0], name)
    return r[1:]


# The extension module checks the tensors and allocates what is not given, for the current stream of their
# device: a call on another stream is the same call with that one as the current stream.


def _current(t) -> int:
    """The current stream's handle on the device of t (what is no device tensor is refused by the call)."""
    dev = t.get_device() if isinstance(t, torch.Tensor) else -1
    return _cuda_getCurrentRawStream(dev) if dev >= 0 else 0


def _on(stream, t):
    """With it the stream, or the one of this handle on the device of t, is the current one there."""
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        return contextlib.nullcontext()       # (refused by the call)
    if not isinstance(stream, torch.cuda.Stream):
        stream = torch.cuda.ExternalStream(int(stream), device=t.device)
    elif stream.device != t.device:
        raise ValueError("stream is on another device than the tensors")
    return torch.cuda.stream(stream)


def gdn_attn_prefill_save(q, k, v, cu_seqlens=None, N=None, window: int = 0, scale=None, o=None,
                          stats=None, stream=None):
    """gdn_attn_prefill that also leaves the statistics gdn_attn_backward needs
    (see include/gdn_hybrid.h).  Returns (o, stats).

    Arguments as gdn_attn_prefill; stats, float32 of total_T * H_q * 2 elements
    (bfloat16 rows: total_T * H_q * (2 + d / 4)), is allocated when not given, as
    o is.
    """
    if stream is not None:
        with _on(stream, q):
            return gdn_attn_prefill_save(q, k, v, cu_seqlens, N, window, scale, o, stats)
    return _done(_native.attn_prefill_save(_fn["gdn_attn_prefill_save"], q, k, v, cu_seqlens, N, window,
                                           scale, o, stats, _current(q)), "gdn_attn_prefill_save")


def gdn_attn_backward_workspace_size(q, k, N: int = 1, window: int = 0) -> int:
    """Workspace bytes gdn_attn_backward needs for q and k of these shapes."""
    T, Hq, d = q.shape
    Hk = k.shape[1]
    if q.dtype not in _DT:
        raise ValueError("q must be float32 or bfloat16")
    io = _DT[q.dtype]
    desc = GdnAttnBwdDesc(N, T, Hq * d, Hk * d, Hk * d, Hq * d, Hk * d, Hk * d, window, Hq, Hk, d, io, io, 1.0)
    return int(lib.gdn_attn_backward_workspace_size(ctypes.byref(desc)))


def gdn_attn_backward(q, k, v, o, d_o, stats, cu_seqlens=None, N=None, window: int = 0, scale=None,
                      dq=None, dk=None, dv=None, grad_dtype=None, workspace=None, stream=None):
    """Gradients of causal attention (see include/gdn_hybrid.h).  Returns (dq, dk, dv).

    q, k, v, cu_seqlens, N, window, scale as for gdn_attn_prefill_save; o and
    stats are what that returned, d_o the upstream gradient (dense, of q's
    type).  dq, dk, dv [total_T, H, d] may be column blocks of one buffer; those
    not given are allocated in grad_dtype (that of q unless given; all are of one
    type, that of q or float32).  `workspace` is a device uint8 tensor of at
    least gdn_attn_backward_workspace_size(...) bytes, allocated when not given.
    """
    if stream is not None:
        with _on(stream, q):
            return gdn_attn_backward(q, k, v, o, d_o, stats, cu_seqlens, N, window, scale, dq, dk, dv, grad_dtype, workspace)
    if grad_dtype is None:
        grad_dtype = getattr(next((t for t in (dq, dk, dv) if t is not None), q), "dtype", None)
    if grad_dtype is not None and grad_dtype not in _DT:      # (without one, what is no tensor is refused by the call)
        raise ValueError("gradients must be float32 or bfloat16")
    return _done(_native.attn_backward(_fn["gdn_attn_backward"], _fn["gdn_attn_backward_workspace_size"],
                                       q, k, v, o, d_o, stats, cu_seqlens, N, window, scale, dq, dk, dv,
                                       grad_dtype == torch.float32, workspace, _current(q)),
                 "gdn_attn_backward")


def gdn_qk_norm_rope_backward_workspace_size(dq=None, dk=None) -> int:
    """Workspace bytes gdn_qk_norm_rope_backward needs for dq and dk of these shapes."""
    one = dk if dq is None else dq
    if one is None or one.dtype not in _DT:
        raise ValueError("dq or dk must be given, float32 or bfloat16")
    rows, _, d = one.shape
    Hq, Hk = (0 if t is None else t.shape[1] for t in (dq, dk))
    desc = GdnQkBwdDesc(rows, Hq * d, Hk * d, Hq * d, Hk * d, Hq, Hk, d, 0, 0, _DT[one.dtype], _DT[one.dtype], 1.0, 0.0)
    return int(lib.gdn_qk_norm_rope_backward_workspace_size(ctypes.byref(desc)))


def gdn_qk_norm_rope_backward(dq, dk, q_raw=None, k_raw=None, positions=None, inv_freq=None,
                              q_weight=None, k_weight=None, interleaved: bool = False,
                              rope_scale: float = 1.0, eps: float = 1e-6, dq_raw=None, dk_raw=None,
                              dq_weight=None, dk_weight=None, workspace=None, stream=None):
    """Gradient of gdn_qk_norm_rope (see include/gdn_hybrid.h).  Returns (dq_raw,
    dk_raw, dq_weight, dk_weight).

    dq [rows, H_q, d], dk [rows, H_k, d], dense, of the raw rows' type or float32
    (either may be None); the other inputs as for gdn_qk_norm_rope (raw rows are
    needed where there is a weight).  dq_raw, dk_raw, of dq's and dk's type, may be
    column blocks of one buffer, or dq, dk themselves, and are allocated when not
    given, as the weights' gradients (fp32 [d]; None without a weight) and the
    workspace are.
    """
    one = dk if dq is None else dq
    if one is None:
        raise ValueError("dq or dk must be given")
    if stream is not None:
        with _on(stream, one):
            return gdn_qk_norm_rope_backward(dq, dk, q_raw, k_raw, positions, inv_freq, q_weight, k_weight, interleaved,
                                             rope_scale, eps, dq_raw, dk_raw, dq_weight, dk_weight, workspace)
    return _done(_native.qk_norm_rope_backward(
        _fn["gdn_qk_norm_rope_backward"], _fn["gdn_qk_norm_rope_backward_workspace_size"], dq, dk, q_raw, k_raw,
        positions, inv_freq, q_weight, k_weight, interleaved, rope_scale, eps, dq_raw, dk_raw, dq_weight,
        dk_weight, workspace, _current(one)), "gdn_qk_norm_rope_backward")


def gdn_add_norm(x, res=None, weight=None, eps: float = 1e-6, group=None, res_out=None, y=None,
                 y_scale=None, stream=None):
    """The residual's addition and the RMS norm behind it (see
    include/gdn_hybrid.h).  Returns (y, y_scale, res_out).

    x [rows, C] (a column block is fine); res [rows, C], of x's type or float32,
    or None; weight fp32 [C] or None.  group None: y has x's type and y_scale is
    None; 0: y is float8_e4m3fn with one scale for a row, 32, 64 or 128: with a
    scale for so many channels (y_scale fp32 [rows, scales of a row]).  y, y_scale
    and, with a res, res_out are allocated when not given; res_out may be res, and
    y may be a dense x.
    """
    if stream is not None:
        with _on(stream, x):
            return gdn_add_norm(x, res, weight, eps, group, res_out, y, y_scale)
    return _done(_native.add_norm(_fn["gdn_add_norm"], x, res, weight, eps, group, res_out, y, y_scale,
                                  _current(x)), "gdn_add_norm")


def gdn_add_norm_backward_workspace_size(dy) -> int:
    """Workspace bytes gdn_add_norm_backward needs for dy of this shape."""
    if dy.dtype not in _DT:
        raise ValueError("dy must be float32 or bfloat16")
    rows, C = dy.shape
    desc = GdnAddNormBwdDesc(rows, C, C, _DT[dy.dtype], _DT[dy.dtype], 0.0)
    return int(lib.gdn_add_norm_backward_workspace_size(ctypes.byref(desc)))


def gdn_add_norm_backward(dy, r, weight=None, d_res_out=None, eps: float = 1e-6, dx=None,
                          d_res=None, d_weight=None, workspace=None, stream=None):
    """Gradient of gdn_add_norm (see include/gdn_hybrid.h).  Returns (dx, d_res,
    d_weight).

    dy [rows, C], dense; r [rows, C], of dy's type or float32: the sum that
    gdn_add_norm left in res_out (or its x, without a res); d_res_out like r, the
    upstream gradient of that sum, or None.  dx has dy's type, d_res that of r;
    where the types are one and dx is not given, dx is d_res.  What is not given
    is allocated (d_weight only with a weight); dx may be dy, d_res may be d_res_out.
    """
    if stream is not None:
        with _on(stream, dy):
            return gdn_add_norm_backward(dy, r, weight, d_res_out, eps, dx, d_res, d_weight, workspace)
    return _done(_native.add_norm_backward(
        _fn["gdn_add_norm_backward"], _fn["gdn_add_norm_backward_workspace_size"], dy, r, weight, d_res_out, eps,
        dx, d_res, d_weight, workspace, _current(dy)), "gdn_add_norm_backward")
