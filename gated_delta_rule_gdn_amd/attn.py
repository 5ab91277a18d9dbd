"""Binding of the attention operators of libgdn.so (the C ABI in
include/gdn_attn.h): argument marshalling only, as in gdn.py.  The tensors are
checked and handed over by the extension module _attn_native (csrc/
attn_bind.cpp); what it refuses raises ValueError.

Tensors of a call are on one device, which need not be the current one; work
goes to that device's current stream, or to the one given.
"""
from __future__ import annotations

import ctypes

import torch
from torch._C import _cuda_getCurrentRawStream

from .gdn import _DT, GDN_OK, GdnError, lib


class _Missing:
    """In place of an extension module that does not load: the attention calls raise,
    the rest of the package needs nothing of it."""

    def __init__(self, why):
        self.why = why

    def __getattr__(self, name):
        raise ImportError(f"the extension module _attn_native is missing or does not load ({self.why}): build it "
                          "with `python gated_delta_rule_gdn_amd/build.py`")


def _load_native():
    # the file's name holds the Python that it is for, the module the torch
    try:
        from . import _attn_native as native
    except ImportError as e:
        return _Missing(e)
    here = torch.__version__.split("+")[0]
    return native if native.torch_version == here else _Missing(f"built for torch {native.torch_version}, this is {here}")


_native = _load_native()

GDN_ROPE_HALF, GDN_ROPE_INTERLEAVED = 0, 1
ATTN_ABI_VERSION = 1
_i64, _i32, _f32, _vp = ctypes.c_int64, ctypes.c_int32, ctypes.c_float, ctypes.c_void_p


class GdnQkDesc(ctypes.Structure):
    _fields_ = [("rows", _i64), ("ld_q", _i64), ("ld_k", _i64), ("H_q", _i32), ("H_k", _i32),
                ("d", _i32), ("rope_dim", _i32), ("rope_mode", _i32), ("io_dtype", _i32),
                ("rope_scale", _f32), ("eps", _f32)]


class GdnKvAppendDesc(ctypes.Structure):
    _fields_ = [("N", _i64), ("total_T", _i64), ("ld_k", _i64), ("ld_v", _i64),
                ("num_pages", _i64), ("max_pages", _i64), ("H_k", _i32), ("d", _i32),
                ("page_size", _i32), ("rope_dim", _i32), ("rope_mode", _i32), ("io_dtype", _i32),
                ("rope_scale", _f32), ("eps", _f32)]


class GdnAttnPrefillDesc(ctypes.Structure):
    _fields_ = [("N", _i64), ("total_T", _i64), ("ld_q", _i64), ("ld_k", _i64), ("ld_v", _i64),
                ("window", _i64), ("H_q", _i32), ("H_k", _i32), ("d", _i32), ("io_dtype", _i32),
                ("scale", _f32)]


class GdnAttnDecodeDesc(ctypes.Structure):
    _fields_ = [("N", _i64), ("num_pages", _i64), ("max_pages", _i64), ("window", _i64),
                ("H_q", _i32), ("H_k", _i32), ("d", _i32), ("page_size", _i32),
                ("io_dtype", _i32), ("scale", _f32)]


# Addresses of the C functions that the calls below run.
_fn = {}


def _use(lib) -> None:
    """Declares the attention entry points of a loaded library and runs them from now on."""
    P = ctypes.POINTER
    lib.gdn_qk_norm_rope.argtypes = [P(GdnQkDesc)] + [_vp] * 9
    lib.gdn_kv_append.argtypes = [P(GdnKvAppendDesc)] + [_vp] * 12
    lib.gdn_attn_prefill.argtypes = [P(GdnAttnPrefillDesc)] + [_vp] * 6
    lib.gdn_attn_decode.argtypes = [P(GdnAttnDecodeDesc)] + [_vp] * 9 + [ctypes.c_size_t, _vp]
    lib.gdn_attn_decode_workspace_size.argtypes = [P(GdnAttnDecodeDesc)]
    lib.gdn_attn_decode_workspace_size.restype = ctypes.c_size_t
    lib.gdn_attn_abi_version.argtypes = []
    for name in ("gdn_qk_norm_rope", "gdn_kv_append", "gdn_attn_prefill", "gdn_attn_decode",
                 "gdn_attn_abi_version"):
        getattr(lib, name).restype = ctypes.c_int
    if lib.gdn_attn_abi_version() != ATTN_ABI_VERSION:
        raise ImportError("libgdn.so attention ABI version mismatch")
    for name in ("gdn_qk_norm_rope", "gdn_kv_append", "gdn_attn_prefill", "gdn_attn_decode",
                 "gdn_attn_decode_workspace_size"):
        _fn[name] = ctypes.cast(getattr(lib, name), _vp).value


_use(lib)


def attn_abi_version() -> int:
    return lib.gdn_attn_abi_version()


def _raw_stream(stream, t) -> int:
    if stream is None:
        dev = t.get_device()
        return _cuda_getCurrentRawStream(dev) if dev >= 0 else 0   # (a host tensor is refused)
    if isinstance(stream, torch.cuda.Stream):
        if stream.device.index != t.get_device():
            raise ValueError("stream is on another device than the tensors")
        return stream.cuda_stream
    return int(stream)


def _empty(shape, dtype, like, stream):
    """An output or workspace that belongs to the stream of the call."""
    device = like.device
    if device.type != "cuda":
        raise ValueError("the tensors of a call must be device tensors")
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=device)
    if not isinstance(stream, torch.cuda.Stream):
        stream = torch.cuda.ExternalStream(int(stream), device=device)
    with torch.cuda.stream(stream):
        return torch.empty(shape, dtype=dtype, device=device)


def gdn_qk_norm_rope(q_raw, k_raw=None, positions=None, inv_freq=None, q_weight=None,
                     k_weight=None, interleaved: bool = False, rope_scale: float = 1.0,
                     eps: float = 1e-6, q=None, k=None, stream=None):
    """RMS norm of each query and key head and the rotary position in one pass
    (see include/gdn_attn.h).  Returns (q, k).

    q_raw [rows, H_q, d], k_raw [rows, H_k, d] (either may be None; column
    blocks of a projection output are fine); positions int64 [rows] and
    inv_freq fp32 [rope_dim / 2], or both None (no rotation); weights fp32 [d]
    or None (that operand is not normed).  q, k are dense, allocated when not
    given, and may be q_raw, k_raw where those are dense.
    """
    one = k_raw if q_raw is None else q_raw
    if one is None:
        raise ValueError("q_raw or k_raw must be given")
    if q is None and q_raw is not None:
        q = _empty(q_raw.shape, q_raw.dtype, q_raw, stream)
    if k is None and k_raw is not None:
        k = _empty(k_raw.shape, k_raw.dtype, k_raw, stream)
    st = _native.qk_norm_rope(_fn["gdn_qk_norm_rope"], q_raw, k_raw, positions, inv_freq, q_weight,
                              k_weight, interleaved, rope_scale, eps, q, k,
                              _raw_stream(stream, one))
    if st != GDN_OK:
        raise GdnError(st, "gdn_qk_norm_rope")
    return q, k


def gdn_kv_append(k_raw, v_raw, k_cache, v_cache, k_scale, v_scale, page_table, seq_lens,
                  cu_seqlens=None, inv_freq=None, k_weight=None, interleaved: bool = False,
                  rope_scale: float = 1.0, eps: float = 1e-6, stream=None) -> None:
    """New keys (normed and rotated) and values into a paged cache of 8-bit
    floats, in place (see include/gdn_attn.h).

    k_raw, v_raw [total_T, H_k, d] (column blocks are fine); k_cache, v_cache
    float8_e4m3fn [num_pages, H_k, page_size, d]; k_scale, v_scale fp32
    [num_pages, H_k]; page_table int32 [N, max_pages]; seq_lens int64 [N], the
    tokens held before the call (not changed); cu_seqlens int64 [N + 1] or
    None for total_T / N new tokens each.
    """
    st = _native.kv_append(_fn["gdn_kv_append"], k_raw, v_raw, k_cache, v_cache, k_scale, v_scale,
                           page_table, seq_lens, cu_seqlens, inv_freq, k_weight, interleaved,
                           rope_scale, eps, _raw_stream(stream, k_raw))
    if st != GDN_OK:
        raise GdnError(st, "gdn_kv_append")


def gdn_attn_prefill(q, k, v, cu_seqlens=None, N=None, window: int = 0, scale=None, o=None,
                     stream=None):
    """Causal attention over whole prompts (see include/gdn_attn.h).  Returns o.

    q [total_T, H_q, d]; k, v [total_T, H_k, d] (column blocks are fine);
    cu_seqlens int64 [N + 1] or None for N sequences of total_T / N tokens (N
    defaults to 1); window 0 (all) or the number of tokens seen; scale
    defaults to 1 / sqrt(d).  o [total_T, H_q, d] is allocated when not given.
    """
    if o is None:
        o = _empty(q.shape, q.dtype, q, stream)
    st = _native.attn_prefill(_fn["gdn_attn_prefill"], q, k, v, cu_seqlens, N, window, scale, o,
                              _raw_stream(stream, q))
    if st != GDN_OK:
        raise GdnError(st, "gdn_attn_prefill")
    return o


def gdn_attn_decode_workspace_size(q, k_cache, page_table, window: int = 0) -> int:
    """Workspace bytes gdn_attn_decode needs for these shapes (0: none)."""
    N, Hq, d = q.shape
    pages, Hk, P = k_cache.shape[:3]
    if q.dtype not in _DT:
        raise ValueError("q must be float32 or bfloat16")
    desc = GdnAttnDecodeDesc(N, pages, page_table.shape[1], window, Hq, Hk, d, P, _DT[q.dtype], 1.0)
    return int(lib.gdn_attn_decode_workspace_size(ctypes.byref(desc)))


def gdn_attn_decode(q, k_cache, v_cache, k_scale, v_scale, page_table, seq_lens, window: int = 0,
                    scale=None, o=None, workspace=None, stream=None):
    """Attention of each sequence's newest token over its paged cache (see
    include/gdn_attn.h).  Returns o.

    q [N, H_q, d]; the cache as for gdn_kv_append; seq_lens int64 [N], the
    tokens held, the newest among them; window 0 (all) or the number of tokens
    seen; scale defaults to 1 / sqrt(d).  `workspace` is a device uint8 tensor
    of at least gdn_attn_decode_workspace_size(...) bytes; it and o are
    allocated when not given.
    """
    if o is None:
        o = _empty(q.shape, q.dtype, q, stream)
    raw = _raw_stream(stream, q)
    st = _native.attn_decode(_fn["gdn_attn_decode"], _fn["gdn_attn_decode_workspace_size"], q,
                             k_cache, v_cache, k_scale, v_scale, page_table, seq_lens, window,
                             scale, o, workspace, raw)
    if st < 0:                              # a workspace of so many bytes is needed
        workspace = _empty((-st,), torch.uint8, q, stream)
        st = _native.attn_decode(_fn["gdn_attn_decode"], _fn["gdn_attn_decode_workspace_size"], q,
                                 k_cache, v_cache, k_scale, v_scale, page_table, seq_lens, window,
                                 scale, o, workspace, raw)
    if st != GDN_OK:
        raise GdnError(st, "gdn_attn_decode")
    return o
