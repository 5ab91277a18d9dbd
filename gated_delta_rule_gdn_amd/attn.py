"""ctypes binding of the attention operators of libgdn.so (the C ABI in
include/gdn_attn.h): argument marshalling only, as in gdn.py.

Tensors of a call are on one device, which need not be the current one; work
goes to that device's current stream, or to the one given.
"""
from __future__ import annotations

import ctypes

import torch
from torch._C import _cuda_getCurrentRawStream

from .gdn import _DT, GDN_OK, GdnError, lib

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


def _declare(lib) -> None:
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


_declare(lib)


def attn_abi_version() -> int:
    return lib.gdn_attn_abi_version()


# A decode step's calls are so short that the host's share decides how fast they
# follow each other, so each tensor is checked in one expression, and what is
# wrong with it is found out only where that fails.

def _refuse(t, name, dev, shape, dtype):
    if not t.is_cuda:
        raise ValueError(f"{name} must be a device tensor")
    if t.get_device() != dev:
        raise ValueError(f"{name} must be on the same device as the other tensors")
    if t.dtype is not dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
    if t.shape != shape:
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")


def _dense(t, name, dev, shape, dtype) -> int:
    """The address of a contiguous tensor of this shape and type (None: 0)."""
    if t is None:
        return 0
    if t.get_device() != dev or t.dtype is not dtype or t.shape != shape or not t.is_contiguous():
        _refuse(t, name, dev, shape, dtype)
        raise ValueError(f"{name} must be contiguous")
    return t.data_ptr()


def _heads(t, name, dev, shape, dtype):
    """The address and row stride (elements) of a [rows, H, d] tensor whose
    rows are dense; a column block of a wider buffer is fine."""
    if t.get_device() != dev or t.dtype is not dtype or t.shape != shape:
        _refuse(t, name, dev, shape, dtype)
    rows, H, d = shape
    ld, sh, sd = t.stride()
    if (sd != 1 or (sh != d and H > 1)) and rows * H:
        raise ValueError(f"{name} must have dense rows of {H} x {d} elements")
    return t.data_ptr(), ld if rows > 1 else H * d


def _first(t, name):
    """Device, dtype and shape of the [rows, H, d] tensor that sets those of a call."""
    dev, io = t.get_device(), t.dtype
    if dev < 0 or not t.is_cuda:
        raise ValueError(f"{name} must be a device tensor")
    if io not in _DT:
        raise ValueError(f"{name} must be float32 or bfloat16")
    if t.dim() != 3:
        raise ValueError(f"{name} must have 3 dimensions (rows, heads, head size)")
    return dev, io, t.shape


def _raw_stream(stream, dev) -> int:
    if stream is None:
        return _cuda_getCurrentRawStream(dev)
    if isinstance(stream, torch.cuda.Stream):
        if stream.device.index != dev:
            raise ValueError("stream is on another device than the tensors")
        return stream.cuda_stream
    return int(stream)


def _empty(shape, dtype, dev, stream):
    """An output or workspace that belongs to the stream of the call."""
    device = torch.device("cuda", dev)
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=device)
    if not isinstance(stream, torch.cuda.Stream):
        stream = torch.cuda.ExternalStream(int(stream), device=device)
    with torch.cuda.stream(stream):
        return torch.empty(shape, dtype=dtype, device=device)


def _call(fn, name, dev, *args):
    if torch.cuda.current_device() == dev:
        st = fn(*args)
    else:
        with torch.cuda.device(dev):
            st = fn(*args)
    if st != GDN_OK:
        raise GdnError(st, name)


def _rope(inv_freq, dev):
    """rope_dim and the address of the frequencies."""
    if inv_freq is None:
        return 0, 0
    if inv_freq.dim() != 1:
        raise ValueError("inv_freq must be a 1-d tensor of rope_dim / 2 frequencies")
    p = _dense(inv_freq, "inv_freq", dev, inv_freq.shape, torch.float32)
    return 2 * inv_freq.shape[0], p


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
    one = q_raw if q_raw is not None else k_raw
    if one is None:
        raise ValueError("q_raw or k_raw must be given")
    dev, io, (rows, _, d) = _first(one, "q_raw" if one is q_raw else "k_raw")
    Hq = Hk = ld_q = ld_k = q_in = k_in = 0
    if q_raw is not None:
        shape = q_raw.shape
        Hq = shape[1]
        q_in, ld_q = _heads(q_raw, "q_raw", dev, shape, io)
        if q is None:
            q = _empty(shape, io, dev, stream)
    elif q is not None:
        raise ValueError("q without q_raw")
    if k_raw is not None:
        Hk = k_raw.shape[1] if k_raw.dim() == 3 else 0
        k_in, ld_k = _heads(k_raw, "k_raw", dev, (rows, Hk, d), io)
        if k is None:
            k = _empty((rows, Hk, d), io, dev, stream)
    elif k is not None:
        raise ValueError("k without k_raw")
    if inv_freq is not None and positions is None:
        raise ValueError("rotation needs positions")
    rope, freqs = _rope(inv_freq, dev)
    pos = _dense(positions, "positions", dev, (rows,), torch.int64)
    desc = GdnQkDesc(rows, ld_q, ld_k, Hq, Hk, d, rope,
                     GDN_ROPE_INTERLEAVED if interleaved else GDN_ROPE_HALF, _DT[io], rope_scale,
                     eps)
    _call(lib.gdn_qk_norm_rope, "gdn_qk_norm_rope", dev, ctypes.byref(desc), q_in, k_in,
          _dense(q_weight, "q_weight", dev, (d,), torch.float32),
          _dense(k_weight, "k_weight", dev, (d,), torch.float32), pos if rope else 0,
          freqs if rope else 0, _dense(q, "q", dev, (rows, Hq, d), io),
          _dense(k, "k", dev, (rows, Hk, d), io), _raw_stream(stream, dev))
    return q, k


def _cache(k_cache, v_cache, k_scale, v_scale, page_table, seq_lens, dev):
    """(shape of the cache, shape of the table, addresses) of a paged cache."""
    if k_cache.dim() != 4:
        raise ValueError("k_cache must be [num_pages, H_k, page_size, d]")
    if page_table.dim() != 2:
        raise ValueError("page_table must be [N, max_pages]")
    shape, table = k_cache.shape, page_table.shape
    scales = shape[:2]
    return shape, table, (
        _dense(k_cache, "k_cache", dev, shape, torch.float8_e4m3fn),
        _dense(v_cache, "v_cache", dev, shape, torch.float8_e4m3fn),
        _dense(k_scale, "k_scale", dev, scales, torch.float32),
        _dense(v_scale, "v_scale", dev, scales, torch.float32),
        _dense(page_table, "page_table", dev, table, torch.int32),
        _dense(seq_lens, "seq_lens", dev, table[:1], torch.int64))


def _packed(cu_seqlens, N, dev):
    """Number of sequences of a packed or equal-length batch, and the offsets' address."""
    if cu_seqlens is None:
        return 1 if N is None else N, 0
    if cu_seqlens.dim() != 1 or cu_seqlens.numel() < 1:
        raise ValueError("cu_seqlens must be a 1-d tensor of N + 1 offsets")
    n = cu_seqlens.shape[0] - 1
    if N is not None and N != n:
        raise ValueError(f"cu_seqlens has {n + 1} offsets, expected N + 1 = {N + 1}")
    return n, _dense(cu_seqlens, "cu_seqlens", dev, (n + 1,), torch.int64)


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
    dev, io, (T, _, _) = _first(k_raw, "k_raw")
    (pages, Hk, P, d), (N, width), (kc, vc, ks, vs, table, lens) = _cache(
        k_cache, v_cache, k_scale, v_scale, page_table, seq_lens, dev)
    k_in, ld_k = _heads(k_raw, "k_raw", dev, (T, Hk, d), io)
    v_in, ld_v = _heads(v_raw, "v_raw", dev, (T, Hk, d), io)
    cu = _packed(cu_seqlens, N, dev)[1]
    rope, freqs = _rope(inv_freq, dev)
    desc = GdnKvAppendDesc(N, T, ld_k, ld_v, pages, width, Hk, d, P, rope,
                           GDN_ROPE_INTERLEAVED if interleaved else GDN_ROPE_HALF, _DT[io],
                           rope_scale, eps)
    _call(lib.gdn_kv_append, "gdn_kv_append", dev, ctypes.byref(desc), cu, lens, table, k_in, v_in,
          _dense(k_weight, "k_weight", dev, (d,), torch.float32), freqs if rope else 0, kc, vc, ks,
          vs, _raw_stream(stream, dev))


def gdn_attn_prefill(q, k, v, cu_seqlens=None, N=None, window: int = 0, scale=None, o=None,
                     stream=None):
    """Causal attention over whole prompts (see include/gdn_attn.h).  Returns o.

    q [total_T, H_q, d]; k, v [total_T, H_k, d] (column blocks are fine);
    cu_seqlens int64 [N + 1] or None for N sequences of total_T / N tokens (N
    defaults to 1); window 0 (all) or the number of tokens seen; scale
    defaults to 1 / sqrt(d).  o [total_T, H_q, d] is allocated when not given.
    """
    dev, io, (T, Hq, d) = _first(q, "q")
    if k.dim() != 3:
        raise ValueError("k must be [total_T, H_k, d]")
    Hk = k.shape[1]
    q_in, ld_q = _heads(q, "q", dev, (T, Hq, d), io)
    k_in, ld_k = _heads(k, "k", dev, (T, Hk, d), io)
    v_in, ld_v = _heads(v, "v", dev, (T, Hk, d), io)
    N, cu = _packed(cu_seqlens, N, dev)
    if o is None:
        o = _empty((T, Hq, d), io, dev, stream)
    desc = GdnAttnPrefillDesc(N, T, ld_q, ld_k, ld_v, window, Hq, Hk, d, _DT[io],
                              d ** -0.5 if scale is None else scale)
    _call(lib.gdn_attn_prefill, "gdn_attn_prefill", dev, ctypes.byref(desc), cu, q_in, k_in, v_in,
          _dense(o, "o", dev, (T, Hq, d), io), _raw_stream(stream, dev))
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
    dev, io, shape = _first(q, "q")
    (pages, Hk, P, d), (N, width), cache = _cache(k_cache, v_cache, k_scale, v_scale, page_table,
                                                  seq_lens, dev)
    Hq = shape[1]
    q_in = _dense(q, "q", dev, (N, Hq, d), io)
    if o is None:
        o = _empty(shape, io, dev, stream)
    desc = GdnAttnDecodeDesc(N, pages, width, window, Hq, Hk, d, P, _DT[io],
                             d ** -0.5 if scale is None else scale)
    ref = ctypes.byref(desc)
    need = lib.gdn_attn_decode_workspace_size(ref)
    ws = nbytes = 0
    if need:
        if workspace is None:
            workspace = _empty((need,), torch.uint8, dev, stream)
        elif workspace.get_device() != dev or not workspace.is_contiguous():
            raise ValueError("workspace must be a contiguous tensor on the device of the others")
        ws, nbytes = workspace.data_ptr(), workspace.numel() * workspace.element_size()
    _call(lib.gdn_attn_decode, "gdn_attn_decode", dev, ref, q_in, *cache,
          _dense(o, "o", dev, shape, io), ws, nbytes, _raw_stream(stream, dev))
    return o
