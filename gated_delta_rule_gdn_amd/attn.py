"""ctypes binding of the attention operators of libgdn.so (the C ABI in
include/gdn_attn.h): argument marshalling only, as in gdn.py.

Tensors of a call are on one device, which need not be the current one; work
goes to that device's current stream, or to the one given.
"""
from __future__ import annotations

import contextlib
import ctypes

import torch

from .gdn import _DT, _ptr, GDN_OK, GdnError, lib

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


def _dev(t, name) -> int:
    if not t.is_cuda:
        raise ValueError(f"{name} must be a device tensor")
    return t.get_device()


def _heads(t, name, dev, rows, H, d, dtype) -> int:
    """A [rows, H, d] device tensor whose rows are dense (a column block of a
    wider buffer is fine).  Returns its row stride in elements."""
    _same(t, name, dev, dtype)
    if t.shape != (rows, H, d):
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {(rows, H, d)}")
    s = t.stride()
    if s[2] != 1 or (H > 1 and s[1] != d):
        if rows * H:
            raise ValueError(f"{name} must have dense rows of {H} x {d} elements")
    return s[0] if rows > 1 else H * d


def _same(t, name, dev, dtype):
    if not t.is_cuda or t.get_device() != dev:
        raise ValueError(f"{name} must be on the same device as the other tensors")
    if t.dtype is not dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")


def _dense(t, name, dev, shape, dtype):
    _same(t, name, dev, dtype)
    if t.shape != shape:
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


def _maybe(t, name, dev, shape, dtype):
    if t is not None:
        _dense(t, name, dev, shape, dtype)


class _On:
    """The device and stream of a call.  Outputs and workspaces that the call
    allocates belong to that stream."""

    def __init__(self, dev, stream):
        self.dev = dev
        self.given = stream
        if stream is None:
            self.raw = torch.cuda.current_stream(dev).cuda_stream
        elif isinstance(stream, torch.cuda.Stream):
            if stream.device.index != dev:
                raise ValueError("stream is on another device than the tensors")
            self.raw = stream.cuda_stream
        else:
            self.raw = int(stream)

    def empty(self, shape, dtype):
        device = torch.device("cuda", self.dev)
        if self.given is None:
            return torch.empty(shape, dtype=dtype, device=device)
        s = self.given if isinstance(self.given, torch.cuda.Stream) else \
            torch.cuda.ExternalStream(self.raw, device=device)
        with torch.cuda.stream(s):
            return torch.empty(shape, dtype=dtype, device=device)

    def call(self, fn, name, *args):
        guard = contextlib.nullcontext() if torch.cuda.current_device() == self.dev else \
            torch.cuda.device(self.dev)
        with guard:
            st = fn(*args, self.raw)
        if st != GDN_OK:
            raise GdnError(st, name)


def _io(t, name):
    if t.dtype not in _DT:
        raise ValueError(f"{name} must be float32 or bfloat16")
    return t.dtype


def _rope(inv_freq, dev):
    if inv_freq is None:
        return 0
    if inv_freq.dim() != 1:
        raise ValueError("inv_freq must be a 1-d tensor of rope_dim / 2 frequencies")
    _dense(inv_freq, "inv_freq", dev, inv_freq.shape, torch.float32)
    return 2 * inv_freq.shape[0]


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
    dev, io = _dev(one, "q_raw"), _io(one, "q_raw")
    if one.dim() != 3:
        raise ValueError("q_raw and k_raw must be [rows, H, d]")
    rows, d = one.shape[0], one.shape[2]
    on = _On(dev, stream)
    Hq = Hk = ld_q = ld_k = 0
    if q_raw is not None:
        Hq = q_raw.shape[1]
        ld_q = _heads(q_raw, "q_raw", dev, rows, Hq, d, io)
        if q is None:
            q = on.empty((rows, Hq, d), io)
        _dense(q, "q", dev, (rows, Hq, d), io)
    elif q is not None:
        raise ValueError("q without q_raw")
    if k_raw is not None:
        if k_raw.dim() != 3:
            raise ValueError("q_raw and k_raw must be [rows, H, d]")
        Hk = k_raw.shape[1]
        ld_k = _heads(k_raw, "k_raw", dev, rows, Hk, d, io)
        if k is None:
            k = on.empty((rows, Hk, d), io)
        _dense(k, "k", dev, (rows, Hk, d), io)
    elif k is not None:
        raise ValueError("k without k_raw")
    _maybe(q_weight, "q_weight", dev, (d,), torch.float32)
    _maybe(k_weight, "k_weight", dev, (d,), torch.float32)
    if inv_freq is not None and positions is None:
        raise ValueError("rotation needs positions")
    rope = _rope(inv_freq, dev)
    _maybe(positions, "positions", dev, (rows,), torch.int64)
    desc = GdnQkDesc(rows, ld_q, ld_k, Hq, Hk, d, rope,
                     GDN_ROPE_INTERLEAVED if interleaved else GDN_ROPE_HALF, _DT[io], rope_scale,
                     eps)
    on.call(lib.gdn_qk_norm_rope, "gdn_qk_norm_rope", ctypes.byref(desc), _ptr(q_raw),
            _ptr(k_raw), _ptr(q_weight), _ptr(k_weight), _ptr(positions) if rope else None,
            _ptr(inv_freq) if rope else None, _ptr(q), _ptr(k))
    return q, k


def _cache(k_cache, v_cache, k_scale, v_scale, page_table, seq_lens, dev):
    """(num_pages, H_k, page_size, d, N, max_pages) of a paged cache."""
    if k_cache.dim() != 4:
        raise ValueError("k_cache must be [num_pages, H_k, page_size, d]")
    if page_table.dim() != 2:
        raise ValueError("page_table must be [N, max_pages]")
    shape = k_cache.shape
    _dense(k_cache, "k_cache", dev, shape, torch.float8_e4m3fn)
    _dense(v_cache, "v_cache", dev, shape, torch.float8_e4m3fn)
    _dense(k_scale, "k_scale", dev, shape[:2], torch.float32)
    _dense(v_scale, "v_scale", dev, shape[:2], torch.float32)
    _dense(page_table, "page_table", dev, page_table.shape, torch.int32)
    _dense(seq_lens, "seq_lens", dev, page_table.shape[:1], torch.int64)
    return (*shape, *page_table.shape)


def _packed(cu_seqlens, N, dev):
    """Number of sequences of a packed or equal-length batch."""
    if cu_seqlens is None:
        return 1 if N is None else N
    if cu_seqlens.dim() != 1 or cu_seqlens.numel() < 1:
        raise ValueError("cu_seqlens must be a 1-d tensor of N + 1 offsets")
    n = cu_seqlens.shape[0] - 1
    if N is not None and N != n:
        raise ValueError(f"cu_seqlens has {n + 1} offsets, expected N + 1 = {N + 1}")
    _dense(cu_seqlens, "cu_seqlens", dev, (n + 1,), torch.int64)
    return n


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
    dev, io = _dev(k_raw, "k_raw"), _io(k_raw, "k_raw")
    pages, Hk, P, d, N, width = _cache(k_cache, v_cache, k_scale, v_scale, page_table, seq_lens,
                                       dev)
    T = k_raw.shape[0]
    ld_k = _heads(k_raw, "k_raw", dev, T, Hk, d, io)
    ld_v = _heads(v_raw, "v_raw", dev, T, Hk, d, io)
    _packed(cu_seqlens, N, dev)
    _maybe(k_weight, "k_weight", dev, (d,), torch.float32)
    rope = _rope(inv_freq, dev)
    desc = GdnKvAppendDesc(N, T, ld_k, ld_v, pages, width, Hk, d, P, rope,
                           GDN_ROPE_INTERLEAVED if interleaved else GDN_ROPE_HALF, _DT[io],
                           rope_scale, eps)
    _On(dev, stream).call(
        lib.gdn_kv_append, "gdn_kv_append", ctypes.byref(desc), _ptr(cu_seqlens), _ptr(seq_lens),
        _ptr(page_table), _ptr(k_raw), _ptr(v_raw), _ptr(k_weight),
        _ptr(inv_freq) if rope else None, _ptr(k_cache), _ptr(v_cache), _ptr(k_scale),
        _ptr(v_scale))


def gdn_attn_prefill(q, k, v, cu_seqlens=None, N=None, window: int = 0, scale=None, o=None,
                     stream=None):
    """Causal attention over whole prompts (see include/gdn_attn.h).  Returns o.

    q [total_T, H_q, d]; k, v [total_T, H_k, d] (column blocks are fine);
    cu_seqlens int64 [N + 1] or None for N sequences of total_T / N tokens (N
    defaults to 1); window 0 (all) or the number of tokens seen; scale
    defaults to 1 / sqrt(d).  o [total_T, H_q, d] is allocated when not given.
    """
    dev, io = _dev(q, "q"), _io(q, "q")
    if q.dim() != 3 or k.dim() != 3:
        raise ValueError("q and k must be [total_T, H, d]")
    T, Hq, d = q.shape
    Hk = k.shape[1]
    ld_q = _heads(q, "q", dev, T, Hq, d, io)
    ld_k = _heads(k, "k", dev, T, Hk, d, io)
    ld_v = _heads(v, "v", dev, T, Hk, d, io)
    N = _packed(cu_seqlens, N, dev)
    on = _On(dev, stream)
    if o is None:
        o = on.empty((T, Hq, d), io)
    _dense(o, "o", dev, (T, Hq, d), io)
    desc = GdnAttnPrefillDesc(N, T, ld_q, ld_k, ld_v, window, Hq, Hk, d, _DT[io],
                              d ** -0.5 if scale is None else scale)
    on.call(lib.gdn_attn_prefill, "gdn_attn_prefill", ctypes.byref(desc), _ptr(cu_seqlens),
            _ptr(q), _ptr(k), _ptr(v), _ptr(o))
    return o


def _decode_desc(q, k_cache, page_table, window, scale):
    N, Hq, d = q.shape
    pages, Hk, P = k_cache.shape[:3]
    return GdnAttnDecodeDesc(N, pages, page_table.shape[1], window, Hq, Hk, d, P, _DT[_io(q, "q")],
                             d ** -0.5 if scale is None else scale)


def gdn_attn_decode_workspace_size(q, k_cache, page_table, window: int = 0) -> int:
    """Workspace bytes gdn_attn_decode needs for these shapes (0: none)."""
    return int(lib.gdn_attn_decode_workspace_size(
        ctypes.byref(_decode_desc(q, k_cache, page_table, window, None))))


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
    dev, io = _dev(q, "q"), _io(q, "q")
    if q.dim() != 3:
        raise ValueError("q must be [N, H_q, d]")
    _, Hk, _, d, N, _ = _cache(k_cache, v_cache, k_scale, v_scale, page_table, seq_lens, dev)
    Hq = q.shape[1]
    _dense(q, "q", dev, (N, Hq, d), io)
    on = _On(dev, stream)
    if o is None:
        o = on.empty((N, Hq, d), io)
    _dense(o, "o", dev, (N, Hq, d), io)
    desc = _decode_desc(q, k_cache, page_table, window, scale)
    need = lib.gdn_attn_decode_workspace_size(ctypes.byref(desc))
    nbytes = 0
    if need:
        if workspace is None:
            workspace = on.empty((need,), torch.uint8)
        if not workspace.is_cuda or workspace.get_device() != dev or not workspace.is_contiguous():
            raise ValueError("workspace must be a contiguous tensor on the device of the others")
        nbytes = workspace.numel() * workspace.element_size()
    on.call(lib.gdn_attn_decode, "gdn_attn_decode", ctypes.byref(desc), _ptr(q), _ptr(k_cache),
            _ptr(v_cache), _ptr(k_scale), _ptr(v_scale), _ptr(page_table), _ptr(seq_lens), _ptr(o),
            _ptr(workspace) if need else None, nbytes)
    return o
