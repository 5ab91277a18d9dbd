"""Gated delta rule (GDN-2 / Gated DeltaNet / DeltaNet) on AMD MI355X (gfx950).

The computation lives in libgdn.so (C ABI, include/gdn.h and, for the
softmax-attention layers of hybrids and their residual stream, include/gdn_attn.h
and include/gdn_hybrid.h), built from the HIP sources under csrc/.  This package
holds the thin bindings only: ctypes, and for the calls of those two headers an
extension module (attn.py, hybrid.py), without which they alone raise.
"""
from .gdn import (  # noqa: F401
    GDN_BF16, GDN_ERR_CHECK, GDN_ERR_HIP, GDN_ERR_INVALID_ARG, GDN_ERR_UNSUPPORTED, GDN_F32,
    GDN_GATES_CHANNEL, GDN_GATES_SCALAR, GDN_OK, GdnBwdDesc, GdnBwdVarlenDesc, GdnConvDesc, GdnDecodeDesc, GdnError,
    GdnFwdDesc, GdnGateDesc, GdnNormDesc, GdnRawGates, GdnVarlenDesc, abi_version, check_selftest, gdn_backward,
    gdn_backward_noalloc, gdn_backward_noalloc_max_bytes, gdn_backward_saved,
    gdn_backward_varlen, gdn_backward_varlen_saved, gdn_backward_workspace_size, gdn_chunk_fwd,
    gdn_chunk_fwd_gated, gdn_chunk_fwd_save, gdn_chunk_fwd_varlen, gdn_chunk_fwd_varlen_save, gdn_decode_step, gdn_gates, gdn_output_gate, gdn_short_conv, lib,
    status_string,
)
from .attn import (  # noqa: F401
    GDN_ROPE_HALF, GDN_ROPE_INTERLEAVED, GdnAttnDecodeDesc, GdnAttnPrefillDesc, GdnKvAppendDesc, GdnQkDesc,
    attn_abi_version, gdn_attn_decode, gdn_attn_decode_workspace_size, gdn_attn_prefill,
    gdn_kv_append, gdn_qk_norm_rope,
)
from .hybrid import (  # noqa: F401
    GdnAddNormBwdDesc, GdnAddNormDesc, GdnAttnBwdDesc, GdnQkBwdDesc, gdn_add_norm, gdn_add_norm_backward,
    gdn_add_norm_backward_workspace_size, gdn_attn_backward, gdn_attn_backward_workspace_size, gdn_attn_prefill_save,
    gdn_qk_norm_rope_backward, gdn_qk_norm_rope_backward_workspace_size, hybrid_abi_version,
)
