"""MI355X-native Kimi Delta Attention (KDA): chunkwise prefill, its training backward and
recurrent decode; and, for the full-attention layers of a hybrid stack, rotary positions, a
paged KV cache, attention over it and its pages' bookkeeping.

The operators live in libkda.so (hand-written HIP kernels for gfx950, C ABI in include/kda.h
and include/kda_paged.h); this package is their thin Python binding.
"""
from ._binding import (KDA_DTYPE_BF16, KDA_DTYPE_F32, LIB_PATH, OPT_BETA_LOGITS,
                       OPT_GATE_LOGITS, OPT_L2NORM_QK, OPT_SCALAR_GATE, KdaError,
                       bwd_workspace_size, chunk_bwd, chunk_fwd, chunk_fwd_noalloc,
                       chunk_fwd_scan, ckpt_empty, ckpt_interval, decode_step,
                       declared_functions, lib, workspace_size)
from ._paged import (attn_paged, attn_workspace_size, cache_append, pages_alloc, pages_compact,
                     pages_copy, pages_fork, pages_free, rope, rope_bwd, rope_freqs)

__all__ = ["chunk_fwd", "chunk_fwd_noalloc", "chunk_fwd_scan", "chunk_bwd", "decode_step",
           "workspace_size", "bwd_workspace_size", "ckpt_interval", "ckpt_empty", "KdaError", "lib", "LIB_PATH",
           "declared_functions", "KDA_DTYPE_BF16", "KDA_DTYPE_F32", "OPT_SCALAR_GATE",
           "OPT_GATE_LOGITS", "OPT_BETA_LOGITS", "OPT_L2NORM_QK", "rope_freqs", "rope", "rope_bwd",
           "cache_append", "attn_paged", "attn_workspace_size", "pages_alloc", "pages_fork",
           "pages_free", "pages_compact", "pages_copy"]
