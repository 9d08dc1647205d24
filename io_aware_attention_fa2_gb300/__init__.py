"""Fused exact attention forward for GB300 (sm_103a).

O = softmax(scale * Q K^T [+ causal mask]) V over [B, N, H, d] bf16/fp16 tensors, computed
tile by tile with online softmax so that the N x N score matrix never reaches HBM, plus the
per-row fp32 log-sum-exp, its backward, and a paged key-value cache for decoding (``paged``), for
drafted tokens and for branching sequences (``draft``).
The computation runs in hand-written CUDA kernels behind a C ABI
(``include/fa.h``); this package is a thin ctypes binding over that library.

Importing the package does not load the CUDA library; the first call does, and raises if the
library has not been built (there is no fallback path).
"""
from .binding import (FaError, attention_backward, attention_forward, available,
                      bwd_workspace_size, device_error, error_string, fa_bwd, fa_fwd,
                      fa_fwd_splitkv, library_path, load_library, splitkv_num_splits,
                      splitkv_workspace_size)
from .draft import (Forked, PagePool, fa_paged_accept, fa_paged_copy, fa_paged_fork,
                    fa_paged_resize, fa_paged_tree, new_page_pool, paged_accept, paged_fork,
                    paged_resize, paged_tree_attention, paged_tree_workspace_size)
from .paged import (fa_key_weights, fa_paged_append, fa_paged_decode, fa_paged_evict, key_weights,
                    key_weights_workspace_size, paged_attention, paged_decode_workspace_size,
                    paged_evict)

__all__ = ["FaError", "Forked", "PagePool", "attention_backward", "attention_forward",
           "available", "bwd_workspace_size", "device_error", "error_string", "fa_bwd", "fa_fwd",
           "fa_fwd_splitkv", "fa_key_weights", "fa_paged_accept", "fa_paged_append",
           "fa_paged_copy", "fa_paged_decode", "fa_paged_evict", "fa_paged_fork",
           "fa_paged_resize", "fa_paged_tree", "key_weights", "key_weights_workspace_size",
           "library_path", "load_library", "new_page_pool", "paged_accept", "paged_attention",
           "paged_decode_workspace_size", "paged_evict", "paged_fork", "paged_resize",
           "paged_tree_attention", "paged_tree_workspace_size", "splitkv_num_splits",
           "splitkv_workspace_size"]
