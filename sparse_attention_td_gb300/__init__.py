"""GB300-native TidalDecode decode step (Position Persistent Sparse Attention).

A thin Python binding of ``libtd.so`` (C ABI in ``include/td.h``).  It only
marshals arguments -- tensor pointers, shapes and the current CUDA stream --
and checks that tensors are CUDA tensors of the declared shapes, so the C
library never sees a host pointer or a short buffer.  Every step of the
computation runs in the library's CUDA kernels; there is no fallback.

Entry points (same names as the C ABI):
  td_full_attn_select  one full-attention layer, optionally selecting top-k
  td_topk_select       the selection step alone, from given scores
  td_sparse_attn       one PPSA layer over a given index set
  td_decode_step       one decode step over an L-layer schedule
  Plan                 a decode step captured into a CUDA graph
Speculative decoding over the same cache, contiguous or paged (make_cache):
  td_block_tables      block tables and slot map of a batch from its lengths
  td_kv_append_slots   new K/V rows into the cache through the slot map
  td_tree_attn         one full layer for a tree of drafted tokens
  td_tree_sparse_attn  one PPSA layer for a tree of drafted tokens
  td_tree_commit       keep the accepted rows of every layer
Small caches:
  td_window_attn       new tokens (prompts or one each) with a sliding window and sinks
  td_q4_append         new K/V rows into a 4-bit cache (make_q4_cache)
  td_q4_attn           td_window_attn over a 4-bit cache
  td_q4_sparse_attn    one PPSA layer over a 4-bit cache
  td_weights_attn      attention that adds up each cached position's weight
  td_evict             keep the first, the recent and the heaviest positions
"""
from ._lib import (  # noqa: F401
    MODE_FULL, MODE_FULL_SELECT, MODE_SPARSE, FLAG_INDEX_OUT_OF_RANGE,
    FLAG_SEQ_LEN_OUT_OF_RANGE, FLAG_WAIT_TIMEOUT, FLAG_TREE_OUT_OF_RANGE, FLAG_PAGE_OUT_OF_RANGE,
    FLAG_PAGES_EXHAUSTED, MAX_TREE, NOALLOC_SCRATCH_BYTES, TdError, Shape, Workspace, Plan, lib, lib_path,
    td_status_string, td_workspace_size, td_workspace_init, td_workspace_status,
    td_full_attn_select, td_full_attn_select_coverage, td_topk_select, td_index_overlap, td_kv_append, td_probe_layer_reads, td_sparse_attn, td_sparse_attn_noalloc, td_decode_step, td_set_tuning, td_query_splits, td_kernel_name,
    td_tree_workspace_size, td_tree_attn, td_tree_sparse_attn, td_tree_commit, td_kv_append_slots,
    td_block_tables, td_cache_workspace_size, td_window_attn, td_q4_append, td_q4_attn,
    td_q4_sparse_attn, td_weights_attn, td_evict, Q4Cache, make_q4_cache, Cache, make_cache, make_shape, default_scale,
)
