"""streaming_kv_cache_gb300 -- streaming view-major KV-cache attention on GB300.

A C-ABI library (libskv.so, hand-written CUDA for sm_103a) with three calls
on the streaming path -- kv_stream_insert, stream_attn_prefill and
stream_attn_verify -- plus the tail-token and whole-window prefills; a paged
cache for requests of different lengths (kv_paged_plan, kv_paged_write,
paged_attn), bounded by eviction of the tokens that get the least attention
(paged_attn_weight, kv_evict_plan, kv_evict_move, kv_paged_trim); sampled
verification of drafts (verify_sampled); attention to an encoder's states
(cross_attn); and a thin ctypes binding.  Build it with
streaming_kv_cache_gb300.build.build().
"""
from . import synth  # noqa: F401
from .skv import (EXPORTS, PagedCache, PagedPlan, PagedScores, SkvError, StreamCache, attn_workspace,  # noqa: F401
                  cross_attn, kv_evict_move, kv_evict_plan, kv_paged_plan, kv_paged_trim, kv_paged_write, kv_stream_insert,
                  kv_stream_insert_noalloc, kv_write_rows,
                  lib, paged_attn, paged_attn_weight, skv_build_rope_table, skv_row_cap, skv_verify_workspace_bytes,
                  skv_build_mrope_table, status_string, stream_attn_prefill,
                  stream_attn_prefill_insert, stream_attn_prefill_tail, stream_attn_verify,
                  stream_attn_window, verify_sampled, verify_workspace)
