"""Ragged mixed-batch step for GB300: Python face of the librb C ABI (include/rb.h).

    prepare_inputs   persistent batch -> input_ids, positions, query_start_loc, seq_lens,
                     slot_mapping, logits_indices (+ max_query_len, max_seq_len, error word)
    kv_write         new K/V rows -> paged cache by slot_mapping
    paged_attention  varlen causal GQA attention through the page table
    paged_attention_cascade  the same when all requests share a prefix (read once), with
                     cascade_prefix_len giving the usable prefix length
    paged_attention_scored  the same with score rules (ScoreRules): capped scores, a distance
                     bias, packed documents and windows, bidirectional prefixes
    gather_rows      hidden rows at logits_indices
    PersistentBatch  device-resident rows of the resident requests; ``apply`` merges one
                     step's scheduler output (remove, append, install, condense) on the GPU
    PagePool         reference counts of the cache's pages: copy, fork, free, compact
    token_logprobs   log probability and rank of given tokens, entropy, top alternatives
    pad_for_graph    smallest captured graph size >= the token count

All compute runs in the library's sm_103a kernels; tensors are caller-owned CUDA tensors.
"""
from ._binding import (Dims, RbError, EBIT_ATTN_META, EBIT_BLOCK_ID, EBIT_NUM_COMPUTED,
                       EBIT_NUM_SCHEDULED, EBIT_ROW_INDEX, EBIT_SEQ_LEN, EBIT_SLOT, EBIT_TIMEOUT,
                       EBIT_TOKEN_SUM, LIB_PATH, gather_rows, kv_write, launch_count, lib,
                       pad_for_graph, paged_attention, prepare_inputs, status_string,
                       workspace_size, cascade_prefix_len, cascade_workspace_size,
                       paged_attention_cascade, ScoreRules, paged_attention_scored)
from ._binding import (EBIT_BATCH_ID, EBIT_BATCH_SIZE, EBIT_LOGITS, EBIT_NO_PAGE,
                       EBIT_PAGE_PAIR, EBIT_PAGE_REF, EBIT_ROW, EBIT_TOKEN_ID)
from .logprobs import MAX_TOP_LOGPROBS, TokenLogprobs, token_logprobs
from .pages import PagePool, pages_workspace_size
from .persistent_batch import PersistentBatch, batch_workspace_size
from .step import StepBuffers, run_step, run_step_fused, run_step_host, run_step_host_async

__all__ = ["Dims", "RbError", "gather_rows", "kv_write", "launch_count", "lib", "pad_for_graph",
           "paged_attention", "prepare_inputs", "status_string", "workspace_size", "StepBuffers",
           "run_step", "run_step_fused", "run_step_host", "run_step_host_async", "LIB_PATH", "PersistentBatch", "batch_workspace_size",
           "cascade_prefix_len", "cascade_workspace_size", "paged_attention_cascade", "ScoreRules",
           "paged_attention_scored", "PagePool",
           "pages_workspace_size", "TokenLogprobs", "token_logprobs", "MAX_TOP_LOGPROBS"]
