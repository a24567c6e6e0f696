"""MLA chunked-context prefill for NVIDIA GB300 (sm_103a).

The computation lives in ``libmla_gb300.so`` (hand-written CUDA kernels behind
a C ABI, ``include/mla_chunked_context.h``).  This package is the thin Python
binding: the functions below carry the C entry points' names and only
marshal arguments; PyTorch provides device memory and streams.
"""

from ._lib import (Chunk, Dims, MlaError, lib, merge_attn_states, mla_chunk_kv_dtype,
                   mla_chunk_workspace_bytes, mla_device_error_flags,
                   mla_chunked_prefill, mla_context_chunk_attn, mla_context_chunk_attn_noalloc,
                   mla_fill_empty_rows,
                   mla_gather_context_rows, mla_has_tcgen05, mla_kv_up_proj,
                   mla_mask_empty_context, mla_plan_context_chunks, mla_prefill_workspace_bytes,
                   mla_varlen_attn, MLA_STATUS_BAD_BLOCK, mla_plan_equal_window_chunks,
                   mla_prefill_equal_window_workspace_bytes, mla_chunked_prefill_equal_window,
                   mla_selftest_bounded_wait, mla_kernel_launches,
                   mla_fused_attn_workspace_bytes, mla_fused_context_attn,
                   mla_fused_attn_plan, mla_prefill_pinned_bytes, mla_profile_begin,
                   mla_profile_end, mla_set_pipeline_overlap, MLA_STATUS_FP16_RANGE,
                   MLA_STATUS_BAD_POSITION, mla_append_latent, mla_absorb_query,
                   mla_expand_output, mla_latent_attn, mla_latent_attn_workspace_bytes)

__all__ = ["Chunk", "Dims", "MlaError", "lib", "merge_attn_states", "mla_chunk_kv_dtype",
           "mla_chunk_workspace_bytes", "mla_device_error_flags",
           "mla_chunked_prefill", "mla_context_chunk_attn", "mla_context_chunk_attn_noalloc",
           "mla_fill_empty_rows",
           "mla_gather_context_rows", "mla_has_tcgen05", "mla_kv_up_proj",
           "mla_mask_empty_context", "mla_plan_context_chunks", "mla_prefill_workspace_bytes",
           "mla_varlen_attn", "MLA_STATUS_BAD_BLOCK", "mla_plan_equal_window_chunks",
           "mla_prefill_equal_window_workspace_bytes", "mla_chunked_prefill_equal_window",
           "mla_selftest_bounded_wait", "mla_kernel_launches", "mla_fused_attn_workspace_bytes",
           "mla_fused_context_attn", "mla_fused_attn_plan", "mla_prefill_pinned_bytes",
           "mla_profile_begin", "mla_profile_end", "mla_set_pipeline_overlap",
           "MLA_STATUS_FP16_RANGE", "ChunkedPrefill", "MLA_STATUS_BAD_POSITION",
           "mla_append_latent", "mla_absorb_query", "mla_expand_output", "mla_latent_attn",
           "mla_latent_attn_workspace_bytes", "LatentDecode"]


class ChunkedPrefill:
    """Holds the device workspace (a torch uint8 tensor) and the pinned host
    metadata scratch for one batch shape and runs ``mla_chunked_prefill`` on
    them."""

    def __init__(self, dims: Dims, context_lens, query_lens, row_budget: int,
                 max_context_chunk: int, split_alignment: int, device="cuda"):
        import torch
        self.dims = dims
        self.context_lens = [int(x) for x in context_lens]
        self.query_lens = [int(x) for x in query_lens]
        self.row_budget = int(row_budget)
        self.max_context_chunk = int(max_context_chunk)
        self.split_alignment = int(split_alignment)
        self.workspace_bytes = mla_prefill_workspace_bytes(
            dims, self.context_lens, self.query_lens, self.row_budget, self.max_context_chunk,
            self.split_alignment)
        self.workspace = torch.empty(max(1, self.workspace_bytes), dtype=torch.uint8,
                                     device=device)
        pinned = mla_prefill_pinned_bytes(dims, self.context_lens, self.query_lens,
                                          self.row_budget, self.max_context_chunk,
                                          self.split_alignment)
        self.pinned = torch.empty(max(16, pinned), dtype=torch.uint8, pin_memory=True)

    def __call__(self, q, new_latent, kv_cache, block_table, w_kv_b, out, out_lse=None,
                 dev_status=None, stream=None):
        mla_chunked_prefill(self.dims, self.context_lens, self.query_lens, self.row_budget,
                            self.max_context_chunk, self.split_alignment, q, new_latent,
                            kv_cache, block_table, w_kv_b, self.workspace, out, out_lse,
                            dev_status, stream, pinned_scratch=self.pinned)
        return out


class LatentDecode:
    """Holds the absorbed queries, latent outputs and workspace for decode
    steps of up to max_tokens new tokens and max_seqs sequences, and runs a
    layer's step on them: absorb the queries, append to the cache, attend,
    expand.  The lengths are read on the device, so one captured step can be
    replayed as they grow.  One instance serves one step at a time."""

    def __init__(self, dims: Dims, max_tokens: int, max_seqs: int, device="cuda"):
        import torch
        self.dims, self.max_tokens, self.max_seqs = dims, int(max_tokens), int(max_seqs)
        H, L, P = dims.num_heads, dims.kv_lora_rank, dims.qk_rope_dim
        self.q_latent = torch.empty(self.max_tokens, H, L + P, dtype=dims.dtype, device=device)
        self.o_latent = torch.empty(self.max_tokens, H, L, dtype=dims.dtype, device=device)
        self.workspace = torch.empty(
            max(16, mla_latent_attn_workspace_bytes(dims, self.max_tokens, self.max_seqs)),
            dtype=torch.uint8, device=device)

    def __call__(self, q, kv_a, query_start_loc, seq_lens, rope_table, kv_cache, block_table,
                 w_kv_b, out, lse=None, norm_weight=None, norm_eps=1e-6, positions=None,
                 interleaved=False, causal=True, dev_status=None, stream=None):
        """q [T, H, Dn+P] before rotation, kv_a [T, L+P] before norm and
        rotation; out [T, H, Dv], lse [H, T].  Rows of no sequence are left
        out of the cache; what out holds for them is not specified.  A token
        that the append skips (a rope position outside the table, more new
        tokens than seq_lens says) attends with its rope columns unrotated,
        and its cache slot keeps what it held: pass dev_status to learn of
        positions outside the table."""
        T, dims = q.shape[0], self.dims
        if T > self.max_tokens or seq_lens.shape[0] > self.max_seqs:
            raise ValueError(f"LatentDecode: {T} tokens of {seq_lens.shape[0]} sequences, room "
                             f"for {self.max_tokens} of {self.max_seqs}")
        q_lat, o_lat = self.q_latent[:T], self.o_latent[:T]
        # The rope columns come with the absorption first, so that a token that
        # the append skips has its own there and not an earlier step's.
        mla_absorb_query(dims, q, w_kv_b, q_lat, stream=stream)
        mla_append_latent(dims, kv_a, query_start_loc, seq_lens, rope_table, kv_cache,
                          block_table, norm_weight, norm_eps, positions, interleaved, q=q,
                          q_pe_out=q_lat[..., dims.kv_lora_rank:], dev_status=dev_status,
                          stream=stream)
        mla_latent_attn(dims, causal, query_start_loc, seq_lens, q_lat, kv_cache, block_table,
                        self.workspace, o_lat, lse, dev_status, stream)
        mla_expand_output(dims, o_lat, w_kv_b, out, stream)
        return out
