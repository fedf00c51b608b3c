"""Strict, batch-invariant token logprob on GB300 (sm_103a).

The compute lives in ``lib/librlk_logp.so`` (CUDA kernels behind a C ABI,
declared in ``include/rlk_logp.h``, ``include/rlk_norm.h`` and ``include/rlk_rollout.h``); this
package is its thin Python binding.
"""

from ._binding import (VOCAB_PADDED, VOCAB_REAL, NUM_SHARDS, SHARD_WIDTH, RlkError, LogpArgs,
                       ShardArgs, EXPORTS, load_library, logp_full, logp_pair, logp_restricted,
                       logp_kl, logp_kl_ref, logp_kl_host, logp_kl_host_workspace_bytes, logp_backward, logp_pair_save, logp_backward_saved,
                       logp_autograd, shard_summary,
                       shard_counts, logp_merge, logp_sharded, shard_counts_window,
                       logp_merge_resumable, merge_state, sample, linear_logp, linear_logp_pair,
                       NORM_BINS, norm_bins, sqnorm_accumulate, sqnorm_finalize, reduce_bins_,
                       grad_norm, KVCache, BTHStrides, RopeArgs, rope, rope_autograd, kv_append, kv_append_rope, paged_attention,
                       paged_attention_workspace_bytes, PrefixGroups, prefix_attention, prefix_attention_workspace_bytes,
                       VerifyArgs, verify_drafts, verify_workspace_bytes)

__all__ = ["VOCAB_PADDED", "VOCAB_REAL", "NUM_SHARDS", "SHARD_WIDTH", "RlkError", "LogpArgs",
           "ShardArgs",
           "EXPORTS", "load_library", "logp_full", "logp_pair", "logp_restricted", "logp_kl", "logp_kl_ref",
           "logp_kl_host", "logp_kl_host_workspace_bytes",
           "logp_backward", "logp_pair_save", "logp_backward_saved", "logp_autograd", "shard_summary", "shard_counts", "logp_merge", "shard_counts_window", "logp_merge_resumable", "merge_state",
           "logp_sharded", "sample", "linear_logp", "linear_logp_pair", "NORM_BINS", "norm_bins", "sqnorm_accumulate",
           "sqnorm_finalize", "reduce_bins_", "grad_norm",
           "KVCache", "BTHStrides", "RopeArgs", "rope", "rope_autograd", "kv_append", "kv_append_rope", "paged_attention", "paged_attention_workspace_bytes",
           "PrefixGroups", "prefix_attention", "prefix_attention_workspace_bytes", "VerifyArgs", "verify_drafts", "verify_workspace_bytes"]
