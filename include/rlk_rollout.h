/*
 * rlk_rollout.h -- C ABI of the rollout's serving operators for GB300
 * (sm_103a), part of librlk_logp.so: the paged key-value cache (append, and
 * the attention of new tokens over it) and the verification of drafted
 * tokens.  One speculative rollout step is
 *
 *   rlk_kv_append -> rlk_paged_attention -> the rest of the model's layers,
 *   the LM head -> rlk_verify_drafts,
 *
 * whose emitted tokens and logprobs are the rollout side that rlk_logp_pair
 * reproduces at training time ("Configurable H100 consistency runs": the
 * rollout engine's decode, sampling flags and logprobs).
 *
 * Conventions: those of rlk_logp.h.  Device pointers owned by the caller,
 * work enqueued on `stream`, nothing allocated or synchronised, host-checkable
 * faults returned before anything is enqueued (RLK_EINVAL, RLK_EALIGN), B == 0
 * or n == 0 a no-op.  What only the device can see (lengths, page numbers,
 * per-sequence parameters) is checked there, before anything is read or
 * written through it: a sequence that fails gets the outputs stated at each
 * call and raises *err_count (optional device int32) by at least one.
 *
 * Results do not depend on the batch: a token's attention output, and a
 * sequence's verification, have the same bits whatever B, the sequence's place
 * in the batch, the pages that hold it, the width of the page table, and (for
 * attention) whether the token comes alone or as one of several new tokens.
 */
#ifndef RLK_ROLLOUT_H
#define RLK_ROLLOUT_H

#include <stddef.h>
#include <stdint.h>

#include "rlk_logp.h"
#include "rlk_norm.h"

#ifdef __cplusplus
extern "C" {
#endif

/* A paged key-value cache and a batch of sequences in it.
 *
 * Token t of sequence b lies in page page_table[b * table_stride +
 * t / page_size], at place t % page_size; element d of its head h at
 *   page * page_stride + place * token_stride + h * head_stride + d
 * of k and of v.  The strides order pages, tokens and heads as the caller
 * likes ([pages][page_size][kv_heads][head_dim] and [pages][kv_heads]
 * [page_size][head_dim] are both ordinary). */
typedef struct rlk_kv_cache {
  void* k;                      /* dtype elements, 16-byte aligned */
  void* v;
  int64_t num_pages;            /* page numbers are 0 .. num_pages - 1 */
  int64_t page_stride;          /* elements; multiples of 8, the same for k and v */
  int64_t token_stride;
  int64_t head_stride;
  int32_t page_size;            /* tokens per page, any number >= 1 */
  int32_t kv_heads;             /* 1 .. 1024 */
  int32_t head_dim;             /* 64 or 128 */
  int32_t dtype;                /* RLK_DT_BF16 or RLK_DT_F16 */
  const int32_t* page_table;    /* [B][table_stride]; only entries of pages that are used are read */
  int64_t table_stride;         /* >= max_pages */
  int32_t max_pages;            /* entries per sequence; max_pages * page_size < 2^31 */
  int64_t B;                    /* sequences, < 2^16 */
  const int32_t* lens;          /* [B] tokens of each sequence, the new ones included */
  const int32_t* new_lens;      /* [B] new tokens of each sequence, 0 .. n, or NULL: n each */
  int32_t n;                    /* new tokens per sequence at most, 0 .. 65535 */
  int32_t* err_count;           /* optional device counter of rejected sequences */
} rlk_kv_cache;

/* Element strides of a [B][n][heads][head_dim] tensor with unit stride in the
 * last place; multiples of 8. */
typedef struct rlk_bth_strides {
  int64_t batch, token, head;
} rlk_bth_strides;

/* Write the keys and values of the new tokens into their pages: new token i of
 * sequence b (i < new_lens[b]) is token lens[b] - new_lens[b] + i.
 *   k, v: [B][n][kv_heads][head_dim] of the cache's dtype, 16-byte aligned.
 * A sequence is rejected, and nothing of it written, if lens[b] < new_lens[b],
 * lens[b] > max_pages * page_size or new_lens[b] is not in 0 .. n; a new token
 * whose page number is out of range is left out and counted.  Tokens of
 * different sequences that share a place are the caller's fault to avoid. */
rlk_status rlk_kv_append(const rlk_kv_cache* cache, const void* k, const rlk_bth_strides* k_strides,
                         const void* v, const rlk_bth_strides* v_strides, void* stream);

/* Attention of the new tokens over the cache (which already holds them).
 * Query i of sequence b stands at pos = lens[b] - new_lens[b] + i and sees the
 * tokens j <= pos; with window > 0 only those with j > pos - window, and the
 * first `sinks` tokens of the sequence.  Query head h reads kv head
 * h / (q_heads / kv_heads).  With s_j = scale * (q . k_j):
 *   out = sum_j exp(s_j - lse) v_j,   lse = ln sum_j exp(s_j).
 *   q:   [B][n][q_heads][head_dim] of the cache's dtype, 16-byte aligned;
 *        q_heads a multiple of kv_heads, at most 128 * kv_heads.
 *   out: the same shape and dtype, 16-byte aligned, strides of its own.
 *   out_lse: float [B][n][q_heads] (contiguous), or NULL.
 *   scale: finite.  window: 0 (off) or > 0.  sinks: >= 0, ignored without a
 *     window.
 *   workspace: device scratch of the size that rlk_paged_attention_workspace
 *     gives for max_tokens = max_pages * page_size, 16-byte aligned (NULL will
 *     do where that is 0).  No contents are expected or kept; calls that
 *     overlap on the GPU need one each.
 * Places i >= new_lens[b], and queries that see only tokens of score -inf, get
 * out = 0 and lse = -inf.  NaN and infinite keys, values or queries spread to the
 * outputs that see them only (the value of a masked token is never used; an
 * infinite one at a weight that is 0 in float32 makes NaN).  A rejected
 * sequence gets NaN in out and lse: for all its places if its lengths are at
 * fault (as in rlk_kv_append), for its places i < new_lens[b] if the page
 * number of a visible token is out of range.
 * The call's cost goes by n, and by the keys and values that a sequence's new
 * tokens see together: prompts and single tokens want calls of their own.
 * Scores, softmax statistics and output sums are held in float32, and out is
 * rounded once at the end.  The weights exp(s_j - max) go into the product with
 * V as two elements of the cache's dtype: 16 bits in bf16, whatever their size;
 * 22 bits in f16, but no finer than 2^-44 of the row's largest weight. */
rlk_status rlk_paged_attention(const rlk_kv_cache* cache, const void* q, const rlk_bth_strides* q_strides,
                               int32_t q_heads, float scale, int32_t window, int32_t sinks, void* out,
                               const rlk_bth_strides* out_strides, float* out_lse, void* workspace,
                               void* stream);

/* *bytes = the scratch that rlk_paged_attention needs for these sizes. */
rlk_status rlk_paged_attention_workspace(int64_t B, int32_t n, int32_t q_heads, int32_t kv_heads, int32_t head_dim,
                                         int64_t max_tokens, size_t* bytes);

/* Verification of drafted tokens by rejection sampling: what comes out is
 * distributed as the target's own tokens, whatever the draft model.
 *
 * Row b * (n + 1) + i of `logits` is the target model's at the place of draft i
 * of sequence b (i = n, or num_drafts[b]: the place after the last draft); row
 * b * n + i of `draft_logits` is the draft model's.  p_i and q_i are their
 * distributions as rlk_sample draws from them: temperature, top-k then top-p,
 * renormalised; temperature 0 puts all on the argmax.  Without draft_logits the
 * drafts are point masses: q_i is 1 at draft_token[b][i].  With
 * u_i = (accept_uniform[b][i] >> 8) / 2^24, for i = 0, 1, ...:
 *   draft i is accepted iff u_i q_i(d_i) < p_i(d_i);
 *   at the first one that is not (a), the token there is drawn from
 *     max(p_a - q_a, 0), renormalised (from p_a, where that has no mass);
 *   if all num_drafts[b] are accepted (a = num_drafts[b]), it is drawn from p_a.
 * The draw is the sampler's: the first column, in column order, at which the
 * running fixed-point mass exceeds U = draw_uniform[b] / 2^32 of the total.  A
 * filtered row's p_a draw is the token that rlk_sample gives for that word. */
typedef struct rlk_verify_args {
  int64_t B;                    /* sequences; B * (2 n + 1) < 2^28 */
  int32_t n;                    /* drafts per sequence at most, 0 .. 1024 */
  int32_t vocab_real;           /* must be RLK_VOCAB_REAL */
  int32_t vocab_padded;         /* must be RLK_VOCAB_PADDED */
  const void* logits;           /* bf16 [B * (n + 1)][row_stride], as in rlk_logp_args */
  int64_t row_stride;
  const void* draft_logits;     /* bf16 [B * n][draft_row_stride], or NULL: point masses */
  int64_t draft_row_stride;
  const int32_t* draft_token;   /* [B][n] */
  const int32_t* num_drafts;    /* [B], 0 .. n, or NULL: n each; rows past them are not read */
  /* the target's sampling parameters: by sequence [B], or NULL for the scalar */
  const float* temperature;  float temperature_scalar;
  const float* top_p;        float top_p_scalar;
  const int32_t* top_k;      int32_t top_k_scalar;
  /* the draft model's (ignored without draft_logits) */
  const float* draft_temperature;  float draft_temperature_scalar;
  const float* draft_top_p;        float draft_top_p_scalar;
  const int32_t* draft_top_k;      int32_t draft_top_k_scalar;
  const uint32_t* accept_uniform;   /* [B][n] random words */
  const uint32_t* draw_uniform;     /* [B] random words */
  int32_t* err_count;           /* optional device counter of rejected sequences */
} rlk_verify_args;

#define RLK_VERIFY_WORKSPACE_BYTES(B, n) ((size_t)(B) * (((size_t)(n) + 1u) * 2464u + (size_t)(n) * 32u))

/* out_token: int32 [B][n + 1], the accepted drafts, then the drawn token, then
 *   -1; out_accepted: int32 [B], a.
 * out_restr, out_full (optional): float [B][n + 1], the target's restricted and
 *   full logprobs of those tokens (bit-identical to rlk_logp_pair), then 0.
 * workspace: RLK_VERIFY_WORKSPACE_BYTES(B, n) bytes of device scratch, 16-byte
 *   aligned.
 * A sequence that comes to a row it cannot use (parameters or drafted token out
 * of their domains, logits that rlk_logp_pair answers with NaN, num_drafts[b]
 * out of range: then at place 0) stops there: token -1 and NaN logprobs at place
 * a, and err_count is raised by one.  Rows it does not come to are of no account. */
rlk_status rlk_verify_drafts(const rlk_verify_args* args, int32_t* out_token, int32_t* out_accepted,
                             float* out_restr, float* out_full, void* workspace, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* RLK_ROLLOUT_H */
