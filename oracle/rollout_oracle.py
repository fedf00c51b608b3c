"""Plain CPU oracle for the rollout's serving operators: the paged key-value
cache (append, attention) and the verification of drafted tokens.

TEST INFRASTRUCTURE ONLY.  It shares no code with the CUDA path.  Everything
is numpy in float64, one query at a time, in the order in which
``include/rlk_rollout.h`` states the operators:

* new token i of sequence b is its token ``lens[b] - new[b] + i``; token t lies
  in page ``table[b][t // page_size]`` at place ``t % page_size``;
* a query at position pos sees the tokens j <= pos, with a window only those
  with j > pos - window and the first ``sinks`` of the sequence;
* out = sum_j exp(s_j - lse) v_j with s_j = scale q.k_j, lse = ln sum exp(s_j);
  a query that sees nothing gets 0 and -inf.
"""

from __future__ import annotations

import math

import numpy as np

from . import logp_oracle as lo


def token_place(table_row, t: int, page_size: int):
    return int(table_row[t // page_size]), t % page_size


def kv_append(k_cache, v_cache, table, lens, new, k, v):
    """Copies of the caches [pages, page_size, heads, dim] with the new tokens written."""
    k_cache, v_cache = np.array(k_cache), np.array(v_cache)
    for b in range(len(lens)):
        for i in range(new[b]):
            page, place = token_place(table[b], lens[b] - new[b] + i, k_cache.shape[1])
            k_cache[page, place] = k[b, i]
            v_cache[page, place] = v[b, i]
    return k_cache, v_cache


def visible(pos: int, window: int, sinks: int) -> np.ndarray:
    """Positions that a query at ``pos`` sees, ascending."""
    j = np.arange(pos + 1)
    return j if window == 0 else j[(j > pos - window) | (j < sinks)]


def attend(q, keys, values, scale: float):
    """(out, lse, bound) of one query over the rows of ``keys`` and ``values``.

    ``bound`` is what a result of limited precision is held to: sum_j p_j |v_j|
    per element, and sum_d |q_d k_jd| scale at its largest over j."""
    q, keys, values = (np.asarray(a, dtype=np.float64) for a in (q, keys, values))
    if len(keys) == 0:
        return np.zeros(values.shape[1]), -math.inf, (np.zeros(values.shape[1]), 0.0)
    s = scale * (keys @ q)
    m = s.max()
    e = np.exp(s - m)
    lse = m + math.log(e.sum())
    p = np.exp(s - lse)
    return p @ values, lse, (p @ np.abs(values), float((np.abs(keys) @ np.abs(q)).max()) * abs(scale))


def paged_attention(q, k_cache, v_cache, table, lens, new, scale: float, window: int = 0, sinks: int = 0):
    """(out [B, n, heads, dim], lse [B, n, heads], weight bound like out, score bound like lse) in float64."""
    B, n, heads, dim = q.shape
    page_size, kv_heads = k_cache.shape[1], k_cache.shape[2]
    group = heads // kv_heads
    out, lse = np.zeros((B, n, heads, dim)), np.full((B, n, heads), -math.inf)
    wb, sb = np.zeros((B, n, heads, dim)), np.zeros((B, n, heads))
    for b in range(B):
        pages = [int(p) for p in table[b][:-(-int(lens[b]) // page_size)]]
        keys = k_cache[pages].reshape(-1, kv_heads, dim)
        values = v_cache[pages].reshape(-1, kv_heads, dim)
        for i in range(new[b]):
            j = visible(int(lens[b]) - int(new[b]) + i, window, sinks)
            for h in range(heads):
                o, z, (w, x) = attend(q[b, i, h], keys[j, h // group], values[j, h // group], scale)
                out[b, i, h], lse[b, i, h], wb[b, i, h], sb[b, i, h] = o, z, w, x
    return out, lse, wb, sb


# ------------------------------------------------------------ verification of drafts

def restricted_row(bits_row, tau: float, top_p: float, top_k: int):
    """(probabilities, restricted logprobs, full logprobs) of a row's real tokens; None for
    a row that has no distribution (NaN or +inf logits, all -inf)."""
    x = lo.bf16_bits_to_f32(np.asarray(bits_row, dtype=np.uint16)[:lo.VREAL])
    if np.any(np.isnan(x)) or np.any(np.isposinf(x)) or np.all(np.isneginf(x)):
        return None
    if tau == 0.0:
        p = np.zeros(lo.VREAL)
        p[int(np.argmax(x))] = 1.0
        with np.errstate(divide="ignore"):
            return p, np.log(p), np.log(p)
    full, restr, S = lo.row_logprobs_all(bits_row, tau, top_p, top_k)
    return np.where(S, np.exp(restr), 0.0), restr, full


def draw_set(mass, word: int, eps: float):
    """Columns that the inverse CDF at U = word / 2^32 may give when the CDF is known to
    ``eps``: the first column whose running mass exceeds U of the total, and those whose
    interval comes within eps of it."""
    cols = np.nonzero(mass > 0)[0]
    cdf = np.cumsum(mass[cols]) / math.fsum(mass[cols])
    u = word / 2.0**32
    before = np.concatenate([[0.0], cdf[:-1]])
    return {int(c) for c in cols[(before - eps <= u) & (u < cdf + eps)]}


def verify_outcomes(target_rows, draft_rows, drafts, accept_words, draw_word: int, eps: float = 0.0):
    """Every (accepted, token) that rejection sampling may give with probabilities known to
    a relative ``eps`` (0: the one outcome).  target_rows: len(drafts) + 1 probability
    vectors; draft_rows: as many as drafts, or None (point masses at the drafts)."""
    out = set()
    for i, d in enumerate(drafts):
        q = np.zeros_like(target_rows[i])
        q[d] = 1.0
        q = q if draft_rows is None else draft_rows[i]
        left, right = (accept_words[i] >> 8) / 2.0**24 * q[d], target_rows[i][d]
        gap = eps * max(left, right)
        if left >= right - gap:                                 # may be refused
            r = np.maximum(target_rows[i] - q, 0.0)
            mass = math.fsum(r)
            # what is left after a cancellation is known to eps of p, not of itself
            out |= {(i, c) for c in (draw_set(r, draw_word, eps / mass) if mass > eps else
                                     draw_set(target_rows[i], draw_word, eps))}
            if left >= right + gap:                             # is refused
                return out
    return out | {(len(drafts), c) for c in draw_set(target_rows[-1], draw_word, eps)}
