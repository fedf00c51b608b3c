"""A speculative rollout with the serving operators, end to end on one GPU.

A model of one attention layer and an LM head continues a few prompts (random weights;
its LM head likes to go round cycles of eight tokens, so that there is something to guess).  Each step drafts tokens for every sequence by
looking its last token up in what the sequence already holds, and then runs

    kv_append  ->  paged_attention  ->  LM head  ->  verify_drafts

over the pending token and its drafts.  The tokens that come out are distributed as
those of a rollout without drafts, and their logprobs are logp_pair's, bit for bit:
what the training side recomputes.

    python examples/rollout_step.py [--drafts 3] [--tokens 48] [--temperature 1.0]
"""

import argparse
import os
import sys

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import torch

import rollout_consistent_vocab_gb300 as rlk

VPAD, VREAL = rlk.VOCAB_PADDED, rlk.VOCAB_REAL
HIDDEN, Q_HEADS, KV_HEADS, HEAD_DIM, PAGE = 256, 4, 2, 64, 16


class Model:
    """One attention layer and the LM head.  Every step has the same shapes, drafts or none,
    so a row of the library's matrix products has the same bits whatever the others hold."""

    def __init__(self, seed=0, device="cuda"):
        g = torch.Generator(device=device)
        g.manual_seed(seed)

        def weight(rows, cols, size):
            return (size * torch.randn((rows, cols), generator=g, device=device)).to(torch.bfloat16)

        self.embedding = weight(VREAL, HIDDEN, 1.0)
        self.wq = weight(HIDDEN, Q_HEADS * HEAD_DIM, HIDDEN**-0.5)
        self.wk = weight(HIDDEN, KV_HEADS * HEAD_DIM, HIDDEN**-0.5)
        self.wv = weight(HIDDEN, KV_HEADS * HEAD_DIM, HIDDEN**-0.5)
        self.wo = weight(Q_HEADS * HEAD_DIM, HIDDEN, HIDDEN**-0.5)
        t = torch.arange(VREAL, device=device)
        self.head = torch.zeros((VPAD, HIDDEN), dtype=torch.bfloat16, device=device)
        self.head[:VREAL] = 0.06 * self.embedding[t - t % 8 + (t + 7) % 8]       # t follows this one

    def keys_values(self, x):
        B, n = x.shape[:2]
        return (x @ self.wk).view(B, n, KV_HEADS, HEAD_DIM), (x @ self.wv).view(B, n, KV_HEADS, HEAD_DIM)


class Rollout:
    """Sequences in a paged cache.  The cache holds each sequence's tokens but the last one,
    which goes in with the step that reads its logits."""

    def __init__(self, model, prompts, max_tokens, drafts, device="cuda"):
        self.model, self.drafts, self.device = model, drafts, device
        self.tokens = [list(p) for p in prompts]
        self.logprobs = [[] for _ in prompts]
        B, pages = len(prompts), -(-(max(map(len, prompts)) + max_tokens + drafts + 1) // PAGE)
        self.k_cache = torch.empty((B * pages, PAGE, KV_HEADS, HEAD_DIM), dtype=torch.bfloat16, device=device)
        self.v_cache = torch.empty_like(self.k_cache)
        self.table = torch.randperm(B * pages, device=device).to(torch.int32).view(B, pages)
        self.errors = torch.zeros(1, dtype=torch.int32, device=device)
        self.workspace = torch.empty(rlk.paged_attention_workspace_bytes(
            B, drafts + 1, Q_HEADS, KV_HEADS, HEAD_DIM, pages * PAGE), dtype=torch.uint8, device=device)
        # the prompts' keys and values (one layer: they need no attention of their own)
        new = [len(p) - 1 for p in prompts]
        x = self._embed([p[:-1] for p in prompts], max(max(new), 1))
        k, v = model.keys_values(x)
        lens = self._ints(new)
        rlk.kv_append(self.k_cache, self.v_cache, self.table, lens, k, v, new_lens=lens, err_count=self.errors)

    def _ints(self, values):
        return torch.tensor(values, dtype=torch.int32, device=self.device)

    def _embed(self, rows, width):
        ids = torch.zeros((len(rows), width), dtype=torch.long)
        for b, r in enumerate(rows):
            ids[b, :len(r)] = torch.tensor(r, dtype=torch.long)
        return self.model.embedding[ids.to(self.device)]

    def _look_up(self, seq, most):
        """What followed the last token where the sequence held it before."""
        for at in range(len(seq) - 2, -1, -1):
            if seq[at] == seq[-1]:
                return seq[at + 1:at + 1 + most]
        return []

    def step(self, temperature, top_p, top_k, generator, speculate=True):
        """One step of all sequences; returns (logits, emitted tokens by sequence, accepted)."""
        m, n, B = self.model, self.drafts, len(self.tokens)
        drafts = [self._look_up(s, n) if speculate else [] for s in self.tokens]
        x = self._embed([[s[-1]] + d for s, d in zip(self.tokens, drafts)], n + 1)
        new = self._ints([1 + len(d) for d in drafts])
        lens = self._ints([len(s) + len(d) for s, d in zip(self.tokens, drafts)])
        k, v = m.keys_values(x)
        rlk.kv_append(self.k_cache, self.v_cache, self.table, lens, k, v, new_lens=new, err_count=self.errors)
        q = (x @ m.wq).view(B, n + 1, Q_HEADS, HEAD_DIM)
        a, _ = rlk.paged_attention(q, self.k_cache, self.v_cache, self.table, lens, new_lens=new,
                                   workspace=self.workspace, err_count=self.errors)
        h = x + a.view(B, n + 1, -1) @ m.wo
        logits = h.view(B * (n + 1), HIDDEN) @ m.head.T
        words = torch.randint(-2**31, 2**31, (B * (n + 1),), generator=generator, device=self.device).to(torch.int32)
        token, accepted, restr, full = rlk.verify_drafts(
            logits, self._ints([d + [0] * (n - len(d)) for d in drafts]).view(B, n), temperature, top_p, top_k,
            num_drafts=self._ints([len(d) for d in drafts]), accept_uniform=words[:B * n].view(B, n),
            draw_uniform=words[B * n:], err_count=self.errors)
        token, accepted, full = token.tolist(), accepted.tolist(), full.tolist()
        emitted = [t[:a + 1] for t, a in zip(token, accepted)]
        # what was not accepted stays in the cache past the sequence's end, and is written over
        for b, t in enumerate(emitted):
            self.tokens[b] += t
            self.logprobs[b] += full[b][:len(t)]
        return logits, emitted, accepted


def prompts_of(count, seed=0):
    """Prompts that repeat a phrase, of different lengths."""
    g = torch.Generator()
    g.manual_seed(seed)
    out = []
    for b in range(count):
        phrase = torch.randint(0, VREAL, (5 + 3 * b,), generator=g).tolist()
        out.append(phrase * 3 + phrase[:2])
    return out


def main(argv=None):
    p = argparse.ArgumentParser(description=__doc__.split("\n")[0])
    p.add_argument("--sequences", type=int, default=4)
    p.add_argument("--drafts", type=int, default=3)
    p.add_argument("--tokens", type=int, default=48, help="new tokens of the longest sequence, at least")
    p.add_argument("--temperature", type=float, default=1.0)
    p.add_argument("--top-p", type=float, default=0.95)
    p.add_argument("--top-k", type=int, default=20)
    a = p.parse_args(argv)
    prompts = prompts_of(a.sequences)
    r = Rollout(Model(), prompts, a.tokens + a.drafts, a.drafts)
    g = torch.Generator(device="cuda")
    g.manual_seed(1)
    steps = accepted = 0
    while max(len(s) - len(q) for s, q in zip(r.tokens, prompts)) < a.tokens:
        _, _, acc = r.step(a.temperature, a.top_p, a.top_k, g)
        steps, accepted = steps + 1, accepted + sum(acc)
    assert int(r.errors) == 0
    made = sum(len(s) - len(q) for s, q in zip(r.tokens, prompts))
    print(f"{len(prompts)} sequences, {steps} steps, {made} tokens ({accepted} of them drafted), "
          f"mean logprob {sum(map(sum, r.logprobs)) / made:.3f}")
    return r


if __name__ == "__main__":
    main()
