"""GPU: the serving operators together, as the example runs them."""

import os
import sys

import numpy as np
import pytest
import torch

import rollout_consistent_vocab_gb300 as pkg

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def example():
    from rollout_consistent_vocab_gb300.build import build_library
    build_library()
    pkg.load_library()
    import rollout_step
    return rollout_step


def _words(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def test_greedy_tokens_do_not_depend_on_the_drafts(example):
    """Temperature 0: the rollout with drafts emits what the one without does."""
    model, prompts = example.Model(), example.prompts_of(3)
    fast, slow = (example.Rollout(model, prompts, 40, 3) for _ in range(2))
    taken = 0
    for _ in range(10):
        taken += sum(fast.step(0.0, 1.0, -1, _words(1))[2])
    while min(len(s) - len(f) for s, f in zip(slow.tokens, fast.tokens)) < 0:
        slow.step(0.0, 1.0, -1, _words(1), speculate=False)
    assert taken > 0                     # some drafts stood
    for f, s, lf, ls in zip(fast.tokens, slow.tokens, fast.logprobs, slow.logprobs):
        assert s[:len(f)] == f
        assert ls[:len(lf)] == lf
    assert int(fast.errors) == 0 and int(slow.errors) == 0


@pytest.mark.parametrize("temperature,top_p,top_k", [(1.0, 0.95, 20), (0.7, 1.0, -1)])
def test_logprobs_are_those_of_the_training_side(example, temperature, top_p, top_k):
    """Every emitted token's logprob is logp_pair's on the step's logits."""
    r = example.Rollout(example.Model(seed=2), example.prompts_of(2, seed=3), 30, 2)
    g = _words(5)
    for _ in range(6):
        had = [len(p) for p in r.logprobs]
        logits, emitted, accepted = r.step(temperature, top_p, top_k, g)
        n = r.drafts + 1
        for b, toks in enumerate(emitted):
            assert len(toks) == accepted[b] + 1 and all(0 <= t < pkg.VOCAB_REAL for t in toks)
            target = torch.tensor(toks, dtype=torch.int32, device="cuda")
            full, restr, support = pkg.logp_pair(logits[b * n:b * n + len(toks)].contiguous(), target, temperature,
                                                 top_p, top_k)
            assert full.tolist() == r.logprobs[b][had[b]:]
            assert bool(torch.isfinite(restr).all()) and int(support.min()) >= 1
    assert int(r.errors) == 0


def test_command_runs(example, capsys):
    r = example.main(["--sequences", "2", "--drafts", "2", "--tokens", "12"])
    assert max(map(len, r.logprobs)) >= 12
    assert np.isfinite(np.concatenate([np.array(p) for p in r.logprobs])).all()
    assert "2 sequences" in capsys.readouterr().out
