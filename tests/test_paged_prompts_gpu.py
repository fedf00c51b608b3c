"""GPU: paged attention of prompts (many tiles of query rows), of batches that mix them with
single tokens, and under windows: against the float64 oracle, and the same bits however the
tokens are brought together.  Inputs and tolerances as in test_paged_gpu.py."""

import math

import pytest
import torch

import rollout_consistent_vocab_gb300 as pkg
from test_paged_gpu import DEV, compare, i32, make, run

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _library():
    from rollout_consistent_vocab_gb300.build import build_library
    build_library()
    pkg.load_library()


@pytest.mark.parametrize("window,sinks", [(0, 0), (100, 4), (1, 0), (600, 1)])
@pytest.mark.parametrize("dim,dtype,heads,kv_heads,page", [(128, "bf16", 4, 2, 16), (64, "f16", 3, 1, 24), (64, "bf16", 2, 2, 100)])
def test_prompts_match_the_oracle(dim, dtype, heads, kv_heads, page, window, sinks):
    # a whole prompt, a chunk after a prefix, a single token, an empty sequence
    lens, new, n = [610, 900, 700, 0, 33], [610, 300, 1, 0, 33], 610
    c = make(lens, n, heads, kv_heads, dim, page, dtype, seed=dim + heads)
    out, lse = run(c, new, window=window, sinks=sinks)
    compare(c, out, lse, new, dtype, window=window, sinks=sinks)
    for b, m in enumerate(new):
        assert not out[b, m:].any() and torch.all(lse[b, m:] == -math.inf)


@pytest.mark.parametrize("window,sinks", [(0, 0), (700, 3), (64, 0)])
@pytest.mark.parametrize("dim,dtype", [(128, "bf16"), (64, "f16")])
def test_a_prompt_in_chunks_and_token_by_token(dim, dtype, window, sinks):
    """2600 tokens at once, in chunks of every kind, and single tokens: the same bits."""
    n = 2600
    c = make([n], n, 8, 2, dim, 16, dtype, seed=50)
    whole, lse = run(c, window=window, sinks=sinks)
    at = 0
    for m in (1, 5, 506, 512, 511, 1000, 64, 1):
        o, z = pkg.paged_attention(c["q"][:, at:at + m], c["k"], c["v"], c["table"], i32([at + m]), window=window, sinks=sinks)
        assert torch.equal(o, whole[:, at:at + m]) and torch.equal(z, lse[:, at:at + m]), (at, m)
        at += m
    assert at == n
    # beside other sequences, with fewer new tokens than the call has places for
    q = torch.zeros((3, 700, 8, dim), dtype=c["q"].dtype, device=DEV)
    q[0, :3], q[1], q[2, :1] = c["q"][0, 1500:1503], c["q"][0, 1900:], c["q"][0, 77:78]
    o, z = pkg.paged_attention(q, c["k"], c["v"], c["table"].repeat(3, 1), i32([1503, 2600, 78]), new_lens=i32([3, 700, 1]),
                               window=window, sinks=sinks)
    for b, (a, m) in enumerate(((1500, 3), (1900, 700), (77, 1))):
        assert torch.equal(o[b, :m], whole[0, a:a + m]) and torch.equal(z[b, :m], lse[0, a:a + m]), b


def test_a_long_prompt():
    """More than 2^16 query rows of a kv head."""
    n = 5000
    c = make([n], n, 16, 1, 64, 64, "bf16", seed=51)
    whole, lse = run(c)
    for at in (0, 1, 511, 512, 2049, 4096, 4999):
        o, z = pkg.paged_attention(c["q"][:, at:at + 1], c["k"], c["v"], c["table"], i32([at + 1]))
        assert torch.equal(o, whole[:, at:at + 1]) and torch.equal(z, lse[:, at:at + 1]), at
    assert torch.isfinite(whole).all()
