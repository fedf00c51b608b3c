"""GPU: attention over a shared prefix where lengths cross a bound of the parts that own tokens are
cut into, and what a call that fails leaves behind.

Inputs, float64 results and tolerances as in test_prefix_gpu.py; bits are compared as bits.
"""

import math

import pytest
import torch

import rollout_consistent_vocab_gb300 as pkg
from rollout_consistent_vocab_gb300 import _binding as b
from test_prefix_gpu import DEV, DT, U, bits, compare, i32, make, run

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _library():
    from rollout_consistent_vocab_gb300.build import build_library
    build_library()
    pkg.load_library()


# own tokens that the last of five new ones takes past the end of a part, and past lengths from which on parts are longer
OWN = [258, 4099, 8194, 8193, 16387, 32770]


@pytest.mark.parametrize("dtype,dim,page", [("bf16", 128, 16), ("f16", 64, 24)])
def test_drafted_tokens_have_the_bits_of_single_ones_where_parts_grow(dtype, dim, page):
    c = make([(2, 64), (1, 700)], OWN, 5, 8, 2, dim, page, dtype, seed=41)
    out, lse = run(c)
    compare(c, out, lse, [5] * len(OWN))
    for i in range(5):
        d = dict(c, q=c["q"][:, i:i + 1], lens=c["lens"] - 4 + i)
        o, z = run(d)
        assert torch.equal(bits(o[:, 0]), bits(out[:, i])) and torch.equal(bits(z[:, 0]), bits(lse[:, i])), i
    # the first three alone, in a call with room for five
    o, z = run(dict(c, lens=c["lens"] - 2), [3] * len(OWN))
    assert torch.equal(bits(o[:, :3]), bits(out[:, :3])) and torch.equal(bits(z[:, :3]), bits(lse[:, :3]))


def test_every_sequence_that_a_missing_page_rejects_is_counted():
    c = make([(20, 64), (3, 64)], [9] * 24, 1, 1, 1, 64, 16, "bf16", seed=42)
    err, pages = i32([0]), c["k"].shape[0]

    def count(d, new=None):
        err.zero_()
        out, lse = run(d, new, err_count=err)
        nan = torch.isnan(out).flatten(1).all(1)
        assert torch.equal(nan, torch.isnan(lse).flatten(1).all(1)) and torch.equal(nan, torch.isnan(out).flatten(1).any(1))
        return int(err), int(nan.sum())

    assert count(c) == (0, 0)
    for page in (-1, pages, 2**31 - 1):
        table = c["table"].clone()
        table[0, 1] = page                                       # a shared one
        raised, rejected = count(dict(c, table=table))
        assert rejected == 20 and raised >= 20
        table = c["table"].clone()
        table[21, 4] = table[23, 0] = page                       # own ones
        raised, rejected = count(dict(c, table=table))
        assert rejected == 2 and raised >= 2
    # sequences without new tokens have nothing to reject
    table = c["table"].clone()
    table[0, 1] = -1
    raised, rejected = count(dict(c, table=table), [1 if b % 2 else 0 for b in range(24)])
    assert rejected == 10 and raised >= 10


@pytest.mark.parametrize("dim,most,page", [(128, 64, 64), (64, 64, 16), (128, 0, 16)])
def test_a_refused_cache_leaves_the_workspace_alone(dim, most, page):
    # strides of 2^39 elements have no tensor map: nothing may be under way when the call says so
    c = make([(3, 64)], [9, 9, 9], 1, 4, 2, dim, page, "bf16", seed=43)
    tokens = page * c["table"].shape[1]
    ws = torch.full((pkg.prefix_attention_workspace_bytes(3, 1, 4, 2, dim, tokens, 1, most),), 255, dtype=torch.uint8, device=DEV)
    cache = b._make_cache(c["k"], c["v"], c["table"], c["lens"], None, 1, None)
    groups = b.PrefixGroups(c["start"].data_ptr(), c["shared"].data_ptr(), 1, most)
    out, strides = torch.zeros_like(c["q"]), b.BTHStrides(4 * dim, 0, dim)

    def call():
        status = pkg.load_library().rlk_prefix_attention(cache, groups, c["q"].data_ptr(), strides, 4, 0.1, out.data_ptr(), strides, None,
                                                         ws.data_ptr(), torch.cuda.current_stream().cuda_stream)
        torch.cuda.synchronize()
        return status

    cache.page_stride, stride = 2**40, cache.page_stride
    assert call() == b.RLK_EINVAL and bool((ws == 255).all()) and not out.any()
    cache.page_stride = stride
    assert call() == b.RLK_OK and not bool((ws == 255).all())


def test_a_bound_past_32_bits_is_refused():
    c = make([(2, 64)], [3, 4], 1, 4, 2, 64, 16, "bf16", seed=44)
    for most in (2**31, 2**32, 2**32 + 64, -2**32 + 64, -2**63):
        with pytest.raises(pkg.RlkError):
            run(c, max_shared=most)


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("bad", [math.inf, -math.inf, math.nan])
def test_values_that_are_not_finite_are_not_lost_for_their_weight(bad, dtype):
    """At a token whose weight is 0 in float32, shared or not, wherever it stands beside the weights that count."""
    shared, n, page, dim = 5000, 9000, 64, 64
    k = torch.zeros((-(-n // page) * page, 1, dim), dtype=DT[dtype], device=DEV)
    table, q = torch.arange(k.shape[0] // page, dtype=torch.int32, device=DEV)[None], torch.zeros((1, 1, 1, dim), dtype=DT[dtype], device=DEV)
    q[..., 0] = 1.0

    def attended(scores, values):
        k[:n, 0, 0] = scores.to(DT[dtype])
        v = torch.ones_like(k)
        v[:n, 0] = values.to(DT[dtype])[:, None]
        out, lse = pkg.prefix_attention(q, k.view(-1, page, 1, dim), v.view(-1, page, 1, dim), table, i32([n]), i32([0, 1]), i32([shared]),
                                        scale=1.0)
        return out[0, 0, 0], lse[0, 0, 0]

    for low in (-400.0, -math.inf):
        for at, heavy in ((0, 8999), (8999, 0), (600, 10), (10, 600), (3, 40), (40, 3), (2500, 100), (4990, 5010), (5300, 8000), (6000, 5998)):
            for every in (True, False):                          # all the others as light, or only those around
                scores, values = torch.full((n,), low if every else 0.0, device=DEV), torch.ones(n, device=DEV)
                scores[at // 512 * 512:at // 512 * 512 + 512] = low
                scores[heavy] = 0.0
                clean, lse = attended(scores, values)
                assert bool(((clean - 1.0).abs() <= 2 * U[dtype]).all()), (low, at, heavy, every)
                values[at] = bad
                got, z = attended(scores, values)
                assert not bool(torch.isfinite(got).any()), (low, at, heavy, every)
                assert torch.equal(bits(z), bits(lse))


def test_prompts_behind_a_shared_prefix():
    """Hundreds of new tokens of each sequence, some of their rows against the oracle, and the bits of all."""
    n, new = 300, [300, 277, 0, 1]
    c = make([(3, 700)], [300, 310, 5, 2], n, 8, 2, 64, 16, "bf16", seed=45)
    c["lens"] = i32([700 + 300, 700 + 310, 700 + 5, 2])
    out, lse = run(c, new)
    for b in (0, 1, 3):
        for i in sorted({0, new[b] // 2, new[b] - 1}):
            lens = c["lens"][b:b + 1] - new[b] + 1 + i
            d = dict(c, q=c["q"][b:b + 1, i:i + 1], table=c["whole"][b:b + 1].to(DEV), whole=c["whole"][b:b + 1], lens=lens, start=i32([0, 1]),
                     shared=i32([c["of"][b]]), of=c["of"][b:b + 1])
            o, z = run(d)
            compare(d, o, z, [1])
            assert torch.equal(bits(o[0, 0]), bits(out[b, i])) and torch.equal(bits(z[0, 0]), bits(lse[b, i])), (b, i)
        assert not out[b, new[b]:].any()


def test_many_sequences_with_a_few_long_ones():
    """More sequences than the plan has threads, own parts of three lengths, a workspace of just the size."""
    B, page, dim = 1500, 64, 64
    long = {0: 40000, 7: 16384, 8: 16385, 700: 33000, 1023: 32768, 1024: 32769, 1499: 20000}
    tails = [long.get(b, 1 + (37 * b) % 90) for b in range(B)]
    c = make([(700, 640), (500, 100)], tails, 1, 4, 2, dim, page, "bf16", seed=46, before=5)
    need = pkg.prefix_attention_workspace_bytes(B, 1, 4, 2, dim, page * c["table"].shape[1], 2, 640)
    ws = torch.full((need + 256,), 255, dtype=torch.uint8, device=DEV)
    out, lse = run(c, workspace=ws[:need], max_shared=640)
    assert bool((ws[need:] == 255).all()) and bool(torch.isfinite(out).all())
    compare(c, out, lse, [1] * B, rows=slice(0, B, 150))
    for b in (0, 5, 7, 8, 700, 1023, 1024, 1200, 1499):
        d = dict(c, q=c["q"][b:b + 1], table=c["whole"][b:b + 1].to(DEV), whole=c["whole"][b:b + 1], lens=c["lens"][b:b + 1], start=i32([0, 1]),
                 shared=i32([c["of"][b]]), of=c["of"][b:b + 1])
        o, z = run(d)
        compare(d, o, z, [1])
        assert torch.equal(bits(o[0]), bits(out[b])) and torch.equal(bits(z[0]), bits(lse[b])), b


def test_a_captured_step_that_grows_past_a_length_of_parts():
    c = make([(2, 64)], [16390, 32775, 16384], 2, 8, 2, 64, 16, "f16", seed=47)
    lens = c["lens"].clone()
    out, lse = run(c)
    g = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(g):
        run(c, out=out, out_lse=lse)
    for back in (20, 8, 5, 2, 0, 16300, 1):
        c["lens"].copy_(lens - back)
        g.replay()
        want, z = run(c)
        torch.cuda.synchronize()
        assert torch.equal(bits(out), bits(want)) and torch.equal(bits(lse), bits(z))
        compare(c, out, lse, [2] * 3)
