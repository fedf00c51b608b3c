"""GPU: paged attention where single weights, values or lengths lie at the edge of their formats.

Inputs, float64 results and tolerances as in test_paged_gpu.py; what a test adds to them
is stated beside it.
"""

import math

import numpy as np
import pytest
import torch

import rollout_consistent_vocab_gb300 as pkg
from oracle import rollout as ro
from test_paged_gpu import DEV, DT, U, i32, np64

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _library():
    from rollout_consistent_vocab_gb300.build import build_library
    build_library()
    pkg.load_library()


def row_of(scores, values, dtype, dim, page=64):
    """One query whose score of token j is scores[j] (scale 1), over values[j] in every place."""
    n = len(scores)
    pages = -(-n // page)
    k = torch.zeros((pages * page, 1, dim), dtype=DT[dtype], device=DEV)
    v = torch.full_like(k, math.nan)
    k[:n, 0, 0] = torch.as_tensor(scores, device=DEV).to(DT[dtype])
    v[:n, 0] = torch.as_tensor(values, device=DEV).to(DT[dtype])[:, None]
    q = torch.zeros((1, 1, 1, dim), dtype=DT[dtype], device=DEV)
    q[..., 0] = 1.0
    table = torch.arange(pages, dtype=torch.int32, device=DEV)[None]
    got = pkg.paged_attention(q, k.view(pages, page, 1, dim), v.view(pages, page, 1, dim), table, i32([n]), scale=1.0)
    return got, np64(q)[0, 0, 0], np64(k)[:n, 0], np64(v)[:n, 0]


def attended(scores, values, dtype, dim=64):
    (out, lse), _, _, _ = row_of(scores, values, dtype, dim)
    return np64(out)[0, 0, 0], float(lse[0, 0, 0])


def one_row(scores, values, dtype, dim=64):
    """(result, float64 result, tolerance, values)"""
    (out, _), q, k, v = row_of(scores, values, dtype, dim)
    want, _, (A, X) = ro.attend(q, k, v, 1.0)
    ds = 2 * (dim + 4) * 2.0**-24 * X + 2.0**-18
    tol = U[dtype] * np.abs(want) + (U[dtype] + ds) * A * (1 + 2.0**-7)
    return np64(out)[0, 0, 0], want, tol, v


# f16: a weight is held to 22 bits, but to no less than 2^-44 of the row's largest
STEP = 2.0**-44


@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("gap", [16.0, 20.75, 23.5, 27.0])
@pytest.mark.parametrize("tokens", [40, 2000, 131071])
def test_f16_weights_far_below_the_largest(tokens, gap, dim):
    """A first token that takes all the weight and has no value: the result is the others'."""
    rng = np.random.default_rng(tokens)
    scores = np.concatenate([[0.0], -gap + rng.uniform(-0.5, 0.5, tokens - 1)])
    values = np.concatenate([[0.0], rng.uniform(500.0, 1500.0, tokens - 1)])
    got, want, tol, v = one_row(scores, values, "f16", dim)
    tol = tol + 2.0**-24 + STEP * np.abs(v).sum(0)
    assert np.all(np.abs(got - want) <= tol), (np.abs(got - want) / tol).max()


def test_f16_values_near_the_largest_on_tokens_of_no_weight():
    for gap in (25.0, 40.0, 60.0):
        for n in (2, 33):
            got, want, tol, v = one_row([0.0] + [-gap] * (n - 1), [1e-3] + [60000.0] * (n - 1), "f16")
            tol = tol + 2.0**-24 + STEP * np.abs(v).sum(0)
            assert np.all(np.abs(got - want) <= tol), (gap, n, got[0], want[0])


def test_f16_infinite_values_in_the_middle_of_a_sequence():
    """An infinite value that every query sees, at a token of ordinary weight."""
    for at in (0, 1, 100, 700):
        for bad in (math.inf, -math.inf):
            values = np.ones(1500)
            values[at] = bad
            k = np.zeros(1500)
            k[::3] = -3.0
            got = one_row(k, values, "f16")[0]
            assert np.all(got == bad), (at, bad, got[:4])


def test_the_longest_sequence():
    """2^31 - 16 tokens, from one page that the table holds again and again."""
    page, width, dim, n = 8176, 262657, 64, 2
    length = page * width
    assert length == 2**31 - 16
    table = torch.zeros((1, width), dtype=torch.int32, device=DEV)
    lens = i32([length])
    g = torch.Generator(device=DEV)
    g.manual_seed(30)
    q = torch.randn((1, n, 2, dim), generator=g, device=DEV).to(torch.bfloat16)
    k = torch.zeros((1, page, 1, dim), dtype=torch.bfloat16, device=DEV)
    v = torch.zeros_like(k)
    for d in range(dim):
        v[0, ::d + 2, 0, d] = 1.0
    # all scores 0: the mean of the values.  Every partial sum is a whole number, exact in float32
    # up to 2^24 of its units of 2048 and more
    once = np64(v)[0, :, 0]
    for kw in ({}, {"window": 5, "sinks": 2**31 - 1}):
        out, lse = pkg.paged_attention(q, k, v, table, lens, **kw)
        for i in range(n):
            seen = length - n + 1 + i
            want = (width * once.sum(0) - once[page - n + 1 + i:].sum(0)) / seen
            assert np.all(np.abs(np64(out)[0, i] - want) <= (2 * U["bf16"] + 2.0**-20) * want)     # rounded once
            assert np.all(np.abs(np64(lse)[0, i] - math.log(seen)) <= 2.0**-18 + 2.0**-23 * math.log(seen))
    # a window at the end, and the first tokens
    k.copy_(torch.randn(k.shape, generator=g, device=DEV))
    v.copy_(torch.randn(v.shape, generator=g, device=DEV))
    for window, sinks in ((1000, 4), (1, 0), (3000, 600)):
        out, lse = pkg.paged_attention(q, k, v, table, lens, window=window, sinks=sinks)
        for i in range(n):
            pos = length - n + i
            j = np.concatenate([np.arange(sinks), np.arange(pos - window + 1, pos + 1)]) % page
            for h in range(2):
                o, z, (A, X) = ro.attend(np64(q)[0, i, h], np64(k)[0, j, 0], np64(v)[0, j, 0], dim**-0.5)
                ds = 2 * (dim + 4) * 2.0**-24 * X + 2.0**-18
                tol = U["bf16"] * np.abs(o) + (U["bf16"] + ds) * A * (1 + 2.0**-7)
                assert np.all(np.abs(np64(out)[0, i, h] - o) <= tol)
                assert abs(float(lse[0, i, h]) - z) <= ds + 2.0**-23 * abs(z)
    # the last token's place
    new = torch.randn((1, 1, 1, dim), generator=g, device=DEV).to(torch.bfloat16)
    pkg.kv_append(k, v, table, lens, new, -new)
    assert torch.equal(k[0, page - 1, 0], new[0, 0, 0]) and torch.equal(v[0, page - 1, 0], -new[0, 0, 0])


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("bad", [math.inf, -math.inf, math.nan])
def test_values_that_are_not_finite_are_not_lost_for_their_weight(bad, dtype):
    """At a token whose weight is 0 in float32, wherever it stands beside the weights that count."""
    n = 9000
    for low in (-400.0, -math.inf):
        for at, heavy in ((0, 8999), (8999, 0), (600, 10), (10, 600), (3, 40), (40, 3), (2500, 100), (100, 2500), (33, 33 + 32)):
            for every in (True, False):      # all the others as light, or only those around
                scores = np.full(n, low) if every else np.zeros(n)
                scores[at // 512 * 512:at // 512 * 512 + 512] = low
                scores[heavy] = 0.0
                values = np.ones(n)
                clean, lse = attended(scores, values, dtype)
                assert np.all(np.abs(clean - 1.0) <= 2 * U[dtype]), (low, at, heavy, every)
                values[at] = bad
                got, z = attended(scores, values, dtype)
                assert not np.isfinite(got).any(), (low, at, heavy, every, got[:4])
                assert z == lse


def test_a_page_table_without_pages():
    """[B, 0]: every sequence is still empty."""
    for pages in (4, 0):
        k = torch.zeros((pages, 16, 2, 64), dtype=torch.bfloat16, device=DEV)
        table = torch.zeros((3, 0), dtype=torch.int32, device=DEV)
        q = torch.ones((3, 2, 8, 64), dtype=torch.bfloat16, device=DEV)
        err = torch.zeros(1, dtype=torch.int32, device=DEV)
        pkg.kv_append(k, k, table, i32([0, 0, 0]), q[:, :, :2], q[:, :, :2], new_lens=i32([0, 0, 0]), err_count=err)
        out, lse = pkg.paged_attention(q, k, k, table, i32([0, 0, 0]), new_lens=i32([0, 0, 0]), err_count=err)
        assert not out.any() and torch.all(lse == -math.inf) and int(err) == 0
        out, lse = pkg.paged_attention(q, k, k, table, i32([0, 1, 0]), new_lens=i32([0, 1, 0]), err_count=err)
        assert torch.isnan(out[1]).all() and torch.isnan(lse[1]).all() and not out[[0, 2]].any() and int(err) >= 1


def test_a_call_without_its_workspace_is_refused():
    k = torch.zeros((4, 16, 2, 64), dtype=torch.bfloat16, device=DEV)
    q = torch.ones((1, 1, 8, 64), dtype=torch.bfloat16, device=DEV)
    with pytest.raises(ValueError):
        pkg.paged_attention(q, k, k, i32([[0, 1]]), i32([3]), workspace=torch.empty(0, dtype=torch.uint8, device=DEV))
