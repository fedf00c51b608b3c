"""Pins of the rollout oracle: closed forms, a torch restatement in float64, and
planted mistakes that the pins must catch (CPU)."""

import math

import numpy as np
import pytest
import torch

from oracle import rollout as ro


def _case(seed=0, B=3, n=2, heads=4, kv_heads=2, dim=8, page=3, pages=20, lens=(7, 2, 11), new=(2, 2, 1)):
    r = np.random.default_rng(seed)
    table = np.stack([r.permutation(pages)[:5] for _ in range(B)])
    for b in range(1, B):                                       # pages of different sequences are distinct
        table[b] = np.setdiff1d(np.arange(pages), table[:b])[:5][r.permutation(5)]
    return dict(q=r.standard_normal((B, n, heads, dim)), k=r.standard_normal((pages, page, kv_heads, dim)),
                v=r.standard_normal((pages, page, kv_heads, dim)), table=table, lens=np.array(lens), new=np.array(new))


@pytest.mark.parametrize("window,sinks", [(0, 0), (3, 0), (3, 2), (1, 1), (100, 4)])
def test_attention_against_a_masked_softmax(window, sinks):
    c = _case()
    out, lse, wb, sb = ro.paged_attention(c["q"], c["k"], c["v"], c["table"], c["lens"], c["new"], 0.3, window, sinks)
    for b in range(3):
        keys = torch.from_numpy(c["k"][c["table"][b]].reshape(15, 2, 8))
        values = torch.from_numpy(c["v"][c["table"][b]].reshape(15, 2, 8))
        for i in range(2):
            pos = c["lens"][b] - c["new"][b] + i
            for h in range(4):
                x = 0.3 * keys[:, h // 2] @ torch.from_numpy(c["q"][b, i, h])
                ok = torch.tensor([j <= pos and (not window or j > pos - window or j < sinks) for j in range(15)])
                x = torch.where(ok, x, torch.tensor(-math.inf, dtype=torch.float64))
                if i >= c["new"][b]:
                    assert lse[b, i, h] == -math.inf and not out[b, i, h].any()
                    continue
                assert abs(lse[b, i, h] - torch.logsumexp(x, 0).item()) < 1e-12
                np.testing.assert_allclose(out[b, i, h], (torch.softmax(x, 0) @ values[:, h // 2]).numpy(), atol=1e-12)
                assert np.all(wb[b, i, h] + 1e-12 >= np.abs(out[b, i, h])) and sb[b, i, h] > 0


def test_attention_closed_forms():
    # equal scores: the mean of the values, lse = s + ln(count)
    out, lse, _ = ro.attend(np.zeros(4), np.ones((5, 4)), np.arange(20.0).reshape(5, 4), 1.0)
    np.testing.assert_allclose(out, [8.0, 9.0, 10.0, 11.0])
    assert abs(lse - math.log(5)) < 1e-15
    # one token: its value and its score
    out, lse, _ = ro.attend(np.array([2.0, 0.0]), np.array([[3.0, 1.0]]), np.array([[5.0, 7.0]]), 0.5)
    assert out.tolist() == [5.0, 7.0] and lse == 3.0
    out, lse, _ = ro.attend(np.ones(2), np.ones((0, 2)), np.ones((0, 2)), 1.0)
    assert out.tolist() == [0.0, 0.0] and lse == -math.inf


def test_visible_sets():
    assert ro.visible(4, 0, 3).tolist() == [0, 1, 2, 3, 4]
    assert ro.visible(9, 3, 2).tolist() == [0, 1, 7, 8, 9]
    assert ro.visible(2, 3, 2).tolist() == [0, 1, 2]
    assert ro.visible(5, 1, 0).tolist() == [5]


def test_append_places():
    c = _case()
    k = np.random.default_rng(1).standard_normal((3, 2, 2, 8))
    v = np.random.default_rng(2).standard_normal((3, 2, 2, 8))
    kc, vc = ro.kv_append(c["k"], c["v"], c["table"], c["lens"], c["new"], k, v)
    flat = lambda x, b: x[c["table"][b]].reshape(15, 2, 8)      # noqa: E731
    changed = 0
    for b in range(3):
        for t in range(15):
            i = t - (c["lens"][b] - c["new"][b])
            is_new = 0 <= i < c["new"][b]
            changed += is_new
            np.testing.assert_array_equal(flat(kc, b)[t], k[b, i] if is_new else flat(c["k"], b)[t])
            np.testing.assert_array_equal(flat(vc, b)[t], v[b, i] if is_new else flat(c["v"], b)[t])
    assert changed == 5 and (kc != c["k"]).any(axis=(2, 3)).sum() == 5


def _mutants():
    good = ro.visible
    return {
        "sees its successor": lambda pos, w, s: good(pos + 1, w, s),
        "not itself": lambda pos, w, s: good(pos, w, s)[:-1],
        "window one too wide": lambda pos, w, s: good(pos, w + 1 if w else 0, s),
        "no sinks": lambda pos, w, s: good(pos, w, 0),
    }


@pytest.mark.parametrize("name", list(_mutants()))
def test_planted_mistakes_are_caught(monkeypatch, name):
    monkeypatch.setattr(ro, "visible", _mutants()[name])
    with pytest.raises((AssertionError, IndexError)):
        for w, s in ((0, 0), (3, 2)):
            test_attention_against_a_masked_softmax(w, s)


# ------------------------------------------------------------ verification

def _probs(r, n, zeros=0):
    p = r.random(n) + 0.05
    p[r.permutation(n)[:zeros]] = 0.0
    return p / p.sum()


def _accept_word(u):
    return int(u * 2**24) << 8


def test_verification_emits_the_target_distribution():
    """Summed over a grid of random numbers and over drafts weighted by q, the first token has
    the target's probabilities: the identity min(p, q) + max(p - q, 0) = p."""
    r = np.random.default_rng(3)
    n, grid = 5, 400
    p, q = _probs(r, n, 1), _probs(r, n, 1)
    got = np.zeros(n)
    for d in range(n):
        if q[d] == 0:
            continue
        for a in range(grid):
            u = (a + 0.5) / grid
            word = [_accept_word(u)]
            if u * q[d] < p[d]:
                assert {x for x, _ in ro.verify_outcomes([p, p], [q], [d], word, 0)} == {1}
                got[d] += q[d] / grid
                continue
            for c in range(20):
                (res,) = ro.verify_outcomes([p, p], [q], [d], word, int((c + 0.5) / 20 * 2**32))
                assert res[0] == 0
                got[res[1]] += q[d] / grid / 20
    assert np.abs(got - p).max() < 0.03
    assert got[p == 0].sum() == 0


def test_verification_by_hand():
    p = np.array([0.5, 0.25, 0.25, 0.0])
    q = np.array([0.25, 0.25, 0.25, 0.25])
    w = lambda u: [_accept_word(u)] * 2                                  # noqa: E731
    # p >= q: accepted at every u; the bonus token by the inverse CDF
    assert ro.verify_outcomes([p, p, p], [q, q], [0, 1], w(0.999), int(0.6 * 2**32)) == {(2, 1)}
    # p = 0: refused at every u, and the residual is all at column 0
    assert ro.verify_outcomes([p, p, p], [q, q], [3, 1], w(0.0), int(0.9 * 2**32)) == {(0, 0)}
    # a point mass: refused at u >= p(d), the rest renormalised over the others
    assert ro.verify_outcomes([p, p], None, [0], w(0.4999)[:1], 0) == {(1, 0)}
    assert ro.verify_outcomes([p, p], None, [0], w(0.5)[:1], int(0.49 * 2**32)) == {(0, 1)}
    assert ro.verify_outcomes([p, p], None, [0], w(0.5)[:1], int(0.51 * 2**32)) == {(0, 2)}
    # no drafts: a plain draw, the word at an edge goes to the next column
    assert ro.verify_outcomes([p], None, [], [], 0) == {(0, 0)}
    assert ro.verify_outcomes([p], None, [], [], 2**31) == {(0, 1)}
    assert ro.verify_outcomes([p], None, [], [], 2**31, eps=1e-6) == {(0, 0), (0, 1)}


def test_verification_mutants(monkeypatch):
    src = ro.verify_outcomes
    mutants = {
        "accepts on >": lambda t, q, d, a, w, eps=0.0: src(t, q, d, [2**32 - 1 - x for x in a], w, eps),
        "draws from p": lambda t, q, d, a, w, eps=0.0: {(i, next(iter(ro.draw_set(t[i], w, 0)))) for i, _ in src(t, q, d, a, w, eps)},
        "bonus from the last draft's row": lambda t, q, d, a, w, eps=0.0: src(t[:-1] + [1 - t[-1]], q, d, a, w, eps),
    }
    for name, m in mutants.items():
        monkeypatch.setattr(ro, "verify_outcomes", m)
        with pytest.raises(AssertionError):
            test_verification_by_hand()
    monkeypatch.setattr(ro, "verify_outcomes", src)
    test_verification_by_hand()


def test_restricted_row_is_the_pinned_one():
    from oracle import logp_oracle as lo
    x = np.full(lo.VPAD, -4.0, dtype=np.float32)
    x[[3, 10, 11]] = [2.0, 1.0, 1.0]
    x[lo.VREAL:] = np.nan
    bits = (x.view(np.uint32) >> 16).astype(np.uint16)
    p, lr, lf = ro.restricted_row(bits, 1.0, 1.0, 2)                     # ties at the k-th value are kept
    e = np.exp(-1.0)
    assert np.count_nonzero(p) == 3 and abs(p[3] - 1 / (1 + 2 * e)) < 1e-12 and abs(p[10] - e / (1 + 2 * e)) < 1e-12
    assert abs(lr[3] - np.log(p[3])) < 1e-12 and lr[5] == -np.inf and np.isfinite(lf[5])
    p, lr, lf = ro.restricted_row(bits, 0.0, 1.0, -1)
    assert p[3] == 1.0 and p.sum() == 1.0 and lr[3] == lf[3] == 0.0
    x[0] = np.nan
    assert ro.restricted_row((x.view(np.uint32) >> 16).astype(np.uint16), 1.0, 1.0, -1) is None
