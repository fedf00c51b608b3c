"""GPU: the verification of drafted tokens against the float64 oracle.

A decision is compared where it is not within 4e-6 (relative, for acceptances;
of the CDF, for draws) of an edge: float32 probabilities carry a few 1e-7, as do
the sampler's draws, which are counted within 2e-6.  Within it either outcome
stands.  Logprobs: the library's tolerance for rlk_logp_pair (2e-5), and bit for
bit what rlk_logp_pair gives for the same tokens.
"""

import math

import numpy as np
import pytest
import torch

import oracle
import rollout_consistent_vocab_gb300 as pkg
from _support import bits_of, param_at
from oracle import rollout as ro

pytestmark = pytest.mark.gpu
DEV = "cuda"
EPS = 4e-6


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from rollout_consistent_vocab_gb300.build import build_library
    build_library()
    pkg.load_library()


def make(B, n, seed, noise=0.5, hot=64, pick=20):
    """Target and draft rows that are near one another, and drafts that the draft model would give."""
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    x = 4.0 * torch.randn((B, n + 1, oracle.VPAD), generator=g, device=DEV)
    x += 12.0 * (torch.rand(x.shape, generator=g, device=DEV) < hot / oracle.VREAL)
    y = x[:, :n] + noise * torch.randn((B, n, oracle.VPAD), generator=g, device=DEV)
    x[..., oracle.VREAL:] = math.nan                                     # padded columns are never read
    y[..., oracle.VREAL:] = math.inf
    x = x.reshape(-1, oracle.VPAD).to(torch.bfloat16)
    y = y.reshape(-1, oracle.VPAD).to(torch.bfloat16)
    top = y[:, :oracle.VREAL].float().topk(pick, dim=1)
    noise = -torch.log(-torch.log(torch.rand(top.values.shape, generator=g, device=DEV).clamp(1e-9)))
    d = top.indices.gather(1, (top.values / 1.5 + noise).argmax(1, keepdim=True)).reshape(B, n).to(torch.int32)
    words = lambda *s: torch.randint(-2**31, 2**31, s, generator=g, device=DEV, dtype=torch.int64).to(torch.int32)  # noqa: E731
    return dict(x=x, y=y, d=d, a=words(B, n), w=words(B))


def run(c, tau=1.0, p=1.0, k=-1, draft=True, **kw):
    return pkg.verify_drafts(c["x"], c["d"], tau, p, k, draft_logits=c["y"] if draft else None,
                             accept_uniform=c["a"], draw_uniform=c["w"], **kw)


def u32(t):
    return t.cpu().numpy().view(np.uint32).astype(np.int64)


def rows_of(bits, b, per, m, tau, p, k):
    out = [ro.restricted_row(bits[b * per + i], float(np.float32(param_at(tau, b))), float(np.float32(param_at(p, b))),
                             int(param_at(k, b))) for i in range(m)]
    return out


def compare(c, got, tau, p, k, draft=True, num=None, dtau=None, dp=None, dk=None):
    """Token, accepted and logprobs of every sequence against the oracle; returns the number of
    sequences with more than one outcome within EPS."""
    token, accepted, restr, full = (t.cpu().numpy() for t in got)
    B, n = c["d"].shape
    xb, yb = bits_of(c["x"]), bits_of(c["y"]) if draft else None
    d, a, w = c["d"].cpu().numpy(), u32(c["a"]), u32(c["w"])
    near = 0
    for b in range(B):
        m = n if num is None else num[b]
        t_rows = rows_of(xb, b, n + 1, m + 1, tau, p, k)
        q_rows = rows_of(yb, b, n, m, tau if dtau is None else dtau, p if dp is None else dp,
                         k if dk is None else dk) if draft else None
        want = ro.verify_outcomes([r[0] for r in t_rows], [r[0] for r in q_rows] if draft else None,
                                  d[b, :m].tolist(), a[b].tolist(), int(w[b]), EPS)
        near += len(want) > 1
        at = int(accepted[b])
        assert (at, int(token[b, at])) in want, (b, at, int(token[b, at]), sorted(want)[:8])
        assert token[b, :at].tolist() == d[b, :at].tolist()
        assert np.all(token[b, at + 1:] == -1)
        assert not restr[b, at + 1:].any() and not full[b, at + 1:].any()
        for i in range(at + 1):
            tok = int(token[b, i])
            assert abs(restr[b, i] - t_rows[i][1][tok]) <= 2e-5 and abs(full[b, i] - t_rows[i][2][tok]) <= 2e-5
    return near


SETTINGS = [(0.7, 0.95, 50), (1.3, 0.99, 128), (1.0, 1.0, 20), (1.3, 0.9, -1), (0.6, 1.0, 1), (1.0, 1.0, 2000),
            (0.0, 1.0, -1)]


@pytest.mark.parametrize("tau,p,k", SETTINGS)
@pytest.mark.parametrize("draft", [True, False])
def test_verification_matches_the_oracle(tau, p, k, draft):
    c = make(7, 3, seed=int(10 * tau) + k + 2)
    if tau == 0.0:                                             # greedy drafts: some the target's own
        best = c["y"][:, :oracle.VREAL].float().argmax(1).to(torch.int32).reshape(7, 3)
        c["d"] = torch.where(torch.arange(7, device=DEV)[:, None] % 2 == 0, best, c["d"])
    got = run(c, tau, p, k, draft)
    assert compare(c, got, tau, p, k, draft) <= 2


def test_unfiltered_rows():
    c = make(6, 2, seed=30)
    for draft in (True, False):
        got = run(c, 1.0, 1.0, -1, draft)
        compare(c, got, 1.0, 1.0, -1, draft)


def test_settings_by_sequence_and_ragged_drafts():
    B, n = 12, 4
    c = make(B, n, seed=31)
    pick = [SETTINGS[i % len(SETTINGS)] for i in range(B)]
    tau = torch.tensor([v[0] for v in pick], device=DEV)
    p = torch.tensor([v[1] for v in pick], device=DEV)
    k = torch.tensor([v[2] for v in pick], dtype=torch.int32, device=DEV)
    best = c["y"][:, :oracle.VREAL].float().argmax(1).to(torch.int32).reshape(B, n)
    c["d"] = torch.where((tau == 0)[:, None], best, c["d"])
    num = [i % (n + 1) for i in range(B)]
    for b in range(B):                                         # what lies past a sequence's drafts is not read
        c["x"][b * (n + 1) + num[b] + 1:(b + 1) * (n + 1)] = math.nan
        c["y"][b * n + num[b]:(b + 1) * n] = math.nan
        c["d"][b, num[b]:] = -5
    got = run(c, tau, p, k, num_drafts=torch.tensor(num, dtype=torch.int32, device=DEV))
    compare(c, got, tau, p, k, num=num)
    # the draft model's own settings
    dtau, dk = 1.1, 40
    got = run(c, tau, p, k, num_drafts=torch.tensor(num, dtype=torch.int32, device=DEV), draft_temperature=dtau,
              draft_top_p=1.0, draft_top_k=dk)
    compare(c, got, tau, p, k, num=num, dtau=dtau, dp=1.0, dk=dk)


def test_greedy_draft_for_a_sampling_target():
    c = make(8, 2, seed=32)
    c["d"] = c["y"][:, :oracle.VREAL].float().argmax(1).to(torch.int32).reshape(8, 2)
    got = run(c, 1.2, 1.0, 100, draft_temperature=0.0)
    compare(c, got, 1.2, 1.0, 100, dtau=0.0)


def test_no_drafts_is_the_sampler():
    c = make(40, 0, seed=33)
    for tau, p, k in ((0.7, 0.95, 50), (1.3, 0.99, 128), (1.3, 0.99, -1), (0.0, 1.0, -1)):
        token, accepted, restr, full = pkg.verify_drafts(c["x"], c["d"], tau, p, k, accept_uniform=c["a"], draw_uniform=c["w"])
        t, r, f, _ = pkg.sample(c["x"], tau, p, k, uniform=c["w"])
        assert torch.equal(token[:, 0], t) and torch.equal(restr[:, 0], r) and torch.equal(full[:, 0], f)
        assert not accepted.any()


def test_logprobs_are_the_pair_passs():
    c = make(10, 4, seed=34)
    for tau, p, k in ((0.7, 0.95, 50), (1.3, 0.99, -1), (1.0, 1.0, -1)):
        token, accepted, restr, full = run(c, tau, p, k)
        there = (token >= 0).reshape(-1)
        f, r, _ = pkg.logp_pair(c["x"], token.reshape(-1).clamp(min=0), tau, p, k)
        assert torch.equal(full.reshape(-1)[there], f[there]) and torch.equal(restr.reshape(-1)[there], r[there])
        assert int(there.sum()) == int(accepted.sum()) + 10


def test_same_draft_and_target_accepts_all():
    c = make(6, 3, seed=35, noise=0.0)
    c["a"].fill_(-1)                                           # the largest random word
    for tau, p, k in ((1.0, 1.0, 20), (1.3, 0.99, -1), (0.9, 1.0, -1)):
        _, accepted, _, _ = run(c, tau, p, k)
        assert torch.all(accepted == 3)


def test_residual_without_mass_falls_back_to_the_target():
    # a draft from outside its own row's support: q = 0 and p = 0, refused, and p - q is 0 everywhere
    c = make(5, 1, seed=36, noise=0.0)
    order = c["x"].reshape(5, 2, -1)[:, 0, :oracle.VREAL].float()
    c["d"] = order.argmin(1, keepdim=True).to(torch.int32)
    token, accepted, _, _ = run(c, 1.0, 1.0, 30)
    t, _, _, _ = pkg.sample(c["x"].reshape(5, 2, -1)[:, 0].contiguous(), 1.0, 1.0, 30, uniform=c["w"])
    assert not accepted.any() and torch.equal(token[:, 0], t)


def test_extreme_random_words():
    c = make(8, 2, seed=37)
    for a, w in ((0, 0), (-1, -1), (0, -1), (-1, 0)):
        c["a"].fill_(a), c["w"].fill_(w)
        for draft in (True, False):
            compare(c, run(c, 1.3, 0.99, 128, draft), 1.3, 0.99, 128, draft)


def test_a_support_below_the_first_window():
    # 60 distinct values far apart: the k-th lies beyond 8 binades, the row is resolved by further windows
    c = make(3, 2, seed=38)
    vals = torch.zeros(oracle.VPAD, device=DEV)
    vals[:] = -60.0
    vals[1000:1040] = torch.logspace(-3.5, 1.2, 40, device=DEV)
    for i in range(9):
        c["x"][i] = vals.roll(i * 17).to(torch.bfloat16)
    for i in range(6):
        c["y"][i] = vals.roll(i * 17 + 3).to(torch.bfloat16)
    c["d"] = torch.tensor([[1039 + 17 * (3 * b + i) for i in range(2)] for b in range(3)], dtype=torch.int32, device=DEV)
    for draft in (True, False):
        compare(c, run(c, 20.0, 1.0, 45, draft), 20.0, 1.0, 45, draft)


def test_same_bits_in_any_batch():
    c = make(9, 3, seed=39)
    whole = run(c, 1.3, 0.99, 128)
    for b in (0, 4, 8):
        one = dict(x=c["x"][4 * b:4 * b + 4], y=c["y"][3 * b:3 * b + 3], d=c["d"][b:b + 1], a=c["a"][b:b + 1], w=c["w"][b:b + 1])
        for u, v in zip(run(one, 1.3, 0.99, 128), whole):
            assert torch.equal(u[0], v[b])
    # wider rows, another stream
    wide = torch.zeros((36, oracle.VPAD + 64), dtype=torch.bfloat16, device=DEV)
    wide[:, :oracle.VPAD] = c["x"]
    st = torch.cuda.Stream()
    torch.cuda.synchronize()
    got = pkg.verify_drafts(wide, c["d"], 1.3, 0.99, 128, draft_logits=c["y"], accept_uniform=c["a"], draw_uniform=c["w"], stream=st)
    st.synchronize()
    for u, v in zip(got, whole):
        assert torch.equal(u, v)


def test_rejected_sequences():
    B, n = 9, 2
    c = make(B, n, seed=40)
    c["a"].zero_()                                             # accept whatever has any probability
    want = run(c, 1.0, 1.0, 1000)
    assert torch.all(want[1] >= 0)
    tau = torch.ones(B, device=DEV)
    num = torch.full((B,), n, dtype=torch.int32, device=DEV)
    tau[0] = -1.0                                              # its rows cannot be used
    c["x"][3 * 1, 77] = math.nan                               # first row of sequence 1
    c["d"][2, 0] = oracle.VREAL                                # not a token
    num[3] = n + 1
    num[4] = -1
    c["y"][2 * 5 + 1, 5] = math.inf                            # second draft row of sequence 5
    c["x"][3 * 6 + 2, 9] = math.nan                            # the row after the last draft of sequence 6
    c["x"][3 * 7] = -math.inf
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    token, accepted, restr, full = run(c, tau, 1.0, 1000, num_drafts=num, err_count=err)
    bad_at = {0: 0, 1: 0, 2: 0, 3: 0, 4: 0, 7: 0}
    bad_at[5] = min(1, int(want[1][5]))
    bad_at[6] = int(want[1][6])
    count = 0
    for b in range(B):
        hit = b in bad_at and not (b == 5 and bad_at[b] == 0) and not (b == 6 and bad_at[b] < 2)
        if not hit:
            for u, v in zip((token, accepted, restr, full), want):
                assert torch.equal(u[b], v[b]), b
            continue
        count += 1
        at = bad_at[b]
        assert int(accepted[b]) == at and torch.all(token[b, at:] == -1), b
        assert math.isnan(restr[b, at]) and math.isnan(full[b, at]) and not restr[b, at + 1:].any()
        assert torch.equal(token[b, :at], want[0][b, :at]) and torch.equal(restr[b, :at], want[2][b, :at])
    assert int(err) == count and count >= 6


def test_a_large_uneven_batch_has_the_right_distribution():
    """Drafts sampled from q, verified against p: the first tokens are distributed as p (chi-square)."""
    n_seq, k = 4000, 12
    g = torch.Generator(device=DEV)
    g.manual_seed(41)
    x = torch.full((2, oracle.VPAD), -30.0, device=DEV)
    cols = torch.tensor([5, 900, 19071, 19072, 40000, 60001, 80002, 100003, 120004, 140005, 151000, 151935], device=DEV)
    x[0, cols] = 1.5 * torch.randn(k, generator=g, device=DEV)
    x[1, cols] = x[0, cols] + torch.randn(k, generator=g, device=DEV)
    x = x.to(torch.bfloat16)
    p = torch.softmax(x[0, cols].double(), 0)
    q = torch.softmax(x[1, cols].double(), 0)
    drafts = cols[torch.multinomial(q, n_seq, replacement=True, generator=g)].to(torch.int32)[:, None]
    words = lambda *s: torch.randint(-2**31, 2**31, s, generator=g, device=DEV, dtype=torch.int64).to(torch.int32)  # noqa: E731
    seen = torch.zeros(k, device=DEV)
    for a in range(0, n_seq, 500):
        token, _, _, _ = pkg.verify_drafts(x[:1].expand(1000, -1).contiguous(), drafts[a:a + 500], 1.0, 1.0, k,
                                           draft_logits=x[1:].expand(500, -1).contiguous(),
                                           accept_uniform=words(500, 1), draw_uniform=words(500))
        seen += (token[:, :1] == cols).sum(0)
    assert int(seen.sum()) == n_seq
    chi = float((((seen - n_seq * p) ** 2) / (n_seq * p)).sum())
    assert chi < 40.0, chi                                     # 11 degrees of freedom: P < 4e-5


def test_binding_refuses():
    c = make(2, 2, seed=42)
    for kw in (dict(x=c["x"][:5]), dict(x=c["x"].half()), dict(x=c["x"][:, :1000]), dict(y=c["y"][:3]), dict(d=c["d"].long()),
               dict(d=c["d"][0]), dict(a=c["a"][:, :1]), dict(w=c["w"][:1]), dict(w=c["w"].cpu())):
        with pytest.raises((ValueError, pkg.RlkError)):
            run(c | kw)
    for kw in (dict(tau=-1.0), dict(p=0.0), dict(k=0), dict(draft_temperature=math.nan), dict(draft_top_p=2.0),
               dict(draft_top_k=-3), dict(num_drafts=torch.zeros(3, dtype=torch.int32, device=DEV))):
        with pytest.raises((ValueError, pkg.RlkError)):
            run(c, **kw)
    got = pkg.verify_drafts(c["x"][:0], c["d"][:0], accept_uniform=c["a"][:0], draw_uniform=c["w"][:0])
    assert got[0].shape == (0, 3)
