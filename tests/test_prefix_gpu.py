"""GPU: attention of groups that share a prefix, against the float64 oracle.

Tolerances are those of paged attention (the same scores, statistics and sums, weights of
16 bits in bf16 and 22 in f16, one rounding of the result), but for the smallest weights of
shared tokens in f16: known to 2^-37 of the row's largest weight among its piece, so that N
shared tokens add at most N 2^-37 max|v|.
"""

import math

import numpy as np
import pytest
import torch

import rollout_consistent_vocab_gb300 as pkg
from oracle import rollout as ro

pytestmark = pytest.mark.gpu
DEV = "cuda"
DT = {"bf16": torch.bfloat16, "f16": torch.float16}
U = {"bf16": 2.0**-9, "f16": 2.0**-12}


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from rollout_consistent_vocab_gb300.build import build_library
    build_library()
    pkg.load_library()


def i32(v):
    return torch.tensor(v, dtype=torch.int32, device=DEV)


def np64(t):
    return t.double().cpu().numpy()


def make(groups, tails, n=1, heads=8, kv_heads=2, dim=128, page=16, dtype="bf16", order="token", seed=0, before=0, qmul=2.0,
         own_pages=False, width=None):
    """groups: (members, shared tokens) of each; `before` sequences ahead of them are in none, nor are those that the
    tails leave over.  Every unused place of the pages is NaN or infinite.  Shared full pages are named by all members'
    rows (own_pages: only by the first's; the others name pages of infinities there)."""
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    start, of, first = [before], [0] * before, list(range(before))
    for members, shared in groups:
        start.append(start[-1] + members)
        of += [shared] * members
        first += [start[-2]] * members
    B = len(tails)
    of, first = of + [0] * (B - len(of)), first + list(range(len(first), B))
    lens = [a + b for a, b in zip(of, tails)]
    need = [-(-t // page) for t in lens]
    pages = 1 + sum(need) + 2
    shape = (pages, page, kv_heads, dim) if order == "token" else (pages, kv_heads, page, dim)
    k, v = (torch.randn(shape, generator=g, device=DEV).to(DT[dtype]) for _ in range(2))
    if order == "head":
        k, v = k.transpose(1, 2), v.transpose(1, 2)
    perm, at = torch.randperm(pages - 1, generator=g, device=DEV).tolist(), 0        # (the last page stays bad)
    width = max(1, max(need)) if width is None else width
    table = torch.full((B, width), -7, dtype=torch.int32)
    used = torch.zeros((pages, page), dtype=torch.bool)
    for b, m in enumerate(need):
        full = 0 if first[b] == b else of[b] // page
        table[b, :full] = table[first[b], :full]
        table[b, full:m] = torch.tensor(perm[at:at + m - full], dtype=torch.int32)
        at += m - full
        if first[b] != b and of[b] % page:                       # a copy of the page that the shared tokens fill in part
            k[table[b, full].item(), :of[b] % page] = k[table[first[b], full].item(), :of[b] % page]
            v[table[b, full].item(), :of[b] % page] = v[table[first[b], full].item(), :of[b] % page]
        for t in range(lens[b]):
            used[table[b, t // page], t % page] = True
    k[~used.to(DEV)] = math.nan
    v[~used.to(DEV)] = math.inf
    whole = table.clone()
    if own_pages:
        for b in range(B):
            if first[b] != b:
                table[b, :of[b] // 32 * 32 // page] = pages - 1
    q = (qmul * torch.randn((B, n, heads, dim), generator=g, device=DEV)).to(DT[dtype])
    return dict(q=q, k=k, v=v, table=table.to(DEV), whole=whole, lens=i32(lens), start=i32(start), shared=i32([s for _, s in groups]),
                of=of, dtype=dtype)


def run(c, new=None, **kw):
    return pkg.prefix_attention(c["q"], c["k"], c["v"], c["table"], c["lens"], c["start"], c["shared"],
                                new_lens=None if new is None else i32(new), **kw)


def compare(c, out, lse, new, scale=None, rows=slice(None)):
    dim, dtype = c["q"].shape[-1], c["dtype"]
    scale = float(np.float32(dim**-0.5 if scale is None else scale))
    o, z, A, X = ro.paged_attention(np64(c["q"])[rows], np64(c["k"]), np64(c["v"]), c["whole"].numpy()[rows],
                                    c["lens"].cpu().numpy()[rows], np.array(new)[rows], scale)
    ds = 2 * (dim + 4) * 2.0**-24 * X + 2.0**-18
    tol = U[dtype] * np.abs(o) + (U[dtype] + ds[..., None]) * A * (1 + 2.0**-7)
    if dtype == "f16":
        v = np64(c["v"])
        tol += 2.0**-24 + np.array(c["of"])[rows, None, None, None] * 2.0**-37 * np.abs(v[np.isfinite(v)]).max()
    got, gl = np64(out)[rows], np64(lse)[rows]
    assert np.all(np.abs(got - o) <= tol), (np.abs(got - o) - tol).max()
    fin = np.isfinite(z)
    assert np.array_equal(gl[~fin], z[~fin])
    assert np.all(np.abs(gl - z)[fin] <= (ds + 2.0**-23 * np.abs(z))[fin]), np.abs(gl - z)[fin].max()


CASES = [
    # groups, tails, n, heads, kv_heads, dim, page, dtype, order
    ([(1, 32)], [1], 1, 1, 1, 64, 16, "bf16", "token"),
    ([(2, 33)], [1, 40], 1, 8, 2, 128, 16, "bf16", "token"),
    ([(3, 31), (2, 64), (2, 100)], [5, 1, 700, 3, 3, 60, 2], 1, 8, 2, 128, 24, "f16", "head"),
    ([(4, 512), (4, 513), (3, 545)], [1, 2, 3, 4, 5, 6, 7, 8, 9, 600, 11], 1, 32, 8, 128, 64, "bf16", "token"),
    ([(20, 1100)], list(range(1, 21)), 1, 8, 1, 128, 16, "bf16", "token"),                     # 160 rows: two tiles
    ([(5, 1500), (3, 96)], [5, 9, 20, 5, 31, 700, 5, 8], 5, 32, 8, 128, 16, "bf16", "head"),
    ([(9, 700)], [9] * 9, 9, 7, 1, 64, 100, "f16", "token"),                                    # 567 rows: three blocks
    ([(2, 4099)], [1, 3], 1, 4, 2, 128, 7, "f16", "token"),
    ([(3, 130)], [2, 2, 300], 2, 28, 4, 128, 1, "bf16", "token"),
    ([(6, 8200)], [3, 1, 1, 2, 1, 1], 1, 8, 2, 64, 1000, "bf16", "token"),                       # pieces of 1024
    ([(2, 600), (0, 500), (1, 0), (4, 255)], [1, 2, 3, 4, 5, 6, 7], 1, 16, 16, 64, 32, "f16", "head"),
    ([(3, 400)], [17, 20, 33], 17, 128, 1, 64, 128, "bf16", "token"),
]


@pytest.mark.parametrize("case", CASES, ids=[f"{c[0][0][0]}x{c[0][0][1]}n{c[2]}h{c[3]}-{c[4]}d{c[5]}p{c[6]}{c[7]}{c[8]}" for c in CASES])
def test_attention_matches_the_oracle(case):
    groups, tails, n, heads, kv_heads, dim, page, dtype, order = case
    c = make(groups, tails, n, heads, kv_heads, dim, page, dtype, order, seed=len(tails) + n)
    out, lse = run(c)
    compare(c, out, lse, [n] * len(tails))


def test_a_very_long_prefix():
    c = make([(2, 34000)], [1, 2], 1, 8, 2, 128, 64, "bf16", seed=5)                            # pieces of 2048
    out, lse = run(c)
    compare(c, out, lse, [1, 1])


RUNS = [
    # more pieces than CTAs: runs that hold pieces side by side, end anywhere, and go from group to group
    ([(2, 4600), (1, 4100), (3, 2080), (0, 700), (2, 5000), (1, 0), (2, 4608), (1, 3000)], 8, 8, 64, 16, "bf16"),
    ([(3, 4600), (2, 1570), (4, 3300), (3, 4096), (1, 9000)], 16, 8, 128, 64, "f16"),
    ([(40, 1700), (2, 2300), (33, 1600), (1, 4500), (70, 1100), (2, 4200)], 16, 4, 64, 64, "bf16"),    # one tile of rows and two
    ([(33, 2600), (3, 9300), (34, 2000), (1, 8900), (33, 1700), (2, 3000)], 32, 8, 128, 24, "bf16"),
    ([(1, 32 + 544 * (i % 9)) for i in range(40)], 8, 8, 128, 128, "bf16"),
    ([(40, 20000), (2, 16384), (3, 1500), (33, 33000), (1, 700), (2, 16383), (5, 1024), (4, 1023)], 16, 4, 64, 64, "bf16"),    # of all lengths
]


@pytest.mark.parametrize("groups,heads,kv_heads,dim,page,dtype", RUNS)
def test_runs_of_many_pieces(groups, heads, kv_heads, dim, page, dtype):
    tails = [1 + (7 * i) % 40 for i in range(sum(m for m, _ in groups))]
    c = make(groups, tails, 1, heads, kv_heads, dim, page, dtype, seed=30)
    out, lse = run(c)
    compare(c, out, lse, [1] * len(tails))
    for _ in range(5):
        o, z = run(c)
        assert torch.equal(o, out) and torch.equal(z, lse)


def test_sequences_without_queries_and_fewer_new_tokens():
    c = make([(5, 700), (3, 300)], [4, 9, 4, 30, 5, 4, 4, 4, 7, 9], 4, 8, 2, 128, 24, "bf16", seed=7, before=1)
    new = [3, 4, 0, 1, 2, 4, 0, 0, 0, 4]
    out, lse = run(c, new)
    compare(c, out, lse, new)
    for b, m in enumerate(new):
        assert not out[b, m:].any() and bool((lse[b, m:] == -math.inf).all())


def test_shared_pages_come_from_the_first_row():
    kw = dict(n=2, heads=8, kv_heads=2, dim=64, page=8, dtype="bf16", seed=9)
    groups, tails = [(3, 333), (2, 64)], [9, 30, 2, 5, 4]
    a, b = make(groups, tails, **kw), make(groups, tails, own_pages=True, **kw)
    (o, z), (p, y) = run(a), run(b)
    compare(b, p, y, [2] * 5)
    assert torch.equal(o, p) and torch.equal(z, y)


@pytest.mark.parametrize("scale", [0.3, -0.2, 0.0, 4.0])
def test_scales(scale):
    c = make([(3, 600)], [2, 3, 40], 1, 8, 2, 64, 16, "bf16", seed=11, qmul=1.0)
    out, lse = run(c, scale=scale)
    compare(c, out, lse, [1] * 3, scale=scale)


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_scores_that_rise_and_fall(dtype):
    """The maximum comes late, early, and far above the rest."""
    c = make([(4, 1024)], [2, 3, 4, 5], 1, 8, 2, 64, 16, dtype, seed=12, qmul=1.0)
    table = c["whole"].tolist()
    ramp = torch.linspace(-3.0, 3.0, 1024, device=DEV)
    for t in range(1024):
        page, place = table[0][t // 16], t % 16
        c["k"][page, place, 0] = (c["k"][page, place, 0] * 0.1 + ramp[t]).to(DT[dtype])
        c["k"][page, place, 1] = (c["k"][page, place, 1] * 0.1 - ramp[t]).to(DT[dtype])
    c["q"] += 1.0
    out, lse = run(c)
    compare(c, out, lse, [1] * 4)


def test_small_weights_in_half_precision():
    """One shared token takes nearly all the weight and its value is small: the others' still count."""
    c = make([(2, 2048)], [1, 1], 1, 2, 1, 64, 16, "f16", seed=13)
    table = c["whole"].tolist()
    c["q"].fill_(1.0)
    c["k"][...] = 0.0
    c["v"][...] = 8.0
    c["k"][table[0][3], 5] = 2.0                                 # score 16 = 64 * 2 / 8: the others weigh e^-16 = 2^-23
    c["v"][table[0][3], 5] = 0.0
    out, lse = run(c)
    compare(c, out, lse, [1, 1])


# ------------------------------------------------------------ the batch does not matter

def bits(t):
    return t.contiguous().view(torch.int16 if t.element_size() == 2 else torch.int32)


def test_a_sequence_has_its_bits_in_any_group():
    c = make([(40, 1700), (3, 900)], [1 + 37 * i % 600 for i in range(44)], 1, 8, 2, 128, 16, "bf16", seed=14, before=1)
    out, lse = run(c)
    for b in (1, 17, 40, 42):
        lead = 1 if b < 41 else 41
        rows = sorted({lead, b})
        d = dict(c, q=c["q"][rows], table=c["table"][rows], lens=c["lens"][rows], start=i32([0, len(rows)]),
                 shared=c["shared"][:1] if b < 41 else c["shared"][1:])
        o, z = run(d)
        assert torch.equal(bits(o[-1]), bits(out[b])) and torch.equal(bits(z[-1]), bits(lse[b])), b
    # and with idle members beside it
    new = [1 if b in (5, 42) else 0 for b in range(44)]
    o, z = run(c, new)
    for b in (5, 42):
        assert torch.equal(bits(o[b]), bits(out[b])) and torch.equal(bits(z[b]), bits(lse[b]))


def test_drafted_tokens_have_the_bits_of_single_ones():
    c = make([(7, 800)], [40] * 7, 5, 32, 8, 128, 16, "bf16", seed=15)
    out, lse = run(c)
    for i in (0, 4):
        d = dict(c, q=c["q"][:, i:i + 1], lens=c["lens"] - 4 + i)
        o, z = run(d)
        assert torch.equal(bits(o[:, 0]), bits(out[:, i])) and torch.equal(bits(z[:, 0]), bits(lse[:, i]))


def test_a_sequence_in_no_group():
    c = make([(2, 31), (3, 0), (2, 640)], [600, 1, 5000, 3, 9, 2, 2, 77, 9234], 2, 8, 2, 128, 16, "bf16", seed=16, before=1)
    new = [2, 1, 2, 2, 2, 2, 2, 2, 2]
    out, lse = run(c, new)
    compare(c, out, lse, new)
    # without any groups: the bits of those that share nothing a call knows of
    d = dict(c, start=i32([0]), shared=i32([]))
    p, y = run(d, new)
    compare(c, p, y, new)
    for b in (0, 1, 2, 3, 4, 5, 8):
        assert torch.equal(bits(p[b]), bits(out[b])) and torch.equal(bits(y[b]), bits(lse[b])), b
    # alone, in a wider table
    wide = torch.full((1, c["table"].shape[1] + 300), -7, dtype=torch.int32, device=DEV)
    wide[:, :c["table"].shape[1]] = c["table"][8:]
    p, y = run(dict(c, q=c["q"][8:], table=wide, lens=c["lens"][8:], start=i32([0]), shared=i32([])))
    assert torch.equal(bits(p[0]), bits(out[8])) and torch.equal(bits(y[0]), bits(lse[8]))


@pytest.mark.parametrize("dtype,dim,n", [("bf16", 128, 1), ("f16", 64, 3), ("bf16", 64, 9), ("f16", 128, 5)])
def test_long_tails(dtype, dim, n):
    """Parts of more than 256 tokens, one of them with a single token."""
    c = make([(2, 64)], [8193 + 256, 4096, 16385 - 64, 300], n, 4, 2, dim, 24, dtype, seed=27)
    out, lse = run(c)
    compare(c, out, lse, [n] * 4)


# ------------------------------------------------------------ what is not finite, what is rejected

def test_values_that_are_not_finite():
    c = make([(3, 200), (2, 100)], [2, 3, 4, 5, 6], 1, 4, 2, 64, 16, "bf16", seed=17)
    table = c["whole"].tolist()
    c["k"][table[0][0], 3, 0] = math.nan                         # kv head 0 of the first group
    c["v"][table[3][1], 2, 1, 5] = math.inf                      # one element of kv head 1 of the second
    out, lse = run(c)
    assert bool(torch.isnan(out[:3, 0, :2]).all()) and bool(torch.isnan(lse[:3, 0, :2]).all())
    assert bool(torch.isfinite(out[:3, 0, 2:]).all()) and bool(torch.isfinite(lse[3:]).all())
    inf = torch.zeros_like(out, dtype=torch.bool)
    inf[3:, 0, 2:, 5] = True
    inf[:3, 0, :2] = True
    assert torch.equal(~torch.isfinite(out), inf) and bool((out[3:, 0, 2:, 5] == math.inf).all())


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_a_prefix_whose_scores_are_all_minus_infinity(dtype):
    c = make([(3, 600)], [2, 3, 300], 1, 4, 2, 64, 16, dtype, seed=18)
    table = c["whole"].tolist()
    c["q"][..., 0] = 1.0
    for t in range(600):
        c["k"][table[0][t // 16], t % 16, :, 0] = -math.inf
    for b in range(3):                                           # (the copies of the last shared page)
        c["k"][table[b][37], :8, :, 0] = -math.inf
    out, lse = run(c)
    # the rest alone
    own, z, _, _ = zip(*(ro.paged_attention(np64(c["q"])[b:b + 1], np.where(np.isfinite(np64(c["k"])), np64(c["k"]), -1e30),
                                            np64(c["v"]), c["whole"].numpy()[b:b + 1], c["lens"].cpu().numpy()[b:b + 1], [1],
                                            float(np.float32(0.125))) for b in range(3)))
    # (half a step of the result, and as much of the values' size for everything else)
    assert np.allclose(np64(out), np.concatenate(own), rtol=U[dtype], atol=U[dtype] * 6)
    assert np.allclose(np64(lse), np.concatenate(z), atol=1e-4)


def test_rejected_sequences_and_groups():
    c = make([(3, 64), (2, 96), (2, 128)], [9, 9, 9, 9, 9, 9, 9, 4], 2, 4, 2, 64, 16, "bf16", seed=19)
    err = i32([0])
    good, gl = run(c, err_count=err)
    assert int(err) == 0
    compare(c, good, gl, [2] * 8)

    def check(bad, count, d, new=None, **kw):
        err.zero_()
        out, lse = run(d, new, err_count=err, **kw)
        assert int(err) >= count > 0
        for b in range(8):
            if b in bad:
                assert bool(torch.isnan(out[b]).all()) and bool(torch.isnan(lse[b]).all()), b
            else:
                assert torch.equal(bits(out[b]), bits(good[b])) and torch.equal(bits(lse[b]), bits(gl[b])), b

    # new tokens that are not behind the shared ones; lengths that do not agree with the new ones, or the table
    lens = c["lens"].clone()
    lens[1], lens[4], lens[6] = 65, 1, 1000
    check({1, 4, 6}, 3, dict(c, lens=lens))
    for bad in (-1, 10**6, 129):
        shared = c["shared"].clone()
        shared[1] = bad
        check({3, 4}, 2, dict(c, shared=shared), max_shared=128)
    for start in ([0, 3, 2, 7], [0, 3, 5, 9], [-1, 3, 5, 7], [3, 0, 5, 7]):
        check(set(range(8)), 8, dict(c, start=i32(start)))
    table = c["table"].clone()
    table[3, 2] = c["k"].shape[0]
    check({3, 4}, 1, dict(c, table=table))
    table[3, 2] = -1
    check({3, 4}, 1, dict(c, table=table))
    table = c["table"].clone()
    table[6, 8] = 2**31 - 1                                      # its own
    check({6}, 1, dict(c, table=table))
    # what an idle sequence's lengths say of the shared tokens is of no account
    lens = c["lens"].clone()
    lens[5] = 0
    err.zero_()
    new = [2] * 8
    new[5] = 0
    out, lse = run(dict(c, lens=lens), new, err_count=err)
    assert int(err) == 0 and torch.equal(bits(out[6]), bits(good[6])) and not out[5].any()


def test_refusals():
    c = make([(2, 64)], [3, 4], 1, 4, 2, 64, 16, "bf16", seed=20)
    for kw in (dict(shared=c["shared"].long()), dict(start=c["start"][:1]), dict(start=c["start"].cpu()), dict(shared=c["shared"][None]),
               dict(start=i32([0, 0, 2])), dict(q=c["q"].half())):
        with pytest.raises(ValueError):
            run(dict(c, **kw))
    for kw in (dict(max_shared=-1), dict(max_shared=16 * c["table"].shape[1] + 1), dict(scale=math.nan)):
        with pytest.raises(pkg.RlkError):
            run(c, **kw)
    with pytest.raises(ValueError):
        run(c, workspace=torch.empty(1000, dtype=torch.uint8, device=DEV))
    with pytest.raises(pkg.RlkError):
        run(dict(c, q=c["q"][:, :, :3].contiguous()))


# ------------------------------------------------------------ in use

def test_outputs_and_workspace_given():
    c = make([(3, 700)], [2, 3, 4], 2, 8, 2, 64, 16, "bf16", seed=21)
    want, z = run(c)
    need = pkg.prefix_attention_workspace_bytes(3, 2, 8, 2, 64, 16 * c["table"].shape[1], 1, 16 * c["table"].shape[1])
    ws = torch.full((need + 48,), 255, dtype=torch.uint8, device=DEV)
    out = torch.full((3, 8, 4, 64), 7.0, dtype=torch.bfloat16, device=DEV).transpose(1, 2)
    lse = torch.empty((3, 2, 8), device=DEV)
    o, y = run(c, out=out[:, 1:3], out_lse=lse, workspace=ws[16:16 + need])
    assert o.data_ptr() == out[:, 1:3].data_ptr() and torch.equal(o, want) and torch.equal(y, z)
    assert bool((out[:, 0] == 7.0).all()) and bool((out[:, 3] == 7.0).all())
    assert bool((ws[:16] == 255).all()) and bool((ws[16 + need:] == 255).all())
    small = pkg.prefix_attention_workspace_bytes(3, 2, 8, 2, 64, 16 * c["table"].shape[1], 1, 700)
    assert small <= need
    o, y = run(c, max_shared=700, workspace=torch.empty(small, dtype=torch.uint8, device=DEV))
    assert torch.equal(o, want) and torch.equal(y, z)


def test_a_captured_step_with_other_lengths_and_groups():
    c = make([(4, 600), (3, 1200)], [40, 41, 42, 43, 44, 45, 46], 1, 8, 2, 128, 16, "bf16", seed=22)
    out, lse = run(c)
    g = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(g):
        run(c, out=out, out_lse=lse)
    for step in range(3):
        c["lens"] -= 3
        if step == 1:
            c["shared"][0] = 320                                 # less of it taken as shared
        if step == 2:
            c["start"].copy_(i32([0, 2, 2]))                     # fewer members, and a group without any
        out.fill_(0)
        g.replay()
        want, z = run(c)
        torch.cuda.synchronize()
        assert torch.equal(out, want) and torch.equal(lse, z)
        compare(c, out, lse, [1] * 7)


def test_two_calls_at_once():
    c = make([(16, 3000)], [20] * 16, 1, 32, 8, 128, 16, "bf16", seed=23)
    d = make([(9, 900), (5, 5000)], [300] * 14, 2, 8, 2, 64, 24, "f16", seed=24)
    want = run(c), run(d)
    streams = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    got = [[run(x, stream=s) for x, s in zip((c, d), streams)] for _ in range(10)]
    torch.cuda.synchronize()
    for pair in got:
        for (o, z), (p, y) in zip(pair, want):
            assert torch.equal(o, p) and torch.equal(z, y)


def test_many_small_groups():
    members = [(1 + i % 3, 32 * (i % 7)) for i in range(700)]
    tails = [1 + (5 * i) % 50 for i in range(sum(m for m, _ in members))]
    c = make(members, tails, 1, 2, 1, 64, 16, "bf16", seed=25)
    out, lse = run(c)
    compare(c, out, lse, [1] * len(tails))


def test_many_own_tokens_in_a_large_batch():
    # more chunks of own tokens than warps, and more elements of the result than threads at once: the bits are
    # those of each sequence alone
    tails = [1 + (211 * i) % 2900 for i in range(200)]
    c = make([(9, 1500), (120, 600)], tails, 1, 64, 2, 64, 16, "bf16", seed=31, before=3)
    out, lse = run(c)
    compare(c, out, lse, [1] * 200, rows=slice(0, 200, 9))
    assert bool(torch.isfinite(out).all())
    for b in (0, 3, 11, 70, 131, 199):
        d = dict(c, q=c["q"][b:b + 1], table=c["table"][b:b + 1], lens=c["lens"][b:b + 1], start=i32([0, 1]), shared=i32([c["of"][b]]))
        o, z = run(d)
        assert torch.equal(bits(o[0]), bits(out[b])) and torch.equal(bits(z[0]), bits(lse[b])), b


def test_a_cache_past_32_bits():
    """Pages whose elements lie past 2^31 (and bytes past 2^32)."""
    page, kv_heads, dim = 64, 8, 128
    pages = 2**32 // (page * kv_heads * dim * 2) + 40
    k, v = (torch.empty((pages, page, kv_heads, dim), dtype=torch.bfloat16, device=DEV) for _ in range(2))
    last = torch.arange(pages - 24, pages, device=DEV)
    g = torch.Generator(device=DEV)
    g.manual_seed(26)
    for x in (k, v):
        x[last] = torch.randn((24, page, kv_heads, dim), generator=g, device=DEV).to(torch.bfloat16)
    table = torch.zeros((2, 12), dtype=torch.int32)
    table[0] = torch.arange(pages - 12, pages)
    table[1, :10], table[1, 10:] = table[0, :10], torch.arange(pages - 24, pages - 22)
    c = dict(q=torch.randn((2, 1, 16, dim), generator=g, device=DEV).to(torch.bfloat16), k=k, v=v, table=table.to(DEV), whole=table,
             lens=i32([700, 710]), start=i32([0, 2]), shared=i32([640]), of=[640, 640], dtype="bf16")
    out, lse = run(c)
    small = dict(c, k=k[last], v=v[last], whole=table - (pages - 24))
    compare(small, out, lse, [1, 1])
