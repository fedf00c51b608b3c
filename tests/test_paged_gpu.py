"""GPU: the paged key-value cache (append, attention) against the float64 oracle.

Tolerances, from the formats and not from a run.  With u half the cache dtype's
unit roundoff (2^-9 bf16, 2^-12 f16), A = sum_j p_j |v_j| and X the largest
scale * sum_d |q_d k_jd|:
  * a score carries at most (D + 4) 2^-24 X of float32 rounding, so a weight's
    relative error is at most ds = 2 (D + 4) 2^-24 X + 2^-18 (maximum and
    normaliser; ex2 and the rescalings of the join);
  * the result is rounded to the dtype once: 2 u |out| <= u |out| + u A, which leaves no
    room for weights of the dtype's precision: they have to carry twice its bits;
  * f16: results below its normal range are rounded at 2^-25 (weights are held
    scaled up, so that theirs is 2^-37 per token of the largest): 2^-24 in all.
  lse: ds alone (its sum is of unrounded weights).
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


def make(lens, n=1, heads=8, kv_heads=2, dim=128, page=16, dtype="bf16", order="token", seed=0, spare=2,
         width=None, qmul=2.0):
    """Sequences of these lengths in shuffled pages, every unused place of the pages NaN."""
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    need = [-(-t // page) for t in lens]
    pages = sum(need) + spare
    shape = (pages, page, kv_heads, dim) if order == "token" else (pages, kv_heads, page, dim)
    k = torch.randn(shape, generator=g, device=DEV).to(DT[dtype])
    v = torch.randn(shape, generator=g, device=DEV).to(DT[dtype])
    if order == "head":
        k, v = k.transpose(1, 2), v.transpose(1, 2)
    perm = torch.randperm(pages, generator=g, device=DEV).tolist()
    width = max(1, max(need)) if width is None else width
    table = torch.full((len(lens), width), -7, dtype=torch.int32)     # entries past the end are never read
    at = 0
    used = torch.zeros((pages, page), dtype=torch.bool)
    for b, m in enumerate(need):
        table[b, :m] = torch.tensor(perm[at:at + m], dtype=torch.int32)
        for t in range(lens[b]):
            used[perm[at + t // page], t % page] = True
        at += m
    k[~used.to(DEV)] = math.nan
    v[~used.to(DEV)] = math.inf
    q = (qmul * torch.randn((len(lens), n, heads, dim), generator=g, device=DEV)).to(DT[dtype])
    return dict(q=q, k=k, v=v, table=table.to(DEV), lens=torch.tensor(lens, dtype=torch.int32, device=DEV))


def i32(v):
    return torch.tensor(v, dtype=torch.int32, device=DEV)


def run(c, new=None, **kw):
    return pkg.paged_attention(c["q"], c["k"], c["v"], c["table"], c["lens"],
                               new_lens=None if new is None else i32(new), **kw)


def np64(t):
    return t.double().cpu().numpy()


def compare(c, out, lse, new, dtype, scale=None, window=0, sinks=0):
    dim = c["q"].shape[-1]
    scale = dim**-0.5 if scale is None else scale
    # the float32 scale that the call takes
    scale = float(np.float32(scale))
    o, z, A, X = ro.paged_attention(np64(c["q"]), np64(c["k"]), np64(c["v"]), c["table"].cpu().numpy(),
                                    c["lens"].cpu().numpy(), new, scale, window, sinks)
    ds = 2 * (dim + 4) * 2.0**-24 * X + 2.0**-18
    tol = U[dtype] * np.abs(o) + (U[dtype] + ds[..., None]) * A * (1 + 2.0**-7) + (2.0**-24 if dtype == "f16" else 0.0)
    got, gl = np64(out), np64(lse)
    assert np.all(np.abs(got - o) <= tol), (np.abs(got - o) - tol).max()
    fin = np.isfinite(z)
    assert np.array_equal(gl[~fin], z[~fin])
    assert np.all(np.abs(gl - z)[fin] <= (ds + 2.0**-23 * np.abs(z))[fin]), np.abs(gl - z)[fin].max()


CASES = [
    # lens, n, heads, kv_heads, dim, page, dtype, order
    ([1], 1, 1, 1, 64, 16, "bf16", "token"),
    ([1, 2, 15, 16, 17], 1, 8, 2, 128, 16, "bf16", "token"),
    ([31, 32, 33, 63, 64, 65, 127, 129], 1, 4, 4, 64, 24, "f16", "head"),
    ([255, 256, 257, 511, 512, 513], 1, 32, 8, 128, 16, "bf16", "token"),
    ([5, 300, 1025], 5, 32, 8, 128, 64, "bf16", "head"),
    ([4099], 3, 8, 1, 128, 7, "f16", "token"),
    ([1000, 8], 8, 8, 1, 64, 100, "bf16", "head"),
    ([700, 64], 8, 64, 1, 128, 128, "bf16", "token"),
    ([260, 17], 17, 7, 7, 64, 1, "f16", "token"),
    ([90, 600], 2, 28, 4, 128, 1000, "bf16", "token"),
    ([40, 515], 3, 128, 1, 64, 16, "bf16", "token"),
]


@pytest.mark.parametrize("case", CASES, ids=[f"{c[0][-1]}x{c[1]}h{c[2]}-{c[3]}d{c[4]}p{c[5]}{c[6]}{c[7]}" for c in CASES])
def test_attention_matches_the_oracle(case):
    lens, n, heads, kv_heads, dim, page, dtype, order = case
    c = make(lens, n, heads, kv_heads, dim, page, dtype, order, seed=len(lens) + n)
    out, lse = run(c)
    compare(c, out, lse, [n] * len(lens), dtype)


@pytest.mark.parametrize("dim,dtype", [(128, "bf16"), (64, "f16")])
@pytest.mark.parametrize("window,sinks", [(1, 0), (1, 1), (5, 3), (64, 4), (300, 0), (300, 280), (1000000, 7), (2048, 1)])
def test_window_and_sinks(window, sinks, dim, dtype):
    lens = [1, 5, 6, 70, 305, 700, 5000]
    c = make(lens, 1, 8, 2, dim, 24, dtype, seed=3)
    out, lse = run(c, window=window, sinks=sinks)
    compare(c, out, lse, [1] * len(lens), dtype, window=window, sinks=sinks)
    c = make([9, 600], 6, 8, 2, dim, 24, dtype, seed=4)
    out, lse = run(c, window=window, sinks=sinks)
    compare(c, out, lse, [6, 6], dtype, window=window, sinks=sinks)


def test_the_largest_windows_and_sinks_hide_nothing():
    c = make([1, 33, 700, 1300], 2, 8, 2, 64, 16, "bf16", seed=21, width=90)
    c["lens"][0] = 2                                           # (both tokens in the first page)
    c["k"][c["table"][0, 0].long(), 1] = 0.5
    c["v"][c["table"][0, 0].long(), 1] = 0.25
    out, lse = run(c)
    top = 2**31 - 1
    for window, sinks in ((top, 0), (top, top), (1, top), (5, 5000), (5, top)):
        o, z = run(c, window=window, sinks=sinks)
        assert torch.equal(o, out) and torch.equal(z, lse), (window, sinks)


def test_garbage_in_unused_places_counts_for_nothing():
    """Infinities and NaN past the end, before the window and between sinks and window."""
    for dim, dtype in ((128, "bf16"), (64, "f16")):
        c = make([77, 1500, 600], 3, 8, 2, dim, 24, dtype, seed=22)
        clean = {k: c[k].clone() for k in ("k", "v")}
        used = torch.zeros(c["k"].shape[:2], dtype=torch.bool, device=DEV)
        for b, t in enumerate(c["lens"].tolist()):
            for j in range(t):
                used[c["table"][b, j // 24].long(), j % 24] = True
        clean["k"][~used], clean["v"][~used] = 0.0, 0.0
        z = dict(c, **clean)
        for kw in ({}, {"window": 100, "sinks": 5}):
            a, b = run(c, **kw), run(z, **kw)
            assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
            assert torch.isfinite(a[0]).all()


def test_long_sequence_and_a_wide_table():
    c = make([40001, 20000, 3], 2, 4, 1, 64, 48, "bf16", seed=5, width=3000)
    out, lse = run(c)
    compare(c, out, lse, [2, 2, 2], "bf16")


def test_ragged_new_tokens_and_empty_sequences():
    c = make([6, 0, 40, 5, 300], 4, 8, 2, 128, 16, "bf16", seed=6)
    new = [4, 0, 1, 0, 3]
    out, lse = run(c, new)
    compare(c, out, lse, new, "bf16")
    for b, m in enumerate(new):
        assert not out[b, m:].any() and torch.all(lse[b, m:] == -math.inf)


def test_scales_and_large_scores():
    # scores of hundreds: nearly one-hot rows; scale 0: the mean; negative scale
    for scale, qmul in ((0.5, 30.0), (0.0, 2.0), (-0.125, 2.0), (1e-30, 1.0)):
        c = make([400, 37], 2, 8, 2, 64, 16, "bf16", seed=7, qmul=qmul)
        out, lse = run(c, scale=scale)
        compare(c, out, lse, [2, 2], "bf16", scale=scale)


def test_same_bits_in_any_batch_and_as_drafts():
    lens, n = [700, 33, 2049, 520], 5
    c = make(lens, n, 32, 8, 128, 16, "bf16", seed=8)
    out, lse = run(c)
    # one sequence at a time, in other pages of another cache order, in a wider table
    for b, t in enumerate(lens):
        m = -(-t // 16)
        k = torch.full((m + 9, 8, 16, 128), math.nan, dtype=torch.bfloat16, device=DEV)
        v = torch.full_like(k, math.nan)
        pages = torch.arange(m + 8, 8, -1, device=DEV)
        k[pages] = c["k"][c["table"][b, :m].long()].transpose(1, 2)
        v[pages] = c["v"][c["table"][b, :m].long()].transpose(1, 2)
        table = torch.full((1, m + 50), 10**6, dtype=torch.int32, device=DEV)
        table[0, :m] = pages
        o, z = pkg.paged_attention(c["q"][b:b + 1], k.transpose(1, 2), v.transpose(1, 2), table, i32([t]))
        assert torch.equal(o[0], out[b]) and torch.equal(z[0], lse[b])
        # each new token decoded alone, when it was the last one
        for i in range(n):
            o, z = pkg.paged_attention(c["q"][b:b + 1, i:i + 1], c["k"], c["v"], c["table"][b:b + 1], i32([t - n + 1 + i]))
            assert torch.equal(o[0, 0], out[b, i]) and torch.equal(z[0, 0], lse[b, i]), (b, i)
    for _ in range(3):
        o, z = run(c)
        assert torch.equal(o, out) and torch.equal(z, lse)


@pytest.mark.parametrize("n,group", [(1, 8), (3, 3), (2, 8), (1, 17), (4, 6), (5, 5), (4, 8), (11, 3), (9, 5), (1, 64)])
@pytest.mark.parametrize("dim,dtype", [(128, "bf16"), (64, "f16")])
def test_every_number_of_query_rows(n, group, dim, dtype):
    """8 to 64 rows of a kv head, in tiles of 8, 16, 24 and 32, some of them without a query."""
    lens = [n, 40 + n, 530, 1100]
    new = [n, max(1, n // 2), 0, n]
    c = make(lens, n, 2 * group, 2, dim, 16, dtype, seed=n * group)
    out, lse = run(c, new)
    compare(c, out, lse, new, dtype)
    for b, i in ((0, n - 1), (1, 0), (3, n // 2)):             # decoded alone: the same bits
        o, z = pkg.paged_attention(c["q"][b:b + 1, i:i + 1], c["k"], c["v"], c["table"][b:b + 1],
                                   i32([lens[b] - new[b] + 1 + i]))
        assert i >= new[b] or (torch.equal(o[0, 0], out[b, i]) and torch.equal(z[0, 0], lse[b, i]))
    # an infinite value among the new tokens: it reaches the queries at and after it, and only them
    t = lens[3] - 1 - n // 2
    c["v"][int(c["table"][3, t // 16]), t % 16, 1] = math.inf
    got, gl = run(c, new)
    assert torch.equal(got[:3], out[:3]) and torch.equal(gl, lse)
    first = n - 1 - n // 2
    assert torch.equal(got[3, :first], out[3, :first]) and torch.equal(got[3, first:, :group], out[3, first:, :group])
    assert torch.all(got[3, first:, group:] == math.inf)


@pytest.mark.parametrize("dim", [64, 128])
def test_bad_values_in_masked_places_stay_there(dim):
    # a drafted token with NaN key and infinite value: only the queries that see it are NaN
    c = make([200, 90], 4, 8, 2, dim, 16, "bf16", seed=9)
    out, _ = run(c)
    t = 198                                                    # the third of the four new tokens
    page = int(c["table"][0, t // 16])
    c["k"][page, t % 16] = math.nan
    c["v"][page, t % 16] = math.inf
    got, lse = run(c)
    assert torch.equal(got[1], out[1]) and torch.equal(got[0, :2], out[0, :2])
    assert torch.isnan(got[0, 2:]).all() and torch.isnan(lse[0, 2:]).all() and torch.isfinite(lse[0, :2]).all()
    # only the value is infinite
    c = make([200], 4, 8, 2, dim, 16, "bf16", seed=9)
    out, want = run(c)
    c["v"][int(c["table"][0, t // 16]), t % 16] = -math.inf
    got, lse = run(c)
    assert torch.equal(got[0, :2], out[0, :2]) and torch.equal(lse, want)
    assert torch.all(got[0, 2:] == -math.inf)
    # before the window, and between the sinks and the window
    c = make([200], 4, 8, 2, dim, 16, "bf16", seed=10)
    out, want = run(c, window=50, sinks=3)
    for t in (3, 9, 100, 146):                                 # the first query sees from 147 on
        c["k"][int(c["table"][0, t // 16]), t % 16] = math.nan
        c["v"][int(c["table"][0, t // 16]), t % 16] = math.nan
    got, lse = run(c, window=50, sinks=3)
    assert torch.equal(got, out) and torch.equal(lse, want)
    t = 148                                                    # seen by the first two queries only
    c["v"][int(c["table"][0, t // 16]), t % 16] = math.inf
    got, _ = run(c, window=50, sinks=3)
    assert torch.all(got[0, :2] == math.inf) and torch.equal(got[0, 2:], out[0, 2:])


def test_lowest_and_infinite_keys():
    c = make([70], 1, 4, 2, 64, 16, "bf16", seed=11)
    low = torch.finfo(torch.bfloat16).min
    c["q"].fill_(1.0)
    flat = c["table"][0].long()
    c["k"][flat[0]] = low                                      # scores far below all others: no weight
    o1, z1 = run(c)
    c["k"][flat[0]] = -math.inf                                # score -inf: no weight either
    o2, z2 = run(c)
    assert torch.isfinite(o1).all() and torch.equal(o1, o2) and torch.equal(z1, z2)
    c["k"][flat[0]] = math.inf
    o3, z3 = run(c)
    assert torch.isnan(o3).all()


def test_rejected_sequences():
    c = make([50, 40, 30, 20, 10], 2, 8, 2, 128, 16, "bf16", seed=12)
    out, lse = run(c)
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    c["lens"][0] = 16 * c["table"].shape[1] + 1                # beyond the table
    c["lens"][1] = 1                                           # fewer than the new tokens
    c["table"][2, 1] = c["k"].shape[0]                         # no such page
    o, z = run(c, err_count=err)
    for b in (0, 1, 2):
        assert torch.isnan(o[b]).all() and torch.isnan(z[b]).all()
    for b in (3, 4):
        assert torch.equal(o[b], out[b]) and torch.equal(z[b], lse[b])
    assert int(err) >= 3
    err.zero_()
    o, z = run(c, [2, 1, 2, 3, -1], err_count=err)             # more than n, and negative
    for b in (0, 2, 3, 4):
        assert torch.isnan(o[b]).all() and torch.isnan(z[b]).all()
    assert torch.isfinite(o[1]).all() and int(err) >= 4
    # a page out of the window's sight is not looked at
    c = make([400], 1, 8, 2, 128, 16, "bf16", seed=13)
    want, _ = run(c, window=20, sinks=2)
    c["table"][0, 3:20] = -1
    err.zero_()
    o, _ = run(c, window=20, sinks=2, err_count=err)
    assert torch.equal(o, want) and int(err) == 0


def test_strided_inputs_and_outputs():
    c = make([100, 260], 3, 8, 2, 64, 16, "f16", seed=14)
    out, lse = run(c)
    wide = torch.full((3, 2, 10, 192), 7.0, dtype=torch.float16, device=DEV)        # [n, B, heads, 3 * dim]
    wide[:, :, :8, 64:128] = c["q"].transpose(0, 1)
    q = wide.transpose(0, 1)[:, :, :8, 64:128]
    dest = torch.full((2, 8, 3, 72), 7.0, dtype=torch.float16, device=DEV)          # [B, heads, n, dim + 8]
    o, z = pkg.paged_attention(q, c["k"], c["v"], c["table"], c["lens"], out=dest.transpose(1, 2)[..., :64])
    assert torch.equal(dest.transpose(1, 2)[..., :64], out) and torch.equal(z, lse)
    assert torch.all(dest[..., 64:] == 7.0)
    # a table that is a view of a wider one
    table = torch.full((2, 40), -1, dtype=torch.int32, device=DEV)
    table[:, 3:3 + c["table"].shape[1]] = c["table"]
    o, z = pkg.paged_attention(c["q"], c["k"], c["v"], table[:, 3:3 + c["table"].shape[1]], c["lens"])
    assert torch.equal(o, out) and torch.equal(z, lse)


def test_offsets_past_32_bits():
    # one page 2^32 elements after the first (8.6 GB apart)
    dim, page, step = 64, 16, 2**22
    pages = 2**10 + 2
    buf = torch.zeros(pages * step, dtype=torch.bfloat16, device=DEV).as_strided((pages, page, 1, dim), (step, dim, dim, 1))
    c = make([20], 1, 4, 1, dim, page, "bf16", seed=15)
    want, wl = run(c)
    vbuf = torch.zeros(pages * step, dtype=torch.bfloat16, device=DEV).as_strided((pages, page, 1, dim), (step, dim, dim, 1))
    for at, src in ((0, 0), (pages - 1, 1)):
        buf[at] = c["k"][int(c["table"][0, src])]
        vbuf[at] = c["v"][int(c["table"][0, src])]
    o, z = pkg.paged_attention(c["q"], buf, vbuf, i32([[0, pages - 1]]), c["lens"])
    assert torch.equal(o, want) and torch.equal(z, wl)
    new = torch.randn((1, 1, 1, dim), device=DEV).to(torch.bfloat16)
    pkg.kv_append(buf, vbuf, i32([[0, pages - 1]]), i32([18]), new, -new)
    assert torch.equal(buf[pages - 1, 1, 0], new[0, 0, 0]) and torch.equal(vbuf[pages - 1, 1, 0], -new[0, 0, 0])


def test_on_another_stream_and_in_a_graph():
    c = make([300, 1000], 2, 8, 2, 128, 16, "bf16", seed=16)
    want, wl = run(c)
    torch.cuda.synchronize()
    st = torch.cuda.Stream()
    o, z = run(c, stream=st)
    st.synchronize()
    assert torch.equal(o, want) and torch.equal(z, wl)
    out, lse = torch.empty_like(want), torch.empty_like(wl)
    ws = torch.empty(max(1, pkg.paged_attention_workspace_bytes(2, 2, 8, 2, 128, 16 * c["table"].shape[1])),
                     dtype=torch.uint8, device=DEV)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        run(c, out=out, out_lse=lse, workspace=ws)
    for _ in range(2):
        out.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want) and torch.equal(lse, wl)
    # lengths are read when the graph runs
    c["lens"] -= 1
    graph.replay()
    torch.cuda.synchronize()
    short, sl = run(c)
    assert torch.equal(out, short) and torch.equal(lse, sl)


# ------------------------------------------------------------ append

@pytest.mark.parametrize("lens,new,n,kv_heads,dim,page,dtype,order", [
    ([1], [1], 1, 1, 64, 16, "bf16", "token"),
    ([16, 17, 33, 5], [1, 1, 1, 0], 1, 8, 128, 16, "bf16", "head"),
    ([40, 0, 70, 3], [33, 0, 40, 3], 40, 2, 64, 7, "f16", "token"),
    ([600, 90], [513, 90], 513, 3, 128, 100, "bf16", "head"),
    ([2, 3], [2, 1], 5, 5, 64, 1, "f16", "token"),
])
def test_append(lens, new, n, kv_heads, dim, page, dtype, order):
    c = make(lens, 1, kv_heads, kv_heads, dim, page, dtype, order, seed=20)
    kv = torch.randn((len(lens), n, 2, kv_heads + 1, dim), device=DEV).to(DT[dtype])
    kv[0, 0, 0, 0, 0] = math.nan                               # copied as it is
    k, v = kv[:, :, 0, :kv_heads], kv[:, :, 1, 1:]
    bits = lambda t: t.contiguous().view(torch.int16).cpu().numpy()  # noqa: E731
    wk, wv = ro.kv_append(bits(c["k"]), bits(c["v"]), c["table"].cpu().numpy(), lens, new, bits(k), bits(v))
    pkg.kv_append(c["k"], c["v"], c["table"], c["lens"], k, v, new_lens=i32(new))
    assert np.array_equal(bits(c["k"]), wk) and np.array_equal(bits(c["v"]), wv)


def test_append_rejects_on_the_device():
    c = make([20, 20, 20, 20, 20], 1, 2, 2, 64, 16, "bf16", seed=21)
    c["k"].zero_(), c["v"].zero_()
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    k = torch.ones((5, 3, 2, 64), dtype=torch.bfloat16, device=DEV)
    c["lens"][0] = 2                                           # fewer than the new tokens
    c["lens"][1] = 33                                          # beyond the table's two pages
    c["table"][2, 1] = -1                                      # tokens 17, 18, 19 have no page
    pkg.kv_append(c["k"], c["v"], c["table"], c["lens"], k, k, new_lens=i32([3, 3, 3, 4, 3]), err_count=err)
    assert int(err) >= 4
    written = (c["k"] != 0).all(-1).all(-1)
    assert int(written.sum()) == 3 and torch.equal(written, (c["v"] != 0).all(-1).all(-1))
    assert written[int(c["table"][4, 1]), 1:4].all()


def test_append_then_attend_is_the_whole_prompt():
    """A prompt written in pieces, attended token by token, is the prompt written at once."""
    n, page = 45, 16
    g = torch.Generator(device=DEV)
    g.manual_seed(22)
    k, v, q = (torch.randn((1, n, h, 64), generator=g, device=DEV).to(torch.bfloat16) for h in (2, 2, 8))
    table = i32([[2, 0, 1]])
    kc = torch.full((3, page, 2, 64), math.nan, dtype=torch.bfloat16, device=DEV)
    vc = kc.clone()
    got = []
    for a, b in ((0, 1), (1, 20), (20, 37), (37, 38), (38, 45)):
        pkg.kv_append(kc, vc, table, i32([b]), k[:, a:b], v[:, a:b])
        got.append(pkg.paged_attention(q[:, a:b], kc, vc, table, i32([b]))[0])
    whole, _ = pkg.paged_attention(q, kc, vc, table, i32([n]))
    assert torch.equal(torch.cat(got, 1), whole)


# ------------------------------------------------------------ refusals

def test_binding_refuses():
    c = make([20, 30], 2, 8, 2, 64, 16, "bf16", seed=23)
    a = (c["q"], c["k"], c["v"], c["table"], c["lens"])

    def bad(i, t, **kw):
        with pytest.raises((ValueError, pkg.RlkError)):
            pkg.paged_attention(*[t if j == i else x for j, x in enumerate(a)], **kw)

    bad(0, c["q"].half())
    bad(0, c["q"][..., :32])
    bad(0, c["q"][0])
    bad(0, c["q"][:, :, :7])                                   # not a multiple of kv_heads
    bad(1, c["k"].cpu())
    bad(1, c["k"].float())
    bad(2, c["v"][:, :8])
    bad(2, c["v"].transpose(1, 2).contiguous().transpose(1, 2))  # strides differ from k's
    bad(3, c["table"].long())
    bad(3, c["table"][:1])
    bad(4, c["lens"].long())
    bad(4, c["lens"], scale=math.inf)
    bad(4, c["lens"], window=-1)
    bad(4, c["lens"], sinks=-1)
    bad(4, c["lens"], new_lens=i32([1]))
    bad(4, c["lens"], out=torch.empty_like(c["q"]).float())
    bad(4, c["lens"], out_lse=torch.empty((2, 2, 9), device=DEV))
    o, z = pkg.paged_attention(c["q"][:0], c["k"], c["v"], c["table"][:0], c["lens"][:0])
    assert o.shape == (0, 2, 8, 64) and z.shape == (0, 2, 8)
    with pytest.raises((ValueError, pkg.RlkError)):
        pkg.kv_append(c["k"], c["v"], c["table"], c["lens"], c["q"], c["q"])       # 8 heads into 2
    k96 = torch.zeros((4, 16, 2, 96), dtype=torch.bfloat16, device=DEV)
    with pytest.raises(pkg.RlkError):
        pkg.paged_attention(torch.zeros((2, 1, 2, 96), dtype=torch.bfloat16, device=DEV), k96, k96, c["table"], c["lens"])
