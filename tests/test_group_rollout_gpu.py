"""GPU: rotation, append and shared-prefix attention together, as a group rollout calls them,
and each of them on other streams, in captured graphs and with gradients.

Tolerances are those of the operators' own tests: the rotated queries and the cache are compared
with the rotation's oracle, and the attention with its oracle over what the cache then holds.
"""

import pytest
import torch

import rollout_consistent_vocab_gb300 as pkg
import test_prefix_gpu as tp
import test_rope_gpu as tr
import test_streams_gpu as ts

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from rollout_consistent_vocab_gb300.build import build_library
    build_library()
    pkg.load_library()


def i32(v):
    return torch.tensor(v, dtype=torch.int32, device=DEV)


def bits(t):
    return t.contiguous().view(torch.int16 if t.element_size() == 2 else torch.int32)


# ------------------------------------------------------------ together

class Rollout:
    """Groups of samples, each group of one prompt: the first sample's pages hold the prompt, the
    others' rows name its full ones and have a copy of the one that the prompt fills in part."""

    def __init__(self, prompts, samples, steps, heads, kv_heads, dim, page, dtype, n=1, rot=None, seed=0):
        self.prompts, self.samples, self.n, self.page, self.dtype = prompts, samples, n, page, dtype
        self.heads, self.kv_heads, self.dim, self.seed = heads, kv_heads, dim, seed
        self.freq = tr.freq_of(rot or dim)
        B = self.B = samples * len(prompts)
        width = max(-(-(p + steps * n) // page) for p in prompts)
        own = [-(-(p + steps * n) // page) - (0 if b % samples == 0 else p // page) for b, p in enumerate(
            p for p in prompts for _ in range(samples))]
        table, at = torch.full((B, width), -1, dtype=torch.int32), 0
        for b in range(B):
            first, p = b - b % samples, prompts[b // samples]
            full = 0 if b == first else p // page
            table[b, :full] = table[first, :full]
            table[b, full:full + own[b]] = torch.arange(at, at + own[b])
            at += own[b]
        self.table = table.to(DEV)
        # what no token has been written to is not a number
        self.k, self.v = (torch.full((at, page, kv_heads, dim), float("nan"), dtype=tr.DT[dtype], device=DEV) for _ in range(2))
        self.start, self.shared = i32([g * samples for g in range(len(prompts) + 1)]), i32(prompts)
        self.of = [p for p in prompts for _ in range(samples)]
        self.lens = i32(self.of)
        self.x = []                                              # the new q, k and v of each append
        # the prompts: all tokens by the first samples, and the last page's again by the others
        longest = max(prompts)
        k, v = (tr.rand((len(prompts), longest, kv_heads, dim), dtype, seed + i) for i in (1, 2))
        rows = torch.arange(B, device=DEV) // samples
        new = i32([p if b % samples == 0 else p % page for b, p in enumerate(self.of)])
        kk, vv = torch.zeros((2, B, longest, kv_heads, dim), dtype=tr.DT[dtype], device=DEV)
        for b in range(B):
            m = int(new[b])
            kk[b, :m], vv[b, :m] = k[rows[b], self.of[b] - m:self.of[b]], v[rows[b], self.of[b] - m:self.of[b]]
        self.err = i32([0])
        pkg.kv_append_rope(self.k, self.v, self.table, self.lens, kk, vv, self.freq, new_lens=new, err_count=self.err)
        self.prompt_k = k

    def step(self, t, **kw):
        """The new tokens of step t: (what they are, rotated queries, attention and lse)."""
        B, n = self.B, self.n
        qkv = tr.rand((B, n, self.heads + 2 * self.kv_heads, self.dim), self.dtype, 100 * self.seed + 10 + t)
        return (qkv,) + self.attend(qkv, **kw)

    def attend(self, qkv, out=None, lse=None, ws=None):
        q, k, v = qkv.split([self.heads, self.kv_heads, self.kv_heads], dim=2)
        self.lens += self.n
        q = pkg.kv_append_rope(self.k, self.v, self.table, self.lens, k, v, self.freq, q=q, q_out=q, err_count=self.err)
        a, z = pkg.prefix_attention(q, self.k, self.v, self.table, self.lens, self.start, self.shared, out=out, out_lse=lse,
                                    max_shared=max(self.prompts), workspace=ws, err_count=self.err)
        return q, a, z

    def case(self, q):
        return dict(q=q, k=self.k, v=self.v, table=self.table, whole=self.table.cpu().clamp(min=0), lens=self.lens, start=self.start,
                    shared=self.shared, of=self.of, dtype=self.dtype)


SETUPS = [
    # prompts, samples, steps, heads, kv_heads, dim, page, dtype, n, rot
    ([700, 45, 1031], 8, 6, 32, 8, 128, 16, "bf16", 1, None),
    ([333, 2100], 5, 4, 8, 1, 64, 24, "f16", 3, 32),
    ([64], 1, 3, 4, 4, 128, 64, "bf16", 2, None),
]


@pytest.mark.parametrize("prompts,samples,steps,heads,kv_heads,dim,page,dtype,n,rot", SETUPS)
def test_a_rollout_of_groups(prompts, samples, steps, heads, kv_heads, dim, page, dtype, n, rot):
    r = Rollout(prompts, samples, steps, heads, kv_heads, dim, page, dtype, n, rot)
    table = r.table.cpu()
    # the prompts' keys in the cache
    for g, p in enumerate(prompts):
        for b in (g * samples, (g + 1) * samples - 1):
            at = torch.arange(p)
            got = r.k[table[b, at // page].long().to(DEV), (at % page).to(DEV)]
            tr.compare(got[None], r.prompt_k[g:g + 1, :p], r.freq, at[None], dtype)
    for t in range(steps):
        before = tr.rand((r.B, n, heads + 2 * kv_heads, dim), dtype, 10 + t)
        _, q, a, z = r.step(t)
        pos = r.lens[:, None] - n + torch.arange(n, dtype=torch.int32, device=DEV)
        tr.compare(q, before[:, :, :heads], r.freq, pos, dtype)
        page_of = r.table.gather(1, (pos // page).long()).long()
        assert torch.equal(r.v[page_of, (pos % page).long()], before[:, :, heads + kv_heads:])
        tr.compare(r.k[page_of, (pos % page).long()], before[:, :, heads:heads + kv_heads], r.freq, pos, dtype)
        tp.compare(r.case(q), a, z, [n] * r.B)
    assert int(r.err) == 0


def test_the_steps_captured():
    # one graph, replayed: the lengths grow on the device
    a, b = (Rollout([500, 90], 6, 8, 8, 2, 128, 16, "bf16", 1) for _ in range(2))
    need = pkg.prefix_attention_workspace_bytes(12, 1, 8, 2, 128, 16 * a.table.shape[1], 2, 500)
    ws = torch.empty(need, dtype=torch.uint8, device=DEV)
    qkv = tr.rand((12, 1, 12, 128), "bf16", 10)
    out, lse = torch.empty((12, 1, 8, 128), dtype=torch.bfloat16, device=DEV), torch.empty((12, 1, 8), device=DEV)
    lens, k, v = a.lens.clone(), tr.copy(a.k), tr.copy(a.v)
    given = qkv.clone()
    a.attend(given, out, lse, ws)                                # (warm)
    for t, u in ((a.lens, lens), (a.k, k), (a.v, v)):
        t.copy_(u)
    g = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(g):
        a.attend(given, out, lse, ws)
    for step in range(8):
        x = tr.rand((12, 1, 12, 128), "bf16", 10 + step)
        given.copy_(x)
        g.replay()
        q, o, z = b.attend(x)
        torch.cuda.synchronize()
        assert torch.equal(bits(out), bits(o)) and torch.equal(bits(lse), bits(z)) and torch.equal(given[:, :, :8], q)
        assert torch.equal(bits(a.k), bits(b.k)) and torch.equal(bits(a.v), bits(b.v))
    assert int(a.err) == int(b.err) == 0


def test_a_rollout_has_its_bits_without_the_others():
    # a group of a batch, on its own, and a sample of it on its own
    whole = Rollout([700, 600], 4, 3, 8, 2, 64, 16, "bf16", 1)
    _, q, a, z = whole.step(0)
    for lo, hi in ((4, 8), (5, 6)):
        o, y = pkg.prefix_attention(q[lo:hi], whole.k, whole.v, whole.table[lo:hi], whole.lens[lo:hi].contiguous(), i32([0, hi - lo]),
                                    whole.shared[1:])
        assert torch.equal(bits(o), bits(a[lo:hi])) and torch.equal(bits(y), bits(z[lo:hi]))


# ------------------------------------------------------------ graphs and streams

def test_two_graphs_with_one_workspace():
    c = tp.make([(6, 1500), (2, 40)], [30, 1, 2, 3, 4, 5, 900, 7], 1, 32, 8, 128, 16, "bf16", seed=1)
    d = tp.make([(3, 4000)], [3, 2, 1], 2, 8, 2, 64, 16, "f16", seed=2)
    want = tp.run(c), tp.run(d)
    size = max(pkg.prefix_attention_workspace_bytes(x["q"].shape[0], x["q"].shape[1], x["q"].shape[2], x["k"].shape[2], x["q"].shape[3],
                                                    16 * x["table"].shape[1], x["shared"].shape[0], 16 * x["table"].shape[1]) for x in (c, d))
    ws = torch.empty(size, dtype=torch.uint8, device=DEV)
    graphs, outs = [], [(torch.empty_like(o), torch.empty_like(z)) for o, z in want]
    torch.cuda.synchronize()
    for x, (o, z) in zip((c, d), outs):
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            tp.run(x, out=o, out_lse=z, workspace=ws)
    for order in ((0, 1), (1, 0), (0, 0), (1, 1)):
        for o, z in outs:
            o.zero_()
            z.zero_()
        ws.fill_(255)
        for i in order:
            graphs[i].replay()
        torch.cuda.synchronize()
        for i in set(order):
            # (by their bits: the second one's last sequence has fewer tokens of its own than new ones, which is NaN)
            assert all(torch.equal(bits(a), bits(b)) for a, b in zip(outs[i], want[i]))


def test_the_result_where_the_queries_were():
    c = tp.make([(5, 800), (1, 300)], [3, 40, 2, 9, 1, 5, 70], 2, 8, 2, 128, 16, "bf16", seed=3)
    want, z = tp.run(c)
    out, lse = tp.run(c, out=c["q"])
    # (by their bits: a sequence with fewer tokens of its own than new ones is NaN)
    assert out.data_ptr() == c["q"].data_ptr() and torch.equal(bits(out), bits(want)) and torch.equal(bits(lse), bits(z))
    assert bool(torch.isfinite(out[[0, 1, 2, 3, 5, 6]]).all())


def rotation():
    x, pos = tr.rand((50, 7, 8, 128), "bf16", 4), tr.places((50, 7), 5)
    return lambda **kw: pkg.rope(x, tr.freq_of(128), pos, **kw), 1


def append():
    c = tr.make([40, 17, 300], 3, 8, 2, 128, 16, "bf16", seed=6)
    return lambda **kw: tr.append(c, tr.freq_of(128), **kw), 1


def attention():
    c = tp.make([(9, 2000)], [30] * 9, 1, 32, 8, 128, 16, "bf16", seed=7)
    tokens = 16 * c["table"].shape[1]
    return lambda **kw: tp.run(c, **kw), pkg.prefix_attention_workspace_bytes(9, 1, 32, 8, 128, tokens, 1, tokens)


CALLS = [rotation, append, attention]


@pytest.mark.parametrize("make", CALLS)
def test_memory_given_out_while_the_call_waits(make):
    ts.test_memory_given_out_while_the_call_waits(make)


@pytest.mark.parametrize("make", CALLS)
def test_memory_that_the_current_stream_still_reads(make):
    ts.test_memory_that_the_current_stream_still_reads(make)


@pytest.mark.parametrize("make", CALLS)
def test_outputs_dropped_while_the_current_stream_reads_them(make):
    ts.test_outputs_dropped_while_the_current_stream_reads_them(make)


# ------------------------------------------------------------ few and many

@pytest.mark.parametrize("B,n", [(0, 1), (0, 0), (3, 0)])
def test_nothing_to_do(B, n):
    k, v = (tr.rand((4, 16, 2, 64), "bf16", s) for s in (19, 20))
    table, lens = torch.zeros((B, 2), dtype=torch.int32, device=DEV), torch.full((B,), 5, dtype=torch.int32, device=DEV)
    q, kn = tr.rand((B, n, 4, 64), "bf16", 21), tr.rand((B, n, 2, 64), "bf16", 22)
    before = k.clone()
    assert pkg.kv_append_rope(k, v, table, lens, kn, kn, tr.freq_of(64), q=q).shape == q.shape
    out, lse = pkg.prefix_attention(q, k, v, table, lens, i32([0, B]), i32([5]))
    assert out.shape == q.shape and lse.shape == (B, n, 4) and torch.equal(k, before)


def test_no_groups_and_one_page():
    # all on their own; and a cache of a single page, which the shared and the own tokens are in
    c = tp.make([], [1, 40, 300, 17], 1, 8, 2, 128, 16, "bf16", seed=23)
    tp.compare(c, *tp.run(c), [1] * 4)
    tp.compare(c, *tp.run(c, max_shared=0), [1] * 4)
    k, v = (tr.rand((1, 200, 2, 64), "f16", s) for s in (24, 25))
    q = tr.rand((1, 2, 8, 64), "f16", 26)
    d = dict(q=q, k=k, v=v, table=i32([[0]]), whole=torch.zeros((1, 1), dtype=torch.int32), lens=i32([190]), start=i32([0, 1]),
             shared=i32([170]), of=[170], dtype="f16")
    tp.compare(d, *tp.run(d), [2])


def test_thousands_of_groups():
    members = [(1 + i % 2, 32 * (i % 4)) for i in range(2500)]
    tails = [1 + (7 * i) % 20 for i in range(sum(m for m, _ in members))]
    c = tp.make(members, tails, 1, 2, 1, 64, 16, "bf16", seed=27)
    err = i32([0])
    out, lse = tp.run(c, err_count=err)
    assert int(err) == 0
    tp.compare(c, out, lse, [1] * len(tails))
    c["start"][1700] += 4000                                     # (past the next one's begin)
    out, lse = tp.run(c, err_count=err)
    assert int(err) >= len(tails) and bool(torch.isnan(out).all()) and bool(torch.isnan(lse).all())


# ------------------------------------------------------------ gradients

def test_a_captured_gradient():
    # differences of x: the map is linear, its transpose the turn back
    x, freq, pos = tr.rand((3, 20, 4, 64), "f32", 8).requires_grad_(), tr.freq_of(64), tr.places((3, 20), 9)
    w = tr.rand((3, 20, 4, 64), "f32", 10)

    def step():
        (got,) = torch.autograd.grad((pkg.rope_autograd(x, freq, pos) * w).sum(), x)
        return got

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        got = step()
    for seed in (11, 12):
        pos.copy_(tr.places((3, 20), seed))
        w.copy_(tr.rand((3, 20, 4, 64), "f32", seed))
        g.replay()
        tr.compare(got, w, freq, pos, "f32", inverse=True)


def test_a_capture_beside_a_graph_of_the_same_leaf_is_refused():
    x, freq, pos = tr.rand((1, 5, 2, 32), "bf16", 13).requires_grad_(), tr.freq_of(32), tr.places((1, 5), 14)
    y = pkg.rope_autograd(x, freq, pos)
    again = pkg.rope_autograd(x, freq, pos)                      # (one more, on the same stream, is nothing to refuse)
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        pkg.rope_autograd(x, freq, pos)                          # (nor is one on another, without a capture)
    torch.cuda.synchronize()
    z = torch.zeros(4, device=DEV)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        z += 1.0
        with pytest.raises(RuntimeError, match="leaf"):
            pkg.rope_autograd(x, freq, pos)
    g.replay()
    y.sum().backward()
    assert x.grad is not None and bool((z == 1.0).all())
    x.grad = None
    del y, again
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):                                    # and with them gone there is nothing to refuse
        pkg.rope_autograd(x, freq, pos)
    g.replay()


def test_gradients_of_gradients():
    x, freq, pos = tr.rand((2, 3, 2, 32), "f32", 15).requires_grad_(), tr.freq_of(32), tr.places((2, 3), 16)
    w, u = (tr.rand((2, 3, 2, 32), "f32", s).requires_grad_(s == 17) for s in (17, 18))
    (g,) = torch.autograd.grad((pkg.rope_autograd(x, freq, pos) * w).sum(), x, create_graph=True)
    (h,) = torch.autograd.grad((g * u).sum(), w)                 # of the turn back: the turn
    tr.compare(h, u, freq, pos, "f32")
