"""GPU: the rotation of heads by position, alone and on the way into the paged cache,
against the float64 oracle.

Tolerance, from the formats and not from a run.  With S = |x| + |y| of an element's pair:
  * the angle: the frequency as a fraction of a turn is off by 2^-52 of itself at most (a
    product with a rounded constant), so |position frequency| 2^-52; cut to 2^-32 of a turn,
    2^-29; an eighth of a turn at most, rounded to float32: 2^-24.  Sine and cosine are within one
    step, 2^-24.  In all |position frequency| 2^-52 + 2^-22.9 of S;
  * two roundings of the products: 2^-23 of S; so 2^-22 + |position frequency| 2^-52 covers both;
  * the result is rounded once: half a step, and half of the smallest number in f16 (2^-25)
    and of the smallest normal ones of the others.
"""

import math

import numpy as np
import pytest
import torch

import rollout_consistent_vocab_gb300 as pkg
from oracle import rope_oracle as ro

pytestmark = pytest.mark.gpu
DEV = "cuda"
DT = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
SMALLEST = {"bf16": 2.0**-126, "f16": 2.0**-25, "f32": 2.0**-126}


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from rollout_consistent_vocab_gb300.build import build_library
    build_library()
    pkg.load_library()


def np64(t):
    return t.double().cpu().numpy()


def freq_of(rot, theta=1e4):
    return theta ** (-torch.arange(rot // 2, dtype=torch.float64) / (rot // 2))


def rand(shape, dtype, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return torch.randn(shape, generator=g, device=DEV).to(DT[dtype])


def places(shape, seed, lo=0, hi=5000):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return torch.randint(lo, hi, shape, generator=g, device=DEV).to(torch.int32)


def compare(got, x, freq, positions, dtype, pair_axis=None, interleaved=False, inverse=False):
    f = freq.numpy()
    pos = positions.cpu().numpy().reshape((-1,) + tuple(positions.shape[-2:]))
    axis = None if pair_axis is None else pair_axis.numpy()
    want, size = ro.rope(np64(x), f, pos, axis, interleaved, inverse)
    far = float(np.abs(pos.astype(np.float64)).max(initial=0.0) * np.abs(f).max())
    tol = (2.0**-22 + far * 2.0**-52) * size + torch.finfo(DT[dtype]).eps / 2 * np.abs(want) * (1 + 2.0**-10) + SMALLEST[dtype]
    rot = 2 * len(f)
    assert np.array_equal(np64(got)[..., rot:], np64(x)[..., rot:])
    off = np.abs(np64(got) - want)
    assert np.all(off <= tol), (off - tol).max()


CASES = [
    # B, n, heads, dim, rot, axes, interleaved, dtype
    (1, 1, 1, 64, 64, 1, False, "bf16"),
    (3, 5, 2, 128, 128, 1, False, "bf16"),
    (2, 7, 28, 128, 64, 1, True, "f16"),
    (2, 33, 3, 64, 16, 1, True, "f32"),
    (1, 130, 5, 128, 48, 2, False, "f32"),
    (2, 9, 40, 64, 64, 3, False, "f16"),
    (5, 3, 1, 80, 80, 4, True, "bf16"),
    (1, 17, 2, 256, 256, 3, False, "f32"),
    (4, 2, 9, 256, 192, 1, True, "bf16"),
    (7, 11, 1, 16, 16, 1, False, "bf16"),
    (1, 4, 300, 128, 128, 1, False, "f16"),
]


@pytest.mark.parametrize("inverse", [False, True])
@pytest.mark.parametrize("case", CASES, ids=["x".join(map(str, c)) for c in CASES])
def test_rope_matches_the_oracle(case, inverse):
    B, n, heads, dim, rot, axes, interleaved, dtype = case
    x, freq = rand((B, n, heads, dim), dtype, 1), freq_of(rot)
    pos = places((axes, B, n), 2) if axes > 1 else places((B, n), 2)
    axis = (torch.arange(rot // 2) % axes).to(torch.uint8) if axes > 1 else None
    got = pkg.rope(x, freq, pos, pair_axis=axis, interleaved=interleaved, inverse=inverse)
    compare(got, x, freq, pos, dtype, axis, interleaved, inverse)
    same = x.clone()
    assert pkg.rope(same, freq, pos, pair_axis=axis, interleaved=interleaved, inverse=inverse, out=same) is same
    assert torch.equal(same, got)


def test_far_and_negative_positions():
    pos = torch.tensor([[0, 1, -1, 131071, 2**24 + 1, -(2**24) - 1, 2**31 - 1, -2**31]], dtype=torch.int32, device=DEV)
    for theta in (1e4, 1e6):
        x, freq = rand((1, 8, 3, 128), "f32", 3), freq_of(128, theta)
        compare(pkg.rope(x, freq, pos), x, freq, pos, "f32")
    # frequencies of more than a turn a position, negative ones and none at all
    x, freq = rand((1, 8, 3, 64), "f32", 4), torch.cat([torch.linspace(-7.0, 7.0, 30, dtype=torch.float64), torch.tensor([0.0, -1e-30])])
    compare(pkg.rope(x, freq, pos[:, :4].repeat(1, 2)), x, freq, pos[:, :4].repeat(1, 2), "f32")


def test_views_and_what_lies_beside_them():
    wide = rand((3, 10, 12, 128), "bf16", 5)
    x, freq, pos = wide[:, 1:8, 2:9, 64:], freq_of(32), places((3, 7), 6)
    big = torch.full((3, 12, 9, 80), 7.0, dtype=torch.bfloat16, device=DEV)
    out = big.permute(0, 2, 1, 3)[:, 1:8, 3:10, 8:72]            # (heads before tokens)
    before = wide.clone()
    assert pkg.rope(x, freq, pos, out=out) is out
    compare(out, x, freq, pos, "bf16")
    assert torch.equal(wide, before)
    out.fill_(7.0)
    assert bool((big == 7.0).all())
    with pytest.raises(pkg.RlkError):                            # not on a 16-byte boundary
        pkg.rope(wide[:, 1:8, 2:9, 60:124], freq, pos)
    with pytest.raises(ValueError):                              # no unit stride
        pkg.rope(wide[..., ::2], freq, places((3, 10), 6))
    # expanded inputs may be read
    got = pkg.rope(x[:, :1].expand(3, 7, 7, 64), freq, pos)
    compare(got, x[:, :1].expand(3, 7, 7, 64), freq, pos, "bf16")


def test_empty():
    freq = freq_of(64)
    for shape in ((0, 3, 2, 64), (2, 0, 2, 64), (2, 3, 0, 64)):
        x = torch.empty(shape, dtype=torch.bfloat16, device=DEV)
        assert pkg.rope(x, freq, places(shape[:2], 1)).shape == shape


def test_a_token_has_its_bits_in_any_batch():
    freq, x, pos = freq_of(128), rand((40, 50, 6, 128), "bf16", 7), places((40, 50), 8, 0, 131072)
    got = pkg.rope(x, freq, pos)
    for b, i in ((0, 0), (39, 49), (17, 23)):
        assert torch.equal(pkg.rope(x[b:b + 1, i:i + 1], freq, pos[b:b + 1, i:i + 1].contiguous())[0, 0], got[b, i])
        assert torch.equal(pkg.rope(x[b:b + 1, i:i + 1, 2:3], freq, pos[b:b + 1, i:i + 1].contiguous())[0, 0, 0], got[b, i, 2])


def test_infinities_stay_with_their_pair():
    x, freq, pos = rand((1, 3, 2, 64), "bf16", 9), freq_of(64), places((1, 3), 10, 1)
    x[0, 1, 1, 5], x[0, 2, 0, 40] = math.inf, math.nan
    y = pkg.rope(x, freq, pos)
    bad = ~torch.isfinite(y)
    want = torch.zeros_like(bad)
    for i, h, j in ((1, 1, 5), (2, 0, 8)):
        want[0, i, h, j] = want[0, i, h, j + 32] = True
    assert torch.equal(bad, want)


@pytest.mark.parametrize("interleaved", [False, True])
def test_gradient(interleaved):
    B, n, heads, dim, rot = 2, 3, 2, 32, 16
    x, freq, pos = rand((B, n, heads, dim), "f32", 11), freq_of(rot), places((3, B, n), 12)
    axis = (torch.arange(rot // 2) % 3).to(torch.uint8)
    kw = dict(pair_axis=axis, interleaved=interleaved)
    w = rand(x.shape, "f32", 13)
    x.requires_grad_()
    y = pkg.rope_autograd(x, freq, pos, **kw)
    assert torch.equal(y, pkg.rope(x.detach(), freq, pos, **kw))
    (y * w).sum().backward()
    compare(x.grad, w, freq, pos, "f32", axis, interleaved, inverse=True)
    # against differences: the map is linear, so that a step of 1 has no error but rounding (each result is
    # within 2^-21 of its size, at most 5 + 1 here; two of them, times |w| <= 5, in 32 places a head that differ
    # in two elements only)
    z = x.detach()
    for at in ((0, 0, 0, 0), (1, 2, 1, 9), (1, 0, 1, 15), (0, 1, 0, 20)):
        hi, lo = z.clone(), z.clone()
        hi[at] += 1.0
        lo[at] -= 1.0
        d = ((pkg.rope(hi, freq, pos, **kw).double() - pkg.rope(lo, freq, pos, **kw).double()) * w.double()).sum() / 2
        assert abs(float(d) - float(x.grad[at])) <= 2 * 2 * 6 * 5 * 2.0**-21
    # an expanded gradient, and one of views
    x.grad = None
    pkg.rope_autograd(x, freq, pos, **kw).sum().backward()
    compare(x.grad, torch.ones_like(x), freq, pos, "f32", axis, interleaved, inverse=True)
    x.grad = None
    pkg.rope_autograd(x, freq, pos, **kw)[..., 1:].transpose(1, 2).contiguous().mul(2.0).sum().backward()
    ones = torch.full_like(x, 2.0)
    ones[..., 0] = 0.0
    compare(x.grad, ones, freq, pos, "f32", axis, interleaved, inverse=True)


def test_gradient_refuses_changed_positions():
    x, freq, pos = rand((1, 3, 2, 32), "f32", 14).requires_grad_(), freq_of(32), places((1, 3), 15)
    y = pkg.rope_autograd(x, freq, pos)
    pos += 1
    with pytest.raises(RuntimeError):
        y.sum().backward()


# ------------------------------------------------------------ on the way into the cache

def make(lens, n, heads, kv_heads, dim, page, dtype, order="token", seed=0):
    need = [-(-t // page) for t in lens]
    pages = sum(need) + 2
    shape = (pages, page, kv_heads, dim) if order == "token" else (pages, kv_heads, page, dim)
    k, v = rand(shape, dtype, seed), rand(shape, dtype, seed + 1)
    if order == "head":
        k, v = k.transpose(1, 2), v.transpose(1, 2)
    perm, at = torch.randperm(pages, generator=torch.Generator().manual_seed(seed)).tolist(), 0
    table = torch.full((len(lens), max(1, max(need, default=1))), -7, dtype=torch.int32)
    for b, m in enumerate(need):
        table[b, :m] = torch.tensor(perm[at:at + m], dtype=torch.int32)
        at += m
    qkv = rand((len(lens), n, heads + 2 * kv_heads, dim), dtype, seed + 2)
    q, kn, vn = qkv.split([heads, kv_heads, kv_heads], dim=2)
    return dict(k=k, v=v, table=table.to(DEV), lens=torch.tensor(lens, dtype=torch.int32, device=DEV), q=q, kn=kn, vn=vn)


def append(c, freq, new=None, **kw):
    kw = dict(q=c["q"]) | kw
    return pkg.kv_append_rope(c["k"], c["v"], c["table"], c["lens"], c["kn"], c["vn"], freq,
                              new_lens=None if new is None else torch.tensor(new, dtype=torch.int32, device=DEV), **kw)


def copy(t):
    """The same values in memory that lies the same."""
    out = torch.empty_strided(t.shape, t.stride(), dtype=t.dtype, device=t.device)
    out.copy_(t)
    return out


APPENDS = [
    # lens, n, new, heads, kv_heads, dim, page, dtype, order, rot, interleaved, axes (0: none given)
    ([1], 1, None, 1, 1, 64, 16, "bf16", "token", 64, False, 0),
    ([5, 40, 17], 3, [3, 0, 2], 8, 2, 128, 16, "bf16", "token", 128, False, 0),
    ([200, 77, 0, 9], 9, [9, 5, 0, 9], 28, 4, 128, 24, "f16", "head", 64, True, 1),
    ([1000] * 5, 100, None, 32, 8, 128, 7, "bf16", "token", 128, False, 3),
    ([64, 63], 64, [64, 1], 3, 1, 64, 1, "f16", "token", 48, True, 4),
    ([31], 30, None, 130, 2, 64, 1000, "bf16", "head", 16, False, 0),
    ([10] * 200, 1, None, 16, 16, 128, 16, "f16", "token", 128, False, 0),
]


@pytest.mark.parametrize("case", APPENDS, ids=[f"{c[0][0]}x{c[1]}h{c[3]}-{c[4]}d{c[5]}p{c[6]}{c[7]}{c[8]}r{c[9]}" for c in APPENDS])
def test_append_has_the_bits_of_rope_and_append(case):
    lens, n, new, heads, kv_heads, dim, page, dtype, order, rot, interleaved, axes = case
    c = make(lens, n, heads, kv_heads, dim, page, dtype, order, seed=20)
    B, freq, m = len(lens), freq_of(rot), [n] * len(lens) if new is None else new
    kw = dict(interleaved=interleaved)
    if axes:
        kw["positions"] = places((axes, B, n), 21)
        kw["pair_axis"] = (torch.arange(rot // 2) % axes).to(torch.uint8)
        at = kw["positions"]
    else:
        at = torch.tensor([[t - a + i for i in range(n)] for t, a in zip(lens, m)], dtype=torch.int32, device=DEV)
    turned = {x: pkg.rope(c[x], freq, at, pair_axis=kw.get("pair_axis"), interleaved=interleaved) for x in ("q", "kn")}
    k, v = copy(c["k"]), copy(c["v"])
    ml = torch.tensor(m, dtype=torch.int32, device=DEV)
    pkg.kv_append(k, v, c["table"], c["lens"], turned["kn"], c["vn"], new_lens=ml)
    before = c["q"].clone()
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    k0, v0 = copy(c["k"]), copy(c["v"])
    q = append(c, freq, new, err_count=err, **kw)
    assert torch.equal(c["k"], k) and torch.equal(c["v"], v) and int(err) == 0
    there = torch.arange(n, device=DEV) < ml[:, None]
    want = turned["q"].masked_fill(~there[..., None, None], 0.0)
    assert torch.equal(q, want) and torch.equal(c["q"], before)
    # queries in place, as views of the wider row; and the keys and values alone
    c["k"].copy_(k0)
    c["v"].copy_(v0)
    assert append(c, freq, new, q_out=c["q"], **kw) is c["q"]
    assert torch.equal(c["q"], want) and torch.equal(c["k"], k) and torch.equal(c["v"], v)
    c["k"].copy_(k0)
    c["v"].copy_(v0)
    assert append(c, freq, new, q=None, **kw) is None
    assert torch.equal(c["k"], k) and torch.equal(c["v"], v)


def test_append_matches_the_oracle():
    c = make([300, 12, 4097], 4, 4, 2, 128, 16, "bf16", seed=30)
    freq = freq_of(128, 1e6)
    q = append(c, freq)
    at = torch.tensor([[t - 4 + i for i in range(4)] for t in (300, 12, 4097)], dtype=torch.int32)
    compare(q, c["q"], freq, at, "bf16")
    table = c["table"].tolist()
    for b, t in enumerate((300, 12, 4097)):
        for i in range(4):
            p = t - 4 + i
            compare(c["k"][table[b][p // 16], p % 16][None, None], c["kn"][b:b + 1, i:i + 1], freq, at[b:b + 1, i:i + 1], "bf16")


def test_append_rejects():
    c = make([20, 9, 30, 16], 2, 4, 2, 64, 8, "bf16", seed=40)
    c["lens"].copy_(torch.tensor([20, 1, 33, 16]))               # fewer than new; more than the table holds
    c["table"][3, 1] = c["k"].shape[0]                           # the page of the last sequence's new tokens
    k0, v0, freq = copy(c["k"]), copy(c["v"]), freq_of(64)
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    q = append(c, freq, err_count=err)
    assert int(err) == 1 + 1 + 2
    at = torch.tensor([[18, 19], [0, 0], [0, 0], [14, 15]], dtype=torch.int32, device=DEV)
    want = pkg.rope(c["q"], freq, at)
    assert torch.equal(q[0], want[0]) and torch.equal(q[3], want[3])
    assert bool(torch.isnan(q[1]).all()) and bool(torch.isnan(q[2]).all())
    changed = (c["k"] != k0).any(-1).any(-1)
    places_ = {(int(c["table"][0, 2]), p) for p in (2, 3)}
    assert {tuple(x) for x in changed.nonzero().tolist()} == places_
    assert {tuple(x) for x in (c["v"] != v0).any(-1).any(-1).nonzero().tolist()} == places_


def test_append_refuses():
    c, freq = make([20], 2, 4, 2, 64, 8, "bf16", seed=50), freq_of(64)
    bad = [dict(q=None, q_out=c["q"]), dict(q=c["q"][0]), dict(q=c["q"].half()), dict(q_out=c["q"][:, :1]),
           dict(positions=places((1, 3), 1)), dict(positions=places((1, 2), 1).cpu()), dict(positions=places((1, 2), 1).long())]
    for kw in bad:
        with pytest.raises(ValueError):
            append(c, freq, **kw)
    with pytest.raises(pkg.RlkError):
        append(c, freq_of(128))
    with pytest.raises(ValueError):
        append(c, freq.to(DEV))


def test_a_captured_step():
    c = make([100, 300], 1, 8, 2, 128, 16, "bf16", seed=60)
    freq, out = freq_of(128), torch.empty((2, 1, 8, 128), dtype=torch.bfloat16, device=DEV)
    x, pos = rand((2, 1, 8, 128), "bf16", 61), places((2, 1), 62)
    y = torch.empty_like(x)
    append(c, freq, q_out=out)
    g = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(g):
        append(c, freq, q_out=out)
        pkg.rope(x, freq, pos, out=y)
    freq.zero_()                                                 # (read during the call, so no longer of account)
    for step in range(2):
        c["lens"] -= 1
        pos += 100
        k0 = copy(c["k"])
        g.replay()
        f = freq_of(128)
        want, k = append(c, f), copy(c["k"])
        c["k"].copy_(k0)
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want) and torch.equal(c["k"], k) and torch.equal(y, pkg.rope(x, f, pos))


def test_a_rotation_of_billions_of_bytes():
    # element offsets past 2^31: the last token of 2^17 + 1 with a stride of 2^14 + 8 elements
    n, stride = 2**17 + 1, 2**14 + 8
    flat = torch.zeros(n * stride, dtype=torch.bfloat16, device=DEV)
    x = flat.as_strided((1, n, 2, 64), (n * stride, stride, 64, 1))
    x[0, -1] = rand((2, 64), "bf16", 70)
    pos, freq = places((1, n), 71, 0, 131072), freq_of(64)
    y = pkg.rope(x, freq, pos)
    compare(y[:, -1:], x[:, -1:], freq, pos[:, -1:], "bf16")
    assert not y[0, :-1].any()
