"""Pins of the rotation's oracle, and what its C entry points refuse on the host before
anything is enqueued (runs without a GPU)."""

import ctypes
import math

import numpy as np
import pytest

import rollout_consistent_vocab_gb300 as pkg
from oracle import rope_oracle as ro
from rollout_consistent_vocab_gb300 import _binding as b
from rollout_consistent_vocab_gb300.build import build_library
from test_rollout_abi_cpu import BAD, cache


@pytest.fixture(scope="module")
def lib():
    build_library()
    return pkg.load_library()


# ------------------------------------------------------------ the oracle

def test_angles_of_far_positions():
    assert ro.angle(0, 1.0) == 0.0
    assert abs(ro.angle(3, 0.5) - 1.5) < 1e-15
    assert abs(ro.angle(-4, 1.0) - (2 * math.pi - 4)) < 1e-14
    # a frequency that is a binary fraction of a radian: math.sin reduces its argument exactly
    for p in (131071, 2**31 - 1, -2**31):
        assert abs(math.sin(ro.angle(p, 0.375)) - math.sin(p * 0.375)) < 1e-14
        assert abs(math.cos(ro.angle(p, 0.375)) - math.cos(p * 0.375)) < 1e-14


@pytest.mark.parametrize("interleaved", [False, True])
def test_rotation_as_complex_numbers(interleaved):
    r = np.random.default_rng(1)
    x, f = r.standard_normal((2, 3, 2, 24)), 10.0 ** -np.arange(8)
    pos, axis = r.integers(0, 5000, (3, 2, 3)), r.integers(0, 3, 8)
    y, size = ro.rope(x, f, pos, axis, interleaved)
    z = x[..., 0:16:2] + 1j * x[..., 1:16:2] if interleaved else x[..., :8] + 1j * x[..., 8:16]
    z = z * np.exp(1j * np.moveaxis(pos[axis], 0, -1) * f)[:, :, None]
    re, im = (y[..., 0:16:2], y[..., 1:16:2]) if interleaved else (y[..., :8], y[..., 8:16])
    np.testing.assert_allclose(re, z.real, atol=1e-11)
    np.testing.assert_allclose(im, z.imag, atol=1e-11)
    assert np.array_equal(y[..., 16:], x[..., 16:]) and np.all(size + 1e-12 >= np.abs(y))
    back, _ = ro.rope(y, f, pos, axis, interleaved, inverse=True)
    np.testing.assert_allclose(back, x, atol=1e-14)
    # a planted mistake: the sign of the angle
    wrong, _ = ro.rope(x, f, pos, axis, interleaved, inverse=True)
    assert np.abs(wrong - y).max() > 0.1


# ------------------------------------------------------------ refusals

FREQ = (ctypes.c_double * 128)(*[1.0 / (1 + j) for j in range(128)])


def args(freq=FREQ, axis=None, rot=64, interleaved=0, positions=0x90000, axes=1):
    return b.RopeArgs(None if freq is None else ctypes.addressof(freq), axis, rot, interleaved, positions, axes)


def freqs(bad):
    f = (ctypes.c_double * 64)(*[0.5] * 64)
    f[31] = bad
    return f


BAD_FREQ = [freqs(math.inf), freqs(math.nan)]
BAD_AXIS, GOOD_AXIS = (ctypes.c_uint8 * 64)(*[0] * 31 + [3] * 33), (ctypes.c_uint8 * 64)(*[0] * 31 + [1] * 33)
ROPES = [
    (dict(freq=None), b.RLK_EINVAL), (dict(rot=0), b.RLK_EINVAL), (dict(rot=8), b.RLK_EINVAL), (dict(rot=24), b.RLK_EINVAL),
    (dict(rot=-16), b.RLK_EINVAL), (dict(rot=144), b.RLK_EINVAL), (dict(interleaved=2), b.RLK_EINVAL),
    (dict(axes=0), b.RLK_EINVAL), (dict(axes=5), b.RLK_EINVAL), (dict(positions=0x90002), b.RLK_EALIGN),
    (dict(freq=BAD_FREQ[0]), b.RLK_EINVAL), (dict(freq=BAD_FREQ[1]), b.RLK_EINVAL),
    (dict(axis=ctypes.addressof(BAD_AXIS), axes=3), b.RLK_EINVAL), (dict(axis=ctypes.addressof(GOOD_AXIS)), b.RLK_EINVAL),
]


@pytest.mark.parametrize("kw,status", ROPES)
def test_rotation_is_checked(lib, kw, status):
    st = ctypes.byref(b.BTHStrides(512, 256, 128))
    r = args(**kw)
    assert lib.rlk_rope(ctypes.byref(r), 3, 2, 2, 128, b.RLK_DT_BF16, 0x60000, st, 0x70000, st, 0, None) == status
    assert lib.rlk_kv_append_rope(ctypes.byref(cache()), ctypes.byref(r), 0x60000, st, 0x70000, st, 0xA0000, st, 2, 0xB0000, st,
                                  None) == status
    assert lib.rlk_last_error()


def test_rope_call_is_checked(lib):
    good = b.BTHStrides(512, 256, 128)

    def call(r=args(), B=3, n=2, heads=2, dim=128, dtype=b.RLK_DT_BF16, x=0x60000, xs=good, out=0x70000, os=good, inverse=0):
        ref = lambda s: None if s is None else ctypes.byref(s)  # noqa: E731
        return lib.rlk_rope(ref(r), B, n, heads, dim, dtype, x, ref(xs), out, ref(os), inverse, None)

    for kw in (dict(r=None), dict(B=-1), dict(n=-1), dict(heads=-1), dict(dim=0), dict(dim=72), dict(dim=272), dict(dim=48),
               dict(dtype=7), dict(x=None), dict(xs=None), dict(out=None), dict(os=None), dict(inverse=2), dict(B=1 << 32, n=1),
               dict(B=1 << 16, n=1 << 16), dict(r=args(positions=None)), dict(out=0x60000, os=b.BTHStrides(512, 256, 256))):
        assert call(**kw) == b.RLK_EINVAL, kw
    for kw in (dict(x=0x60008), dict(out=0x70002), dict(xs=b.BTHStrides(512, 252, 128)), dict(os=b.BTHStrides(4, 256, 128)),
               dict(dtype=b.RLK_DT_F32, xs=b.BTHStrides(512, 256, 130))):
        assert call(**kw) == b.RLK_EALIGN, kw
    # nothing to do
    for kw in (dict(B=0), dict(n=0), dict(heads=0)):
        assert call(x=None, xs=None, out=None, os=None, r=args(positions=None), **kw) == b.RLK_OK, kw


@pytest.mark.parametrize("kw,status", BAD)
def test_append_checks_the_cache(lib, kw, status):
    st = ctypes.byref(b.BTHStrides(512, 256, 128))
    r = args()
    assert lib.rlk_kv_append_rope(ctypes.byref(cache(**kw)), ctypes.byref(r), 0x60000, st, 0x70000, st, None, None, 0, None, None,
                                  None) == status


def test_append_call_is_checked(lib):
    good = b.BTHStrides(512, 256, 128)

    def call(c=cache(), r=args(), k=0x60000, ks=good, v=0x70000, vs=good, q=0xA0000, qs=good, heads=2, out=0xB0000, os=good):
        ref = lambda s: None if s is None else ctypes.byref(s)  # noqa: E731
        return lib.rlk_kv_append_rope(ref(c), ref(r), k, ref(ks), v, ref(vs), q, ref(qs), heads, out, ref(os), None)

    for kw in (dict(c=None), dict(r=None), dict(k=None), dict(ks=None), dict(v=None), dict(vs=None), dict(q=None), dict(qs=None),
               dict(out=None), dict(os=None), dict(heads=-1), dict(heads=257), dict(c=cache(head_dim=64), r=args(rot=80)),
               dict(out=0xA0000, os=b.BTHStrides(512, 128, 256))):
        assert call(**kw) == b.RLK_EINVAL, kw
    for kw in (dict(k=0x60008), dict(q=0xA0004), dict(out=0xB0002), dict(qs=b.BTHStrides(512, 250, 128)),
               dict(os=b.BTHStrides(512, 256, 12))):
        assert call(**kw) == b.RLK_EALIGN, kw
    for c in (cache(B=0), cache(n=0), cache(B=0, k=None, lens=None, page_table=None)):
        assert call(c=c, k=None, ks=None, v=None, vs=None, q=None, qs=None, out=None, os=None) == b.RLK_OK


def test_binding_refuses():
    import torch
    f = torch.ones(32, dtype=torch.float64)
    pos = torch.zeros((2, 3), dtype=torch.int32)
    good = b._rope_args(f, None, False, pos, 2, 3, -1)
    assert good.rot_dim == 64 and good.axes == 1
    assert b._rope_args(f, None, True, pos[None].repeat(3, 1, 1), 2, 3, -1).axes == 3
    axis = torch.zeros(32, dtype=torch.uint8)
    for kw in (dict(inv_freq=f.float()), dict(inv_freq=f[None]), dict(inv_freq=torch.ones(64, dtype=torch.float64)[::2]),
               dict(pair_axis=axis.int()), dict(pair_axis=axis[:31]), dict(pair_axis=torch.zeros(64, dtype=torch.uint8)[::2]),
               dict(positions=pos.long()), dict(positions=pos[:1]), dict(positions=pos[0]), dict(positions=pos.T),
               dict(positions=torch.zeros((3, 2), dtype=torch.int32).T)):
        with pytest.raises(ValueError):
            b._rope_args(**dict(inv_freq=f, pair_axis=None, interleaved=False, positions=pos, B=2, n=3, dev=-1) | kw)
    with pytest.raises(ValueError):
        b._rope_args(f, None, False, pos, 2, 3, 0)
    with pytest.raises(ValueError):
        pkg.rope(torch.zeros((2, 3, 1, 64)), f, pos)
