"""The shared-prefix attention's C entry points refuse bad arguments on the host before
anything is enqueued, and its scratch sizes (runs without a GPU)."""

import ctypes
import math

import pytest

import rollout_consistent_vocab_gb300 as pkg
from rollout_consistent_vocab_gb300 import _binding as b
from rollout_consistent_vocab_gb300.build import build_library
from test_rollout_abi_cpu import BAD, cache


@pytest.fixture(scope="module")
def lib():
    build_library()
    return pkg.load_library()


def attend(lib, c=cache(), start=0xA0000, shared=0xB0000, groups=2, most=40, pg=True, q=0x60000, qs=b.BTHStrides(512, 256, 128), heads=4,
           scale=0.1, out=0x70000, os=b.BTHStrides(512, 256, 128), lse=None, ws=0x80000):
    ref = lambda s: None if s is None else ctypes.byref(s)  # noqa: E731
    g = b.PrefixGroups(start, shared, groups, most)
    return lib.rlk_prefix_attention(ref(c), ref(g if pg else None), q, ref(qs), heads, scale, out, ref(os), lse, ws, None)


@pytest.mark.parametrize("kw,status", BAD)
def test_cache_is_checked(lib, kw, status):
    assert attend(lib, c=cache(**kw)) == status
    assert lib.rlk_last_error()


def test_call_is_checked(lib):
    for kw in (dict(c=None), dict(pg=False), dict(start=None), dict(shared=None), dict(groups=-1), dict(groups=1 << 16), dict(most=-1),
               dict(most=65), dict(q=None), dict(qs=None), dict(out=None), dict(os=None), dict(heads=0), dict(heads=3),
               dict(heads=258), dict(scale=math.inf), dict(scale=math.nan), dict(ws=None)):
        assert attend(lib, **kw) == b.RLK_EINVAL, kw
    for kw in (dict(start=0xA0002), dict(shared=0xB0001), dict(q=0x60008), dict(out=0x70004), dict(lse=0x90002), dict(ws=0x80008),
               dict(os=b.BTHStrides(512, 256, 130))):
        assert attend(lib, **kw) == b.RLK_EALIGN, kw
    # places a step past the last token are still of 32 bits; so are the steps of all sequences
    for c in (cache(page_size=1, max_pages=2**31 - 64, table_stride=2**31), cache(page_size=1 << 20, max_pages=2047, B=65535, table_stride=2048)):
        assert attend(lib, c=c) == b.RLK_EINVAL
    for c in (cache(B=0), cache(n=0), cache(B=0, k=None, lens=None, page_table=None)):
        assert attend(lib, c=c, q=None, qs=None, out=None, os=None, ws=None, start=None, shared=None) == b.RLK_OK


def test_workspace_formula(lib):
    size = ctypes.c_size_t()
    call = lib.rlk_prefix_attention_workspace
    for B, n, heads, kv, dim, tokens, groups, most in (
            (1, 1, 8, 8, 128, 16, 1, 16), (1, 1, 8, 1, 64, 256, 0, 0), (64, 1, 32, 8, 128, 16384, 4, 31), (64, 1, 32, 8, 128, 16384, 4, 32),
            (64, 1, 32, 8, 128, 16384, 1, 8191), (64, 1, 32, 8, 128, 16384, 1, 8192), (64, 1, 32, 8, 128, 16384, 1, 9000),
            (3, 5, 8, 2, 64, 140000, 3, 32767), (3, 5, 8, 2, 64, 140000, 3, 32800), (3, 5, 8, 2, 64, 140000, 3, 131071),
            (0, 1, 1, 1, 64, 500, 0, 100), (2, 1, 1, 1, 64, 2**31 - 1, 65535, 2**31 - 1), (65535, 1, 32, 4, 128, 70000, 300, 700)):
        assert call(B, n, heads, kv, dim, tokens, groups, most, ctypes.byref(size)) == b.RLK_OK
        assert b.prefix_attention_workspace_bytes(B, n, heads, kv, dim, tokens, groups, most) == size.value
    for bad in ((-1, 1, 1, 1, 64, 1, 0, 0), (1, 1, 3, 2, 64, 1, 0, 0), (1, 1, 1, 1, 64, 10, -1, 0), (1, 1, 1, 1, 64, 10, 1 << 16, 0),
                (1, 1, 1, 1, 64, 10, 1, 11), (1, 1, 1, 1, 64, 10, 1, -1)):
        assert call(*bad, ctypes.byref(size)) == b.RLK_EINVAL, bad
    assert call(1, 1, 1, 1, 64, 1, 0, 0, None) == b.RLK_EINVAL
