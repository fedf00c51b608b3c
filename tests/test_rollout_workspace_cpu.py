"""The workspace of paged attention at the C entry point (runs without a GPU)."""

import ctypes

import pytest

import rollout_consistent_vocab_gb300 as pkg
from rollout_consistent_vocab_gb300 import _binding as b
from rollout_consistent_vocab_gb300.build import build_library
from test_rollout_abi_cpu import cache


@pytest.fixture(scope="module")
def lib():
    build_library()
    return pkg.load_library()


def test_workspace_is_checked(lib):
    c, st = cache(), b.BTHStrides(512, 256, 128)

    def attend(ws):
        s = ctypes.byref(st)
        return lib.rlk_paged_attention(ctypes.byref(c), 0x60000, s, 4, 0.1, 0, 0, 0x70000, s, None, ws, None)

    assert attend(None) == b.RLK_EINVAL
    assert attend(0x80008) == b.RLK_EALIGN


def test_no_tokens_need_no_workspace(lib):
    size = ctypes.c_size_t(7)
    for B, n, heads, tokens in ((3, 2, 8, 0), (0, 2, 8, 100), (3, 0, 8, 100)):
        assert lib.rlk_paged_attention_workspace(B, n, heads, 2, 64, tokens, ctypes.byref(size)) == b.RLK_OK
        assert size.value == 0 == b.paged_attention_workspace_bytes(B, n, heads, 2, 64, tokens)
