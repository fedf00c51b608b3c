"""The rollout operators' C entry points refuse bad arguments on the host
before anything is enqueued (runs without a GPU)."""

import ctypes
import math

import pytest

import rollout_consistent_vocab_gb300 as pkg
from rollout_consistent_vocab_gb300 import _binding as b
from rollout_consistent_vocab_gb300.build import build_library


@pytest.fixture(scope="module")
def lib():
    build_library()
    return pkg.load_library()


def cache(**kw):
    c = b.KVCache(0x10000, 0x20000, 8, 4096, 256, 128, 16, 2, 128, b.RLK_DT_BF16, 0x30000, 4, 4, 3, 0x40000,
                  None, 2, None)
    for k, v in kw.items():
        setattr(c, k, v)
    return c


BAD = [
    (dict(k=None), b.RLK_EINVAL), (dict(v=None), b.RLK_EINVAL), (dict(page_table=None), b.RLK_EINVAL),
    (dict(lens=None), b.RLK_EINVAL), (dict(B=-1), b.RLK_EINVAL), (dict(B=1 << 16), b.RLK_EINVAL),
    (dict(n=-1), b.RLK_EINVAL), (dict(n=1 << 16), b.RLK_EINVAL), (dict(head_dim=96), b.RLK_EINVAL),
    (dict(dtype=b.RLK_DT_F32), b.RLK_EINVAL), (dict(kv_heads=0), b.RLK_EINVAL), (dict(page_size=0), b.RLK_EINVAL),
    (dict(max_pages=-1), b.RLK_EINVAL), (dict(table_stride=3), b.RLK_EINVAL), (dict(num_pages=-1), b.RLK_EINVAL),
    (dict(page_size=1 << 30, max_pages=4), b.RLK_EINVAL), (dict(kv_heads=1025), b.RLK_EINVAL),
    (dict(k=0x10008), b.RLK_EALIGN), (dict(page_stride=4100), b.RLK_EALIGN), (dict(token_stride=4), b.RLK_EALIGN),
    (dict(head_stride=130), b.RLK_EALIGN), (dict(lens=0x40002), b.RLK_EALIGN), (dict(page_table=0x30001), b.RLK_EALIGN),
    (dict(new_lens=0x50002), b.RLK_EALIGN), (dict(err_count=0x50001), b.RLK_EALIGN),
]


@pytest.mark.parametrize("kw,status", BAD)
def test_cache_is_checked(lib, kw, status):
    st = b.BTHStrides(512, 256, 128)
    c = cache(**kw)
    s = ctypes.byref(st)
    assert lib.rlk_kv_append(ctypes.byref(c), 0x60000, s, 0x70000, s, None) == status
    assert lib.rlk_paged_attention(ctypes.byref(c), 0x60000, s, 4, 0.1, 0, 0, 0x70000, s, None, 0x80000, None) == status
    assert lib.rlk_last_error()


def test_calls_are_checked(lib):
    c, st = cache(), b.BTHStrides(512, 256, 128)

    def append(k=0x60000, ks=st, v=0x70000, vs=st, c=c):
        return lib.rlk_kv_append(None if c is None else ctypes.byref(c), k, None if ks is None else ctypes.byref(ks), v,
                                 None if vs is None else ctypes.byref(vs), None)

    assert append(c=None) == b.RLK_EINVAL
    assert append(k=None) == b.RLK_EINVAL
    assert append(vs=None) == b.RLK_EINVAL
    assert append(v=0x70004) == b.RLK_EALIGN
    assert append(ks=b.BTHStrides(512, 250, 128)) == b.RLK_EALIGN

    def attend(q=0x60000, qs=st, heads=4, scale=0.1, window=0, sinks=0, out=0x70000, os=st, lse=None, ws=0x80000):
        return lib.rlk_paged_attention(ctypes.byref(c), q, ctypes.byref(qs), heads, scale, window, sinks, out,
                                       ctypes.byref(os), lse, ws, None)

    assert attend(q=None) == b.RLK_EINVAL
    assert attend(out=None) == b.RLK_EINVAL
    for heads in (0, 3, -2, 2 * 128 + 2):
        assert attend(heads=heads) == b.RLK_EINVAL
    for scale in (math.inf, math.nan):
        assert attend(scale=scale) == b.RLK_EINVAL
    assert attend(window=-1) == b.RLK_EINVAL
    assert attend(sinks=-1) == b.RLK_EINVAL
    assert attend(q=0x60008) == b.RLK_EALIGN
    assert attend(os=b.BTHStrides(512, 256, 132)) == b.RLK_EALIGN
    assert attend(lse=0x90002) == b.RLK_EALIGN


def test_empty_calls_are_no_ops(lib):
    st = b.BTHStrides(0, 0, 0)
    s = ctypes.byref(st)
    for c in (cache(B=0), cache(n=0), cache(B=0, k=None, lens=None, page_table=None)):
        assert lib.rlk_kv_append(ctypes.byref(c), None, s, None, s, None) == b.RLK_OK
        assert lib.rlk_paged_attention(ctypes.byref(c), None, s, 4, 0.1, 0, 0, None, s, None, None, None) == b.RLK_OK


def test_workspace_formula(lib):
    size = ctypes.c_size_t()
    for B, n, heads, kv, dim, tokens in ((1, 1, 8, 8, 128, 16), (1, 1, 8, 1, 64, 256), (3, 2, 4, 2, 128, 257),
                                         (2, 1, 32, 8, 128, 16384), (2, 9, 32, 8, 128, 16385), (1, 5, 7, 7, 64, 131072),
                                         (1, 1, 1, 1, 64, 2**31 - 1), (0, 1, 1, 1, 64, 500), (4, 8, 64, 8, 128, 1),
                                         (4, 17, 64, 8, 128, 5000), (65535, 1, 32, 4, 128, 70000)):
        assert lib.rlk_paged_attention_workspace(B, n, heads, kv, dim, tokens, ctypes.byref(size)) == b.RLK_OK
        assert b.paged_attention_workspace_bytes(B, n, heads, kv, dim, tokens) == size.value
    assert lib.rlk_paged_attention_workspace(-1, 1, 1, 1, 64, 1, ctypes.byref(size)) == b.RLK_EINVAL
    assert lib.rlk_paged_attention_workspace(1, 1, 3, 2, 64, 1, ctypes.byref(size)) == b.RLK_EINVAL
    assert lib.rlk_paged_attention_workspace(1, 1, 3, 0, 64, 1, ctypes.byref(size)) == b.RLK_EINVAL
    assert lib.rlk_paged_attention_workspace(1, 1, 1, 1, 64, 1, None) == b.RLK_EINVAL


def verify_args(**kw):
    a = b.VerifyArgs(3, 2, b.VOCAB_REAL, b.VOCAB_PADDED, 0x10000, b.VOCAB_PADDED, 0x20000, b.VOCAB_PADDED, 0x30000, None,
                     None, 0.7, None, 0.95, None, 50, None, 0.7, None, 0.95, None, 50, 0x40000, 0x50000, None)
    for k, v in kw.items():
        setattr(a, k, v)
    return a


@pytest.mark.parametrize("kw,status", [
    (dict(B=-1), b.RLK_EINVAL), (dict(n=-1), b.RLK_EINVAL), (dict(n=1025), b.RLK_EINVAL), (dict(B=1 << 28), b.RLK_EINVAL),
    (dict(B=1 << 27), b.RLK_EINVAL), (dict(vocab_real=7), b.RLK_EINVAL), (dict(logits=None), b.RLK_EINVAL),
    (dict(logits=0x10008), b.RLK_EALIGN), (dict(row_stride=100), b.RLK_EINVAL), (dict(draft_logits=0x20004), b.RLK_EALIGN),
    (dict(draft_row_stride=152580), b.RLK_EALIGN), (dict(draft_token=None), b.RLK_EINVAL), (dict(accept_uniform=None), b.RLK_EINVAL),
    (dict(draw_uniform=None), b.RLK_EINVAL), (dict(draw_uniform=0x50002), b.RLK_EALIGN), (dict(num_drafts=0x60001), b.RLK_EALIGN),
    (dict(temperature_scalar=-1.0), b.RLK_EINVAL), (dict(top_p_scalar=0.0), b.RLK_EINVAL), (dict(top_k_scalar=0), b.RLK_EINVAL),
    (dict(draft_temperature_scalar=math.inf), b.RLK_EINVAL), (dict(draft_top_p_scalar=1.5), b.RLK_EINVAL),
    (dict(draft_top_k_scalar=-2), b.RLK_EINVAL), (dict(temperature=0x70002), b.RLK_EALIGN), (dict(draft_top_k=0x70002), b.RLK_EALIGN),
    (dict(err_count=0x70002), b.RLK_EALIGN),
])
def test_verify_is_checked(lib, kw, status):
    a = verify_args(**kw)
    assert lib.rlk_verify_drafts(ctypes.byref(a), 0x80000, 0x90000, None, None, 0xA0000, None) == status
    assert lib.rlk_last_error()


def test_verify_outputs_are_checked(lib):
    def call(token=0x80000, accepted=0x90000, restr=None, full=None, ws=0xA0000, a=verify_args()):
        return lib.rlk_verify_drafts(None if a is None else ctypes.byref(a), token, accepted, restr, full, ws, None)

    assert call(a=None) == b.RLK_EINVAL
    assert call(token=None) == b.RLK_EINVAL
    assert call(accepted=None) == b.RLK_EINVAL
    assert call(ws=None) == b.RLK_EINVAL
    assert call(ws=0xA0008) == b.RLK_EALIGN
    assert call(restr=0x81002) == b.RLK_EALIGN
    assert call(full=0x81001) == b.RLK_EALIGN
    # the draft model's parameters are of no account without its logits; an empty batch is a no-op
    assert call(a=verify_args(B=0, draft_logits=None, draft_top_p_scalar=9.0)) == b.RLK_OK


def test_verify_workspace_macro():
    import os
    import re
    text = open(os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "include", "rlk_rollout.h")).read()
    m = re.search(r"#define\s+RLK_VERIFY_WORKSPACE_BYTES\(B, n\)\s+(.+)", text).group(1)
    for B, n in ((1, 0), (3, 4), (128, 7)):
        assert eval(re.sub(r"\(size_t\)|(?<=\d)u\b", "", m), {"B": B, "n": n}) == b.verify_workspace_bytes(B, n)
