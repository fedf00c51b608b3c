"""The rollout calls refuse tensors that are not on the GPU where the others are, before anything
is enqueued.  (A second GPU is stood in for by objects that say so; nothing is launched.)"""

import types

import pytest
import torch

import rollout_consistent_vocab_gb300 as pkg
from rollout_consistent_vocab_gb300 import _binding as b


class Elsewhere:
    """What the checks look at of a tensor on cuda:1."""
    dtype, device = torch.int32, torch.device("cuda", 1)

    def get_device(self):
        return 1

    def numel(self):
        return 1

    def data_ptr(self):
        return 0x1000


def test_tensors_on_another_gpu():
    b._placed(Elsewhere(), 1, "x")
    assert b._err_ptr(Elsewhere(), 1) == 0x1000
    for call in (lambda: b._placed(Elsewhere(), 0, "x"), lambda: b._err_ptr(Elsewhere(), 0),
                 lambda: b._placed(torch.zeros(1), 0, "x"), lambda: b._err_ptr(torch.zeros(1, dtype=torch.int32), 0),
                 lambda: b._err_ptr(torch.zeros(1), -1), lambda: b._err_ptr(torch.zeros(0, dtype=torch.int32), -1)):
        with pytest.raises(ValueError):
            call()


def test_the_current_gpu_and_the_stream(monkeypatch):
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    with pytest.raises(ValueError):
        b._stream(None, 1)
    st = types.SimpleNamespace(cuda_stream=77, device=torch.device("cuda", 1))
    assert b._stream(st, 1) == b._stream(st) == 77
    with pytest.raises(ValueError):
        b._stream(st, 0)


# ------------------------------------------------------------ on a GPU: host tensors

@pytest.fixture(scope="module")
def lib():
    from rollout_consistent_vocab_gb300.build import build_library
    build_library()
    pkg.load_library()


def i32(v, device="cuda"):
    return torch.tensor(v, dtype=torch.int32, device=device)


@pytest.mark.gpu
def test_attention_and_append_refuse_host_tensors(lib):
    k = torch.zeros((4, 16, 2, 64), dtype=torch.bfloat16, device="cuda")
    q = torch.zeros((2, 1, 8, 64), dtype=torch.bfloat16, device="cuda")
    a = dict(q=q, k_cache=k, v_cache=k.clone(), page_table=i32([[0], [1]]), lens=i32([3, 4]))
    need = pkg.paged_attention_workspace_bytes(2, 1, 8, 2, 64, 16)
    more = dict(new_lens=i32([1, 1]), out=torch.empty_like(q), out_lse=torch.empty((2, 1, 8), device="cuda"),
                workspace=torch.empty(need, dtype=torch.uint8, device="cuda"), err_count=i32([0]))
    pkg.paged_attention(**a, **more)
    for name in (*a, *more):
        kw = {**a, **more}
        kw[name] = kw[name].cpu()
        with pytest.raises(ValueError):
            pkg.paged_attention(**kw)
    for err in (torch.zeros(1, device="cuda"), i32([]), i32([0]).long()):
        with pytest.raises(ValueError):
            pkg.paged_attention(**a, err_count=err)
    del a["q"]
    a |= dict(k=q[:, :, :2], v=q[:, :, 2:4], new_lens=i32([1, 1]), err_count=i32([0]))
    pkg.kv_append(**a)
    for name in a:
        with pytest.raises(ValueError):
            pkg.kv_append(**{**a, name: a[name].cpu()})


@pytest.mark.gpu
def test_verification_refuses_host_tensors(lib):
    B, n = 2, 1
    a = dict(logits=torch.zeros((B * (n + 1), pkg.VOCAB_PADDED), dtype=torch.bfloat16, device="cuda"), draft_token=i32([[1], [2]]),
             draft_logits=torch.zeros((B * n, pkg.VOCAB_PADDED), dtype=torch.bfloat16, device="cuda"),
             accept_uniform=i32([[5], [6]]), draw_uniform=i32([7, 8]), num_drafts=i32([1, 1]))
    for name in ("temperature", "top_p", "draft_temperature", "draft_top_p"):
        a[name] = torch.ones(B, device="cuda")
    for name in ("top_k", "draft_top_k"):
        a[name] = i32([20, 20])
    a |= dict(out_token=i32([[0, 0], [0, 0]]), out_accepted=i32([0, 0]), out_restr=torch.empty((B, n + 1), device="cuda"),
              out_full=torch.empty((B, n + 1), device="cuda"), err_count=i32([0]),
              workspace=torch.empty(pkg.verify_workspace_bytes(B, n), dtype=torch.uint8, device="cuda"))
    pkg.verify_drafts(**a)
    for name in a:
        with pytest.raises(ValueError):
            pkg.verify_drafts(**{**a, name: a[name].cpu()})
