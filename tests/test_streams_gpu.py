"""GPU: calls on a stream that is not the current one, with scratch and outputs of their own.

What a call allocates for itself may be neither memory that earlier work of the current
stream still uses, nor memory that its later work gets while the call runs.  A wait of some
ten milliseconds on one of the streams makes the order certain.
"""

import pytest
import torch

import rollout_consistent_vocab_gb300 as pkg
import test_paged_gpu
import test_verify_gpu

pytestmark = pytest.mark.gpu
DEV = "cuda"
WAIT = 60_000_000                        # clock cycles


@pytest.fixture(scope="module", autouse=True)
def _library():
    from rollout_consistent_vocab_gb300.build import build_library
    build_library()
    pkg.load_library()


def attention():
    c = test_paged_gpu.make([5000, 1200, 40], 3, 8, 2, 128, 16, "bf16", seed=40)
    return (lambda **kw: test_paged_gpu.run(c, **kw),
            pkg.paged_attention_workspace_bytes(3, 3, 8, 2, 128, 16 * c["table"].shape[1]))


def verification():
    c = test_verify_gpu.make(5, 3, seed=41)
    return lambda **kw: test_verify_gpu.run(c, 1.0, 0.95, 50, **kw), pkg.verify_workspace_bytes(5, 3)


def _logits(T=6, seed=42):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    x = 4.0 * torch.randn((T, pkg.VOCAB_PADDED), generator=g, device=DEV)
    return x.to(torch.bfloat16), torch.arange(T, dtype=torch.int32, device=DEV) * 1000


def pair():
    x, t = _logits()
    return lambda **kw: pkg.logp_pair(x, t, 0.8, 0.9, 50, **kw), 256


def backward():
    x, t = _logits()
    g = torch.linspace(-1.0, 1.0, 6, device=DEV)
    return lambda **kw: pkg.logp_backward(x, t, 0.8, 0.9, 50, grad_full=g, grad_restr=g, **kw), 256


def sampler():
    x, t = _logits()
    u = t * 12345                        # (made before the call: its stream does not wait for the current one)
    return lambda **kw: pkg.sample(x, 0.8, 0.9, 50, uniform=u, **kw), pkg._binding.sample_workspace_bytes(6)


def _head(H=128):
    g = torch.Generator(device=DEV)
    g.manual_seed(43)
    w, h = (0.3 * torch.randn((n, H), generator=g, device=DEV) for n in (pkg.VOCAB_PADDED, 6))
    return h.to(torch.bfloat16), w.to(torch.bfloat16), torch.arange(6, dtype=torch.int32, device=DEV) * 1000


def head():
    h, w, t = _head()
    return lambda **kw: pkg.linear_logp(h, w, t, 0.8, **kw), pkg._binding.linear_workspace_bytes(6)


def head_pair():
    h, w, t = _head()
    return (lambda **kw: pkg.linear_logp_pair(h, w, t, 0.8, 0.9, 50, **kw),
            pkg._binding.linear_pair_workspace_bytes(6))


def sharded():
    x, t = _logits()
    shards = [x[:, r * pkg.SHARD_WIDTH:(r + 1) * pkg.SHARD_WIDTH].contiguous() for r in range(pkg.NUM_SHARDS)]
    return lambda **kw: pkg.logp_sharded(shards, t, 0.8, 0.9, 50, **kw), 8 * 6 * 1024 * 4


def norm():
    x = [torch.linspace(-2.0, 3.0, n, device=DEV) for n in (1000, 77)]
    return lambda **kw: pkg.grad_norm(x, **kw), 8 * pkg.NORM_BINS


CALLS = [attention, verification, pair, backward, sampler, head, head_pair, sharded, norm]


def outputs(got):
    return [got] if isinstance(got, torch.Tensor) else list(got)


def sizes(want, scratch):
    return [scratch] + [t.numel() * t.element_size() for t in want]


@pytest.mark.parametrize("make", CALLS)
def test_memory_given_out_while_the_call_waits(make):
    call, scratch = make()
    want = outputs(call())
    st = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(st):
        torch.cuda._sleep(WAIT)
    got = outputs(call(stream=st))
    blocks = [torch.full((n,), 77, dtype=torch.uint8, device=DEV) for n in sizes(want, scratch) for _ in range(3)]
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    assert all(bool((b == 77).all()) for b in blocks)


@pytest.mark.parametrize("make", CALLS)
def test_memory_that_the_current_stream_still_reads(make):
    call, scratch = make()
    want = outputs(call())
    st = torch.cuda.Stream()
    blocks = [torch.full((n,), 77, dtype=torch.uint8, device=DEV) for n in sizes(want, scratch) for _ in range(3)]
    torch.cuda.synchronize()
    torch.cuda._sleep(WAIT)
    copies = [b.clone() for b in blocks]
    del blocks
    got = outputs(call(stream=st))
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    assert all(bool((b == 77).all()) for b in copies)


@pytest.mark.parametrize("make", CALLS)
def test_outputs_dropped_while_the_current_stream_reads_them(make):
    call, _ = make()
    want = outputs(call())
    st = torch.cuda.Stream()
    torch.cuda.synchronize()
    got = outputs(call(stream=st))
    torch.cuda.current_stream().wait_stream(st)
    torch.cuda._sleep(WAIT)
    copies = [t.clone() for t in got]
    del got
    with torch.cuda.stream(st):
        blocks = [torch.full((t.numel() * t.element_size(),), 77, dtype=torch.uint8, device=DEV) for t in want]
    torch.cuda.synchronize()
    assert len(blocks) == len(want)
    assert all(torch.equal(a, b) for a, b in zip(copies, want))
