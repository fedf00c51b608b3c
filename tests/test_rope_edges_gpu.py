"""GPU: the rotation of heads at the edges of its arguments' formats.

Float64 results and tolerances as in test_rope_gpu.py.
"""

import pytest
import torch

import rollout_consistent_vocab_gb300 as pkg
from test_rope_gpu import DEV, compare, freq_of, places, rand

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _library():
    from rollout_consistent_vocab_gb300.build import build_library
    build_library()
    pkg.load_library()


def test_small_negative_frequencies_at_far_positions():
    pos = torch.tensor([[0, 1, -1, 131071, 2**24 + 1, -(2**24) - 1, 2**31 - 1, -2**31]], dtype=torch.int32, device=DEV)
    x = rand((1, 8, 3, 64), "f32", 21)
    for first, last in ((-1.0, -3.0), (-3.0, -6.0), (-6.0, -12.0)):
        freq = -torch.logspace(first, last, 32, dtype=torch.float64)
        compare(pkg.rope(x, freq, pos), x, freq, pos, "f32")
        compare(pkg.rope(x, freq, pos, inverse=True), x, freq, pos, "f32", inverse=True)


@pytest.mark.parametrize("kept", ["graph", "node"])
def test_a_gradient_captured_beside_what_another_stream_made(kept):
    """A stream other than the default one joins the capture for the sum of the leaf's gradient: nothing to refuse,
    whether a graph of the leaf lives or a wrapper keeps its accumulation node."""
    x, freq, pos = rand((2, 5, 3, 64), "f32", 22).requires_grad_(), freq_of(64), places((2, 5), 23)
    w = rand((2, 5, 3, 64), "f32", 24)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        old = pkg.rope_autograd(x, freq, pos)
        if kept == "node":
            node = torch.autograd.graph.get_gradient_edge(x).node
            old.sum().backward()
            del old
    torch.cuda.synchronize()

    def step():
        x.grad = None
        (pkg.rope_autograd(x, freq, pos) * w).sum().backward()

    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    got = x.grad
    for seed in (25, 26):
        pos.copy_(places((2, 5), seed))
        w.copy_(rand((2, 5, 3, 64), "f32", seed))
        g.replay()
        torch.cuda.synchronize()
        compare(got, w, freq, pos, "f32", inverse=True)
    if kept == "node":
        assert node.metadata                                     # (it lived through all of this)
    else:
        assert bool(torch.isfinite(old).all())
