"""GPU: the rotation of heads at the edges of its arguments' formats.

Float64 results and tolerances as in test_rope_gpu.py.
"""

import pytest
import torch

import rollout_consistent_vocab_gb300 as pkg
from test_rope_gpu import DEV, compare, rand

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
