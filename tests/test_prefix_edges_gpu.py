"""GPU: attention over a shared prefix where lengths cross a bound of the parts that own tokens are
cut into, and what a call that fails leaves behind.

Inputs, float64 results and tolerances as in test_prefix_gpu.py; bits are compared as bits.
"""

import pytest
import torch

import rollout_consistent_vocab_gb300 as pkg
from test_prefix_gpu import DEV, bits, compare, i32, make, run

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _library():
    from rollout_consistent_vocab_gb300.build import build_library
    build_library()
    pkg.load_library()


# own tokens that the last of five new ones takes past the end of a part, and past lengths from which on parts are longer
OWN = [258, 4099, 8194, 8193, 16387, 32770]


@pytest.mark.parametrize("dtype,dim,page", [("bf16", 128, 16), ("f16", 64, 24)])
def test_drafted_tokens_have_the_bits_of_single_ones_where_parts_grow(dtype, dim, page):
    c = make([(2, 64), (1, 700)], OWN, 5, 8, 2, dim, page, dtype, seed=41)
    out, lse = run(c)
    compare(c, out, lse, [5] * len(OWN))
    for i in range(5):
        d = dict(c, q=c["q"][:, i:i + 1], lens=c["lens"] - 4 + i)
        o, z = run(d)
        assert torch.equal(bits(o[:, 0]), bits(out[:, i])) and torch.equal(bits(z[:, 0]), bits(lse[:, i])), i
    # the first three alone, in a call with room for five
    o, z = run(dict(c, lens=c["lens"] - 2), [3] * len(OWN))
    assert torch.equal(bits(o[:, :3]), bits(out[:, :3])) and torch.equal(bits(z[:, :3]), bits(lse[:, :3]))
