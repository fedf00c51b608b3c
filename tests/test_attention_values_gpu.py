"""GPU: what a value that is not finite makes of the rows that see it at a weight next to 0, in paged
attention and over a shared prefix: the same whether the row's token comes alone or among new ones.
"""

import math

import pytest
import torch

import rollout_consistent_vocab_gb300 as pkg
from test_prefix_gpu import DEV, DT, bits, i32

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _library():
    from rollout_consistent_vocab_gb300.build import build_library
    build_library()
    pkg.load_library()


def paged(q, k, v, table, lens):
    return pkg.paged_attention(q, k, v, table, lens, scale=1.0)


def prefix(q, k, v, table, lens):
    return pkg.prefix_attention(q, k, v, table, lens, i32([0, 1]), i32([64]), scale=1.0)


@pytest.mark.parametrize("attention", [paged, prefix])
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("bad", [math.inf, -math.inf, math.nan])
def test_a_row_has_its_bits_alone(attention, dtype, bad):
    n, length, page, dim = 40, 600, 24, 64
    table, q = torch.arange(25, dtype=torch.int32, device=DEV)[None], torch.zeros((1, n, 2, dim), dtype=DT[dtype], device=DEV)
    q[..., 0] = 1.0
    # of no weight in float32; f16: on either side of where a part of one is 0 (2^-32 of the largest), and where both are (2^-45)
    for low in (-math.inf, -400.0, -31.0, -31.5, -22.0, -22.5, -20.0):
        for at in (70, 100, 543, 545, 559, 560, 575, 585, 598, 599):
            k, v = torch.zeros((600, 1, dim), dtype=DT[dtype], device=DEV), torch.ones((600, 1, dim), dtype=DT[dtype], device=DEV)
            k[at, 0, 0], v[at, 0, ::3] = low, bad
            c = (k.view(25, page, 1, dim), v.view(25, page, 1, dim), table)
            out, lse = attention(q, *c, i32([length]))
            seen = torch.arange(length - n, length, device=DEV) >= at
            assert torch.equal(~torch.isfinite(out[0, :, :, ::3]).any(-1), seen[:, None].expand(n, 2)), (low, at)
            assert bool(torch.isfinite(out[..., 1::3]).all()) and bool(torch.isfinite(out[..., 2::3]).all())
            if low < -300.0:                                     # 0 times an infinite value
                assert bool(torch.isnan(out[0, seen][..., ::3]).all()), (low, at)
            for i in (0, 1, 17, n - 1):
                o, z = attention(q[:, :1], *c, i32([length - n + 1 + i]))
                assert torch.equal(bits(o[0, 0]), bits(out[0, i])) and torch.equal(bits(z[0, 0]), bits(lse[0, i])), (low, at, i)
