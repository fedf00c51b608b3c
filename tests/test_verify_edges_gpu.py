"""GPU: verification of many drafts a sequence.  Inputs, comparison and tolerances as in
test_verify_gpu.py."""

import pytest
import torch

import oracle
import rollout_consistent_vocab_gb300 as pkg
from test_verify_gpu import DEV, compare, make, run

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _library():
    from rollout_consistent_vocab_gb300.build import build_library
    build_library()
    pkg.load_library()


@pytest.mark.parametrize("draft", [True, False])
def test_more_drafts_than_a_warp_has_lanes(draft):
    """The first refusal among the first 32, the next 32 and the last ones, and none."""
    stops, n = (31, 32, 65, None), 66
    c = make(len(stops), n, seed=50, noise=0.0)
    rows = c["x"].reshape(len(stops), n + 1, -1)
    c["a"].zero_()                                             # accept whatever has any probability
    c["d"] = rows[:, :n, :oracle.VREAL].float().argmax(-1).to(torch.int32)
    for b, i in enumerate(stops):
        if i is not None:                                      # a draft without any
            c["d"][b, i] = int(rows[b, i, :oracle.VREAL].float().argmin())
    got = run(c, 0.8, 1.0, 50, draft)
    assert got[1].tolist() == [n if i is None else i for i in stops]
    compare(c, got, 0.8, 1.0, 50, draft)
    num = [32, 10, 64, 65]
    got = run(c, 0.8, 1.0, 50, draft, num_drafts=torch.tensor(num, dtype=torch.int32, device=DEV))
    assert got[1].tolist() == [m if i is None else min(i, m) for i, m in zip(stops, num)]
    token = got[0].cpu()
    for b, a in enumerate(got[1].tolist()):
        assert token[b, :a].tolist() == c["d"][b, :a].tolist() and token[b, a] >= 0 and torch.all(token[b, a + 1:] == -1)
