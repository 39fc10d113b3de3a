"""kamera_attention_mass: blocks of many units, one after another."""
import math

import pytest
import torch

from tests.chunk_testlib import LAYOUTS
from tests.test_gpu_attention_mass import Masses, check

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _cuda(cuda_ok):
    return cuda_ok


@pytest.mark.parametrize("name", ["gqa128-group7", "gqa64-group3", "mha64-page5", "mla-16-heads"])
@pytest.mark.parametrize("reqs", [[(700, 900)], [(1, 2500)] * 24])
def test_units_one_after_another(name, reqs):
    # log-sum-exps pass through two places, each filled again as soon as all have read it
    b = Masses(name, reqs, seed=20).run()
    check(b)
    want = b.mass.clone()
    for _ in range(30):
        b.call()
        assert torch.equal(b.mass.nan_to_num(-1), want.nan_to_num(-1))
    assert int(b.st.item()) == 0


@pytest.mark.parametrize("name", sorted(LAYOUTS))
@pytest.mark.parametrize("reqs", [[(40, 300), (1, 270)], [(300, 290)]])
@pytest.mark.parametrize("negative", [False, True])
def test_keys_that_all_scores_shut_out(name, reqs, negative):
    # keys with an infinity that makes their score minus infinity for every query head: nothing is
    # laid on their tokens, whatever the number of query rows that a tile of them has
    b = Masses(name, reqs, seed=21, scale=-0.1 if negative else None)
    heads = torch.arange(b.hq) * b.dk
    b.q_full[:, heads] = b.q_full[:, heads].abs() + 0.5
    for r in range(len(reqs)):
        for u in (3, 130, 255):
            slot = int(b.slots(r)[u])
            b.k[:, slot, torch.arange(b.H) * b.dk] = math.inf if negative else -math.inf
    for r in range(len(reqs)):
        x, bound, _ = b.exact(r)
        assert bool((x[:, :, 3] == -math.inf).all())
        b.scores[r] = (x, bound)
        b.lse_in[int(b.start[r]):int(b.start[r + 1])] = torch.logsumexp(x, -1).float().cpu()
    assert bool(torch.isfinite(b.lse_in[:int(b.start[-1])]).all())
    check(b.run())
    assert bool((b.mass[:, [3, 130, 255]] == 0).all())
