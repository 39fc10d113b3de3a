"""kamera_attention_mass: blocks of many units, one after another."""
import pytest
import torch

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
