"""Arguments of kamera_append that the binding refuses, or takes as they are, on the device."""
import pytest
import torch

from tests.test_gpu_append import Run

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _cuda(cuda_ok):
    return cuda_ok


@pytest.mark.parametrize("name", ["mrope-blocked", "mla-mrope"])
def test_positions_by_section_are_refused(name):
    r = Run(name, [9, 4])
    right = r.pos
    for wrong in (right.T.copy(), right.reshape(-1), right[None]):
        r.pos = wrong
        with pytest.raises(ValueError):
            r.call()
    torch.cuda.synchronize()
    assert torch.all(r.out == -7) and int(r.st.item()) == 0
    r.pos = right
    assert r.call() == 0
    r.check(r.want())
