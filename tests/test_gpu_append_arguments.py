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


@pytest.mark.parametrize("name", ["gqa128", "mla"])
def test_one_token_of_any_stride(name):
    r = Run(name, [1])
    n, dk, hq, hk = r.q.stride(0), r.q.shape[2], r.hq, r.k.shape[1]
    whole = torch.zeros(3, n + 4, dtype=torch.bfloat16, device="cuda")
    whole[0, :n] = torch.as_strided(r.q, (n,), (1,))

    def heads(first, count):
        return torch.as_strided(whole, (1, count, dk), (n + 4, dk, 1), first * dk)

    r.q, r.k = heads(0, hq), heads(hq, hk)
    if r.v is not None:
        r.v = heads(hq + hk, hk)
    assert r.q.stride(0) % 8 != 0
    assert r.call() == 0
    r.check(r.want())
