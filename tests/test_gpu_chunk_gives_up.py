"""A tcgen05 kernel over chunks that gave up waiting: the call reports it and writes nothing. With a
limit of zero every CTA gives up before its first copy or product, so nothing is ever in flight."""
import ctypes

import pytest
import torch

import position_independent_multimodal_gb300 as km
from tests.chunk_checks import check_rows
from tests.chunk_testlib import Chunks
from tests.test_gpu_attention_mass import Masses, check

pytestmark = pytest.mark.gpu

TENSOR = ["gqa128-group7", "gqa64-group3", "mla-16-heads", "mla-130-heads-page3"]
REQS = [(1, 700), (90, 300), (0, 9), (1, 127), (300, 0)]


@pytest.fixture(scope="module", autouse=True)
def _cuda(cuda_ok):
    return cuda_ok


@pytest.fixture
def limit():
    v = ctypes.c_ulonglong.in_dll(km.lib(), "kamera_chunk_wait_ns")
    was = v.value
    assert was == 2_000_000_000
    yield v
    v.value = was


@pytest.mark.parametrize("name", TENSOR)
def test_attention_writes_nothing(limit, name):
    b = Chunks(name, REQS, seed=30).dev()
    limit.value = 0
    b.call()
    torch.cuda.synchronize()
    assert int(b.st.item()) == km.KAMERA_DEVICE_TIMEOUT
    assert bool((b.out == -7).all()) and bool((b.lse == -7).all())
    # the next call in the same workspace is not touched by it
    limit.value = 2_000_000_000
    b.st.zero_()
    b.call()
    torch.cuda.synchronize()
    check_rows(b)


def test_other_widths_have_no_such_waits(limit):
    limit.value = 0
    check_rows(Chunks("gqa80", REQS, seed=31).run())


@pytest.mark.parametrize("name", TENSOR)
@pytest.mark.parametrize("decay", [0.0, 0.5])
def test_masses_stay(limit, name, decay):
    # (no window: the tokens before one only fade, by a kernel that waits for nothing)
    b = Masses(name, REQS, seed=32, decay=decay).dev()
    limit.value = 0
    b.call()
    torch.cuda.synchronize()
    assert int(b.st.item()) == km.KAMERA_DEVICE_TIMEOUT
    assert torch.equal(b.mass.cpu().nan_to_num(-1), b.before.nan_to_num(-1))
    limit.value = 2_000_000_000
    b.st.zero_()
    b.call()
    torch.cuda.synchronize()
    check(b)


def test_masses_of_other_widths_have_no_such_waits(limit):
    limit.value = 0
    check(Masses("gqa80", REQS, seed=33).run())
