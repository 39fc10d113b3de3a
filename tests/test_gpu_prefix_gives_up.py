"""A wide block's kernel that gave up waiting: the call reports it and writes no output. With a
limit of zero every CTA gives up before its first copy or product, so nothing is ever in flight."""
import ctypes

import pytest
import torch

import position_independent_multimodal_gb300 as km
from tests.test_gpu_prefix_attention import Batch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _cuda(cuda_ok):
    return cuda_ok


@pytest.fixture
def limit():
    v = ctypes.c_ulonglong.in_dll(km.lib(), "kamera_prefix_wait_ns")
    was = v.value
    assert was == 2_000_000_000
    yield v
    v.value = was


@pytest.mark.parametrize("groups", [
    [(900, [5] * 40)],                          # wide blocks alone
    [(900, [300, 0, 7] * 5), (0, [70, 900])],   # thin ones too, and requests of thin blocks alone
])
@pytest.mark.parametrize("name", ["gqa128-group7", "gqa64-group3", "mla-16-heads", "mla-128-heads"])
def test_nothing_is_written(limit, name, groups):
    b = Batch(name, groups, seed=len(groups))
    b.dev()
    limit.value = 0
    b.call()
    torch.cuda.synchronize()
    assert int(b.st.item()) == km.KAMERA_DEVICE_TIMEOUT
    assert torch.all(b.out == -7) and torch.all(b.lse == -7)
    # the next call in the same workspace is not touched by it
    limit.value = 2_000_000_000
    b.st.zero_()
    b.call()
    torch.cuda.synchronize()
    assert int(b.st.item()) == 0
    b.check(reqs=[0, 1, len(b.ctx) - 1])


def test_kernels_without_such_waits_work_on(limit):
    limit.value = 0
    for name, groups in (("gqa80", [(900, [5] * 12)]), ("gqa128-group7", [(300, [5, 9])])):
        b = Batch(name, groups, seed=3)
        assert b.run() == 0
        b.check()
