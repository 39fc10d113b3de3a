"""Plans of kamera_prefix_attention with more groups, listed prefixes and listed requests than its
kernel has threads (256) or keeps in shared memory (1024). The bounds are those of
test_gpu_prefix_attention."""
import numpy as np
import pytest
import torch

import position_independent_multimodal_gb300 as km
from tests import test_gpu_prefix_attention as base

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _cuda(cuda_ok):
    return cuda_ok


SMALL = {  # one layer; seven query heads to a KV head, so that six requests make a wide block
    "gqa128": (base.gqa(128, 1, layers=1), 7),
    "gqa64": (base.gqa(64, 2, layers=1), 14),
    "any": (base.gqa(48, 1, layers=1), 3),
    "mla": (base.mla(512, 64, layers=1), 16),
    "mla-wide": (base.mla(512, 64, layers=1), 128),
}


def run(monkeypatch, name, groups, seed):
    monkeypatch.setitem(base.LAYOUTS, name, SMALL[name])
    b = base.Batch(name, groups, seed=seed, layer=0)
    assert b.run() == 0
    R = len(b.ctx)
    rs = np.random.RandomState(seed)
    b.check(reqs=sorted({0, 1, 255, 256, 1023, 1024, R - 2, R - 1} & set(range(R)) |
                        set(rs.randint(0, R, 24).tolist())))
    # none was left out, and a request without tokens says so
    lse = b.lse.cpu()
    assert torch.all(torch.isneginf(lse).all(1) == torch.as_tensor(b.ctx == 0))
    assert torch.all(torch.isfinite(lse).all(1) == torch.as_tensor(b.ctx > 0))
    assert not torch.any(lse == -7)
    return b


@pytest.mark.parametrize("count", [1024, 1025, 1500])
@pytest.mark.parametrize("name", ["gqa128", "any", "mla"])
def test_many_thin_groups(monkeypatch, name, count):
    rs = np.random.RandomState(count)
    groups = [(int(rs.randint(0, 40)), [int(rs.randint(0, 20)) if rs.rand() < 0.9 else None
                                        for _ in range(rs.randint(1, 3))]) for _ in range(count)]
    run(monkeypatch, name, groups, seed=count)


@pytest.mark.parametrize("own", [0, 9])
@pytest.mark.parametrize("count", [256, 257, 300, 1100])
@pytest.mark.parametrize("name", ["gqa128", "gqa64"])
def test_many_wide_prefixes(monkeypatch, name, count, own):
    # of one length and of several; with thin own blocks and without
    groups = [(20 + (17 * g % 150 if own else 0), [own and (g + i) % own for i in range(6)])
              for g in range(count)]
    run(monkeypatch, name, groups, seed=count + own)


@pytest.mark.parametrize("count", [1024, 1025, 1100])
def test_many_wide_requests(monkeypatch, count):
    rs = np.random.RandomState(count)
    own = [int(x) for x in rs.randint(1, 30, count - 41)]
    run(monkeypatch, "mla-wide", [(0, own), (33, [3, None] * 20 + [1])], seed=count)


def test_groups_in_the_thousands_that_are_no_partition(monkeypatch):
    monkeypatch.setitem(base.LAYOUTS, "gqa128", SMALL["gqa128"])
    b = base.Batch("gqa128", [(3, [1])] * 1300, seed=4, layer=0)
    b.dev()
    b.args[1][1200] = 1199 - 5
    b.call()
    torch.cuda.synchronize()
    assert int(b.st.item()) == km.KAMERA_DEVICE_BAD_ITEM and torch.all(b.out == -7) and torch.all(b.lse == -7)
