"""The serving calls refuse a page table that is a slice of columns: beside it lies what is not of
the table, and the page calls write the table."""
import numpy as np
import pytest
import torch

import position_independent_multimodal_gb300 as km
from tests.test_gpu_pages import Model, items, run_compact
from tests.test_gpu_prefix_attention import Batch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _cuda(cuda_ok):
    return cuda_ok


@pytest.mark.parametrize("cols", [slice(1, 7), slice(0, 6), slice(1, 8)])
def test_page_calls_refuse_a_slice_of_columns(cols):
    # column 0 and the last ones hold numbers of the caller's that happen to be live pages
    m = Model("gqa", 30, 3, 6)
    m.hold(0, 70)
    m.hold(1, 90)
    m.to_device()
    whole = np.tile(np.flatnonzero(m.refs)[-8:].astype(np.int32), (3, 1))
    whole[:, cols][:, :6] = m.table
    back = torch.as_tensor(whole).cuda()
    before = back.clone()
    pool = km.Pool(m.dk, m.dv, back[:, cols])
    live = torch.full((1,), -9, dtype=torch.int32, device="cuda")
    x = items([(0, 2, 40)])
    for call in (lambda: km.kamera_compact(m.h, pool, m.dr, live, m.ws(0), m.st),
                 lambda: km.kamera_fork(m.h, pool, x, m.dr, m.ws(1), m.st),
                 lambda: km.kamera_extend(m.h, pool, x, m.dr, m.ws(1), m.st),
                 lambda: km.kamera_free(m.h, pool, x, m.dr, m.st),
                 lambda: km.kamera_copy_pages(m.h, pool, x[0, :1], x[0, 1:2], m.st)):
        with pytest.raises(ValueError):
            call()
    m.check()
    assert torch.equal(back, before) and int(live.item()) == -9
    run_compact(m)  # a contiguous table of the same entries


def test_attention_refuses_a_slice_of_columns():
    b = Batch("gqa128-group7", [(40, [5, 60]), (0, [1])], seed=1)
    b.dev()
    wide = torch.zeros(3, b.stride + 2, dtype=torch.int32, device="cuda")
    wide[:, 1:-1] = b.pool.page_table
    whole = b.pool
    b.pool = km.Pool(whole.k, whole.v, wide[:, 1:-1])
    with pytest.raises(ValueError):
        b.call()
    assert torch.all(b.out == -7) and int(b.st.item()) == 0
    b.pool = km.Pool(whole.k, whole.v, wide[:, 1:-1].contiguous())
    b.call()
    torch.cuda.synchronize()
    assert int(b.st.item()) == 0
    b.check()
