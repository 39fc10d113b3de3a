"""A page-table entry whose page ends past the pool, up to the largest int32, is refused by every
call that resolves slots: the rows stay as they were and KAMERA_DEVICE_SLOT_OOB is set."""
import numpy as np
import pytest
import torch

import position_independent_multimodal_gb300 as km
import workloads as wl
from tests import kamera_testlib as tl

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _cuda(cuda_ok):
    return cuda_ok


@pytest.mark.parametrize("page", [8, 2 ** 31 - 2, 2 ** 31 - 1, -1, -2 ** 31])
@pytest.mark.parametrize("call", ["relocate", "reuse", "batch", "batch-workspace", "inplace"])
def test_page_past_the_pool(call, page):
    lay = wl.Layout(kind=wl.GQA, num_layers=2, page_size=16, num_kv_heads=2, head_dim=64,
                    rope_dim=64, rope_theta=1e4)
    w = wl.reuse_workload("ids", lay, n_chunks=1, T=32, placements=[(0, 0, 0, 5)], m=8, l0=0,
                          l1=1, seed=1, strong=True, patch_per_item=True)
    slots = 8 * lay.page_size
    pt = torch.tensor([[3, page]], dtype=torch.int32)
    k, v = tl.sentinel_pool(lay, slots)
    k[:, 48:64] = 0  # page 3: a value that a small patch changes
    h = km.create(lay)
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    pool = km.Pool(k, v, pt.cuda(), slots)
    it = tl.to_device_items(w.items)[0]
    if call == "relocate":
        km.kamera_relocate(h, pool, 0, 0, 32, 7, st)
    elif call == "reuse":
        km.kamera_reuse(h, it, pool, st)
    elif call == "inplace":
        km.kamera_patch_inplace(h, pool, 0, 0, 32, it.patch_u, it.patch_vt, 8, 0, 1, 1, st)
    else:
        if call == "batch-workspace":
            ws = torch.zeros(km.kamera_batch_workspace_bytes(h, 1), dtype=torch.uint8,
                             device="cuda")
            km.kamera_set_batch_workspace(h, ws)
        km.kamera_batch_reuse(h, km.pack_items([it]).cuda(), 1, 32, 8, pool, st)
    torch.cuda.synchronize()
    assert int(st.item()) == km.KAMERA_DEVICE_SLOT_OOB
    kb = wl.bf16_bits(k)
    outside = np.ones(slots, bool)
    outside[48:64] = False
    assert np.all(kb[:, outside] == wl.POOL_SENTINEL_BITS)
    turns = call == "relocate"  # zeros turned are zeros
    assert turns or np.any(kb[:, 48:64] != 0)
