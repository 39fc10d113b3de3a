"""The in-place patch with sign -1, many times over the same rows: the same bits each time. The
factors are negated in shared memory by the threads that copied them there; a thread that negated what
another's copy had yet to bring left a sign wrong in about one run of three of the one-token chunk."""
import dataclasses

import pytest
import torch

import position_independent_multimodal_gb300 as km
from tests import kamera_testlib as tl
from tests.test_gpu_parity import gqa_layout, mla_layout, ragged

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("kind", ["gqa", "mla"])
def test_subtracting_gives_the_same_bits_each_time(cuda_ok, kind):
    lay = gqa_layout() if kind == "gqa" else mla_layout()
    w = ragged(lay, 16, f"again{kind}")
    h = km.create(lay)
    items = tl.to_device_items(w.items)
    clean = [dataclasses.replace(it, patch_m=0, patch_l0=0, patch_l1=0, patch_u=None,
                                 patch_vt=None) for it in items]
    k0, v0, status, (_, pt) = tl.run_batch(h, lay, clean, w.page_table, w.num_slots)
    assert status == 0
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    d_items = km.pack_items(items).cuda()
    longest = max(it.num_tokens for it in items)
    first = None
    for n in range(100):
        k, v = k0.clone(), None if v0 is None else v0.clone()
        pool = km.Pool(k, v, pt, w.num_slots)
        if n % 2:
            km.kamera_batch_patch_inplace(h, d_items, len(items), longest, 16, pool, -1, st)
        else:
            for it in items:
                km.kamera_patch_inplace(h, pool, it.req, it.start_tok, it.num_tokens, it.patch_u,
                                        it.patch_vt, it.patch_m, it.patch_l0, it.patch_l1, -1, st)
        got = [x.view(torch.int16) for x in (k, v) if x is not None]
        first = first or got
        assert all(torch.equal(x, y) for x, y in zip(got, first)), n
    assert int(st.item()) == 0
