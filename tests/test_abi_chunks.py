"""Chunk attention, attention masses and eviction in the C ABI on the host (no GPU needed): sizes
of workspaces, and arguments that are refused before anything is launched. Addresses are made up: no
call gets as far as to use one."""
import ctypes
import math

import pytest

import position_independent_multimodal_gb300 as km
from position_independent_multimodal_gb300 import build as kbuild
import workloads as wl
from tests.test_abi_serving import A, BAD_POOLS, BIG, pool

BAD, NONE = km.KAMERA_ERR_INVALID_ARG, km.KAMERA_ERR_UNSUPPORTED


@pytest.fixture(scope="module")
def lib():
    kbuild.build()
    return km.lib()


@pytest.fixture(scope="module")
def gqa(lib):
    return km.create(wl.Layout(kind=wl.GQA, num_layers=2, page_size=16, num_kv_heads=2, head_dim=64,
                               rope_dim=64))


@pytest.fixture(scope="module")
def mla(lib):
    return km.create(wl.Layout(kind=wl.MLA, num_layers=2, page_size=16, latent_dim=512, rope_dim=64))


@pytest.fixture(scope="module")
def wide(lib):  # keys of 1088 columns
    return km.create(wl.Layout(kind=wl.MLA, num_layers=1, page_size=16, latent_dim=1024, rope_dim=64))


BATCH = dict(layer=1, q=A, q_stride=512, num_tokens=9, num_q_heads=8, start=A, ctx=A, num_reqs=3,
             window=0, scale=0.125)
# what no call takes, whatever comes behind the batch
BAD_BATCHES = [dict(layer=-1), dict(layer=2), dict(q=None), dict(q=A + 8), dict(q_stride=504),
               dict(q_stride=516), dict(q_stride=-512), dict(num_tokens=-1), dict(num_q_heads=0),
               dict(num_q_heads=-8), dict(num_q_heads=7), dict(start=None), dict(start=A + 2),
               dict(ctx=None), dict(ctx=A + 1), dict(num_reqs=-1), dict(num_reqs=5),
               dict(window=-1), dict(scale=math.nan), dict(scale=math.inf), dict(scale=-math.inf),
               dict(status=None)]
LARGE = [dict(num_q_heads=258, q_stride=BIG), dict(num_reqs=65536), dict(q_stride=1 << 39)]


def chunk(lib, h, p=None, out=A, lse=A, ws=A, size=None, status=A, **kw):
    b = dict(BATCH, **kw)
    if size is None:
        size = lib.kamera_chunk_attention_workspace(h, 9, 3, 8)
    return lib.kamera_chunk_attention(h, ctypes.byref(p or pool()), *b.values(), out, lse, ws, size,
                                      status, None)


def mass(lib, h, p=None, lse=A, decay=1.0, to=A, stride=80, ws=A, size=None, status=A, **kw):
    b = dict(BATCH, **kw)
    if size is None:
        size = lib.kamera_attention_mass_workspace(h, 9, 3, 8)
    return lib.kamera_attention_mass(h, ctypes.byref(p or pool()), *b.values(), lse, decay, to,
                                     stride, ws, size, status, None)


@pytest.mark.parametrize("f", [chunk, mass])
@pytest.mark.parametrize("kw", BAD_BATCHES)
def test_batches_refused(lib, gqa, f, kw):
    assert f(lib, gqa.ptr, **kw) == BAD


@pytest.mark.parametrize("f", [chunk, mass])
def test_batches_refused_more(lib, gqa, mla, wide, f):
    for kw in BAD_POOLS:
        assert f(lib, gqa.ptr, p=pool(**kw)) == BAD, kw
    assert f(lib, None, size=BIG) == BAD
    for kw in LARGE:
        assert f(lib, gqa.ptr, p=pool(num_reqs=70000), **kw) == NONE, kw
    for kw in (dict(ws=None), dict(ws=A + 8), dict(size=0)):
        assert f(lib, gqa.ptr, **kw) == BAD, kw
    # MLA: any number of heads, one pool tensor, wider rows of q
    assert f(lib, mla.ptr, p=pool()) == BAD
    assert f(lib, mla.ptr, p=pool(v=None)) == BAD  # rows of 8 * 576 in a stride of 512
    assert f(lib, mla.ptr, p=pool(v=None), num_q_heads=7, num_tokens=0) == km.KAMERA_OK
    assert f(lib, wide.ptr, p=pool(v=None), layer=0, q_stride=8 * 1088) == NONE


@pytest.mark.parametrize("f", [chunk, mass])
@pytest.mark.parametrize("none", [dict(num_tokens=0), dict(num_reqs=0),
                                  dict(num_tokens=0, q=None, start=None, ctx=None, ws=None)])
def test_empty_batches(lib, gqa, f, none):
    assert f(lib, gqa.ptr, **none) == km.KAMERA_OK
    for kw in (dict(layer=2), dict(window=-1), dict(scale=math.nan), dict(num_q_heads=7)):
        assert f(lib, gqa.ptr, **none, **kw) == BAD, kw


def test_workspaces(lib, gqa, mla):
    for f in (lib.kamera_chunk_attention_workspace, lib.kamera_attention_mass_workspace):
        for h in (gqa, mla):
            need = f(h.ptr, 9, 3, 8)
            # a batch's tiles are shared out over a fixed number of workers
            assert need > 0 and f(h.ptr, 1 << 30, 65535, 256) == need
        for sizes in ((-1, 3, 8), (9, -1, 8), (9, 3, -1)):
            assert f(gqa.ptr, *sizes) == 0
        assert f(None, 9, 3, 8) == 0
    for f, g in ((chunk, lib.kamera_chunk_attention_workspace),
                 (mass, lib.kamera_attention_mass_workspace)):
        assert f(lib, gqa.ptr, size=g(gqa.ptr, 9, 3, 8) - 1) == BAD


def test_chunk_attention_refuses(lib, gqa):
    for kw in (dict(out=None), dict(out=A + 8), dict(lse=None), dict(lse=A + 2)):
        assert chunk(lib, gqa.ptr, **kw) == BAD, kw


def test_attention_mass_refuses(lib, gqa):
    for kw in (dict(lse=None), dict(lse=A + 2), dict(to=None), dict(to=A + 1), dict(stride=0),
               dict(stride=-80), dict(decay=-0.5), dict(decay=math.nan), dict(decay=math.inf)):
        assert mass(lib, gqa.ptr, **kw) == BAD, kw


def test_evict_refuses(lib, gqa, mla):
    need = lib.kamera_evict_workspace(gqa.ptr, 3)
    assert need > 0 and lib.kamera_evict_workspace(gqa.ptr, -1) == 0
    assert lib.kamera_evict_workspace(None, 3) == 0

    def evict(h=gqa.ptr, p=None, items=A, n=3, refs=A, to=A, stride=80, kept=A, kept_stride=60, ws=A,
              size=need, status=A):
        return lib.kamera_evict(h, ctypes.byref(p or pool()), items, n, refs, to, stride, kept,
                                kept_stride, ws, size, status, None)

    for kw in (dict(items=None), dict(items=A + 2), dict(n=-1), dict(refs=None), dict(refs=A + 1),
               dict(to=None), dict(to=A + 2), dict(stride=0), dict(stride=-1), dict(kept=None),
               dict(kept=A + 2), dict(kept_stride=0), dict(kept_stride=-60), dict(ws=None),
               dict(ws=A + 8), dict(size=need - 1), dict(status=None), dict(h=None)):
        assert evict(**kw) == BAD, kw
    for kw in BAD_POOLS:
        assert evict(p=pool(**kw)) == BAD, kw
    assert evict(h=mla.ptr) == BAD  # a pool of V
    assert evict(n=65536, size=BIG) == NONE
    assert evict(n=0, items=None) == km.KAMERA_OK
    assert evict(h=mla.ptr, p=pool(v=None), n=0) == km.KAMERA_OK
    assert evict(n=0, stride=0) == BAD
