"""The serving calls of the C ABI on the host (no GPU needed): struct sizes, and arguments that are
refused before anything is launched. Addresses are made up: no call gets as far as to use one."""
import ctypes
import math

import pytest

import position_independent_multimodal_gb300 as km
from position_independent_multimodal_gb300 import _binding as kb
from position_independent_multimodal_gb300 import build as kbuild
import workloads as wl

A = 1 << 20  # an address, aligned to all that is asked for
BIG = 1 << 40


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


def pool(**kw):
    p = dict(k=A, v=A, num_slots=160, page_table=A, num_reqs=4, pt_stride=5)
    p.update(kw)
    return kb.kamera_pool(p["k"], p["v"], p["num_slots"], p["page_table"], p["num_reqs"],
                          p["pt_stride"])


BAD_POOLS = [dict(k=None), dict(v=None), dict(k=A + 8), dict(num_slots=0), dict(num_slots=165),
             dict(page_table=None), dict(page_table=A + 2), dict(num_reqs=0), dict(pt_stride=0)]


def test_struct_sizes():
    assert ctypes.sizeof(kb.kamera_new_tokens) == 120


def tokens(**kw):
    t = dict(q=A, k=A, v=A, q_weight=A, k_weight=A, positions=A, req=A, tok=A, q_out=2 * A,
             q_stride=512, k_stride=128, v_stride=128, q_out_stride=512, num_tokens=9,
             num_q_heads=8, eps=1e-6, reserved=0)
    t.update(kw)
    return kb.kamera_new_tokens(*t.values())


def append(lib, h, p=None, t=None, layer=0, status=A):
    return lib.kamera_append(h.ptr, ctypes.byref(p or pool()), layer, ctypes.byref(t or tokens()),
                             status, None)


BAD_TOKENS = [dict(num_tokens=-1), dict(num_q_heads=-1), dict(reserved=1), dict(eps=-1e-9),
              dict(eps=math.nan), dict(eps=math.inf), dict(k=None), dict(k=A + 2), dict(v=None),
              dict(v=A + 8), dict(q=None), dict(q=A + 4), dict(q_out=None), dict(q_out=A + 2),
              dict(q_stride=504), dict(q_stride=516), dict(k_stride=120), dict(k_stride=132),
              dict(v_stride=0), dict(v_stride=-128), dict(q_out_stride=511), dict(q_weight=A + 2),
              dict(k_weight=A + 4), dict(positions=None), dict(positions=A + 4), dict(req=None),
              dict(req=A + 2), dict(tok=None), dict(tok=A + 1),
              dict(q_out=A, q_out_stride=520)]


@pytest.mark.parametrize("kw", BAD_TOKENS)
def test_append_refuses(lib, gqa, kw):
    assert append(lib, gqa, t=tokens(**kw)) == km.KAMERA_ERR_INVALID_ARG


def test_append_refuses_more(lib, gqa, mla):
    bad = km.KAMERA_ERR_INVALID_ARG
    for kw in BAD_POOLS:
        assert append(lib, gqa, p=pool(**kw)) == bad
    for layer in (-1, 2):
        assert append(lib, gqa, layer=layer) == bad
    assert append(lib, gqa, status=None) == bad
    assert append(lib, gqa, t=tokens(num_q_heads=257, q_stride=BIG, q_out_stride=BIG)) == \
        km.KAMERA_ERR_UNSUPPORTED
    assert append(lib, gqa, t=tokens(num_tokens=0)) == km.KAMERA_OK
    # MLA: no V, no norm of the queries
    wide = dict(q_stride=8 * 576, q_out_stride=8 * 576, k_stride=576)
    p = pool(v=None)
    assert append(lib, mla, p=p, t=tokens(**wide)) == bad
    assert append(lib, mla, p=p, t=tokens(v=None, **wide)) == bad
    assert append(lib, mla, p=p, t=tokens(v=None, q_weight=None, **dict(wide, k_stride=512))) == bad
    assert append(lib, mla, p=p, t=tokens(v=None, num_tokens=0)) == km.KAMERA_OK


def test_page_calls_refuse(lib, gqa):
    bad, none = km.KAMERA_ERR_INVALID_ARG, km.KAMERA_ERR_UNSUPPORTED
    need = lib.kamera_page_workspace(gqa.ptr, 160, 3)
    assert need > 0 and lib.kamera_page_workspace(gqa.ptr, -16, 3) == 0
    assert lib.kamera_page_workspace(gqa.ptr, 160, -1) == 0
    assert lib.kamera_page_workspace(None, 160, 3) == 0

    def planned(f, p=None, items=A, n=3, refs=A, ws=A, size=need, status=A):
        return f(gqa.ptr, ctypes.byref(p or pool()), items, n, refs, ws, size, status, None)

    for f in (lib.kamera_fork, lib.kamera_extend):
        for kw in (dict(items=None), dict(items=A + 2), dict(n=-1), dict(refs=None),
                   dict(refs=A + 1), dict(ws=None), dict(ws=A + 8), dict(size=need - 1),
                   dict(status=None)):
            assert planned(f, **kw) == bad, kw
        for kw in BAD_POOLS:
            assert planned(f, p=pool(**kw)) == bad, kw
        assert planned(f, n=65536, size=BIG) == none
        assert planned(f, items=None, n=0) == km.KAMERA_OK
        assert f(None, ctypes.byref(pool()), A, 3, A, A, need, A, None) == bad

    def free(p=None, items=A, n=3, refs=A, status=A):
        return lib.kamera_free(gqa.ptr, ctypes.byref(p or pool()), items, n, refs, status, None)

    for kw in (dict(items=None), dict(items=A + 2), dict(n=-1), dict(refs=None), dict(status=None)):
        assert free(**kw) == bad, kw
    assert free(n=65536) == none and free(n=0) == km.KAMERA_OK

    def compact(p=None, refs=A, live=A, ws=A, size=need, status=A):
        return lib.kamera_compact(gqa.ptr, ctypes.byref(p or pool()), refs, live, ws, size, status,
                                  None)

    for kw in (dict(refs=None), dict(live=None), dict(live=A + 2), dict(ws=None), dict(ws=A + 4),
               dict(size=8), dict(status=None)):
        assert compact(**kw) == bad, kw

    def copy(p=None, src=A, dst=A, n=3, status=A):
        return lib.kamera_copy_pages(gqa.ptr, ctypes.byref(p or pool()), src, dst, n, status, None)

    for kw in (dict(src=None), dict(dst=None), dict(src=A + 2), dict(dst=A + 1), dict(n=-1),
               dict(status=None)):
        assert copy(**kw) == bad, kw
    assert copy(n=65536) == none and copy(n=0) == km.KAMERA_OK


def test_prefix_attention_refuses(lib, gqa):
    bad, none = km.KAMERA_ERR_INVALID_ARG, km.KAMERA_ERR_UNSUPPORTED
    need = lib.kamera_prefix_attention_workspace(gqa.ptr, 4, 8)
    assert need > 0
    assert lib.kamera_prefix_attention_workspace(None, 4, 8) == 0
    assert lib.kamera_prefix_attention_workspace(gqa.ptr, -1, 8) == 0

    def call(p=None, layer=0, q=A, reqs=4, heads=8, start=A, prefix=A, groups=2, ctx=A, scale=0.1,
             out=A, lse=A, ws=A, size=need, status=A):
        return lib.kamera_prefix_attention(gqa.ptr, ctypes.byref(p or pool()), layer, q, reqs, heads,
                                           start, prefix, groups, ctx, scale, out, lse, ws, size,
                                           status, None)

    for kw in (dict(layer=-1), dict(layer=2), dict(q=None), dict(q=A + 8), dict(reqs=-1),
               dict(reqs=5), dict(heads=0), dict(heads=7), dict(start=None), dict(start=A + 2),
               dict(prefix=None), dict(groups=0), dict(groups=5), dict(ctx=None),
               dict(scale=math.nan), dict(scale=math.inf), dict(out=None), dict(out=A + 8),
               dict(lse=None), dict(lse=A + 2), dict(ws=None), dict(ws=A + 8), dict(size=need - 1),
               dict(status=None)):
        assert call(**kw) == bad, kw
    for kw in BAD_POOLS:
        assert call(p=pool(**kw)) == bad, kw
    assert call(heads=258) == none
    assert call(reqs=65536, p=pool(num_reqs=70000), size=BIG) == none
    assert call(reqs=0) == km.KAMERA_OK
