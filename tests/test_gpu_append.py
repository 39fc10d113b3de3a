"""kamera_append against the definition in float64.

Tolerance per element: |got - y| <= 2^-8 |y| + c 2^-24 S (1 + 2^-8). The first term is one
rounding to bf16 (at most half a step, 2^-8 of the value). S = |a| + |b| of the normed pair that
the element is turned from, the scale of the float32 evaluation, and c counts its relative errors
in units of 2^-24: half the error of the sum of squares (a lane adds up to 32 squares in turn and
a shuffle tree of five levels joins the lanes: (37 + 1) / 2 = 19), 4 for rsqrtf (2 ulps) and its
argument's division, 2 for the two products, 3 for the rotation's products and sum, and 2 pi + 4
for the phase (the angle, at most pi, is rounded once; sincospif is good to 2 ulps): c = 40.
Columns that no arithmetic touches are equal bit for bit.
"""
import dataclasses

import numpy as np
import pytest
import torch

import position_independent_multimodal_gb300 as km
import workloads as wl
from tests import kamera_testlib as tl

pytestmark = pytest.mark.gpu

C = 40 * 2.0 ** -24


@pytest.fixture(scope="module", autouse=True)
def _cuda(cuda_ok):
    return cuda_ok


def gqa(hd, hkv, page=16, **kw):
    return wl.Layout(kind=wl.GQA, num_layers=2, page_size=page, num_kv_heads=hkv, head_dim=hd,
                     rope_dim=hd, rope_theta=1e6, **kw)


def mla(lat, rope, page=16, **kw):
    return wl.Layout(kind=wl.MLA, num_layers=2, page_size=page, latent_dim=lat, rope_dim=rope,
                     rope_theta=1e4, **kw)


LAYOUTS = {
    "gqa128": (gqa(128, 4), 28),
    "gqa64-page5": (gqa(64, 2, page=5), 6),
    "gqa64-interleaved": (gqa(64, 2, rope_style=wl.INTERLEAVED), 4),
    "gqa16": (gqa(16, 1), 3),
    "gqa80-page1": (gqa(80, 3, page=1), 9),
    "gqa256": (gqa(256, 1, page=64), 5),
    "gqa48-interleaved": (gqa(48, 2, rope_style=wl.INTERLEAVED), 2),
    "mrope-blocked": (gqa(128, 2, mrope_section=(16, 24, 24)), 6),
    "mrope-interleaved": (gqa(128, 2, mrope_section=(24, 20, 20),
                              mrope_style=wl.MROPE_INTERLEAVED), 6),
    "mla": (mla(512, 64), 16),
    "mla-small-interleaved": (mla(48, 16, page=3, rope_style=wl.INTERLEAVED), 5),
    "mla-mrope": (mla(128, 32, mrope_section=(4, 6, 6)), 2),
}


def phases(lay, pos):
    """Angles [T][pairs] in float64 from exact integer products is more than these positions
    need: they stay below 2^21, so position times frequency has 2^-32 of a turn to spare."""
    n = lay.rope_dim // 2
    inv = lay.rope_theta ** (-2.0 * np.arange(n) / lay.rope_dim)
    if any(lay.mrope_section):
        t, h, w = lay.mrope_section
        i = np.arange(n)
        if lay.mrope_style == wl.MROPE_INTERLEAVED:
            axis = np.where((i % 3 == 1) & (i < 3 * h), 1, np.where((i % 3 == 2) & (i < 3 * w), 2, 0))
        else:
            axis = np.where(i < t, 0, np.where(i < t + h, 1, 2))
        return pos[:, axis] * inv
    return pos[:, None] * inv


def turned(lay, x, ang):
    """x [T][heads][rope] turned; also the scale |a| + |b| of each element."""
    n = lay.rope_dim // 2
    c, s = np.cos(ang)[:, None], np.sin(ang)[:, None]
    y, S = np.empty_like(x), np.empty_like(x)
    if lay.rope_style == wl.NEOX_HALF:
        ia, ib = np.arange(n), np.arange(n) + n
    else:
        ia, ib = 2 * np.arange(n), 2 * np.arange(n) + 1
    a, b = x[..., ia], x[..., ib]
    y[..., ia], y[..., ib] = a * c - b * s, b * c + a * s
    S[..., ia] = S[..., ib] = np.abs(a) + np.abs(b)
    return y, S


def normed(x, w, eps):
    if w is None:
        return x
    return x / np.sqrt(np.mean(x * x, -1, keepdims=True) + eps) * w


def f64(t):
    return t.detach().double().cpu().numpy()


def expected(lay, q, k, v, qw, kw, pos, eps):
    """(q', K rows, V rows) and their scales; a scale of 0 marks copied columns."""
    ang = phases(lay, pos)
    qw, kw = (None if w is None else f64(w) for w in (qw, kw))
    if lay.kind == wl.GQA:
        yq, Sq = turned(lay, normed(f64(q), qw, eps), ang)
        yk, Sk = turned(lay, normed(f64(k), kw, eps), ang)
        return (yq, Sq), (yk, Sk), f64(v)
    lat = lay.latent_dim

    def row(x, w):
        y, S = turned(lay, x[..., lat:], ang)
        c = normed(x[..., :lat], w, eps)
        return np.concatenate([c, y], -1), np.concatenate([np.abs(c) * (w is not None), S], -1)

    return row(f64(q), None), row(f64(k), kw), None


def check(got, want):
    y, S = want
    tol = np.where(S > 0, 2.0 ** -8 * np.abs(y) + C * S * (1 + 2.0 ** -8) + 2.0 ** -133, 0)
    bad = ~(np.abs(got - y) <= tol)
    assert not bad.any(), (int(bad.sum()), np.argwhere(bad)[:4], got[bad][:4], y[bad][:4])


class Run:
    def __init__(self, name, lens, seed=0, weights=True, eps=1e-6, far=100000, apart=False):
        self.lay, self.hq = lay, hq = LAYOUTS[name]
        g = torch.Generator().manual_seed(seed)
        rs = np.random.RandomState(seed)
        T, R = int(sum(lens)), len(lens)
        self.T = T
        old = rs.randint(0, 2 * lay.page_size + 1, R)
        per = int(max(-(-(o + n) // lay.page_size) for o, n in zip(old, lens))) + 1
        self.pages = R * per
        self.pt = wl.shuffled_page_table(R, per, g)
        self.req = np.repeat(np.arange(R), lens)
        self.tok = np.concatenate([np.arange(o, o + n) for o, n in zip(old, lens)] or [[]]).astype(int)
        shape = (T, 3) if any(lay.mrope_section) else (T,)
        self.pos = rs.randint(-far, far, shape)
        dk = lay.head_dim if lay.kind == wl.GQA else lay.latent_dim + lay.rope_dim
        hk = lay.num_kv_heads if lay.kind == wl.GQA else 1
        x = wl.normal_bf16((T, hq + 2 * hk, dk), 1.0, g, "cpu")
        x = (x.float() * torch.exp(torch.randn(dk, generator=g))).to(torch.bfloat16).cuda()
        if apart:  # each in memory of its own
            self.q, self.k, self.v = (y.contiguous() for y in (x[:, :hq], x[:, hq:hq + hk], x[:, hq + hk:]))
        else:
            self.q, self.k, self.v = x[:, :hq], x[:, hq:hq + hk], x[:, hq + hk:]
        w = wl.normal_bf16((2, dk), 1.0, g, "cpu").cuda()
        self.qw = self.kw = None
        if weights:
            self.kw = w[1]
            if lay.kind == wl.GQA:
                self.qw = w[0]
            else:
                self.kw = w[1][:lay.latent_dim].contiguous()
        if lay.kind == wl.MLA:
            self.v = None
        self.eps = eps
        self.h = km.create(lay)
        self.pk, self.pv = tl.sentinel_pool(lay, self.pages * lay.page_size)
        self.pool = km.Pool(self.pk, self.pv, self.pt.cuda())
        self.out = torch.full((T, hq, dk), -7.0, dtype=torch.bfloat16, device="cuda")
        self.st = torch.zeros(1, dtype=torch.int32, device="cuda")

    def dev(self):
        return (torch.as_tensor(self.pos, dtype=torch.int64).cuda(),
                torch.as_tensor(self.req, dtype=torch.int32).cuda(),
                torch.as_tensor(self.tok, dtype=torch.int32).cuda())

    def call(self, layer=1, out=None, **kw):
        pos, req, tok = self.dev()
        km.kamera_append(self.h, self.pool, layer, self.q, self.k, self.v, self.qw, self.kw, pos,
                         req, tok, self.eps, self.out if out is None else out, self.st, **kw)
        torch.cuda.synchronize()
        return int(self.st.item())

    def want(self):
        return expected(self.lay, self.q, self.k, self.v, self.qw, self.kw,
                        self.pos.astype(np.float64), self.eps)

    def slots(self):
        ps = self.lay.page_size
        return self.pt.numpy()[np.maximum(self.req, 0), self.tok // ps].astype(int) * ps + self.tok % ps

    def check(self, want, rows=None, out=None, q_rows=None, layer=1):
        rows = np.arange(self.T) if rows is None else rows
        q_rows = rows if q_rows is None else q_rows
        q, k, v = want
        out = f64(self.out if out is None else out)
        check(out[q_rows], (q[0][q_rows], q[1][q_rows]))
        sl = self.slots()[rows]
        n = len(rows)
        check(f64(self.pk[layer])[sl].reshape(n, *k[0].shape[1:]), (k[0][rows], k[1][rows]))
        if v is not None:
            assert np.array_equal(f64(self.pv[layer])[sl], v[rows].reshape(n, -1))
        left = np.ones(self.pk.shape[1], bool)
        left[sl] = False
        for p in (self.pk, self.pv):
            if p is not None:
                b = wl.bf16_bits(p)
                assert np.all(b[layer][left] == wl.POOL_SENTINEL_BITS)
                assert np.all(b[1 - layer] == wl.POOL_SENTINEL_BITS)


@pytest.mark.parametrize("weights", [True, False])
@pytest.mark.parametrize("name", sorted(LAYOUTS))
def test_ragged_batch(name, weights):
    r = Run(name, [1, 7, 40, 3], seed=len(name), weights=weights)
    assert r.call() == 0
    r.check(r.want())


@pytest.mark.parametrize("lens", [[1], [2], [1] * 5, [129], [700, 901], [3000]])
@pytest.mark.parametrize("name", ["gqa128", "mrope-blocked", "mla", "gqa80-page1"])
def test_lengths(name, lens):
    r = Run(name, lens, seed=3)
    assert r.call(layer=0) == 0
    r.check(r.want(), layer=0)


@pytest.mark.parametrize("name", ["gqa128", "mla"])
def test_separate_inputs_in_place_and_keys_alone(name):
    r = Run(name, [5, 30], seed=5, apart=True)
    want = r.want()
    q = r.q.clone()
    r.q = q
    assert r.call(out=q) == 0  # in place
    r.check(want, out=q)
    r2 = Run(name, [5, 30], seed=5)
    r2.q = r2.out = None
    pos, req, tok = r2.dev()
    km.kamera_append(r2.h, r2.pool, 1, None, r2.k, r2.v, None, r2.kw, pos, req, tok, r2.eps, None,
                     r2.st)
    assert torch.equal(r2.pk.view(torch.int16), r.pk.view(torch.int16))


@pytest.mark.parametrize("name", ["gqa64-page5", "mla"])
def test_padding_and_bad_rows(name):
    # padding rows, rows outside the table and a page outside the pool, in the midst of good ones
    r = Run(name, [6, 20, 9], seed=6)
    r.req[3] = -1
    r.req[-4:] = -5
    assert r.call() == 0
    keep = r.req >= 0
    r.check(r.want(), rows=np.flatnonzero(keep))
    assert torch.all(r.out[torch.as_tensor(~keep)] == -7)

    r = Run(name, [6, 20, 9], seed=6)
    want = r.want()
    r.req[2], r.tok[8], r.tok[9] = 3, -1, r.pt.shape[1] * r.lay.page_size
    assert r.call() == km.KAMERA_DEVICE_BAD_ITEM
    bad = np.isin(np.arange(r.T), [2, 8, 9])
    r.req[bad], r.tok[bad] = 0, 0
    r.check(want, rows=np.flatnonzero(~bad))
    assert torch.all(r.out[torch.as_tensor(bad)] == -7)

    for page in (-1, r.pages, 2 ** 31 - 1):
        r = Run(name, [6, 20, 9], seed=6)
        want = r.want()
        at = r.tok[0] // r.lay.page_size
        hit = (r.req == 0) & (r.tok // r.lay.page_size == at)
        sl = r.slots()
        r.pool.page_table[0, at] = page
        assert r.call() == km.KAMERA_DEVICE_SLOT_OOB
        r.check(want, rows=np.flatnonzero(~hit), q_rows=np.arange(r.T))
        assert np.all(wl.bf16_bits(r.pk)[1, sl[hit]] == wl.POOL_SENTINEL_BITS)


def test_far_positions_turn_exactly():
    # positions up to 2^62: the float64 angle would be lost, so the phase of each comes from
    # integers: position times the frequency's Q0.64 fraction of a turn, modulo one turn
    r = Run("gqa64-interleaved", [30], seed=8, weights=False)
    r.pos = np.random.RandomState(1).randint(-2 ** 62, 2 ** 62, 30)
    assert r.call() == 0
    d = torch.as_tensor(r.pos).cuda()
    cs = torch.empty(30, 32, 2, device="cuda")
    km.kamera_rope_phases(r.h, d, cs)
    c, s = f64(cs)[:, None, :, 0], f64(cs)[:, None, :, 1]
    x = f64(r.k)
    a, b = x[..., 0::2], x[..., 1::2]
    y = np.stack([a * c - b * s, b * c + a * s], -1).reshape(x.shape)
    S = np.repeat(np.abs(a) + np.abs(b), 2, -1)
    check(f64(r.pk[1])[r.slots()].reshape(y.shape), (y, S))


@pytest.mark.parametrize("name", ["gqa128", "mla"])
def test_zero_rows_large_values_and_non_finite(name):
    r = Run(name, [12], seed=9)
    for x in (r.q, r.k):
        x[0] = 0
        x[1] = x[1] * 2.0 ** 60     # the sum of squares passes float32
        x[2] = x[2] * 2.0 ** -60    # eps rules
    want = r.want()
    r.q[5, 0, 3], r.k[6, 0, 5], r.k[7, 0, 9] = float("nan"), float("inf"), float("nan")
    assert r.call() == 0
    rows = np.array([i for i in range(12) if i not in (5, 6, 7)])
    sl = r.slots()
    q, k, v = want
    check(f64(r.out)[rows], (q[0][rows], q[1][rows]))
    check(f64(r.pk[1])[sl[rows]].reshape(len(rows), *k[0].shape[1:]), (k[0][rows], k[1][rows]))
    # other heads of the token with the NaN are as they were; the head itself carries it
    check(f64(r.out)[5:6, 1:], (q[0][5:6, 1:], q[1][5:6, 1:]))
    assert torch.isnan(r.out[5, 0]).any() and torch.isnan(r.pk[1, sl[7]]).any()
    assert not torch.isfinite(r.pk[1, sl[6]].float()).all()


def test_other_stream_and_graph_replay():
    r = Run("gqa128", [33], seed=11)
    s = torch.cuda.Stream()
    assert r.call(stream=s) == 0
    r.check(r.want())
    pos, req, tok = r.dev()

    def once():
        km.kamera_append(r.h, r.pool, 1, r.q, r.k, r.v, r.qw, r.kw, pos, req, tok, r.eps, r.out,
                         r.st)

    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        once()
    r.q.mul_(0.5)
    r.k.neg_()
    pos.add_(17)
    r.pos += 17
    g.replay()
    torch.cuda.synchronize()
    r.check(r.want())


def test_refusals():
    r = Run("gqa128", [4])
    pos, req, tok = r.dev()

    def call(**kw):
        a = dict(q=r.q, k=r.k, v=r.v, qw=r.qw, kw=r.kw, pos=pos, req=req, tok=tok, eps=1e-6,
                 out=r.out, st=r.st, layer=0)
        a.update(kw)
        km.kamera_append(r.h, r.pool, a["layer"], a["q"], a["k"], a["v"], a["qw"], a["kw"],
                         a["pos"], a["req"], a["tok"], a["eps"], a["out"], a["st"])

    for kw in (dict(q=r.q.float()), dict(q=r.q.cpu()), dict(k=r.k[:, :2]), dict(v=None),
               dict(q=None), dict(out=None), dict(pos=pos.int()), dict(pos=pos[:2]),
               dict(req=req.long()), dict(tok=tok[:3]), dict(qw=r.qw[:64]), dict(qw=r.qw.float()),
               dict(q=r.q.transpose(1, 2).contiguous().transpose(1, 2)), dict(st=r.st.float())):
        with pytest.raises(ValueError):
            call(**kw)
    for kw in (dict(layer=2), dict(layer=-1), dict(eps=-1.0), dict(eps=float("nan"))):
        with pytest.raises(km.KameraError) as e:
            call(**kw)
        assert e.value.status == km.KAMERA_ERR_INVALID_ARG
    torch.cuda.synchronize()
    assert torch.all(r.out == -7) and int(r.st.item()) == 0
    call(q=r.q[:0], k=r.k[:0], v=r.v[:0], pos=pos[:0], req=req[:0], tok=tok[:0], out=r.out[:0])


@pytest.mark.parametrize("name", ["gqa128", "gqa48-interleaved", "mla"])
def test_norm_at_the_ends_of_the_range(name):
    # sums of squares above and below float32's range, without an eps to hide the latter
    r = Run(name, [9], seed=10, eps=0.0)
    for i, e in enumerate((-120, -90, -64, -45, 0, 50, 64, 90, 118)):
        for x in (r.q, r.k):
            x[i] = x[i] * 2.0 ** e
    want = r.want()
    assert r.call() == 0
    r.check(want)


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("name", sorted(LAYOUTS))
def test_many_tokens_with_padding_and_bad_rows(name, in_place):
    # a warp has several tokens here, among them padding, rows outside the table and slots outside
    # the pool; sums of squares beyond float32's range in some
    r = Run(name, [1900, 3, 1, 577], seed=21, apart=True)
    rs = np.random.RandomState(4)
    for i in rs.choice(r.T, 40, replace=False):
        for x in (r.q, r.k):
            x[i] = x[i] * 2.0 ** 80
    want = r.want()
    pad, bad = rs.permutation(r.T)[:200].reshape(2, -1)
    at = r.tok[1899] // r.lay.page_size
    lost = (r.req == 0) & (r.tok // r.lay.page_size == at)
    lost[np.r_[pad, bad]] = False
    sl = r.slots()
    r.pool.page_table[0, at] = r.pages + 3
    r.req[pad], r.req[bad[:50]] = -1, len(r.pt)
    r.tok[bad[50:]] = r.pt.shape[1] * r.lay.page_size
    out = r.q if in_place else r.out
    before = out.clone()
    assert r.call(out=out) == km.KAMERA_DEVICE_BAD_ITEM | km.KAMERA_DEVICE_SLOT_OOB
    skip = np.isin(np.arange(r.T), np.r_[pad, bad])
    r.req[skip], r.tok[skip] = 0, 0
    r.check(want, rows=np.flatnonzero(~skip & ~lost), q_rows=np.flatnonzero(~skip), out=out)
    skip = torch.as_tensor(skip)
    assert torch.equal(out[skip].view(torch.int16), before[skip].view(torch.int16))
    assert np.all(wl.bf16_bits(r.pk)[1, sl[lost]] == wl.POOL_SENTINEL_BITS)


def test_many_keys_alone_and_more_heads_than_fit():
    # keys alone; and 5 / 7 heads of 128, a lane group without a head in its last turn
    for hkv, hq in ((4, 28), (5, 35), (7, 7)):
        LAYOUTS["here"] = (gqa(128, hkv), hq)
        try:
            r, r2 = Run("here", [901], seed=23), Run("here", [901], seed=23)
        finally:
            del LAYOUTS["here"]
        assert r.call() == 0
        r.check(r.want())
        pos, req, tok = r2.dev()
        km.kamera_append(r2.h, r2.pool, 1, None, r2.k, r2.v, None, r2.kw, pos, req, tok, r2.eps,
                         None, r2.st)
        assert torch.equal(r2.pk.view(torch.int16), r.pk.view(torch.int16))
