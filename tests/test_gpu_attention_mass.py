"""kamera_attention_mass against float64 sums of the softmax weights.

Bounds: a score is off by at most B = (Dk + 1) 2^-24 |scale| sum_d |q_d k_ud| (float32 accumulation
of a dot product), and the exponent log2(e) (scale s - lse) is formed from two rounded products and
a difference, each rounded by at most 2^-24 of it, and its power by 2^-22: a weight is off by at
most B + 2^-22 (2 + |scale s| + |lse|) of itself. n weights of one sign are added in float32: n 2^-24
of the sum. The decay's product and sum are two more roundings.
"""
import math

import numpy as np
import pytest
import torch

import position_independent_multimodal_gb300 as km
from tests.chunk_testlib import LAYOUTS, Chunks, i32

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _cuda(cuda_ok):
    return cuda_ok


class Masses(Chunks):
    def __init__(self, name, reqs, decay=0.0, extra=5, **kw):
        super().__init__(name, reqs, **kw)
        self.decay = decay
        R = len(reqs)
        g = torch.Generator().manual_seed(99)
        self.lse_in = torch.full((self.rows, self.hq), math.nan)
        self.scores = []
        for r in range(R):
            if self.new[r]:
                x, b, _ = self.exact(r)
                self.scores.append((x, b))
                self.lse_in[int(self.start[r]):int(self.start[r + 1])] = \
                    torch.logsumexp(x, -1).float().cpu()
            else:
                self.scores.append(None)
        width = int(self.ctx.max()) + extra
        fill = torch.rand(R, width, generator=g)
        self.before = torch.full_like(fill, math.nan) if decay == 0 else fill
        self.mass = self.before.cuda()
        w = km.kamera_attention_mass_workspace(self.h, self.rows, R, self.hq)
        self.ws = torch.full((w,), 0xFF, dtype=torch.uint8, device="cuda")

    def call(self, **kw):
        km.kamera_attention_mass(self.h, self.pool, self.layer, self.q, self.d_start, self.d_ctx,
                                 self.scale, self.lse_in.cuda(), self.decay, self.mass, self.ws,
                                 self.st, window=self.window, **kw)


def check(b, skip=(), status=0):
    assert int(b.st.item()) == status
    got = b.mass.cpu()
    for r in range(len(b.new)):
        c, n = int(b.ctx[r]), int(b.new[r])
        if n == 0 or r in skip:
            assert torch.equal(got[r].nan_to_num(-1), b.before[r].nan_to_num(-1))
            continue
        assert torch.equal(got[r, c:].nan_to_num(-1), b.before[r, c:].nan_to_num(-1))
        x, bound = b.scores[r]
        lse = b.lse_in[int(b.start[r]):int(b.start[r + 1])].cuda().double()[..., None]
        w = torch.where(lse == -math.inf, 0.0, torch.exp(x - torch.where(lse == -math.inf, 0.0, lse)))
        off = bound[..., None] + 2.0 ** -22 * (2 + torch.where(x == -math.inf, 0.0, x.abs()) + lse.abs())
        total = w.sum((0, 1)).cpu()
        tol = torch.where(w > 0, w * off, 0.0).sum((0, 1)).cpu() + total * (n * b.hq * 2.0 ** -24)
        if b.decay:
            old = float(np.float32(b.decay)) * b.before[r, :c].double()
            total = total + old
            tol = tol + 2.0 ** -23 * total
        err = (got[r, :c].double() - total).abs()
        assert bool((err <= tol + 1e-30).all()), (r, float((err / (tol + 1e-30)).max()))


CASES = [(1, 0), (0, 5), (1, 200), (37, 91), (130, 0), (5, 128), (1, 127)]


@pytest.mark.parametrize("name", sorted(LAYOUTS))
def test_layouts(name):
    check(Masses(name, CASES, seed=1).run())


@pytest.mark.parametrize("name", ["gqa128-group7", "mha64-page5", "mla-16-heads", "gqa80"])
@pytest.mark.parametrize("reqs", [[(1, 0)], [(1, 5000)], [(700, 0)], [(3, 0), (1, 1)], [(257, 1300)],
                                  [(1, 255)] * 40, [(0, 0), (2, 126), (0, 3), (129, 127)]])
def test_lengths(name, reqs):
    check(Masses(name, reqs, seed=2).run())


@pytest.mark.parametrize("name", ["gqa128-group7", "gqa64-group3", "mha128-page1", "mla-16-heads",
                                  "gqa80"])
@pytest.mark.parametrize("window", [1, 2, 100, 256, 257, 1000, 2 ** 31 - 1])
@pytest.mark.parametrize("decay", [0.0, 1.0, 0.75])
def test_windows_and_decay(name, window, decay):
    check(Masses(name, [(300, 400), (1, 500), (40, 0), (1, 0), (3, 1100)], window=window,
                 decay=decay, seed=3).run())


@pytest.mark.parametrize("name", ["gqa128-group7", "gqa64-group3", "mla-16-heads", "gqa80"])
def test_pages_outside_the_pool(name):
    b = Masses(name, [(70, 300), (2, 40)], seed=4, decay=0.5)
    b.table[0, 3] = b.k.shape[1] // b.lay.page_size
    b.table[0, 7] = -1
    ps = b.lay.page_size
    x, bound = b.scores[0]
    for p in (3, 7):
        x[..., p * ps:(p + 1) * ps] = -math.inf
    check(b.run(), status=km.KAMERA_DEVICE_SLOT_OOB)


@pytest.mark.parametrize("name", ["gqa128-group7", "gqa64-group3", "mla-16-heads", "gqa80"])
def test_tokens_before_the_window_may_be_released(name):
    b = Masses(name, [(3, 700)], window=100, seed=5)
    b.table[0, :(700 - 99) // b.lay.page_size] = -1
    check(b.run())


@pytest.mark.parametrize("name", ["gqa128-group7", "gqa64-group3", "mla-16-heads", "gqa80"])
def test_what_is_not_seen_lays_nothing(name):
    b = Masses(name, [(150, 400), (1, 30)], seed=6)
    # rows that saw nothing, and a key and a query that are not finite: the last token's key is seen
    # by that token alone
    b.lse_in[3:6] = -math.inf
    last = int(b.slots(0)[-1])
    b.k[:, last] = math.nan
    b.run()
    assert bool(torch.isnan(b.mass[0, 549]))
    b.mass[0, 549] = b.scores[0][0][-1, :, 549].sub(b.lse_in[149].cuda().double()).exp().sum()
    check(b)
    b.q_full[149] = math.nan  # its query reaches all tokens that it sees, the other request's none
    b.run()
    assert bool(torch.isnan(b.mass[0, :550]).all()) and bool(torch.isfinite(b.mass[1, :31]).all())


@pytest.mark.parametrize("name", ["gqa128-group7", "mla-16-heads", "gqa80"])
def test_requests_that_are_refused(name):
    b = Masses(name, [(5, 20), (6, 30), (4, 0)], seed=7, extra=0).dev()
    bad = b.ctx.copy()
    bad[0], bad[1] = 4, 37  # (more than the masses' columns)
    b.d_ctx = i32(bad)
    b.call()
    check(b, skip=(0, 1), status=km.KAMERA_DEVICE_BAD_ITEM)


@pytest.mark.parametrize("start", [[0, 5, 4, 15], [-1, 5, 11, 15], [0, 5, 11, 19]])
def test_calls_that_are_refused(start):
    b = Masses("gqa128-group7", [(5, 20), (6, 30), (4, 0)], seed=8, window=9, decay=0.5).dev()
    b.d_start = i32(start)
    b.call()
    check(b, skip=(0, 1, 2), status=km.KAMERA_DEVICE_BAD_ITEM)


@pytest.mark.parametrize("name", ["gqa128-group7", "mla-16-heads", "gqa80"])
def test_same_call_same_bytes(name):
    b = Masses(name, [(150, 700), (1, 3000), (1, 5)], seed=9).run()
    want = b.mass.clone()
    b.ws.fill_(0x7F)
    for _ in range(3):
        b.call()
        assert torch.equal(b.mass.nan_to_num(-1), want.nan_to_num(-1))


def test_many_requests():
    rs = np.random.RandomState(10)
    check(Masses("gqa64-group3", [(int(rs.randint(0, 3)), int(rs.randint(0, 60)))
                                  for _ in range(1200)], seed=10).run())
