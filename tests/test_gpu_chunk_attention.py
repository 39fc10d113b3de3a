"""kamera_chunk_attention against float64 attention of each new token over what it sees.

Bounds, with B = max_u (Dk + 1) 2^-24 |scale| sum_d |q_d k_ud| (float32 accumulation of a dot
product) and Vm = max_u |V_u|, both over the tokens seen: a score error of B moves a softmax weight
by at most about 2 B, and an output by at most (8 B + 1e-4) Vm with the float32 sums over tiles and
parts (each adds at most n 2^-24 of the mass for n terms; 1e-4 covers the contexts here). Softmax
weights rounded to bf16 are off by at most half a step, 2^-8, and the normaliser is not rounded:
another 2^-8 Vm. The output's own rounding adds 2^-8 |o|. The log-sum-exp takes float32 weights:
4 B + 1e-5 (1 + |lse|).
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


def check(b, skip=(), status=0, only=None):
    """Every output of the call; with `only` (a mask of rows), of those rows alone."""
    assert int(b.st.item()) == status
    written = torch.zeros(b.rows, dtype=torch.bool)
    for r in range(len(b.new)):
        if b.new[r] == 0 or r in skip:
            continue
        rows = slice(int(b.start[r]), int(b.start[r + 1]))
        written[rows] = True
        x, bound, v = b.exact(r)
        n, hq, c = x.shape
        top = x.amax(-1, keepdim=True)
        top = torch.where(top == -math.inf, 0.0, top)
        p = torch.exp(x - top)
        total = p.sum(-1, keepdim=True)
        lse = (top + total.log()).squeeze(-1)
        p = torch.where(total > 0, p / total, 0.0).view(n, b.H, hq // b.H, c)
        o = torch.einsum("nhgc,hcd->nhgd", p, v).flatten(1, 2)
        vm = v.abs().amax((1, 2)).repeat_interleave(hq // b.H)
        got, z = b.out[rows].double(), b.lse[rows].double()
        good = ((8 * bound + 1e-4 + 2.0 ** -8) * vm)[..., None] + 2.0 ** -8 * o.abs() - (got - o).abs()
        fin = torch.isfinite(lse)
        same = torch.where(fin, (z - lse).abs() <= 4 * bound + 1e-5 * (1 + lse.abs()), z == lse)
        if only is not None:
            good, same = good[only[rows]], same[only[rows]]
        assert bool((good >= 0).all()), (r, float(good.min()))
        assert bool(same.all()), r
    assert bool((b.out[~written] == -7).all()) and bool((b.lse[~written] == -7).all())


@pytest.mark.parametrize("name", sorted(LAYOUTS))
def test_layouts(name):
    # decoding and starting requests, none, single tokens of a context of one, pages that end
    # inside tiles
    check(Chunks(name, [(1, 0), (0, 5), (1, 200), (37, 91), (130, 0), (5, 128), (1, 127)],
                 seed=1).run())


@pytest.mark.parametrize("name", ["gqa128-group7", "mha64-page5", "mla-16-heads", "gqa80"])
@pytest.mark.parametrize("reqs", [[(1, 0)], [(1, 5000)], [(700, 0)], [(3, 0), (1, 1)], [(257, 1300)],
                                  [(1, 31)] * 40, [(0, 0), (2, 126), (0, 3), (129, 127)]])
def test_lengths(name, reqs):
    check(Chunks(name, reqs, seed=2).run())


@pytest.mark.parametrize("name", ["gqa128-group7", "gqa64-group3", "mha128-page1", "mla-16-heads",
                                  "gqa80"])
@pytest.mark.parametrize("window", [1, 2, 100, 128, 129, 1000, 2 ** 31 - 1])
def test_windows(name, window):
    check(Chunks(name, [(300, 400), (1, 500), (40, 0), (1, 0)], window=window, seed=3).run())


@pytest.mark.parametrize("name", ["gqa128-group7", "gqa64-group3", "mla-16-heads", "gqa80"])
def test_tokens_before_the_window_may_be_released(name):
    b = Chunks(name, [(3, 700)], window=100, seed=4)
    first = (700 - 99) // b.lay.page_size  # the first page that a token sees
    b.table[0, :first] = -1
    b.run()
    assert int(b.st.item()) == 0
    check(b)


@pytest.mark.parametrize("name", ["gqa128-group7", "gqa64-group3", "mla-16-heads", "gqa80"])
def test_sharp_scores_and_rising_maxima(name):
    b = Chunks(name, [(140, 600), (1, 900)], seed=5, sharp=6.0)
    for r in range(2):  # keys grow along the context: the running maximum rises again and again
        idx = torch.as_tensor(b.slots(r))
        grow = torch.linspace(0.05, 3.0, len(idx))[None, :, None]
        b.k[:, idx] = (b.k[:, idx].float() * grow).bfloat16()
    check(b.run())


@pytest.mark.parametrize("scale", [0.0, -0.1, 3.0])
@pytest.mark.parametrize("name", ["gqa128-group7", "gqa64-group3", "mla-16-heads", "gqa80"])
def test_scales(name, scale):
    check(Chunks(name, [(50, 300), (1, 200)], seed=6, scale=scale).run())


@pytest.mark.parametrize("name", ["gqa128-group7", "gqa64-group3", "mla-16-heads", "gqa80"])
def test_query_strides(name):
    lay, hq = LAYOUTS[name]
    dk = lay.head_dim if lay.head_dim else lay.latent_dim + lay.rope_dim
    check(Chunks(name, [(20, 30), (1, 40)], seed=7, stride=hq * dk + 8, before=5, pad=9).run())


@pytest.mark.parametrize("name", ["gqa128-group7", "gqa64-group3", "mla-16-heads", "gqa80"])
def test_pages_outside_the_pool(name):
    b = Chunks(name, [(70, 300), (2, 40), (1, 15)], seed=8)
    b.table[0, 3] = b.k.shape[1] // b.lay.page_size
    b.table[0, 7] = -1
    b.table[2, 0] = 1 << 30  # all that the token sees
    check(b.run(), status=km.KAMERA_DEVICE_SLOT_OOB)
    assert bool((b.lse[int(b.start[2])] == -math.inf).all())
    assert bool((b.out[int(b.start[2])] == 0).all())


@pytest.mark.parametrize("name", ["gqa128-group7", "mha64-page5", "mla-16-heads", "gqa80"])
@pytest.mark.parametrize("value", [math.nan, math.inf, -math.inf])
def test_values_that_a_token_does_not_see(name, value):
    # the last new token and one that the window leaves behind are not finite: the tokens that do
    # not see them have their outputs
    for reqs in ([(200, 330), (9, 0)], [(1, 0), (90, 2000)]):
        b = Chunks(name, reqs, window=300, seed=9)
        r = int(np.argmax(b.new))
        bad = [int(b.ctx[r]) - 1, int(b.ctx[r]) - int(b.new[r]) - 250]
        idx = torch.as_tensor(b.slots(r)[bad])
        b.k[:, idx] = value
        if b.v is not None:
            b.v[:, idx] = value
        b.run()
        me = np.arange(b.rows) - int(b.start[r]) + int(b.ctx[r]) - int(b.new[r])
        mine = (np.arange(b.rows) >= b.start[r]) & (np.arange(b.rows) < b.start[r + 1])
        sees = np.zeros(b.rows, bool)
        for u in bad:
            sees |= mine & (me >= u) & (me - u < 300)
        assert sees.any() and not sees[mine].all()
        sees = torch.as_tensor(sees).cuda()
        if math.isnan(value):
            assert bool(torch.isnan(b.out[sees]).all()) and bool(torch.isnan(b.lse[sees]).all())
        check(b, only=~sees)


def test_requests_that_are_refused():
    b = Chunks("gqa128-group7", [(5, 20), (6, 30), (4, 0)], seed=10)
    b.dev()
    bad = b.ctx.copy()
    bad[0], bad[1] = 4, b.table.shape[1] * b.lay.page_size + 1
    b.d_ctx = i32(bad)
    b.call()
    torch.cuda.synchronize()
    check(b, skip=(0, 1), status=km.KAMERA_DEVICE_BAD_ITEM)


@pytest.mark.parametrize("start", [[0, 5, 4, 15], [-1, 5, 11, 15], [0, 5, 11, 19], [0, 20, 11, 15]])
@pytest.mark.parametrize("name", ["gqa128-group7", "gqa80"])
def test_calls_that_are_refused(name, start):
    b = Chunks(name, [(5, 20), (6, 30), (4, 0)], seed=11)
    b.dev()
    b.d_start = i32(start)
    b.call()
    torch.cuda.synchronize()
    assert int(b.st.item()) == km.KAMERA_DEVICE_BAD_ITEM
    assert bool((b.out == -7).all()) and bool((b.lse == -7).all())


@pytest.mark.parametrize("name", ["gqa128-group7", "mla-16-heads", "gqa80"])
def test_same_call_same_bytes(name):
    b = Chunks(name, [(150, 700), (1, 3000), (1, 5)], seed=12).run()
    out, lse = b.out.clone(), b.lse.clone()
    b.ws.fill_(0x7F)
    for _ in range(3):
        b.call()
        torch.cuda.synchronize()
        assert torch.equal(b.out, out) and torch.equal(b.lse, lse)


@pytest.mark.parametrize("name", ["gqa128-group7", "mla-16-heads"])
def test_captured_and_replayed(name):
    b = Chunks(name, [(30, 400), (1, 900), (1, 64)], seed=13).run()
    want = b.out.clone()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        b.call()
    b.out.fill_(-7)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(b.out, want)
    # the same graph over another batch of the same sizes
    b.d_ctx.copy_(i32([200, 31, 1]))
    b.d_start.copy_(i32([0, 25, 25, 26]))
    b.out.fill_(-7)
    b.lse.fill_(-7)
    graph.replay()
    torch.cuda.synchronize()
    b.ctx, b.new, b.start = np.array([200, 31, 1]), np.array([25, 0, 1]), np.array([0, 25, 25, 26])
    check(b)


def test_many_requests():
    rs = np.random.RandomState(14)
    reqs = [(int(rs.randint(0, 3)), int(rs.randint(0, 60))) for _ in range(1500)]
    check(Chunks("gqa64-group3", reqs, seed=14).run())
