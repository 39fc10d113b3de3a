"""kamera_evict against a sort on the host: what stays, its order, rows and masses bit for bit."""
import numpy as np
import pytest
import torch

import position_independent_multimodal_gb300 as km
import workloads as wl
from tests.chunk_testlib import LAYOUTS, gqa, i32, mla

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _cuda(cuda_ok):
    return cuda_ok


SHAPES = {
    "gqa128": gqa(128, 4, layers=3),
    "gqa64-page5": gqa(64, 5, page=5),
    "gqa16-page1": gqa(16, 1, page=1),
    "gqa80-page64": gqa(80, 2, page=64, layers=1),
    "mla": mla(512, 64, layers=3),
    "mla-narrow-page3": mla(96, 32, page=3),
    "mha128": LAYOUTS["mha128-page1"][0],
}


class Cache:
    """Requests (tokens, keep, first, last) over a pool; rows carry bits of all kinds."""

    def __init__(self, name, items, seed=0, masses="spread", kept=None, width=None, spare=2):
        self.lay = lay = SHAPES[name]
        rs = np.random.RandomState(seed)
        ps = lay.page_size
        self.items = [(r, *it) for r, it in enumerate(items)]
        tokens = np.array([it[0] for it in items])
        n = -(-tokens // ps)
        pages = int(n.sum()) + 3
        R = len(items) + spare  # rows of the table that no item names
        self.table = np.full((R, max(1, int(n.max())) + 1), -1, np.int64)
        perm, at = rs.permutation(pages), 0
        for r, k in enumerate(n):
            self.table[r, :k] = perm[at:at + k]
            at += k
        self.refs = np.zeros(pages, np.int64)
        self.refs[self.table[self.table >= 0]] = 1
        g = torch.Generator().manual_seed(seed)
        slots = pages * ps

        def bits(row):
            x = torch.randint(0, 1 << 16, (lay.num_layers, slots, row), generator=g)
            return x.to(torch.uint16).view(torch.bfloat16)

        self.k = bits(lay.row_k)
        self.v = bits(lay.row_v) if lay.kind == wl.GQA else None
        w = width or max(1, int(tokens.max())) + 3
        self.mass = torch.as_tensor({
            "spread": lambda: np.exp(2.5 * rs.randn(R, w)),
            "ties": lambda: rs.randint(0, 4, (R, w)),
            "equal": lambda: np.zeros((R, w)),
            "signed": lambda: rs.randn(R, w) * 1e-3,
            "odd": lambda: rs.choice([0.0, -0.0, np.inf, -np.inf, np.nan, 1e-45, 1.0, -1.0], (R, w)),
        }[masses](), dtype=torch.float32)
        kw = kept or max(1, max(min(k, t) for t, k, _, _ in items))
        self.kept = torch.full((len(items), kw), -9, dtype=torch.int32)
        self.h = km.create(lay)
        self.ws = torch.full((km.kamera_evict_workspace(self.h, len(items)),), 0xFF,
                             dtype=torch.uint8, device="cuda")
        self.st = torch.zeros(1, dtype=torch.int32, device="cuda")

    def dev(self):
        self.d = [None if x is None else x.cuda() for x in (self.k, self.v, self.mass, self.kept)]
        self.pool = km.Pool(self.d[0], self.d[1], i32(self.table))
        self.d_items, self.d_refs = i32(self.items), i32(self.refs)
        return self

    def call(self, **kw):
        km.kamera_evict(self.h, self.pool, self.d_items, self.d_refs, self.d[2], self.d[3], self.ws,
                        self.st, **kw)

    def run(self):
        self.dev()
        self.call()
        torch.cuda.synchronize()
        return self

    def want(self, skip=()):
        k, v, mass, kept = (None if x is None else x.clone() for x in (self.k, self.v, self.mass, self.kept))
        ps = self.lay.page_size
        for i, (r, n, keep, first, last) in enumerate(self.items):
            if i in skip:
                continue
            if keep >= n:
                kept[i, :n] = torch.arange(n, dtype=torch.int32)
                continue
            m = self.mass[r, :n].double().numpy().copy()
            rank = [(0 if first <= t < n - last else -1,  # those that are kept in any case
                     0 if np.isnan(m[t]) else 1, 0 if np.isnan(m[t]) else -m[t], t) for t in range(n)]
            to = np.sort(np.array([x[3] for x in sorted(rank)[:keep]], np.int64))
            kept[i, :keep] = torch.as_tensor(to, dtype=torch.int32)
            mass[r, :keep] = self.mass[r, to]
            mass[r, keep:n] = 0
            t = np.arange(keep)
            src = torch.as_tensor(self.table[r, to // ps] * ps + to % ps)
            dst = torch.as_tensor(self.table[r, t // ps] * ps + t % ps)
            for x in (k, v):
                if x is not None and keep:
                    x[:, dst] = x[:, src]
        return k, v, mass, kept


def same(a, b):
    if a is None:
        return b is None
    t = torch.int16 if a.dtype == torch.bfloat16 else torch.int32
    return torch.equal(a.cpu().contiguous().view(t), b.contiguous().view(t))


def check(c, skip=(), status=0):
    assert int(c.st.item()) == status
    for got, want in zip(c.d, c.want(skip)):
        assert same(got, want)


ITEMS = [(1000, 500, 4, 100), (37, 36, 0, 0), (64, 64, 3, 3), (1, 1, 0, 0), (1, 0, 0, 0), (0, 0, 0, 0),
         (0, 5, 2, 3), (200, 1, 0, 0), (200, 1, 1, 0), (200, 1, 0, 1), (131, 130, 60, 70),
         (131, 7, 3, 4), (90, 300, 5, 5), (2500, 2400, 0, 2000), (2500, 129, 16, 0)]


@pytest.mark.parametrize("name", sorted(SHAPES))
@pytest.mark.parametrize("masses", ["spread", "ties"])
def test_layouts(name, masses):
    check(Cache(name, ITEMS, seed=1, masses=masses).run())


@pytest.mark.parametrize("masses", ["equal", "signed", "odd"])
def test_masses_of_all_kinds(masses):
    check(Cache("gqa64-page5", ITEMS, seed=2, masses=masses).run())


@pytest.mark.parametrize("n,keep", [(1023, 511), (1024, 1), (1025, 1024), (33000, 16000),
                                    (70001, 69000), (70001, 10)])
@pytest.mark.parametrize("masses", ["spread", "ties"])
def test_lengths(n, keep, masses):
    check(Cache("gqa16-page1", [(n, keep, 0, 0), (n // 3, keep // 4, 0, 0)], seed=3, masses=masses).run())


def test_nothing_is_kept():
    c = Cache("gqa128", [(50, 0, 0, 0)], seed=4).run()
    check(c)
    assert bool((c.d[2][0, :50] == 0).all())


BAD = [(99, 50, 25, 0, 0), (-1, 50, 25, 0, 0), (1, -1, 0, 0, 0), (1, 50, 25, 20, 6), (1, 50, 25, -1, 0),
       (1, 50, 25, 0, -1), (1, 50, -1, 0, 0), (1, 10 ** 6, 5, 0, 0), (1, 50, 41, 0, 0),
       (1, 50, 2 ** 31 - 1, 2 ** 31 - 1, 2 ** 31 - 1)]


@pytest.mark.parametrize("item", BAD)
def test_items_that_are_refused(item):
    c = Cache("gqa128", [(60, 30, 0, 0), (50, 25, 0, 0), (40, 39, 1, 1)], seed=5, kept=40)
    c.items[1] = item
    check(c.run(), skip=(1,), status=km.KAMERA_DEVICE_BAD_ITEM)


def test_masses_narrower_than_the_tokens():
    c = Cache("gqa128", [(60, 30, 0, 0), (50, 25, 0, 0)], seed=6, width=55)
    c.mass = c.mass[:, :55].contiguous()
    assert c.mass.shape[1] == 55
    check(c.run(), skip=(0,), status=km.KAMERA_DEVICE_BAD_ITEM)


def test_pages_that_are_shared_or_outside():
    # a shared page that stays as it is, one that would be written, one outside the pool, one behind
    # the tokens
    c = Cache("gqa128", [(160, 100, 40, 0), (160, 100, 0, 0), (160, 100, 0, 0), (160, 160, 0, 0),
                         (150, 100, 0, 0)], seed=7, spare=0)
    c.mass[0, 40:60] = 1e9
    c.refs[c.table[0, 0:2]] = 2
    c.mass[1, 0] = -1  # the first token goes: all pages up to the 100th token are written
    c.refs[c.table[1, 2]] = 3
    c.table[2, 9] = -1
    c.table[3, 9] = 10 ** 6
    c.table[4, 10] = 10 ** 6
    check(c.run(), skip=(1, 2), status=km.KAMERA_DEVICE_BAD_ITEM | km.KAMERA_DEVICE_SLOT_OOB)


def test_captured_and_replayed():
    c = Cache("gqa128", [(700, 300, 4, 50), (90, 60, 0, 0)], seed=8).dev()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    c.call()  # (loads the kernels)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        c.call()
    for d, x in zip(c.d, (c.k, c.v, c.mass, c.kept)):
        d.copy_(x)
    graph.replay()
    torch.cuda.synchronize()
    check(c)
