"""Page calls against a plain host model: tables, counts and rows are equal exactly."""
import numpy as np
import pytest
import torch

import position_independent_multimodal_gb300 as km
import workloads as wl

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _cuda(cuda_ok):
    return cuda_ok


LAYOUTS = {
    "gqa": wl.Layout(kind=wl.GQA, num_layers=3, page_size=16, num_kv_heads=2, head_dim=64,
                     rope_dim=64),
    "mla-page5": wl.Layout(kind=wl.MLA, num_layers=2, page_size=5, latent_dim=48, rope_dim=16),
    "page1": wl.Layout(kind=wl.GQA, num_layers=2, page_size=1, num_kv_heads=1, head_dim=16,
                       rope_dim=16),
    "page300": wl.Layout(kind=wl.GQA, num_layers=1, page_size=300, num_kv_heads=8, head_dim=128,
                         rope_dim=128),
}


class Model:
    """The definitions, one entry at a time."""

    def __init__(self, name, pages, reqs, stride, seed=0):
        self.lay = lay = LAYOUTS[name]
        self.ps = lay.page_size
        g = torch.Generator().manual_seed(seed)
        n = pages * self.ps
        self.dk = wl.normal_bf16((lay.num_layers, n, lay.row_k), 1.0, g, "cpu").cuda()
        self.dv = wl.normal_bf16((lay.num_layers, n, lay.row_v), 1.0, g, "cpu").cuda() \
            if lay.kind == wl.GQA else None
        self.table = np.full((reqs, stride), -1, np.int32)
        self.refs = np.zeros(pages, np.int32)
        self.h = km.create(lay)
        self.rs = np.random.RandomState(seed)

    def hold(self, r, tokens, scattered=True):
        free = np.flatnonzero(self.refs == 0)
        n = -(-tokens // self.ps)
        pick = self.rs.permutation(free)[:n] if scattered else free[:n]
        self.table[r, :n] = pick
        self.refs[pick] += 1

    def to_device(self):
        self.dt = torch.as_tensor(self.table).cuda()
        self.dr = torch.as_tensor(self.refs).cuda()
        self.pool = km.Pool(self.dk, self.dv, self.dt)
        self.st = torch.zeros(1, dtype=torch.int32, device="cuda")
        self.k, self.v = wl.bf16_bits(self.dk), None if self.dv is None else wl.bf16_bits(self.dv)

    def ws(self, n):
        b = km.kamera_page_workspace(self.h, self.dk.shape[1], n)
        return torch.full((b,), 0xA5, dtype=torch.uint8, device="cuda")

    def move_rows(self, src, dst, rows):
        for x in (self.k, self.v):
            if x is not None:
                x[:, dst * self.ps:dst * self.ps + rows] = x[:, src * self.ps:src * self.ps + rows]

    def free_pages(self):
        return list(np.flatnonzero(self.refs == 0))

    def fork(self, items):
        st, free = 0, self.free_pages()
        out = False
        todo = []
        for parent, child, n in items:
            R, cap = self.table.shape[0], self.table.shape[1] * self.ps
            if not (0 <= parent < R and 0 <= child < R and parent != child and 0 <= n <= cap):
                st |= km.KAMERA_DEVICE_BAD_ITEM
                continue
            full, rest = divmod(n, self.ps)
            page = None
            if rest:
                out |= not free
                if out:
                    st |= km.KAMERA_DEVICE_NO_PAGES
                    continue
                page = free.pop(0)
            todo.append((parent, child, full, rest, page))
        for parent, child, full, rest, page in todo:
            for i in range(full):
                p = self.table[parent, i]
                self.table[child, i] = p
                if 0 <= p < len(self.refs):
                    self.refs[p] += 1
                else:
                    st |= km.KAMERA_DEVICE_SLOT_OOB
            if rest:
                self.table[child, full], self.refs[page] = page, 1
                src = self.table[parent, full]
                if 0 <= src < len(self.refs):
                    self.move_rows(src, page, rest)
                else:
                    st |= km.KAMERA_DEVICE_SLOT_OOB
        return st

    def span_ok(self, r, a, b):
        return 0 <= r < self.table.shape[0] and 0 <= a <= b <= self.table.shape[1] * self.ps

    def cols(self, a, b):
        return range(-(-a // self.ps), -(-b // self.ps))

    def extend(self, items):
        st, free, used = 0, self.free_pages(), 0
        out = False
        for r, a, b in items:
            if not self.span_ok(r, a, b):
                st |= km.KAMERA_DEVICE_BAD_ITEM
                continue
            c = self.cols(a, b)
            if not len(c):
                continue
            out |= used + len(c) > len(free)
            if out:
                st |= km.KAMERA_DEVICE_NO_PAGES
                continue
            for i in c:
                self.table[r, i] = free[used]
                self.refs[free[used]] = 1
                used += 1
        return st

    def free(self, items):
        st = 0
        for r, a, b in items:
            if not self.span_ok(r, a, b):
                st |= km.KAMERA_DEVICE_BAD_ITEM
                continue
            for i in self.cols(a, b):
                p = self.table[r, i]
                self.table[r, i] = -1
                if not 0 <= p < len(self.refs):
                    st |= km.KAMERA_DEVICE_SLOT_OOB
                elif self.refs[p] <= 0:
                    st |= km.KAMERA_DEVICE_BAD_ITEM
                else:
                    self.refs[p] -= 1
        return st

    def compact(self):
        live = np.flatnonzero(self.refs > 0)
        n = len(live)
        to = {int(s): int(d) for s, d in zip(live[live >= n], np.flatnonzero(self.refs[:n] == 0))}
        for s, d in to.items():
            self.move_rows(s, d, self.ps)
            self.refs[d], self.refs[s] = self.refs[s], 0
        for e in np.ndindex(self.table.shape):
            self.table[e] = to.get(int(self.table[e]), self.table[e])
        return n

    def check(self, st=0):
        torch.cuda.synchronize()
        assert int(self.st.item()) == st
        assert np.array_equal(self.dt.cpu().numpy(), self.table)
        assert np.array_equal(self.dr.cpu().numpy(), self.refs)
        assert np.array_equal(wl.bf16_bits(self.dk), self.k)
        if self.dv is not None:
            assert np.array_equal(wl.bf16_bits(self.dv), self.v)
        self.st.zero_()


def items(x):
    return torch.as_tensor(np.array(x, np.int64).reshape(-1, 3), dtype=torch.int32).cuda()


def run_fork(m, x, **kw):
    km.kamera_fork(m.h, m.pool, items(x), m.dr, m.ws(len(x)), m.st, **kw)
    m.check(m.fork(x))


def run_extend(m, x, **kw):
    km.kamera_extend(m.h, m.pool, items(x), m.dr, m.ws(len(x)), m.st, **kw)
    m.check(m.extend(x))


def run_free(m, x, **kw):
    km.kamera_free(m.h, m.pool, items(x), m.dr, m.st, **kw)
    m.check(m.free(x))


def run_compact(m, **kw):
    live = torch.full((1,), -9, dtype=torch.int32, device="cuda")
    km.kamera_compact(m.h, m.pool, m.dr, live, m.ws(0), m.st, **kw)
    n = m.compact()
    m.check()
    assert int(live.item()) == n


@pytest.mark.parametrize("name", sorted(LAYOUTS))
def test_life_of_a_pool(name):
    # parents of every kind of length, forks, growth, release of some, compaction, and again
    m = Model(name, 97, 14, 9, seed=2)
    ps = m.ps
    for r, n in enumerate([1, ps, ps + 1, 4 * ps - 1]):
        m.hold(r, n)
    m.to_device()
    run_fork(m, [(0, 4, 1), (1, 5, ps), (2, 6, ps + 1), (3, 7, 4 * ps - 1), (3, 8, 3 * ps - 1),
                 (3, 9, 0), (2, 10, 1)])
    run_extend(m, [(4, 1, ps + 3), (5, ps, ps), (7, 4 * ps - 1, 7 * ps), (9, 0, 2 * ps + 1)])
    run_free(m, [(3, 0, 4 * ps - 1), (6, 1, ps + 1), (9, ps + 1, 2 * ps + 1)])
    run_compact(m)
    run_compact(m)  # nothing left to move
    run_fork(m, [(7, 11, 5 * ps - 1), (7, 12, 7 * ps)])
    run_free(m, [(7, 0, 7 * ps), (0, 0, 1), (1, 0, ps)])
    run_compact(m)


@pytest.mark.parametrize("pages", [1, 3, 1023, 1024, 1025, 5000])
def test_sizes_of_the_pool(pages):
    m = Model("page1", pages, 6, 2100, seed=pages)
    rs = np.random.RandomState(pages)
    for r in range(3):
        m.hold(r, min(2000, pages // 4))
    m.to_device()
    n = min(2000, pages // 5)
    run_extend(m, [(3, 0, n), (4, 0, n // 2)])
    run_free(m, [(1, 0, min(2000, pages // 4)), (3, n // 3, n)])
    run_compact(m)


@pytest.mark.parametrize("full", ["none", "all", "low", "high"])
def test_compaction_at_the_ends(full):
    m = Model("gqa", 40, 3, 40)
    if full == "all":
        m.hold(0, 40 * 16)
    elif full != "none":
        m.table[0, :20] = np.arange(20) + (20 if full == "high" else 0)
        m.refs[m.table[0, :20]] = 1
    m.to_device()
    run_compact(m)


def test_stale_entries_do_not_move():
    # an entry that names a page which nothing holds, or none at all, stays as it is
    m = Model("gqa", 30, 2, 8)
    m.table[0, :3] = [29, 4, 11]
    m.refs[[29, 4, 11]] = 1
    m.table[1] = [28, 30, 2 ** 31 - 1, -2 ** 31, -1, 29, 3, 0]
    m.refs[29] += 1
    m.to_device()
    run_compact(m)


def test_pages_run_out():
    m = Model("gqa", 12, 8, 6)
    m.hold(0, 16 * 4 + 5)
    m.hold(1, 16 * 3)
    m.to_device()  # 4 pages are free
    run_extend(m, [(2, 0, 40), (3, 0, 33), (4, 0, 1), (5, 7, 9)])
    run_fork(m, [(0, 4, 64), (0, 5, 65), (0, 6, 33), (0, 7, 48)])
    run_free(m, [(2, 0, 40)])
    run_fork(m, [(0, 2, 50)])


def test_bad_items_are_left_out():
    m = Model("gqa", 20, 5, 4)
    m.hold(0, 50)
    m.hold(1, 20)
    m.to_device()
    big = 2 ** 31 - 1
    run_fork(m, [(0, 0, 20), (-1, 2, 5), (0, 5, 5), (big, 2, 5), (0, big, 5), (0, 3, 65),
                 (0, 3, -1), (0, 3, big), (0, 2, 20)])
    run_extend(m, [(3, 5, 4), (3, -1, 4), (5, 0, 4), (-1, 0, 4), (3, 0, 65), (3, 0, big),
                   (4, 0, 17)])
    run_free(m, [(0, 9, 8), (7, 0, 8), (0, 0, big), (1, 0, 20)])
    run_free(m, [(1, 0, 20)])  # released already: the entries are -1
    m.table[3, 0], m.table[3, 1] = 19, 3
    m.refs[19] = 0
    m.to_device()
    m.check()
    run_free(m, [(3, 0, 16)])  # a page that nothing held
    m.table[0, 1], m.table[0, 2] = 20, -7
    m.to_device()
    run_fork(m, [(0, 4, 40)])  # a parent with pages outside the pool


def test_an_entry_named_twice_is_released_once():
    m = Model("gqa", 20, 3, 8)
    m.hold(0, 100)
    m.to_device()
    run_fork(m, [(0, 1, 96)])
    km.kamera_free(m.h, m.pool, items([(1, 0, 96), (1, 0, 96)]), m.dr, m.st)
    torch.cuda.synchronize()
    m.free([(1, 0, 96)])
    m.st.zero_()  # the second finds -1
    m.check()


@pytest.mark.parametrize("n", [1, 2, 31, 300])
@pytest.mark.parametrize("name", sorted(LAYOUTS))
def test_copies(name, n):
    pages = 2 * n + 3
    m = Model(name, pages, 1, 1, seed=n)
    m.to_device()
    at = m.rs.permutation(pages)
    src, dst = at[:n].copy(), at[n:2 * n].copy()
    src[n // 2] = src[0]  # one page copied twice
    for s, d in zip(src, dst):
        m.move_rows(s, d, m.ps)
    a, b = (torch.as_tensor(x, dtype=torch.int32).cuda() for x in (src, dst))
    km.kamera_copy_pages(m.h, m.pool, a, b, m.st)
    m.check()


def test_copies_outside_the_pool_are_left_out():
    m = Model("gqa", 9, 1, 1)
    m.to_device()
    src = np.array([0, 1, 9, 2, -1, 2 ** 31 - 1, 3])
    dst = np.array([4, 9, 5, -1, 6, 7, 8])
    m.move_rows(0, 4, m.ps)
    m.move_rows(3, 8, m.ps)
    a, b = (torch.as_tensor(x, dtype=torch.int32).cuda() for x in (src, dst))
    km.kamera_copy_pages(m.h, m.pool, a, b, m.st)
    m.check(km.KAMERA_DEVICE_SLOT_OOB)
    km.kamera_copy_pages(m.h, m.pool, a[:0], b[:0], m.st)
    m.check()


def test_table_with_a_wider_stride_and_another_stream():
    m = Model("gqa", 60, 4, 6)
    m.hold(0, 70)
    m.to_device()
    m.table = np.concatenate([m.table, np.full((4, 3), 77, np.int32)], 1)
    m.dt = torch.as_tensor(m.table).cuda()
    m.pool = km.Pool(m.dk, m.dv, m.dt)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    x, w = items([(0, 1, 70), (0, 2, 33)]), m.ws(2)
    torch.cuda.synchronize()
    km.kamera_fork(m.h, m.pool, x, m.dr, w, m.st, stream=s)
    m.check(m.fork([(0, 1, 70), (0, 2, 33)]))


def test_a_captured_step_replays():
    m = Model("gqa", 60, 6, 8)
    m.hold(0, 70)
    m.hold(1, 45)
    m.to_device()
    fork = [(0, 2, 70), (0, 3, 33), (1, 4, 45)]
    grow = [(2, 70, 100), (3, 33, 34), (4, 45, 65)]
    drop = [(2, 0, 100), (3, 0, 34), (4, 0, 65)]
    run_fork(m, fork)
    run_extend(m, grow)
    f, g_, d, w = items(fork), items(grow), items(drop), m.ws(3)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        km.kamera_free(m.h, m.pool, d, m.dr, m.st)
        km.kamera_fork(m.h, m.pool, f, m.dr, w, m.st)
        km.kamera_extend(m.h, m.pool, g_, m.dr, w, m.st)
    for _ in range(3):
        graph.replay()
        m.free(drop)
        m.fork(fork)
        m.extend(grow)
        m.check()


def test_refusals():
    m = Model("gqa", 20, 3, 4)
    m.hold(0, 40)
    m.to_device()
    x, w = items([(0, 1, 20)]), m.ws(1)
    for bad in (dict(x=x.long()), dict(x=x.cpu()), dict(x=x[:, :2]), dict(refs=m.dr[:-1]),
                dict(refs=m.dr.long()), dict(w=w.cpu()), dict(st=m.st.long()),
                dict(pool=km.Pool(m.dk[:2], m.dv[:2], m.dt)),
                dict(pool=km.Pool(m.dk, None, m.dt)), dict(pool=km.Pool(m.dk, m.dv, m.dt.long()))):
        a = dict(x=x, refs=m.dr, w=w, st=m.st, pool=m.pool)
        a.update(bad)
        with pytest.raises(ValueError):
            km.kamera_fork(m.h, a["pool"], a["x"], a["refs"], a["w"], a["st"])
    for short in (w[:-1], None):
        with pytest.raises(km.KameraError) as e:
            km.kamera_fork(m.h, m.pool, x, m.dr, short, m.st)
        assert e.value.status == km.KAMERA_ERR_INVALID_ARG
        with pytest.raises(km.KameraError):
            km.kamera_compact(m.h, m.pool, m.dr, m.st, None if short is None else m.ws(0)[:-1], m.st)
    many = torch.zeros(65536, 3, dtype=torch.int32, device="cuda")
    with pytest.raises(km.KameraError) as e:
        km.kamera_free(m.h, m.pool, many, m.dr, m.st)
    assert e.value.status == km.KAMERA_ERR_UNSUPPORTED
    m.check()
    km.kamera_fork(m.h, m.pool, x[:0], m.dr, None, m.st)
    m.check()
