"""A run of chunk attention, attention masses and eviction together, as a server with a budget of
tokens for each request would make it: a batch of new tokens (pieces of prompts next to requests that
decode) gets room, enters the pool and is attended layer by layer, its softmax weights are added to
the masses of the tokens it looked at, and requests that have outgrown the budget keep the tokens
with the greatest masses and give pages back. Rows are kept on the host by request and token as they
were appended; attention and masses are checked against float64 over what was kept, so a page that
was handed out, given back or drawn together wrongly shows in the outputs."""
import math

import numpy as np
import pytest
import torch

import position_independent_multimodal_gb300 as km
import workloads as wl
from tests.chunk_testlib import Chunks, i32

pytestmark = pytest.mark.gpu

LAYOUTS = {
    "gqa": (wl.Layout(kind=wl.GQA, num_layers=2, page_size=16, num_kv_heads=2, head_dim=128,
                      rope_dim=128, rope_theta=1e6), 14),
    "gqa64-page5": (wl.Layout(kind=wl.GQA, num_layers=2, page_size=5, num_kv_heads=3, head_dim=64,
                              rope_dim=64, rope_theta=1e6), 3),
    "gqa80": (wl.Layout(kind=wl.GQA, num_layers=2, page_size=8, num_kv_heads=1, head_dim=80,
                        rope_dim=80, rope_theta=1e6), 4),
    "mla": (wl.Layout(kind=wl.MLA, num_layers=2, page_size=64, latent_dim=512, rope_dim=64,
                      rope_theta=1e4), 16),
}
R, BUDGET, FIRST, LAST, WIDTH, DECAY = 4, 300, 4, 60, 640, 0.75
PAD = 2  # rows behind the last request's

# new tokens of each request, by step: pieces of prompts, decoding, nothing
STEPS = [(280, 1, 0, 37), (1, 299, 150, 64), (150, 1, 1, 0), (1, 1, 170, 1), (1, 1, 1, 1),
         (1, 0, 1, 310), (29, 1, 1, 1), (1, 1, 129, 1)]


@pytest.fixture(scope="module", autouse=True)
def _cuda(cuda_ok):
    return cuda_ok


def bits(x):
    return x.view(torch.int16 if x.dtype == torch.bfloat16 else torch.int32)


class Window:
    def __init__(self, name, seed=0):
        self.lay, self.hq = lay, hq = LAYOUTS[name]
        self.gqa = lay.kind == wl.GQA
        self.hk = lay.num_kv_heads if self.gqa else 1
        self.dk = lay.head_dim if self.gqa else lay.latent_dim + lay.rope_dim
        self.dv = lay.head_dim if self.gqa else lay.latent_dim
        ps, g = lay.page_size, torch.Generator().manual_seed(seed)
        pages = R * (BUDGET + 340) // ps + R
        slots = pages * ps
        nan = dict(fill_value=math.nan, dtype=torch.bfloat16, device="cuda")
        self.k = torch.full((lay.num_layers, slots, lay.row_k), **nan)
        self.v = torch.full((lay.num_layers, slots, lay.row_v), **nan) if self.gqa else None
        self.pt = torch.full((R + 1, -(-WIDTH // ps)), -1, dtype=torch.int32, device="cuda")
        self.pool = km.Pool(self.k, self.v, self.pt)
        self.refs = torch.zeros(pages, dtype=torch.int32, device="cuda")
        self.mass = torch.full((R + 1, WIDTH), math.nan, device="cuda")
        self.st = torch.zeros(1, dtype=torch.int32, device="cuda")
        self.h, self.scale = km.create(lay), 1 / math.sqrt(self.dk)
        byte = dict(dtype=torch.uint8, device="cuda")
        self.page_ws = torch.empty(km.kamera_page_workspace(self.h, slots, R), **byte)
        most = max(sum(s) for s in STEPS) + PAD
        # the attention's and the masses' calls follow one another on a stream: one workspace
        self.ws = torch.empty(max(km.kamera_chunk_attention_workspace(self.h, most, R, hq),
                                  km.kamera_attention_mass_workspace(self.h, most, R, hq),
                                  km.kamera_evict_workspace(self.h, R)), **byte)
        lens, at = np.zeros(R, int), np.zeros(R, int)  # tokens held, tokens so far
        self.steps = []
        for new in STEPS:
            new = np.array(new)
            T = int(new.sum()) + PAD
            req = np.concatenate([np.repeat(np.arange(R), new), np.full(PAD, -1)])
            tok = np.concatenate([lens[r] + np.arange(n) for r, n in enumerate(new)] + [np.zeros(PAD)])
            pos = np.concatenate([at[r] + np.arange(n) for r, n in enumerate(new)] + [np.zeros(PAD)])
            d = dict(new=new, before=lens.copy(), ctx=lens + new)
            d["extend"] = i32([[r, lens[r], lens[r] + new[r]] for r in range(R)])
            d["req"], d["tok"], d["d_ctx"] = i32(req), i32(tok), i32(d["ctx"])
            d["pos"] = torch.as_tensor(pos.astype(np.int64)).cuda()
            d["start"] = i32(np.concatenate([[0], np.cumsum(new)]))
            d["x"] = wl.normal_bf16((2, T, hq + 2 * self.hk, self.dk), 1.0, g, "cpu").cuda()
            d["q"] = torch.zeros(2, T, hq, self.dk, dtype=torch.bfloat16, device="cuda")
            d["out"] = torch.zeros(2, T, hq, self.dv, dtype=torch.bfloat16, device="cuda")
            d["lse"] = torch.zeros(2, T, hq, device="cuda")
            at, lens = at + new, lens + new
            over = [r for r in range(R) if lens[r] > BUDGET]
            d["over"] = over
            if over:
                d["evict"] = i32([[r, lens[r], BUDGET, FIRST, LAST] for r in over])
                d["kept"] = torch.full((len(over), BUDGET), -9, dtype=torch.int32, device="cuda")
                d["free"] = i32([[r, BUDGET, lens[r]] for r in over])
                lens = np.minimum(lens, BUDGET)
            self.steps.append(d)

    def enter(self, d):
        km.kamera_extend(self.h, self.pool, d["extend"], self.refs, self.page_ws, self.st)

    def layer(self, d, i):
        a, b = self.hq, self.hq + self.hk
        x = d["x"][i]
        km.kamera_append(self.h, self.pool, i, x[:, :a], x[:, a:b], x[:, b:] if self.gqa else None,
                         None, None, d["pos"], d["req"], d["tok"], 0.0, d["q"][i], self.st)
        km.kamera_chunk_attention(self.h, self.pool, i, d["q"][i], d["start"], d["d_ctx"],
                                  self.scale, d["out"][i], d["lse"][i], self.ws, self.st)
        # a step's first call lets what was there fade, the next adds its layer's
        km.kamera_attention_mass(self.h, self.pool, i, d["q"][i], d["start"], d["d_ctx"],
                                 self.scale, d["lse"][i], DECAY if i == 0 else 1.0, self.mass[:R],
                                 self.ws, self.st)

    def leave(self, d):
        if d["over"]:
            km.kamera_evict(self.h, self.pool, d["evict"], self.refs, self.mass, d["kept"], self.ws,
                            self.st)
            km.kamera_free(self.h, self.pool, d["free"], self.refs, self.st)

    def zero_masses(self, d):
        """Tokens that were never attended have no mass yet: the masses of new ones begin at 0."""
        for r in range(R):
            self.mass[r, int(d["before"][r]):int(d["ctx"][r])] = 0

    def run(self):
        for d in self.steps:
            self.zero_masses(d)
            self.enter(d)
            for i in range(2):
                self.layer(d, i)
            self.leave(d)

    def slots(self, r, n):
        ps, t = self.lay.page_size, np.arange(n)
        return torch.as_tensor(self.pt[r].cpu().numpy().astype(np.int64)[t // ps] * ps + t % ps).cuda()

    def rows(self, i, r, n):
        s = self.slots(r, n)
        return self.k[i][s], None if self.v is None else self.v[i][s]


def check_layer(w, d, i, before, kept):
    """Outputs (bounds of test_gpu_chunk_attention.py) and masses (of test_gpu_attention_mass.py) of
    layer i; kept[r]: rows of request r's tokens, before: the masses."""
    for r in range(R):
        n, c = int(d["new"][r]), int(d["ctx"][r])
        if n == 0:
            assert torch.equal(bits(w.mass[r]), bits(before[r]))
            continue
        k, v = kept[r]
        k = k.double().view(c, w.hk, w.dk)
        v = k[..., :w.dv] if v is None else v.double().view(c, w.hk, w.dv)
        a = int(d["start"][r])
        q = d["q"][i][a:a + n].double().view(n, w.hk, -1, w.dk)
        sees = (torch.arange(c)[None] <= torch.arange(c - n, c)[:, None]).cuda()[:, None, None]
        x = torch.where(sees, w.scale * torch.einsum("nhgd,chd->nhgc", q, k), -math.inf)
        b = torch.einsum("nhgd,chd->nhgc", q.abs(), k.abs()) * sees
        b = b.amax(-1) * w.scale * (w.dk + 1) * 2.0 ** -24
        z = torch.logsumexp(x, -1)
        o = torch.einsum("nhgc,chd->nhgd", torch.exp(x - z[..., None]), v)
        vm = v.abs().amax((0, 2))[:, None]
        tol = ((8 * b + 1e-4 + 2.0 ** -8) * vm)[..., None] + 2.0 ** -8 * o.abs()
        got = d["out"][i][a:a + n].double().view(o.shape)
        assert bool(((got - o).abs() <= tol).all()), (r, i)
        lse = d["lse"][i][a:a + n].double().view(z.shape)
        assert bool(((lse - z).abs() <= 4 * b + 1e-5 * (1 + z.abs())).all()), (r, i)
        p = torch.exp(x - lse[..., None])
        off = b[..., None] + 2.0 ** -22 * (2 + torch.where(sees, x.abs(), 0.0) + lse.abs()[..., None])
        total, tol = p.sum((0, 1, 2)), torch.where(sees, p * off, 0.0).sum((0, 1, 2))
        tol += total * (n * w.hq * 2.0 ** -24)
        total += (DECAY if i == 0 else 1.0) * before[r, :c].double()
        tol += 2.0 ** -23 * total
        assert bool(((w.mass[r, :c].double() - total).abs() <= tol + 1e-30).all()), (r, i)
        assert torch.equal(bits(w.mass[r, c:]), bits(before[r, c:]))


@pytest.mark.parametrize("name", sorted(LAYOUTS))
def test_a_run_within_a_budget(name):
    w = Window(name)
    held = [[None] * R, [None] * R]  # by layer and request
    for step, d in enumerate(w.steps):
        w.zero_masses(d)
        w.enter(d)
        for i in range(2):
            before = w.mass.clone()
            w.layer(d, i)
            torch.cuda.synchronize()
            assert int(w.st.item()) == 0, step
            for r in range(R):
                c = int(d["ctx"][r])
                rows, old, n = w.rows(i, r, c), held[i][r], int(d["before"][r])
                for new, was in zip(rows, old or ()):
                    assert new is None or torch.equal(bits(new[:n]), bits(was)), (step, i, r)
                held[i][r] = rows
            check_layer(w, d, i, before, held[i])
        assert bool((d["out"][:, -PAD:] == 0).all()) and bool((d["lse"][:, -PAD:] == 0).all())
        mass = w.mass.cpu().numpy()
        w.leave(d)
        torch.cuda.synchronize()
        assert int(w.st.item()) == 0, step
        for j, r in enumerate(d["over"]):
            n = int(d["ctx"][r])
            among = np.arange(FIRST, n - LAST)
            best = among[np.argsort(-mass[r, among], kind="stable")[:BUDGET - FIRST - LAST]]
            want = np.concatenate([np.arange(FIRST), np.sort(best), np.arange(n - LAST, n)])
            assert np.array_equal(d["kept"][j].cpu().numpy(), want), (step, r)
            assert np.array_equal(w.mass[r, :BUDGET].cpu().numpy(), mass[r, want])
            assert not w.mass[r, BUDGET:n].any()
            pick = torch.as_tensor(want).cuda()
            for i in range(2):
                held[i][r] = tuple(None if x is None else x[pick] for x in held[i][r])
        live = w.pt[w.pt >= 0].cpu().numpy()
        assert np.array_equal(np.bincount(live, minlength=len(w.refs)), w.refs.cpu().numpy())
        assert int(w.refs.max()) == 1


@pytest.mark.parametrize("name", ["gqa", "gqa80", "mla"])
def test_a_captured_run_gives_the_same_bits(name):
    # all steps in a row, on a stream of their own and as a graph that is replayed twice
    a, b = Window(name, seed=1), Window(name, seed=1)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        a.run()
    torch.cuda.synchronize()
    first = [x.clone() for x in (b.k, b.v, b.pt, b.refs, b.mass) if x is not None]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        b.run()
    for _ in range(2):
        for x, y in zip((x for x in (b.k, b.v, b.pt, b.refs, b.mass) if x is not None), first):
            x.copy_(y)
        graph.replay()
        torch.cuda.synchronize()
        assert int(a.st.item()) == int(b.st.item()) == 0
        assert torch.equal(a.pt, b.pt) and torch.equal(a.refs, b.refs)
        for x, y in ((a.k, b.k), (a.v, b.v), (a.mass, b.mass)):
            assert x is None or torch.equal(bits(x), bits(y))
        for d, e in zip(a.steps, b.steps):
            for x in ("q", "out", "lse") + (("kept",) if d["over"] else ()):
                assert torch.equal(bits(d[x]), bits(e[x])), x


def test_two_servers_at_once():
    # on streams of their own, with workspaces of their own
    a, b = Window("gqa", seed=2), Window("gqa", seed=3)
    c, d = Window("gqa", seed=2), Window("gqa", seed=3)
    torch.cuda.synchronize()
    one, two = torch.cuda.Stream(), torch.cuda.Stream()
    with torch.cuda.stream(one):
        a.run()
    with torch.cuda.stream(two):
        b.run()
    torch.cuda.synchronize()
    c.run()
    d.run()
    torch.cuda.synchronize()
    for x, y in ((a, c), (b, d)):
        assert int(x.st.item()) == 0
        assert torch.equal(bits(x.k), bits(y.k)) and torch.equal(bits(x.mass), bits(y.mass))
        for s, t in zip(x.steps, y.steps):
            assert torch.equal(bits(s["out"]), bits(t["out"]))


@pytest.mark.parametrize("name", ["gqa128-group7", "gqa80", "mla-16-heads"])
def test_offsets_past_32_bits(name):
    # a pool of more than 2^31 elements a channel, its last pages in use: attention, masses and an
    # eviction there give what they give in a small pool
    b = Chunks(name, [(40, 300), (1, 500)], seed=15)
    lay, ps = b.lay, b.lay.page_size
    few = b.k.shape[1] // ps
    pages = 2 ** 31 // (lay.num_layers * lay.row_k * ps) + few + 1000
    b.dev()
    small, table = b.pool, b.pool.page_table
    high = torch.where(table >= 0, table + (pages - few), table)

    def grown(x):
        y = torch.empty(lay.num_layers, pages * ps, x.shape[2], dtype=x.dtype, device="cuda")
        assert y.numel() > 2 ** 31
        y[:, -few * ps:] = x
        return y

    big = km.Pool(grown(small.k), None if small.v is None else grown(small.v), high)
    got = []
    for pool, n in ((small, few), (big, pages)):
        b.pool = pool
        b.out.fill_(-7)
        b.lse.fill_(-7)
        b.call()
        ws = torch.empty(max(km.kamera_attention_mass_workspace(b.h, b.rows, 2, b.hq),
                             km.kamera_evict_workspace(b.h, 2)), dtype=torch.uint8, device="cuda")
        mass = torch.zeros(2, 520, device="cuda")
        km.kamera_attention_mass(b.h, pool, 1, b.q, b.d_start, b.d_ctx, b.scale, b.lse, 0.0, mass, ws,
                                 b.st)
        refs = torch.zeros(n, dtype=torch.int32, device="cuda")
        refs[pool.page_table[pool.page_table >= 0].long()] = 1
        kept = torch.zeros(2, 400, dtype=torch.int32, device="cuda")
        km.kamera_evict(b.h, pool, i32([[0, 340, 200, 3, 20], [1, 501, 400, 0, 0]]), refs, mass, kept,
                        ws, b.st)
        torch.cuda.synchronize()
        assert int(b.st.item()) == 0
        got.append((b.out.clone(), b.lse.clone(), mass, kept, pool.k[:, -few * ps:],
                    None if pool.v is None else pool.v[:, -few * ps:]))
    for x, y in zip(*got):
        assert x is None or torch.equal(bits(x.contiguous()), bits(y.contiguous()))


@pytest.mark.parametrize("name", ["gqa128-group7", "gqa64-group3", "mla-16-heads", "gqa80"])
def test_outputs_at_any_16_bytes(name):
    b = Chunks(name, [(40, 300), (1, 500), (150, 0)], seed=16).run()
    out, lse = b.out, b.lse
    wide = torch.full((out.numel() + 8,), -7.0, dtype=torch.bfloat16, device="cuda")
    thin = torch.full((lse.numel() + 1,), -7.0, device="cuda")
    b.out, b.lse = wide[8:].view(out.shape), thin[1:].view(lse.shape)
    b.call()
    torch.cuda.synchronize()
    assert torch.equal(bits(b.out), bits(out)) and torch.equal(bits(b.lse), bits(lse))
    assert bool((wide[:8] == -7).all()) and float(thin[0]) == -7
