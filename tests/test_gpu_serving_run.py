"""A run of the serving calls together: a prompt enters the pool, its request is forked, the
branches decode (room for a token, the token in, attention over the shared prefix and their own
tokens, layer by layer), some are released, the pool is compacted and the rest go on. Rows written
are checked against the formulas in float64 and then kept on the host by request and token;
attention is checked against float64 attention over what was kept, so a page that was copied,
moved, handed out or shared wrongly shows in the outputs."""
import math

import numpy as np
import pytest
import torch

import position_independent_multimodal_gb300 as km
import workloads as wl
from tests import test_gpu_append as ta

pytestmark = pytest.mark.gpu

EPS = 1e-6


@pytest.fixture(scope="module", autouse=True)
def _cuda(cuda_ok):
    return cuda_ok


LAYOUTS = {
    "gqa": (wl.Layout(kind=wl.GQA, num_layers=2, page_size=16, num_kv_heads=2, head_dim=128,
                      rope_dim=128, rope_theta=1e6), 14),
    "mrope-page5": (wl.Layout(kind=wl.GQA, num_layers=2, page_size=5, num_kv_heads=1, head_dim=64,
                              rope_dim=64, rope_theta=1e6, mrope_section=(8, 12, 12)), 3),
    "mla": (wl.Layout(kind=wl.MLA, num_layers=2, page_size=16, latent_dim=512, rope_dim=64,
                      rope_theta=1e4), 16),
}
ROWS, CAP = 12, 2000  # page-table rows, tokens of each


class Server:
    def __init__(self, name, seed=0):
        self.lay, self.hq = lay, hq = LAYOUTS[name]
        self.gqa = lay.kind == wl.GQA
        self.ps = lay.page_size
        self.hk = lay.num_kv_heads if self.gqa else 1
        self.dk = lay.head_dim if self.gqa else lay.latent_dim + lay.rope_dim
        self.dv = lay.head_dim if self.gqa else lay.latent_dim
        self.g = torch.Generator().manual_seed(seed)
        pages = 3 * CAP // self.ps
        n = pages * self.ps
        nan = float("nan")  # a row that no token holds must never matter
        self.k = torch.full((lay.num_layers, n, lay.row_k), nan, dtype=torch.bfloat16, device="cuda")
        self.v = torch.full((lay.num_layers, n, lay.row_v), nan, dtype=torch.bfloat16,
                            device="cuda") if self.gqa else None
        self.pt = torch.full((ROWS, -(-CAP // self.ps)), -1, dtype=torch.int32, device="cuda")
        self.pool = km.Pool(self.k, self.v, self.pt)
        self.refs = torch.zeros(pages, dtype=torch.int32, device="cuda")
        self.h = km.create(lay)
        self.st = torch.zeros(1, dtype=torch.int32, device="cuda")
        self.live = torch.zeros(1, dtype=torch.int32, device="cuda")
        self.page_ws = torch.empty(km.kamera_page_workspace(self.h, n, ROWS), dtype=torch.uint8,
                                   device="cuda")
        self.attn_ws = torch.empty(km.kamera_prefix_attention_workspace(self.h, ROWS, hq),
                                   dtype=torch.uint8, device="cuda")
        w = wl.normal_bf16((2, self.dk), 0.5, self.g, "cpu").cuda() + 1
        self.qw = w[0] if self.gqa else None
        self.kw = w[1] if self.gqa else w[1][:lay.latent_dim].contiguous()
        self.scale = 1 / math.sqrt(self.dk)
        # by request: the rows of its tokens, [layers][tokens][row], as bf16 values on the host
        self.rows = [None] * ROWS

    def items(self, x):
        return torch.tensor(x, dtype=torch.int32, device="cuda").reshape(-1, 3)

    def positions(self, tok):
        """A text position, and for M-RoPE a different one on each axis."""
        p = np.asarray(tok, np.int64) + 1000
        return np.stack([p, p + 7, p - 3], -1) if any(self.lay.mrope_section) else p

    def inputs(self, T):
        x = wl.normal_bf16((T, self.hq + 2 * self.hk, self.dk), 1.0, self.g, "cpu").cuda()
        return x[:, :self.hq], x[:, self.hq:self.hq + self.hk], \
            x[:, self.hq + self.hk:] if self.gqa else None

    def append(self, layer, q, k, v, pos, req, tok, out):
        km.kamera_append(self.h, self.pool, layer, q, k, v, self.qw if q is not None else None,
                         self.kw, pos, req, tok, EPS, out, self.st)

    def slots(self, req, tok):
        pt = self.pt.cpu().numpy().astype(np.int64)
        return pt[req, tok // self.ps] * self.ps + tok % self.ps

    def keep(self, layer, q, k, v, req, tok, out):
        """Checks what an append wrote; the rows as they are now, [T][row] of K and V."""
        want_q, want_k, want_v = ta.expected(self.lay, k if q is None else q, k, v, self.qw,
                                             self.kw, self.positions(tok).astype(np.float64), EPS)
        if q is not None:
            ta.check(ta.f64(out), want_q)
        s = torch.as_tensor(self.slots(req, tok)).cuda()
        rk = ta.f64(self.k[layer][s])
        ta.check(rk.reshape(want_k[0].shape), want_k)
        if v is None:
            return rk, None
        rv = ta.f64(self.v[layer][s])
        assert np.array_equal(rv, want_v.reshape(rv.shape))
        return rk, rv

    def attend(self, layer, q, n, group, prefix, ctx, out, lse):
        km.kamera_prefix_attention(self.h, self.pool, layer, q, group, prefix, ctx, self.scale, out,
                                   lse, self.attn_ws, self.st)

    def check_attention(self, layer, q, n, out, lse):
        """Bounds as derived in test_gpu_prefix_attention.py."""
        for r in range(n):
            if self.rows[r] is None:
                assert torch.all(out[r] == 0) and torch.all(lse[r] == -math.inf)
                continue
            k, v = (None if x is None else torch.as_tensor(x[layer]) for x in self.rows[r])
            k = k.reshape(len(k), self.hk, -1)
            v = k[..., :self.dv] if v is None else v.reshape(len(v), self.hk, -1)
            x = q[r].double().cpu().reshape(self.hk, -1, self.dk)
            s = self.scale * torch.einsum("hgd,thd->hgt", x, k)
            z = torch.logsumexp(s, -1)
            o = torch.einsum("hgt,thd->hgd", torch.exp(s - z[..., None]), v)
            B = (self.dk + 1) * 2.0 ** -24 * self.scale * \
                torch.einsum("hgd,thd->hgt", x.abs(), k.abs()).amax(-1)
            vm = v.abs().amax((0, 2))[:, None]
            tol = ((8 * B + 1e-4 + 2.0 ** -8) * vm)[..., None] + 2.0 ** -8 * o.abs()
            d = (out[r].double().cpu().reshape(o.shape) - o).abs()
            assert torch.all(d <= tol), (r, float((d / tol).max()))
            e = (lse[r].double().cpu().reshape(z.shape) - z).abs()
            assert torch.all(e <= 4 * B + 1e-5 * (1 + z.abs())), r

    def prompt(self, r, P):
        km.kamera_extend(self.h, self.pool, self.items([r, 0, P]), self.refs, self.page_ws, self.st)
        tok = np.arange(P)
        ks, vs = [], []
        for layer in range(self.lay.num_layers):
            _, k, v = self.inputs(P)
            self.append(layer, None, k, v, torch.as_tensor(self.positions(tok)).cuda(),
                        torch.full((P,), r, dtype=torch.int32, device="cuda"),
                        torch.as_tensor(tok, dtype=torch.int32).cuda(), None)
            rk, rv = self.keep(layer, None, k, v, np.full(P, r), tok, None)
            ks.append(rk)
            vs.append(rv)
        self.rows[r] = (np.stack(ks), np.stack(vs) if self.gqa else None)

    def length(self, r):
        return 0 if self.rows[r] is None else self.rows[r][0].shape[1]

    def fork(self, parent, children, n):
        km.kamera_fork(self.h, self.pool, self.items([[parent, c, n] for c in children]), self.refs,
                       self.page_ws, self.st)
        for c in children:
            self.rows[c] = tuple(None if x is None else x[:, :n].copy() for x in self.rows[parent])

    def release(self, reqs):
        km.kamera_free(self.h, self.pool, self.items([[r, 0, self.length(r)] for r in reqs]),
                       self.refs, self.st)
        for r in reqs:
            self.rows[r] = None

    def decode(self, n, groups):
        """A token for each of the live requests below n; groups: (first request, prefix)."""
        lay = self.lay
        who = [r for r in range(n) if self.rows[r] is not None]
        at = np.array([self.length(r) for r in who])
        km.kamera_extend(self.h, self.pool, self.items([[r, a, a + 1] for r, a in zip(who, at)]),
                         self.refs, self.page_ws, self.st)
        # a row for each request; those of empty ones are padding
        req, tok = np.full(n, -1), np.zeros(n, int)
        req[who], tok[who] = who, at
        i32 = lambda x: torch.as_tensor(np.asarray(x), dtype=torch.int32).cuda()  # noqa: E731
        ctx = np.zeros(n, int)
        ctx[who] = at + 1
        start = i32([g for g, _ in groups] + [n])
        prefix = i32([p for _, p in groups])
        for layer in range(lay.num_layers):
            q, k, v = self.inputs(n)
            out = torch.zeros(n, self.hq, self.dk, dtype=torch.bfloat16, device="cuda")
            self.append(layer, q, k, v, torch.as_tensor(self.positions(tok)).cuda(), i32(req),
                        i32(tok), out)
            pick = torch.as_tensor(who).cuda()
            rk, rv = self.keep(layer, q[pick], k[pick], None if v is None else v[pick],
                               np.array(who), at, out[pick])
            for i, r in enumerate(who):
                old = self.rows[r]
                if layer == 0:
                    old = tuple(None if x is None else
                                np.concatenate([x, np.zeros_like(x[:, :1])], 1) for x in old)
                    self.rows[r] = old
                old[0][layer, -1] = rk[i]
                if rv is not None:
                    old[1][layer, -1] = rv[i]
            o = torch.empty(n, self.hq, self.dv, dtype=torch.bfloat16, device="cuda")
            lse = torch.empty(n, self.hq, device="cuda")
            self.attend(layer, out, n, start, prefix, i32(ctx), o, lse)
            self.check_attention(layer, out, n, o, lse)
        assert int(self.st.item()) == 0

    def check_pages(self):
        held = self.pt[self.pt >= 0].cpu().numpy()
        assert np.array_equal(np.bincount(held, minlength=len(self.refs)), self.refs.cpu().numpy())


@pytest.mark.parametrize("name", sorted(LAYOUTS))
def test_a_run_of_the_serving_calls(name):
    s = Server(name)
    s.prompt(0, 701)           # more than a wide tile; the last page is not full
    s.prompt(7, 33)
    s.fork(0, [1, 2, 3, 4, 5, 6], 701)
    s.fork(7, [8, 9], 20)      # off the middle of the other prompt
    s.check_pages()
    groups = [(0, 701), (7, 20)]
    for _ in range(3):
        s.decode(10, groups)
    s.fork(9, [10, 11], s.length(9))  # branches of a branch
    s.check_pages()
    groups = [(0, 701), (7, 20), (9, 23)]
    for _ in range(2):
        s.decode(12, groups)
    s.release([0, 3, 8])       # the parent goes, its pages stay with the branches
    s.check_pages()
    s.decode(12, groups)
    km.kamera_compact(s.h, s.pool, s.refs, s.live, s.page_ws, s.st)
    s.check_pages()
    refs = s.refs.cpu().numpy()
    n = int(s.live.item())
    assert n == int((refs > 0).sum()) and np.all(refs[:n] > 0)
    for _ in range(3):
        s.decode(12, groups)
    s.fork(1, [0, 3], 400)     # into released rows, off the middle of the shared prefix
    s.check_pages()
    groups = [(0, 400), (7, 20), (9, 23)]
    s.decode(12, groups)
    s.release([r for r in range(12) if s.rows[r] is not None])
    assert int(s.st.item()) == 0 and not s.refs.any() and torch.all(s.pt == -1)


def test_a_captured_decode_step_gives_the_same_bits():
    a, b = Server("gqa", seed=3), Server("gqa", seed=3)
    for s in (a, b):
        s.prompt(0, 150)
        s.fork(0, [1, 2, 3], 150)
    n, dev = 4, dict(device="cuda")
    assert torch.equal(a.k.view(torch.int16), b.k.view(torch.int16))
    start = torch.tensor([0, n], dtype=torch.int32, **dev)
    prefix = torch.tensor([150], dtype=torch.int32, **dev)
    req = torch.arange(n, dtype=torch.int32, **dev)
    x = torch.zeros(2, n, a.hq + 2 * a.hk, a.dk, dtype=torch.bfloat16, **dev)
    pos = torch.zeros(n, dtype=torch.int64, **dev)
    tok = torch.zeros(n, dtype=torch.int32, **dev)
    ctx = torch.zeros(n, dtype=torch.int32, **dev)
    items = torch.zeros(n, 3, dtype=torch.int32, **dev)

    def step(s, out, o, lse):
        km.kamera_extend(s.h, s.pool, items, s.refs, s.page_ws, s.st)
        for layer in range(2):
            q, k, v = x[layer, :, :s.hq], x[layer, :, s.hq:s.hq + s.hk], x[layer, :, s.hq + s.hk:]
            s.append(layer, q, k, v, pos, req, tok, out[layer])
            s.attend(layer, out[layer], n, start, prefix, ctx, o[layer], lse[layer])

    def outputs(s):
        return (torch.zeros(2, n, s.hq, s.dk, dtype=torch.bfloat16, **dev),
                torch.zeros(2, n, s.hq, s.dv, dtype=torch.bfloat16, **dev),
                torch.zeros(2, n, s.hq, **dev))

    oa, ob = outputs(a), outputs(b)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step(b, *ob)
    g = torch.Generator().manual_seed(5)
    for t in range(20):  # a page begins on the way
        x.copy_(wl.normal_bf16(tuple(x.shape), 1.0, g, "cpu"))
        at = 150 + t
        pos.fill_(at)
        tok.fill_(at)
        ctx.fill_(at + 1)
        items.copy_(torch.tensor([[r, at, at + 1] for r in range(n)], dtype=torch.int32))
        step(a, *oa)
        graph.replay()
        torch.cuda.synchronize()
        for u, w in zip(oa, ob):
            assert torch.equal(u.view(torch.uint8), w.view(torch.uint8)), t
    assert torch.equal(a.pt, b.pt) and torch.equal(a.refs, b.refs)
    assert torch.equal(a.k.view(torch.int16), b.k.view(torch.int16))
    assert int(a.st.item()) == int(b.st.item()) == 0


@pytest.mark.parametrize("name", ["gqa", "mla"])
def test_offsets_past_32_bits(name):
    # a pool of more than 2^32 bytes and 2^31 elements a channel, its last pages in use
    s = Server(name, seed=8)
    lay, ps, hq = s.lay, s.ps, s.hq
    pages = 2 ** 31 // (lay.num_layers * lay.row_k * ps) + 4000
    shape = (lay.num_layers, pages * ps, lay.row_k)
    s.k = torch.empty(shape, dtype=torch.bfloat16, device="cuda")
    s.v = torch.empty(shape, dtype=torch.bfloat16, device="cuda") if s.gqa else None
    assert s.k.numel() > 2 ** 31
    P, n = 150, -(-150 // ps)
    s.pt[0, :n] = torch.arange(pages - n, pages, dtype=torch.int32).flip(0).cuda()
    s.pool = km.Pool(s.k, s.v, s.pt)
    s.refs = torch.zeros(pages, dtype=torch.int32, device="cuda")
    s.refs[pages - n:] = 1
    s.page_ws = torch.empty(km.kamera_page_workspace(s.h, pages * ps, ROWS), dtype=torch.uint8,
                            device="cuda")
    layer, tok = 1, np.arange(P)
    i32 = lambda x: torch.as_tensor(np.asarray(x), dtype=torch.int32).cuda()  # noqa: E731

    def enter(r, t, q):
        x, k, v = s.inputs(len(t))
        out = torch.zeros_like(x) if q else None
        s.append(layer, x if q else None, k, v, torch.as_tensor(s.positions(t)).cuda(),
                 i32(np.full(len(t), r)), i32(t), out)
        return out, s.keep(layer, x if q else None, k, v, np.full(len(t), r), t, out)

    _, (rk, rv) = enter(0, tok, False)

    def attend(q, rows_k, rows_v):
        o = torch.empty(1, hq, s.dv, dtype=torch.bfloat16, device="cuda")
        lse = torch.empty(1, hq, device="cuda")
        s.attend(layer, q, 1, i32([0, 1]), i32([P]), i32([len(rows_k)]), o, lse)
        s.rows[0] = tuple(None if x is None else np.stack([np.zeros_like(x), x])
                          for x in (rows_k, rows_v))
        s.check_attention(layer, q, 1, o, lse)

    q = s.inputs(1)[0].contiguous()
    attend(q, rk, rv)
    # a copy within the last pages, then the whole request drawn to the front of the pool
    last = [x for x in (s.k, s.v) if x is not None]
    km.kamera_copy_pages(s.h, s.pool, i32([pages - 2]), i32([pages - n - 5]), s.st)
    for x in last:
        a = x.view(lay.num_layers, pages, ps, -1)
        assert torch.equal(a[:, pages - 2].view(torch.int16), a[:, pages - n - 5].view(torch.int16))
    km.kamera_compact(s.h, s.pool, s.refs, s.live, s.page_ws, s.st)
    assert int(s.live.item()) == n and int(s.pt[0, :n].max()) == n - 1
    assert int(s.refs.sum()) == n and torch.all(s.refs[:n] == 1)
    attend(q, rk, rv)
    # and a branch whose new page is among the last: every page between is taken
    s.refs[n:pages - 1] = 1
    s.fork(0, [1], P)
    assert int(s.pt[1, n - 1]) == pages - 1 and int(s.st.item()) == 0
    assert torch.equal(s.k[layer][s.slots(np.full(P, 1), tok)].view(torch.int16),
                       s.k[layer][s.slots(np.full(P, 0), tok)].view(torch.int16))
