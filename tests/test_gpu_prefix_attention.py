"""kamera_prefix_attention against float64 attention over each request's whole context.

Bounds, with B = max_t (Dk + 1) 2^-24 |scale| sum_d |q_d k_td| (float32 accumulation of a dot
product) and Vm = max_t |V_t|: a score error of B moves a softmax weight by at most about 2 B, and
an output by at most (8 B + 1e-4) Vm with the float32 sums over tiles, segments and parts (each
adds at most n 2^-24 of the mass for n terms; 1e-4 covers the contexts here). Softmax weights
rounded to bf16 are off by at most half a step, 2^-8, and the normaliser is not rounded: another
2^-8 Vm on the tensor cores (2^-8 |o| would not do: weights of either sign of V add up). The
output's own rounding adds 2^-8 |o|. The log-sum-exp takes float32 weights on every path:
4 B + 1e-5 (1 + |lse|).
"""
import math

import numpy as np
import pytest
import torch

import position_independent_multimodal_gb300 as km
import workloads as wl

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _cuda(cuda_ok):
    return cuda_ok


def gqa(hd, hkv, page=16, layers=2):
    return wl.Layout(kind=wl.GQA, num_layers=layers, page_size=page, num_kv_heads=hkv,
                     head_dim=hd, rope_dim=hd)


def mla(lat, rope, page=16, layers=2):
    return wl.Layout(kind=wl.MLA, num_layers=layers, page_size=page, latent_dim=lat,
                     rope_dim=rope)


LAYOUTS = {
    "gqa128-group7": (gqa(128, 4), 28),
    "gqa128-group4-page64": (gqa(128, 2, page=64), 8),
    "mha128-page1": (gqa(128, 3, page=1), 3),
    "gqa128-one-kv-head": (gqa(128, 1, page=48), 40),
    "gqa64-group3": (gqa(64, 2), 6),
    "mha64-page5": (gqa(64, 5, page=5), 5),
    "gqa80": (gqa(80, 2), 6),
    "gqa16": (gqa(16, 1), 1),
    "gqa256": (gqa(256, 1, page=128), 9),
    "mla-16-heads": (mla(512, 64), 16),
    "mla-128-heads": (mla(512, 64, page=64), 128),
    "mla-130-heads-page3": (mla(512, 64, page=3), 130),
    "mla-narrow": (mla(96, 32), 5),
}


def tensor_path(lay):
    return (lay.kind == wl.GQA and lay.head_dim in (64, 128)) or \
        (lay.kind == wl.MLA and (lay.latent_dim, lay.rope_dim) == (512, 64))


class Batch:
    """Groups of requests over a pool whose unheld rows are NaN."""

    def __init__(self, name, groups, seed=0, sharp=1.0, outside=float("nan"), layer=1):
        # groups: (prefix, [own tokens of each request; None: an empty context])
        self.lay, self.hq = lay, hq = LAYOUTS[name]
        self.layer = layer
        ps = lay.page_size
        g = torch.Generator().manual_seed(seed)
        rs = np.random.RandomState(seed)
        self.start = np.cumsum([0] + [len(o) for _, o in groups])
        self.prefix = np.array([p for p, _ in groups])
        own = [x for _, o in groups for x in o]
        grp = np.repeat(np.arange(len(groups)), np.diff(self.start))
        self.ctx = np.array([0 if x is None else int(self.prefix[k]) + x for x, k in zip(own, grp)], int)
        R = len(own)
        need = sum(-(-int(p) // ps) for p in self.prefix) + sum(-(-int(c) // ps) + 1 for c in self.ctx)
        pages = need + 3
        self.stride = max([1] + [-(-int(c) // ps) for c in self.ctx]) + 1
        free = list(rs.permutation(pages))
        self.table = np.full((R, self.stride), -1, np.int64)
        self.pages = pages
        n = pages * ps
        self.k = torch.full((lay.num_layers, n, lay.row_k), outside, dtype=torch.bfloat16)
        self.v = torch.full((lay.num_layers, n, lay.row_v), outside, dtype=torch.bfloat16) \
            if lay.kind == wl.GQA else None

        def fill(slots):
            for x in (self.k, self.v):
                if x is not None and len(slots):
                    idx = torch.as_tensor(slots)
                    x[:, idx] = wl.normal_bf16((x.shape[0], len(slots), x.shape[2]), 1.0, g, "cpu")

        for k, (p, o) in enumerate(groups):
            whole = p // ps
            shared = [free.pop() for _ in range(whole)]
            fill((np.array(shared, int)[:, None] * ps + np.arange(ps)).reshape(-1))
            first = None
            for r in range(self.start[k], self.start[k + 1]):
                c = int(self.ctx[r])
                if c == 0:
                    continue
                self.table[r, :whole] = shared
                for i in range(whole, -(-c // ps)):
                    self.table[r, i] = free.pop()
                slots = self.slots(r)
                fill(slots[whole * ps:])
                if first is None:
                    first = slots
                else:  # the prefix's last part, in a page of the request's own
                    a, b = torch.as_tensor(first[whole * ps:p]), torch.as_tensor(slots[whole * ps:p])
                    for x in (self.k, self.v):
                        if x is not None and len(a):
                            x[:, b] = x[:, a]
        self.dk = lay.head_dim if lay.kind == wl.GQA else lay.latent_dim + lay.rope_dim
        self.dv = lay.head_dim if lay.kind == wl.GQA else lay.latent_dim
        self.q = wl.normal_bf16((R, hq, self.dk), sharp, g, "cpu")
        self.scale = 1 / math.sqrt(self.dk)
        self.h = km.create(lay)
        self.out = torch.full((R, hq, self.dv), -7.0, dtype=torch.bfloat16, device="cuda")
        self.lse = torch.full((R, hq), -7.0, device="cuda")
        self.st = torch.zeros(1, dtype=torch.int32, device="cuda")
        w = km.kamera_prefix_attention_workspace(self.h, R, hq)
        self.ws = torch.full((w,), 0xFF, dtype=torch.uint8, device="cuda")

    def slots(self, r):
        t = np.arange(self.ctx[r])
        ps = self.lay.page_size
        return self.table[r, t // ps] * ps + t % ps

    def dev(self):
        i32 = lambda x: torch.as_tensor(np.asarray(x), dtype=torch.int32).cuda()  # noqa: E731
        self.pool = km.Pool(self.k.cuda(), None if self.v is None else self.v.cuda(), i32(self.table))
        self.args = (self.q.cuda(), i32(self.start), i32(self.prefix), i32(self.ctx))

    def call(self, **kw):
        q, start, prefix, ctx = self.args
        km.kamera_prefix_attention(self.h, self.pool, self.layer, q, start, prefix, ctx,
                                   self.scale, self.out, self.lse, self.ws, self.st, **kw)

    def run(self, **kw):
        self.dev()
        torch.cuda.synchronize()
        self.call(**kw)
        torch.cuda.synchronize()
        return int(self.st.item())

    def want(self, r, leave=()):
        """(o, lse, bound of o, bound of lse) of request r, without the tokens in `leave`."""
        lay, hq = self.lay, self.hq
        keep = np.setdiff1d(np.arange(self.ctx[r]), leave)
        s = torch.as_tensor(self.slots(r)[keep])
        H = lay.num_kv_heads if lay.kind == wl.GQA else 1
        k = self.k[self.layer][s].double().reshape(len(keep), H, -1)
        v = k[..., :self.dv] if self.v is None else \
            self.v[self.layer][s].double().reshape(len(keep), H, -1)
        q = self.q[r].double().reshape(H, hq // H, -1)
        x = self.scale * torch.einsum("hgd,thd->hgt", q, k)
        z = torch.logsumexp(x, -1)
        o = torch.einsum("hgt,thd->hgd", torch.exp(x - z[..., None]), v)
        B = (self.dk + 1) * 2.0 ** -24 * abs(self.scale) * \
            torch.einsum("hgd,thd->hgt", q.abs(), k.abs()).amax(-1)
        vm = v.abs().amax((0, 2))[:, None]
        tol = (8 * B + 1e-4 + (2.0 ** -8 if tensor_path(lay) else 0)) * vm
        tol = tol[..., None] + 2.0 ** -8 * o.abs()
        return (o.reshape(hq, -1), z.reshape(hq), tol.reshape(hq, -1),
                (4 * B + 1e-5 * (1 + z.abs())).reshape(hq))

    def check(self, reqs=None, leave=()):
        out, lse = self.out.double().cpu(), self.lse.double().cpu()
        for r in range(len(self.ctx)) if reqs is None else reqs:
            if self.ctx[r] == 0:
                assert torch.all(out[r] == 0) and torch.all(lse[r] == -math.inf), r
                continue
            o, z, to, tz = self.want(r, leave)
            d = (out[r] - o).abs()
            assert torch.all(d <= to), (r, float((d / to).max()), int((~(d <= to)).sum()))
            e = (lse[r] - z).abs()
            assert torch.all(e <= tz), (r, float((e / tz).max()))


@pytest.mark.parametrize("sharp", [1.0, 6.0])
@pytest.mark.parametrize("name", sorted(LAYOUTS))
def test_groups_of_every_kind(name, sharp):
    # no prefix, one token, ends around a tile and a page, an empty own part, empty contexts
    # (the first of a group among them), a group of one, a group that is empty altogether
    b = Batch(name, [(0, [1, 130, None]), (1, [0, 5]), (129, [None, 0, 1, 127, 300, 128]),
                     (640, [17]), (50, [None, None]), (255, [1, 2, 40])], seed=len(name), sharp=sharp)
    assert b.run() == 0
    b.check()


@pytest.mark.parametrize("prefix", [1, 16, 127, 128, 129, 256, 1000])
@pytest.mark.parametrize("name", ["gqa128-group7", "mha64-page5", "mla-16-heads"])
def test_one_request(name, prefix):
    b = Batch(name, [(prefix, [0])], seed=prefix)
    assert b.run() == 0
    b.check()


@pytest.mark.parametrize("ctx", [1, 2, 15, 300, 2500])
@pytest.mark.parametrize("name", ["gqa128-group7", "gqa64-group3", "mla-16-heads", "gqa80"])
def test_nothing_shared(name, ctx):
    b = Batch(name, [(0, [ctx, max(1, ctx // 2), None]), (0, [3])], seed=ctx)
    assert b.run() == 0
    b.check()


@pytest.mark.parametrize("name", ["gqa128-group7", "gqa64-group3", "mla-128-heads", "gqa80"])
def test_many_requests_of_one_prefix(name):
    # more rows than a block, blocks cut between CTAs, a last block of a few rows
    rs = np.random.RandomState(4)
    b = Batch(name, [(1500, [int(x) for x in rs.randint(0, 200, 41)])], seed=1)
    assert b.run() == 0
    b.check()


@pytest.mark.parametrize("name", ["gqa128-group7", "mla-16-heads"])
def test_long_prefix(name):
    b = Batch(name, [(20011, [0, 700, 3]), (4097, [1])], seed=2)
    assert b.run() == 0
    b.check()


def test_many_small_requests():
    # more requests than the plan's threads, most of them empty
    own = [None if i % 5 else i % 7 for i in range(2300)]
    b = Batch("gqa16", [(0, own[:900]), (33, own[900:2299]), (7, own[2299:])], seed=3)
    assert b.run() == 0
    b.check(reqs=range(0, 2300, 17))


@pytest.mark.parametrize("name", ["gqa128-group7", "mla-16-heads", "gqa80"])
def test_scores_that_rise_along_the_context(name):
    # the running maximum rises tile by tile, by more than float32's exponent range in all, and a
    # mid token dominates; then a negative scale, where the smallest product wins
    for scale in (1.0, -1.0):
        b = Batch(name, [(900, [300, 1]), (0, [700])], seed=5)
        for r in range(3):
            s = torch.as_tensor(b.slots(r))
            ramp = (torch.arange(len(s)) / 1200 * 8)[:, None]  # by token: alike in every request
            b.k[:, s] = (b.k[:, s].float().sign() * 0.25 * (1 + ramp)).to(torch.bfloat16)
        b.q = (b.q.float().abs() * 3).to(torch.bfloat16)
        b.scale = scale / 4
        assert b.run() == 0
        b.check()


@pytest.mark.parametrize("name", ["gqa128-group7", "mla-16-heads", "gqa80"])
def test_equal_scores_and_zero_scale(name):
    b = Batch(name, [(200, [100, 0]), (0, [1])], seed=6)
    b.scale = 0.0
    assert b.run() == 0
    b.check()


@pytest.mark.parametrize("outside", [float("inf"), float("-inf"), float("nan"), -3.3895e38])
@pytest.mark.parametrize("name", ["gqa128-group7", "gqa64-group3", "mla-16-heads", "gqa80"])
def test_rows_that_no_token_holds_do_not_matter(name, outside):
    b = Batch(name, [(130, [5, 60]), (0, [1])], seed=7, outside=outside)
    assert b.run() == 0
    b.check()


@pytest.mark.parametrize("name", ["gqa128-group7", "mla-16-heads", "gqa80"])
def test_non_finite_keys_and_values_stay_with_their_requests(name):
    b = Batch(name, [(140, [30, 50, 20]), (5, [60])], seed=8)
    bad = b.slots(1)[150]
    b.k[:, bad, 3] = float("nan")
    minus = b.slots(2)[145]
    b.k[:, minus] = float("-inf")
    b.q[2] = b.q[2].abs() + 0.01  # every score of that token is -inf: it weighs nothing
    if b.v is None:
        b.k[:, minus] = 0  # the row is its own value: a plain row here
    assert b.run() == 0
    b.check(reqs=[0, 3])
    assert torch.isnan(b.out[1, 0].float()).any() and torch.isnan(b.lse[1, 0])
    out = b.out[2].float()
    assert torch.isfinite(out).all() and torch.isfinite(b.lse[2]).all()
    if b.v is not None:
        o, z, to, tz = (x for x in b.want(2, leave=[145]))
        assert torch.all((b.out[2].double().cpu() - o).abs() <= to)


@pytest.mark.parametrize("name", ["gqa128-group7", "mla-16-heads", "gqa80", "mha64-page5"])
def test_pages_outside_the_pool_are_left_out(name):
    for page in (-1, 2 ** 31 - 1, None):
        b = Batch(name, [(200, [100, 30])], seed=9)
        ps = b.lay.page_size
        at = 40 // ps
        b.dev()
        b.pool.page_table[0, at] = b.pages if page is None else page
        b.call()
        torch.cuda.synchronize()
        assert int(b.st.item()) == km.KAMERA_DEVICE_SLOT_OOB
        b.check(leave=np.arange(at * ps, (at + 1) * ps))  # the prefix is read through row 0


@pytest.mark.parametrize("name", ["gqa128-group7", "mla-16-heads", "gqa80"])
def test_contexts_that_break_the_rules_are_not_written(name):
    b = Batch(name, [(100, [10, 20, 30, 0]), (20, [5])], seed=10)
    b.dev()
    ctx = b.args[3]
    ctx[1], ctx[2] = 99, -1
    b.call()
    torch.cuda.synchronize()
    assert int(b.st.item()) == km.KAMERA_DEVICE_BAD_ITEM
    b.check(reqs=[0, 3, 4])
    assert torch.all(b.out[1:3] == -7) and torch.all(b.lse[1:3] == -7)
    for r, c in ((0, b.stride * b.lay.page_size + 1), (4, 2 ** 31 - 1)):
        b = Batch(name, [(100, [10, 20, 30, 0]), (20, [5])], seed=10)
        b.dev()
        b.args[3][r] = c
        b.call()
        torch.cuda.synchronize()
        assert int(b.st.item()) == km.KAMERA_DEVICE_BAD_ITEM
        b.check(reqs=[x for x in range(5) if x != r])
        assert torch.all(b.out[r] == -7)
    for prefix in (-1, 2 ** 31 - 1):
        b = Batch(name, [(100, [10, 20, 30, 0]), (20, [5])], seed=10)
        b.dev()
        b.args[2][0] = prefix
        b.call()
        torch.cuda.synchronize()
        assert int(b.st.item()) == km.KAMERA_DEVICE_BAD_ITEM
        b.check(reqs=[4])
        assert torch.all(b.out[:4] == -7)


@pytest.mark.parametrize("start", [[0, 3, 2, 5], [1, 2, 3, 5], [0, 1, 2, 4], [0, 2, 9, 5],
                                   [0, -1, 2, 5], [0, 1, 2, 6]])
def test_groups_that_are_no_partition_write_nothing(start):
    b = Batch("gqa128-group7", [(10, [1, 2]), (0, [3]), (5, [1, 1])], seed=11)
    b.dev()
    b.args[1].copy_(torch.as_tensor(start, dtype=torch.int32))
    b.call()
    torch.cuda.synchronize()
    assert int(b.st.item()) == km.KAMERA_DEVICE_BAD_ITEM
    assert torch.all(b.out == -7) and torch.all(b.lse == -7)


def test_empty_groups_between_others():
    b = Batch("gqa128-group7", [(10, [1, 2]), (9, []), (0, [3]), (40, []), (5, [1, 1])], seed=12)
    assert b.run() == 0
    b.check()


@pytest.mark.parametrize("name", ["gqa128-group7", "mla-16-heads", "gqa80"])
def test_agrees_with_decode_attention_and_repeats_its_bits(name):
    b = Batch(name, [(300, [40, 1, 200]), (0, [77])], seed=13)
    assert b.run() == 0
    first, lse = b.out.clone(), b.lse.clone()
    R, mx = len(b.ctx), int(b.ctx.max())
    out = torch.empty(R, b.hq, b.dv, device="cuda")
    l2 = torch.empty(R, b.hq, device="cuda")
    w = torch.empty(km.kamera_decode_attention_workspace(b.h, R, b.hq, mx), dtype=torch.uint8,
                    device="cuda")
    km.kamera_decode_attention(b.h, b.pool, b.layer, b.args[0], b.args[3], mx, b.scale, out, l2,
                               w, b.st)
    assert float((out - first.float()).abs().max()) <= 2.0 ** -6 * float(b.k.nan_to_num(0).abs().max())
    assert float((l2 - lse).abs().max()) <= 2.0 ** -7
    b.ws.random_(0, 255)
    b.call()
    assert torch.equal(b.out.view(torch.int16), first.view(torch.int16)) and torch.equal(b.lse, lse)


@pytest.mark.parametrize("name", ["gqa128-group7", "mla-16-heads"])
def test_other_stream_and_graph_replay(name):
    b = Batch(name, [(300, [40, 1, 200]), (0, [77])], seed=14)
    s = torch.cuda.Stream()
    assert b.run(stream=s) == 0
    b.check()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        b.call()
    # another batch in the same buffers: shorter contexts, other queries
    b.ctx = b.ctx - np.array([40, 0, 100, 76])
    b.args[3].copy_(torch.as_tensor(b.ctx, dtype=torch.int32))
    b.q = (b.q.float() * 0.5).to(torch.bfloat16)
    b.args[0].copy_(b.q)
    b.out.fill_(-7)
    graph.replay()
    torch.cuda.synchronize()
    b.check()


def test_two_streams_at_once():
    x = [Batch("gqa128-group7", [(1000, [40, 1, 200]), (0, [77])], seed=20 + i) for i in range(2)]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for b in x:
        b.dev()
    torch.cuda.synchronize()
    for _ in range(5):
        for b, s in zip(x, streams):
            b.call(stream=s)
    torch.cuda.synchronize()
    for b in x:
        assert int(b.st.item()) == 0
        b.check()


def test_refusals():
    b = Batch("gqa128-group7", [(10, [1, 2]), (0, [3])], seed=15)
    b.dev()
    q, start, prefix, ctx = b.args

    def call(q=q, start=start, prefix=prefix, ctx=ctx, out=b.out, lse=b.lse, ws=b.ws, st=b.st,
             layer=0, scale=0.1):
        km.kamera_prefix_attention(b.h, b.pool, layer, q, start, prefix, ctx, scale, out, lse, ws,
                                   st)

    for kw in (dict(q=q.float()), dict(q=q[..., :64].contiguous()), dict(q=q[:, ::2]),
               dict(start=start[:-1]), dict(start=start.long()), dict(prefix=prefix.cpu()),
               dict(ctx=ctx[:2]), dict(out=b.out.float()), dict(lse=b.lse.double()),
               dict(ws=b.ws.cpu()), dict(st=b.st.long())):
        with pytest.raises(ValueError):
            call(**kw)
    for kw in (dict(layer=2), dict(layer=-1), dict(scale=float("inf")), dict(scale=float("nan")),
               dict(ws=b.ws[:-16]), dict(ws=None),
               dict(start=start[[0, 1, 2, 2, 2]].contiguous(), prefix=prefix[[0, 1, 0, 0]].contiguous())):
        with pytest.raises(km.KameraError) as e:
            call(**kw)
        assert e.value.status == km.KAMERA_ERR_INVALID_ARG
    with pytest.raises(km.KameraError):  # heads that the KV heads do not divide
        call(q=q[:, :27].contiguous(), out=b.out[:, :27].contiguous(), lse=b.lse[:, :27].contiguous())
    torch.cuda.synchronize()
    assert torch.all(b.out == -7) and int(b.st.item()) == 0


@pytest.mark.parametrize("groups,prefix,size,step", [
    (1, 3000, 41, 0), (1, 640, 130, 0), (3, 2000, 9, 0), (40, 300, 6, 0), (2, 129, 64, 0),
    (3, 1500, 12, 700), (9, 128, 9, 130), (2, 100, 40, 5000), (20, 400, 7, 37)])
@pytest.mark.parametrize("name", ["gqa128-group7", "gqa64-group3", "mla-16-heads"])
def test_wide_blocks_with_workers_of_their_own(name, groups, prefix, size, step):
    # wide blocks of prefixes alone, of one length and of several: each is shared out among workers
    # of its own where there are workers enough for that
    b = Batch(name, [(prefix + k * step, [(3 * i + k) % 5 for i in range(size)])
                     for k in range(groups)], seed=15)
    assert b.run() == 0
    n = groups * size
    b.check(reqs=sorted({0, 1, size - 1, size // 2, n // 2, n - size, n - 1} & set(range(n))))


@pytest.mark.parametrize("name", ["gqa128-group7", "mla-16-heads", "gqa80"])
def test_workspace_at_any_16_bytes_and_nothing_behind_it(name):
    b = Batch(name, [(300, [40, 1, 200, 7, 9, 4, 4, 4]), (0, [77])], seed=16)
    size = len(b.ws)
    for at in (16, 48, 112, 128):
        room = torch.full((size + 512,), 0x5A, dtype=torch.uint8, device="cuda")
        b.ws = room[at:at + size]
        assert b.run() == 0
        b.check()
        assert torch.all(room[:at] == 0x5A) and torch.all(room[at + size:] == 0x5A)
