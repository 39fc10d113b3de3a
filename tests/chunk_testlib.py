"""Batches of new tokens over a paged pool, and what attention over them is in float64."""
import math

import numpy as np
import torch

import position_independent_multimodal_gb300 as km
import workloads as wl


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
    "gqa128-200-heads": (gqa(128, 1, page=256), 200),
    "gqa64-group3": (gqa(64, 2), 6),
    "mha64-page5": (gqa(64, 5, page=5), 5),
    "gqa80": (gqa(80, 2), 6),
    "gqa16": (gqa(16, 1), 1),
    "gqa256": (gqa(256, 1, page=128), 9),
    "gqa96-100-heads": (gqa(96, 1, page=8), 100),
    "mla-16-heads": (mla(512, 64), 16),
    "mla-128-heads": (mla(512, 64, page=64), 128),
    "mla-130-heads-page3": (mla(512, 64, page=3), 130),
    "mla-narrow": (mla(96, 32), 5),
    "mla-wide": (mla(768, 256, page=7), 3),
}


def tensor_path(lay):
    return (lay.kind == wl.GQA and lay.head_dim in (64, 128)) or \
        (lay.kind == wl.MLA and (lay.latent_dim, lay.rope_dim) == (512, 64))


def i32(x):
    return torch.as_tensor(np.asarray(x), dtype=torch.int32).cuda()


class Chunks:
    """Requests of (new tokens, tokens before them) over a pool whose unheld rows are `outside`."""

    def __init__(self, name, reqs, window=0, seed=0, sharp=1.0, outside=float("nan"), layer=1,
                 pad=3, before=0, stride=None, scale=None):
        self.lay, self.hq = lay, hq = LAYOUTS[name]
        self.layer, self.window = layer, window
        ps = lay.page_size
        g = torch.Generator().manual_seed(seed)
        rs = np.random.RandomState(seed)
        self.new = np.array([n for n, _ in reqs])
        self.ctx = np.array([n + p for n, p in reqs])
        self.start = before + np.cumsum([0] + list(self.new))
        R, rows = len(reqs), int(self.start[-1]) + pad
        n = -(-self.ctx // ps)
        pages = int(n.sum()) + 3
        self.table = np.full((R, int(max(n.max(), 1)) + 1), -1, np.int64)
        perm, at = rs.permutation(pages), 0
        for r, k in enumerate(n):
            self.table[r, :k] = perm[at:at + k]
            at += k
        slots = pages * ps
        self.k = torch.full((lay.num_layers, slots, lay.row_k), outside, dtype=torch.bfloat16)
        self.v = torch.full((lay.num_layers, slots, lay.row_v), outside, dtype=torch.bfloat16) \
            if lay.kind == wl.GQA else None
        for r in range(R):
            idx = torch.as_tensor(self.slots(r))
            for x in (self.k, self.v):
                if x is not None and len(idx):
                    x[:, idx] = wl.normal_bf16((x.shape[0], len(idx), x.shape[2]), 1.0, g, "cpu")
        mk = lay.kind == wl.GQA
        self.H = lay.num_kv_heads if mk else 1
        self.dk = lay.head_dim if mk else lay.latent_dim + lay.rope_dim
        self.dv = lay.head_dim if mk else lay.latent_dim
        self.rows = rows
        wide = stride or hq * self.dk  # elements between tokens
        self.q_full = torch.full((rows, wide), float("nan"), dtype=torch.bfloat16)
        a, b = int(self.start[0]), int(self.start[-1])
        self.q_full[a:b, :hq * self.dk] = wl.normal_bf16((b - a, hq * self.dk), sharp, g, "cpu")
        self.scale = 1 / math.sqrt(self.dk) if scale is None else scale
        self.h = km.create(lay)
        self.out = torch.full((rows, hq, self.dv), -7.0, dtype=torch.bfloat16, device="cuda")
        self.lse = torch.full((rows, hq), -7.0, device="cuda")
        self.st = torch.zeros(1, dtype=torch.int32, device="cuda")
        w = km.kamera_chunk_attention_workspace(self.h, rows, R, hq)
        self.ws = torch.full((w,), 0xFF, dtype=torch.uint8, device="cuda")

    def slots(self, r):
        t = np.arange(self.ctx[r])
        ps = self.lay.page_size
        return self.table[r, t // ps] * ps + t % ps

    def dev(self):
        self.pool = km.Pool(self.k.cuda(), None if self.v is None else self.v.cuda(),
                            i32(self.table))
        self.q = self.q_full.cuda()[:, :self.hq * self.dk].unflatten(1, (self.hq, self.dk))
        self.d_start, self.d_ctx = i32(self.start), i32(self.ctx)
        return self

    def call(self, **kw):
        km.kamera_chunk_attention(self.h, self.pool, self.layer, self.q, self.d_start, self.d_ctx,
                                  self.scale, self.out, self.lse, self.ws, self.st,
                                  window=self.window, **kw)

    def run(self, **kw):
        self.dev()
        self.call(**kw)
        torch.cuda.synchronize()
        return self

    def exact(self, r):
        """(scores [tokens][hq][ctx], -inf where not seen, their error bound B [tokens][hq], values
        [H][ctx][dv], 0 where they are not finite) of request r in float64, on the GPU. Tokens in
        pages outside the pool are not seen."""
        c, n = int(self.ctx[r]), int(self.new[r])
        ps = self.lay.page_size
        t = np.arange(c)
        page = self.table[r, t // ps]
        have = (page >= 0) & (page < self.k.shape[1] // ps)
        slot = torch.as_tensor(np.where(have, page * ps + t % ps, 0))
        k = self.k[self.layer, slot].cuda().double().view(c, self.H, self.dk)
        v = self.v[self.layer, slot].cuda().double().view(c, self.H, self.dv) \
            if self.v is not None else k[..., :self.dv]
        a = int(self.start[r])
        q = self.q_full[a:a + n, :self.hq * self.dk].cuda().double()
        q = q.view(n, self.H, self.hq // self.H, self.dk)
        me = torch.arange(c - n, c)[:, None]
        u = torch.arange(c)[None]
        sees = (u <= me) & torch.as_tensor(have)[None]
        if self.window:
            sees &= u > me - self.window
        sees = sees.cuda()[:, None, None]
        x = self.scale * torch.einsum("nhgd,chd->nhgc", q, k)
        b = torch.einsum("nhgd,chd->nhgc", q.abs(), torch.nan_to_num(k.abs(), 0.0, 0.0))
        b = b * abs(self.scale) * (self.dk + 1) * 2.0 ** -24
        x = torch.where(sees, x, -math.inf).flatten(1, 2)
        b = torch.where(sees, b, 0.0).flatten(1, 2)
        return x, b.amax(-1), torch.nan_to_num(v.permute(1, 0, 2), 0.0, 0.0, 0.0)
