"""Cases and plain forms of the operators around a cache that grows in chunks and is cut back.

Three families, as a serving step uses them one after the other:

* ``chunk``: attention of new tokens over the paged pool. Each request's new tokens are the last of
  its context, from one (decoding) to a whole prompt; each sees the tokens before it and itself, or
  the last ``window`` of them. Requests of both kinds share a batch.
* ``mass``: the attention weight that the new tokens lay on each cached token, summed over their
  query heads (the weights are taken again from the log-sum-exp that attention left).
* ``evict``: requests over their budget keep their first and last tokens and those of the greatest
  mass; the rows that stay are drawn together in every layer, their masses with them.

Layouts are those of the reference workloads: 28 query heads over 4 KV heads of 128 (28 layers),
32 over 8 of 128 (64 layers), 32 heads of 128 each with its own KV head, 6 query heads over 2 KV
heads of 64, and the latent layout of 512 + 64 with 16 heads. The data are bf16 throughout.
"""
import math

import numpy as np
import torch

own = False

PAGE = 16

# query heads, KV heads, head dim; KV heads 0 is the latent layout (512 + 64)
LAYOUTS = {
    "gqa128": (28, 4, 128),
    "gqa128w": (32, 8, 128),
    "mha128": (32, 32, 128),
    "gqa64": (6, 2, 64),
    "mla": (16, 0, 512),
}
LATENT, PE = 512, 64


def listed():
    return [
        # one decode step of a few users over short contexts: latency alone counts
        {"name": "chunk decode 8 x 700", "op": "chunk", "layout": "gqa128", "reqs": 8, "single": 8, "new": 1, "past": 700, "window": 0, "ragged": 1},
        # a full serving batch: most requests decode, a few bring in a piece of their prompt
        {"name": "chunk mixed 40", "op": "chunk", "layout": "gqa128w", "reqs": 40, "single": 36, "new": 511, "past": 8000, "window": 0, "ragged": 2},
        # the next piece of one very long prompt: the largest
        {"name": "chunk 2011 over 60000", "op": "chunk", "layout": "gqa128", "reqs": 1, "single": 0, "new": 2011, "past": 60000, "window": 0, "ragged": 3},
        # whole prompts from nothing, every head with keys of its own
        {"name": "chunk prompts MHA 3 x 4001", "op": "chunk", "layout": "mha128", "reqs": 3, "single": 0, "new": 4001, "past": 0, "window": 0, "ragged": 4},
        # pieces of prompts of a latent-attention model
        {"name": "chunk MLA 4 x 300 over 9003", "op": "chunk", "layout": "mla", "reqs": 4, "single": 0, "new": 300, "past": 9003, "window": 0, "ragged": 5},
        # narrow heads with a sliding window
        {"name": "chunk 64-wide window 1000", "op": "chunk", "layout": "gqa64", "reqs": 5, "single": 1, "new": 3001, "past": 5000, "window": 1000, "ragged": 6},
        # masses of a decoding batch
        {"name": "mass decode 32 x 6001", "op": "mass", "layout": "gqa128", "reqs": 32, "single": 32, "new": 1, "past": 6001, "window": 0, "ragged": 7},
        # a long prompt judged by its last piece
        {"name": "mass 250 over 30000", "op": "mass", "layout": "gqa128", "reqs": 1, "single": 0, "new": 250, "past": 30000, "window": 0, "ragged": 8},
        # the same of latent rows, several requests
        {"name": "mass MLA 6 x 100 over 5000", "op": "mass", "layout": "mla", "reqs": 6, "single": 2, "new": 100, "past": 5000, "window": 0, "ragged": 9},
        # one request a little over its budget
        {"name": "evict 1 x 701 to 600", "op": "evict", "layout": "gqa128", "layers": 28, "reqs": 1, "tokens": 701, "keep": 0.856, "first": 4, "last": 64, "ties": 0, "ragged": 10},
        # a full batch cut to half
        {"name": "evict 20 x 4000 to half", "op": "evict", "layout": "gqa128", "layers": 28, "reqs": 20, "tokens": 4000, "keep": 0.5, "first": 4, "last": 128, "ties": 0, "ragged": 11},
        # long contexts of a latent-attention model cut to a quarter, many masses equal
        {"name": "evict MLA 6 x 30000 to quarter", "op": "evict", "layout": "mla", "layers": 27, "reqs": 6, "tokens": 30000, "keep": 0.25, "first": 16, "last": 500, "ties": 1, "ragged": 12},
    ]


def _log(rng, a, b):
    return int(round(math.exp(rng.uniform(math.log(a), math.log(b)))))


def draw(rng):
    op = rng.choice(["chunk", "chunk", "chunk", "chunk", "mass", "mass", "mass", "evict", "evict"])
    lay = rng.choice(sorted(LAYOUTS))
    if op == "evict":
        tokens = _log(rng, 2, 20000 if lay != "mha128" else 6000)
        layers = rng.randint(1, {"mha128": 6, "gqa128w": 32}.get(lay, 28))
        # at most the rows of the largest listed case
        row = sum(_rows(lay)) * layers
        reqs = rng.randint(1, max(1, min(24, int(1.5e9 / (row * tokens)))))
        first = rng.randint(0, min(tokens // 4, 20))
        return {"op": op, "layout": lay, "layers": layers, "reqs": reqs, "tokens": tokens, "keep": round(rng.uniform(0.05, 1.0), 3),
                "first": first, "last": rng.randint(0, min(tokens // 4, 300)), "ties": rng.randint(0, 1), "ragged": rng.randint(1, 10000)}
    reqs = _log(rng, 1, 60)
    new = _log(rng, 1, 4000 if op == "chunk" else 400)
    past = 0 if rng.random() < 0.2 else _log(rng, 1, {"mha128": 6000, "mla": 12000}.get(lay, 30000))
    c = {"op": op, "layout": lay, "reqs": reqs, "single": rng.randint(0, reqs), "new": new, "past": past,
         "window": _log(rng, 1, 5000) if rng.random() < 0.25 else 0, "ragged": rng.randint(1, 10000)}
    while work(c)["flops"] > (1.6e12 if op == "chunk" else 2e11) or work(c)["bytes"] > 2e9:
        c["new"], c["reqs"] = max(1, c["new"] // 2), max(1, c["reqs"] * 3 // 4)
        c["single"] = min(c["single"], c["reqs"])
    return c


# ---------------------------------------------------------------------------------------
# sizes
# ---------------------------------------------------------------------------------------

def _rows(lay):
    """Widths of a K row and a V row of the pool (V: 0 in the latent layout)."""
    hq, hkv, d = LAYOUTS[lay]
    return (hkv * d, hkv * d) if hkv else (LATENT + PE, 0)


def _widths(lay):
    """(columns of a query head and of its output, KV heads, query heads of one of them)."""
    hq, hkv, d = LAYOUTS[lay]
    return (d, d, hkv, hq // hkv) if hkv else (LATENT + PE, LATENT, 1, hq)


def _ceil(a, b):
    return -(-a // b)


def _lens(case):
    """(new tokens, context) of each request: the first `single` bring one token each, the others
    between half of the case's and all of it; contexts before them likewise."""
    rs = np.random.RandomState(case["ragged"])
    R, n, p = case["reqs"], case["new"], case["past"]
    new = rs.randint(_ceil(n, 2), n + 1, R)
    past = rs.randint(p // 2, p + 1, R)
    new[-1], past[-1] = n, p
    new[:case["single"]] = 1
    return new, past + new


def _kept(case):
    """(tokens, kept tokens, protected first, protected last) of each request."""
    rs = np.random.RandomState(case["ragged"])
    tokens = rs.randint(_ceil(case["tokens"], 2), case["tokens"] + 1, case["reqs"])
    tokens[0] = case["tokens"]
    first, last = np.minimum(case["first"], tokens // 4), np.minimum(case["last"], tokens // 4)
    keep = np.maximum((tokens * case["keep"]).astype(np.int64), first + last)
    return tokens, keep, first, last


def _seen(case):
    """Pairs of a new token and a token that it sees, over the batch."""
    new, ctx = _lens(case)
    total = 0
    for n, c in zip(new, ctx):
        sees = np.arange(c - n + 1, c + 1, dtype=np.int64)
        total += int((np.minimum(sees, case["window"]) if case["window"] else sees).sum())
    return total


def _read(case):
    """Cached tokens that some new token sees, over the batch."""
    new, ctx = _lens(case)
    return int(np.minimum(ctx, case["window"] + new - 1).sum()) if case["window"] else int(ctx.sum())


def work(case):
    lay = case["layout"]
    rk, rv = _rows(lay)
    if case["op"] == "evict":
        tokens, keep, first, last = _kept(case)
        moved = int(np.where(keep < tokens, keep - first, 0).sum())
        return {"bytes": moved * 2 * case["layers"] * 2 * (rk + rv) + int((8 * tokens + 4 * keep).sum()), "flops": 0}
    dk, dv, H, hpk = _widths(lay)
    new, ctx = _lens(case)
    T, hq = int(new.sum()), H * hpk
    if case["op"] == "chunk":
        return {"bytes": _read(case) * 2 * (rk + rv) + T * hq * (2 * dk + 2 * dv + 4) + 4 * int(_ceil(ctx, PAGE).sum()),
                "flops": 2 * hq * (dk + dv) * _seen(case)}
    return {"bytes": _read(case) * 2 * rk + T * hq * (2 * dk + 4) + 4 * int(ctx.sum()) + 4 * int(_ceil(ctx, PAGE).sum()),
            "flops": 2 * hq * dk * _seen(case)}


# ---------------------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------------------

class State:
    pass


def _handle(lay, layers):
    import position_independent_multimodal_gb300 as km

    hq, hkv, d = LAYOUTS[lay]

    class Layout:
        kind = km.KAMERA_GQA if hkv else km.KAMERA_MLA
        num_layers, page_size = layers, PAGE
        num_kv_heads, head_dim = hkv, d if hkv else 0
        latent_dim, rope_dim = 0 if hkv else LATENT, d if hkv else PE
        rope_style, rope_theta = km.KAMERA_ROPE_NEOX_HALF, 1e6

    return km, km.create(Layout)


def _pool(lay, layers, pages, gen):
    rk, rv = _rows(lay)
    k = torch.randn(layers, pages * PAGE, rk, generator=gen, device="cuda", dtype=torch.bfloat16)
    v = torch.randn(layers, pages * PAGE, rv, generator=gen, device="cuda", dtype=torch.bfloat16) if rv else None
    return k, v


def _ints(x, dtype=torch.int32):
    return torch.as_tensor(np.ascontiguousarray(x), dtype=dtype).cuda()


def _table(lens, rs, spare):
    """A page table in which each request's pages lie anywhere, and the pages of its pool."""
    n = _ceil(np.asarray(lens), PAGE)
    pages = int(n.sum()) + spare
    table = np.full((len(n), int(n.max()) + 1), -1, np.int64)
    perm, at = rs.permutation(pages), 0
    for r, k in enumerate(n):
        table[r, :k] = perm[at:at + k]
        at += k
    return table, pages


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    rs = np.random.RandomState(seed % (1 << 31))
    s = State()
    s.case, s.lay = case, case["layout"]
    (_prepare_evict if case["op"] == "evict" else _prepare_attend)(s, case, gen, rs)
    if own:
        s.km, s.handle = _handle(s.lay, s.k.shape[0])
        s.pool = s.km.Pool(s.k, s.v, s.table)
        s.status = torch.zeros(1, dtype=torch.int32, device="cuda")
        if case["op"] == "chunk":
            n = s.km.kamera_chunk_attention_workspace(s.handle, s.q.shape[0], case["reqs"], s.q.shape[1])
        elif case["op"] == "mass":
            n = s.km.kamera_attention_mass_workspace(s.handle, s.q.shape[0], case["reqs"], s.q.shape[1])
        else:
            n = s.km.kamera_evict_workspace(s.handle, case["reqs"])
        s.work = torch.empty(max(n, 1), dtype=torch.uint8, device="cuda")
    return s


def _prepare_attend(s, case, gen, rs):
    dk, dv, H, hpk = _widths(s.lay)
    new, ctx = _lens(case)
    table, pages = _table(ctx, rs, 3)
    s.k, s.v = _pool(s.lay, 2, pages, gen)
    s.layer = 1
    s.new, s.ctx = new, ctx  # what the scheduler knows of the batch
    s.table, s.ctx_len = _ints(table), _ints(ctx)
    s.start = _ints(np.concatenate([[0], np.cumsum(new)]))
    rows = _ceil(int(new.sum()), 8) * 8  # a batch's rows, padded as a captured step keeps them
    hq = H * hpk
    # the queries where the projection left them, keys and values beside them
    wide = hq + 2 * H if s.v is not None else hq
    s.q = (1.5 * torch.randn(rows, wide, dk, generator=gen, device="cuda")).to(torch.bfloat16)[:, :hq]
    s.scale = 1 / math.sqrt(dk if s.v is not None else 192)
    s.out = torch.zeros(rows, hq, dv, dtype=torch.bfloat16, device="cuda")
    s.lse = torch.zeros(rows, hq, dtype=torch.float32, device="cuda")
    if case["op"] == "mass":
        for r, lo, hi, x in _scores(s):
            s.lse[lo:hi] = torch.logsumexp(x, -1).permute(1, 0, 2).flatten(1)
        s.mass = torch.zeros(case["reqs"], int(ctx.max()) + 5, dtype=torch.float32, device="cuda")


def _prepare_evict(s, case, gen, rs):
    tokens, keep, first, last = _kept(case)
    table, pages = _table(tokens, rs, 3)
    s.k, s.v = _pool(s.lay, case["layers"], pages, gen)
    s.table = _ints(table)
    refs = np.zeros(pages, np.int64)
    refs[table[table >= 0]] = 1
    s.refs = _ints(refs)
    s.sizes = list(zip(tokens, keep, first, last))
    s.items = _ints(np.stack([np.arange(len(tokens)), tokens, keep, first, last], 1))
    width = int(tokens.max()) + 3
    # sums of attention weights: a few tokens hold most of the mass
    m = torch.exp(2.5 * torch.randn(len(tokens), width, generator=gen, device="cuda"))
    if case["ties"]:  # as weights that were kept in a few bits, many of them none
        m = torch.floor(4 * m) / 4
    s.mass0 = m * (torch.arange(width, device="cuda") < _ints(tokens)[:, None])
    s.mass = s.mass0.clone()
    s.kept = torch.full((len(tokens), int(keep.max())), -1, dtype=torch.int32, device="cuda")


# ---------------------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------------------

def run(s):
    return {"chunk": _run_chunk, "mass": _run_mass, "evict": _run_evict}[s.case["op"]](s)


def _scores(s):
    """For each request, a piece of its new tokens at a time: (request, first row, end row, scores
    [KV heads][tokens][query heads of one][context]), minus infinity where a token is not seen."""
    dk, dv, H, hpk = _widths(s.lay)
    at = 0
    for r, (n, c) in enumerate(zip(s.new.tolist(), s.ctx.tolist())):
        t = torch.arange(c, device="cuda")
        k = s.k[s.layer][s.table[r].long()[t // PAGE] * PAGE + t % PAGE].float().view(c, H, dk)
        step = max(1, (1 << 28) // (H * hpk * c))
        for lo in range(0, n, step):
            hi = min(n, lo + step)
            q = s.q[at + lo:at + hi].float().view(hi - lo, H, hpk, dk).permute(1, 0, 2, 3)
            x = torch.matmul(q.reshape(H, -1, dk), k.permute(1, 2, 0)).mul_(s.scale).view(H, hi - lo, hpk, c)
            me = torch.arange(c - n + lo, c - n + hi, device="cuda")[:, None]
            hide = t > me
            if s.case["window"]:
                hide |= t <= me - s.case["window"]
            yield r, at + lo, at + hi, x.masked_fill_(hide[:, None], -math.inf)
        at += n


def _run_chunk(s):
    if own:
        s.km.kamera_chunk_attention(s.handle, s.pool, s.layer, s.q, s.start, s.ctx_len, s.scale, s.out, s.lse, s.work, s.status,
                                    window=s.case["window"])
        return {"out": s.out, "lse": s.lse}
    dk, dv, H, hpk = _widths(s.lay)
    for r, lo, hi, x in _scores(s):
        c = x.shape[-1]
        t = torch.arange(c, device="cuda")
        slots = s.table[r].long()[t // PAGE] * PAGE + t % PAGE
        v = (s.k[s.layer][slots, :LATENT] if s.v is None else s.v[s.layer][slots]).float().view(c, H, dv)
        top = x.amax(-1, keepdim=True)
        p = x.sub_(top).exp_()
        total = p.sum(-1, keepdim=True)
        o = torch.matmul(p.flatten(1, 2), v.permute(1, 0, 2)).view(H, hi - lo, hpk, dv) / total
        s.out[lo:hi] = o.permute(1, 0, 2, 3).flatten(1, 2).to(torch.bfloat16)
        s.lse[lo:hi] = (top + total.log())[..., 0].permute(1, 0, 2).flatten(1)
    return {"out": s.out, "lse": s.lse}


def _run_mass(s):
    if own:
        s.km.kamera_attention_mass(s.handle, s.pool, s.layer, s.q, s.start, s.ctx_len, s.scale, s.lse, 0.0, s.mass, s.work, s.status,
                                   window=s.case["window"])
        return {"mass": s.mass}
    dk, dv, H, hpk = _widths(s.lay)
    for r, c in enumerate(s.ctx.tolist()):
        s.mass[r, :c] = 0
    for r, lo, hi, x in _scores(s):
        lse = s.lse[lo:hi].view(hi - lo, H, hpk).permute(1, 0, 2)
        s.mass[r, :x.shape[-1]] += x.sub_(lse[..., None]).exp_().sum((0, 1, 2))
    return {"mass": s.mass}


def _pools(s):
    return {"k": s.k} if s.v is None else {"k": s.k, "v": s.v}


def _run_evict(s):
    s.mass.copy_(s.mass0)
    if own:
        s.km.kamera_evict(s.handle, s.pool, s.items, s.refs, s.mass, s.kept, s.work, s.status)
        return {"kept": s.kept, "mass": s.mass, **_pools(s)}
    for r, (n, keep, first, last) in enumerate(s.sizes):
        if keep >= n:
            s.kept[r, :n] = torch.arange(n, device="cuda", dtype=torch.int32)
            continue
        m = s.mass[r, :n].clone()
        m[:first], m[n - last:] = math.inf, math.inf
        to = torch.sort(torch.sort(m, descending=True, stable=True).indices[:keep]).values
        s.kept[r, :keep] = to.int()
        s.mass[r, :keep] = s.mass[r, to]
        s.mass[r, keep:n] = 0
        t = torch.arange(keep, device="cuda")
        row = s.table[r].long()
        src, dst = row[to // PAGE] * PAGE + to % PAGE, row[t // PAGE] * PAGE + t % PAGE
        for x in (s.k, s.v):
            if x is not None:
                x.index_copy_(1, dst, x.index_select(1, src))
    return {"kept": s.kept, "mass": s.mass, **_pools(s)}


# ---------------------------------------------------------------------------------------
# the definitions in 64 bits
# ---------------------------------------------------------------------------------------

def exact(case, seed):
    if case["op"] == "evict":
        return None  # rows and masses move whole: nothing is computed
    s = prepare(case, seed)
    dk, dv, H, hpk = _widths(s.lay)
    table = s.table.cpu().numpy().astype(np.int64)
    new, ctx = _lens(case)
    out, lse = s.out.double(), s.lse.double()
    mass = s.mass.double() if case["op"] == "mass" else None
    first = 0
    for r in range(len(new)):
        c, n = int(ctx[r]), int(new[r])
        t = np.arange(c)
        slot = torch.as_tensor(table[r, t // PAGE] * PAGE + t % PAGE).cuda()
        keys = s.k[s.layer].index_select(0, slot).double()
        values = keys[:, :LATENT] if s.v is None else s.v[s.layer].index_select(0, slot).double()
        many = max(1, (1 << 26) // c)
        for h in range(H * hpk):
            g = h // hpk
            for i in range(0, n, many):
                rows = slice(first + i, first + min(n, i + many))
                x = s.scale * (s.q[rows, h].double() @ keys[:, g * dk:(g + 1) * dk].T)
                who = np.arange(c - n + i, c - n + min(n, i + many))[:, None]
                sees = (t[None] <= who) & ((t[None] > who - case["window"]) if case["window"] else True)
                x = torch.where(torch.as_tensor(sees).cuda(), x, -math.inf)
                if mass is not None:
                    mass[r, :c] += torch.exp(x - s.lse[rows, h, None].double()).sum(0)
                    continue
                z = torch.logsumexp(x, -1)
                out[rows, h] = torch.exp(x - z[:, None]) @ values[:, g * dv:(g + 1) * dv]
                lse[rows, h] = z
        first += n
    return {"out": out, "lse": lse} if mass is None else {"mass": mass}
