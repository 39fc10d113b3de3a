"""Cases and plain forms of the cache's serving operators.

Three families, as a serving step uses them one after the other:

* ``append``: the new tokens of a batch enter a layer of the paged pool. Queries and keys get
  their per-head RMS norm and the rotation to their positions in one pass (MLA: the norm of the
  latent and the rotation of the k_pe bands); keys and values land in the tokens' slots.
* ``beam``, ``compact``, ``copy``: pages of the pool. A beam step releases the children of the
  last step, forks the survivors (shared pages counted, the last partial page copied) and gives
  the children room to grow; compaction moves the live pages below the number of live pages;
  a copy duplicates listed pages.
* ``attend``: decode attention of a batch whose requests share long prefixes, each group's
  prefix attended once for all its requests, the rest of each context for itself.

Layouts are those of the reference workloads: 28 query heads over 4 KV heads of 128 (28 layers),
32 over 8 of 128 (64 layers), 32 heads of 128 each with its own KV head, 2 KV heads of 64, and
the latent layout of 512 + 64 with 16 heads. The data are bf16 throughout.
"""
import math

import numpy as np
import torch

own = False

PAGE = 16
EPS = 1e-6

# query heads, KV heads, head dim, rope base, M-RoPE sections; KV heads 0 is the latent layout
# (512 + 64)
LAYOUTS = {
    "gqa128": (28, 4, 128, 1e6, (0, 0, 0)),
    "gqa128m": (28, 4, 128, 1e6, (16, 24, 24)),
    "gqa128w": (32, 8, 128, 1e6, (0, 0, 0)),
    "mha128": (32, 32, 128, 1e4, (0, 0, 0)),
    "gqa64": (6, 2, 64, 1e4, (0, 0, 0)),
    "mla": (16, 0, 512, 1e4, (0, 0, 0)),
}
LATENT, PE = 512, 64


def listed():
    return [
        # one decode step of a few users: latency alone counts
        {"name": "append decode 8", "op": "append", "layout": "gqa128", "tokens": 8, "reqs": 8, "far": 30000},
        # a long prompt with image positions (t, h, w), ragged over five requests
        {"name": "append prompt M-RoPE 16381", "op": "append", "layout": "gqa128m", "tokens": 16381, "reqs": 5, "far": 200000},
        # prompts of a latent-attention model
        {"name": "append prompt MLA 5003", "op": "append", "layout": "mla", "tokens": 5003, "reqs": 3, "far": 100000},
        # beam search of one user
        {"name": "beam 2 x 4", "op": "beam", "layout": "gqa128", "layers": 28, "parents": 2, "children": 4, "ctx": 700, "grow": 1, "pages": 600},
        # parallel sampling for a full batch, a large pool
        {"name": "beam 24 x 16", "op": "beam", "layout": "gqa128w", "layers": 64, "parents": 24, "children": 16, "ctx": 1001, "grow": 12, "pages": 2600},
        # a fragmented pool drawn together
        {"name": "compact 9000", "op": "compact", "layout": "gqa128", "layers": 28, "reqs": 60, "ctx": 1700, "pages": 9000},
        # saved pages brought back beside their originals
        {"name": "copy MLA 500 pages", "op": "copy", "layout": "mla", "layers": 27, "n": 500, "pages": 3000},
        # a few users behind one short system prompt: the smallest
        {"name": "attend 4 x 200", "op": "attend", "layout": "gqa128", "reqs": 4, "groups": 1, "prefix": 200, "own": 20, "ragged": 3},
        # a batch behind three documents
        {"name": "attend 48 x 6001", "op": "attend", "layout": "gqa128", "reqs": 48, "groups": 3, "prefix": 6001, "own": 700, "ragged": 4},
        # many samples of one very long context: the largest
        {"name": "attend 128 x 65500", "op": "attend", "layout": "gqa128", "reqs": 128, "groups": 1, "prefix": 65500, "own": 500, "ragged": 5},
        # a latent-attention batch behind two documents
        {"name": "attend MLA 40 x 9003", "op": "attend", "layout": "mla", "reqs": 40, "groups": 2, "prefix": 9003, "own": 300, "ragged": 6},
        # narrow heads
        {"name": "attend 64-wide 33 x 4100", "op": "attend", "layout": "gqa64", "reqs": 33, "groups": 2, "prefix": 4100, "own": 90, "ragged": 7},
    ]


def _log(rng, a, b):
    return int(round(math.exp(rng.uniform(math.log(a), math.log(b)))))


def draw(rng):
    op = rng.choice(["append", "append", "beam", "compact", "copy", "attend", "attend", "attend"])
    lay = rng.choice(sorted(LAYOUTS))
    if op == "append":
        n = _log(rng, 1, 12000 if lay != "mha128" else 6000)
        return {"op": op, "layout": lay, "tokens": n, "reqs": rng.randint(1, min(n, 40)), "far": _log(rng, 10, 1000000)}
    if op == "beam":
        layers = rng.randint(2, 28 if lay != "mha128" else 8)
        p, c, ctx = rng.randint(1, 12), rng.randint(1, 12), _log(rng, 1, 2000)
        grow = rng.randint(0, 50)
        need = p * (-(-ctx // PAGE) + c * (2 + grow // PAGE))
        return {"op": op, "layout": lay, "layers": layers, "parents": p, "children": c, "ctx": ctx, "grow": grow,
                "pages": need + _log(rng, 20, 1500)}
    if op == "compact":
        reqs, ctx = rng.randint(1, 40), _log(rng, 20, 1200)
        return {"op": op, "layout": lay, "layers": rng.randint(1, 16 if lay != "mha128" else 4), "reqs": reqs, "ctx": ctx,
                "pages": reqs * -(-ctx // PAGE) + _log(rng, 10, 1500)}
    if op == "copy":
        n = _log(rng, 1, 600)
        return {"op": op, "layout": lay, "layers": rng.randint(1, 28 if lay != "mha128" else 6), "n": n, "pages": 2 * n + _log(rng, 4, 1000)}
    reqs = _log(rng, 1, 130)
    groups = rng.randint(1, min(reqs, 4))
    prefix = _log(rng, 1, {"mha128": 6000, "mla": 20000}.get(lay, 30000))
    return {"op": op, "layout": lay, "reqs": reqs, "groups": groups, "prefix": prefix,
            "own": _log(rng, 1, 900 if lay != "mha128" else 200), "ragged": rng.randint(1, 10000)}


# ---------------------------------------------------------------------------------------
# sizes
# ---------------------------------------------------------------------------------------

def _rows(lay):
    """Widths of a K row and a V row of the pool (V: 0 in the latent layout)."""
    hq, hkv, d, _, _ = LAYOUTS[lay]
    return (hkv * d, hkv * d) if hkv else (LATENT + PE, 0)


def _ceil(a, b):
    return -(-a // b)


def _attend_lens(case):
    """(first request of each group and the end, prefix of each group, context of each request):
    groups of nearly equal size, prefixes from 60 % of the case's, own tokens from one up."""
    rs = np.random.RandomState(case["ragged"])
    R, G = case["reqs"], case["groups"]
    start = np.array([R * g // G for g in range(G + 1)])
    prefix = np.maximum(1, (case["prefix"] * (1 - 0.4 * rs.rand(G))).astype(np.int64))
    prefix[0] = case["prefix"]
    group = np.repeat(np.arange(G), np.diff(start))
    ctx = prefix[group] + rs.randint(1, case["own"] + 1, R)
    return start, prefix, ctx


def _split(n, parts):
    """n tokens over `parts` requests, unevenly, none empty where there are enough."""
    w = np.arange(1, parts + 1, dtype=np.float64)
    c = np.maximum(1, np.floor(n * w / w.sum()).astype(np.int64))
    c[-1] += n - c.sum()
    return c if c[-1] > 0 else np.array([n // parts + (i < n % parts) for i in range(parts)])


def work(case):
    lay = case["layout"]
    hq, hkv, d, _, sec = LAYOUTS[lay]
    rk, rv = _rows(lay)
    if case["op"] == "append":
        T = case["tokens"]
        dq = d if hkv else LATENT + PE
        pos = 24 if sum(sec) else 8
        return {"bytes": T * (2 * 2 * (hq * dq + rk + rv) + pos + 8), "flops": T * 6 * (hq * dq + rk)}
    if case["op"] == "beam":
        ctx, n = _beam_ctx(case), case["children"]
        rows = sum(int(c) % PAGE for c in ctx) * n
        table = sum(_ceil(int(c), PAGE) for c in ctx) * n
        return {"bytes": rows * 2 * case["layers"] * 2 * (rk + rv) + 16 * table + 4 * case["pages"], "flops": 0}
    if case["op"] == "compact":
        refs, _ = _scattered(case, 0)
        live = int((refs > 0).sum())
        moved = int((refs[live:] > 0).sum())
        return {"bytes": moved * PAGE * case["layers"] * 2 * 2 * (rk + rv) + 8 * case["pages"] + 8 * int(refs.sum()), "flops": 0}
    if case["op"] == "copy":
        return {"bytes": case["n"] * (PAGE * case["layers"] * 2 * 2 * (rk + rv) + 8), "flops": 0}
    start, prefix, ctx = _attend_lens(case)
    group = np.repeat(np.arange(len(prefix)), np.diff(start))
    dk, dv = (d, d) if hkv else (LATENT + PE, LATENT)
    read = int(prefix.sum() + (ctx - prefix[group]).sum())
    return {"bytes": read * 2 * (rk + rv) + len(ctx) * hq * (2 * dk + 2 * dv + 4) + 4 * int(_ceil_all(ctx).sum()),
            "flops": 2 * hq * (dk + dv) * int(ctx.sum())}


def _ceil_all(x):
    return -(-x // PAGE)


def _beam_ctx(case):
    """Contexts of a beam step's parents: ragged, ending inside pages."""
    p = case["parents"]
    return np.array([max(1, case["ctx"] - (37 * i) % (1 + case["ctx"] // 2)) for i in range(p)])


def _scattered(case, seed):
    """(use counts of the pages, pages of each request) of a pool in which requests have come and
    gone: live pages lie anywhere, and pairs of neighbouring requests share their first half.
    The lengths and how many pages move go by the case alone, the places by the seed too."""
    rs = np.random.RandomState(1)
    lens = [max(1, int(case["ctx"] * (0.5 + 0.5 * rs.rand()))) for _ in range(case["reqs"])]
    n = [_ceil(x, PAGE) for x in lens]
    rows, taken = [], 0
    perm = rs.permutation(case["pages"])
    for r, k in enumerate(n):
        share = min(k, n[r - 1]) // 2 if r % 2 else 0
        mine = perm[taken:taken + k - share]
        taken += k - share
        rows.append(np.concatenate([rows[r - 1][:share], mine]) if share else mine)
    refs = np.zeros(case["pages"], np.int64)
    for row in rows:
        refs[row] += 1
    if seed:  # the same counts on each side of the border, elsewhere
        live = int((refs > 0).sum())
        rs = np.random.RandomState(seed % (1 << 31))
        to = np.concatenate([rs.permutation(live), live + rs.permutation(case["pages"] - live)])
        rows = [to[row] for row in rows]
        refs = np.zeros(case["pages"], np.int64)
        for row in rows:
            refs[row] += 1
    return refs, rows


# ---------------------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------------------

class State:
    pass


def _handle(lay, layers):
    import position_independent_multimodal_gb300 as km

    hq, hkv, d, theta, sec = LAYOUTS[lay]

    class Layout:
        kind = km.KAMERA_GQA if hkv else km.KAMERA_MLA
        num_layers, page_size = layers, PAGE
        num_kv_heads, head_dim = hkv, d if hkv else 0
        latent_dim, rope_dim = 0 if hkv else LATENT, d if hkv else PE
        rope_style, rope_theta = km.KAMERA_ROPE_NEOX_HALF, theta
        mrope_section, mrope_style = sec, km.KAMERA_MROPE_CONTIGUOUS

    return km, km.create(Layout)


def _pool(lay, layers, pages, gen):
    rk, rv = _rows(lay)
    k = torch.randn(layers, pages * PAGE, rk, generator=gen, device="cuda", dtype=torch.bfloat16)
    v = torch.randn(layers, pages * PAGE, rv, generator=gen, device="cuda", dtype=torch.bfloat16) if rv else None
    return k, v


def _ints(x, dtype=torch.int32):
    return torch.as_tensor(np.ascontiguousarray(x), dtype=dtype).cuda()


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    rs = np.random.RandomState(seed % (1 << 31))
    s = State()
    s.case, s.lay = case, case["layout"]
    hq, hkv, d, _, sec = LAYOUTS[s.lay]
    {"append": _prepare_append, "beam": _prepare_beam, "compact": _prepare_compact,
     "copy": _prepare_copy, "attend": _prepare_attend}[case["op"]](s, case, gen, rs, seed)
    if own:
        s.km, s.handle = _handle(s.lay, s.k.shape[0])
        s.pool = s.km.Pool(s.k, s.v, s.table)
        s.status = torch.zeros(1, dtype=torch.int32, device="cuda")
        if case["op"] == "attend":
            n = s.km.kamera_prefix_attention_workspace(s.handle, case["reqs"], hq)
            s.work = torch.empty(max(n, 1), dtype=torch.uint8, device="cuda")
        elif case["op"] in ("beam", "compact"):
            items = case["parents"] * case["children"] if case["op"] == "beam" else 0
            n = s.km.kamera_page_workspace(s.handle, s.k.shape[1], items)
            s.work = torch.empty(max(n, 1), dtype=torch.uint8, device="cuda")
    return s


def _prepare_append(s, case, gen, rs, seed):
    hq, hkv, d, _, sec = LAYOUTS[s.lay]
    T, R = case["tokens"], case["reqs"]
    new = _split(T, R)
    old = 7 * np.arange(R) % 40  # tokens that the requests hold already
    stride = int(max(_ceil(int(a + b), PAGE) for a, b in zip(old, new)))
    pages = R * stride
    s.table = _ints(rs.permutation(pages).reshape(R, stride))
    s.k, s.v = _pool(s.lay, 2, pages, gen)
    s.layer = 1
    req = np.repeat(np.arange(R), new)
    tok = np.concatenate([np.arange(a, a + b) for a, b in zip(old, new)])
    s.req, s.tok = _ints(req), _ints(tok)
    far = rs.randint(0, case["far"], R)[req]
    if sum(sec):  # image patches: t moves slowly, h and w walk a grid
        pos = np.stack([far + tok // 400, far + tok // 20 % 20, far + tok % 20], 1)
    else:
        pos = far + tok
    s.pos = _ints(pos, torch.int64)
    std = torch.exp(torch.randn(d if hkv else LATENT + PE, generator=gen, device="cuda") * 0.5)
    dq = d if hkv else LATENT + PE
    q = torch.randn(T, hq, dq, generator=gen, device="cuda") * std
    k = torch.randn(T, max(hkv, 1), dq, generator=gen, device="cuda") * std
    # the projection's output, one row for a token: queries, keys and values side by side
    if hkv:
        v = torch.randn(T, hkv, d, generator=gen, device="cuda")
        x = torch.cat([q, k, v], 1).to(torch.bfloat16)
        s.q, s.kn, s.vn = x[:, :hq], x[:, hq:hq + hkv], x[:, hq + hkv:]
        s.qw = (1 + 0.2 * torch.randn(d, generator=gen, device="cuda")).to(torch.bfloat16)
        s.kw = (1 + 0.2 * torch.randn(d, generator=gen, device="cuda")).to(torch.bfloat16)
    else:
        s.q, s.kn, s.vn, s.qw = q.to(torch.bfloat16), k.to(torch.bfloat16), None, None
        s.kw = (1 + 0.2 * torch.randn(LATENT, generator=gen, device="cuda")).to(torch.bfloat16)
    s.out = torch.empty(T, hq, dq, dtype=torch.bfloat16, device="cuda")


def _prepare_beam(s, case, gen, rs, seed):
    p, c, pages = case["parents"], case["children"], case["pages"]
    ctx = _beam_ctx(case)
    n = [_ceil(int(x), PAGE) for x in ctx]
    stride = _ceil(int(ctx.max()) + case["grow"], PAGE) + 2
    table = np.full((p * (1 + c), stride), -1, np.int64)
    refs = np.zeros(pages, np.int64)
    perm = rs.permutation(pages)[:sum(n)]
    at = 0
    for i, k in enumerate(n):
        table[i, :k] = perm[at:at + k]
        at += k
    refs[perm] = 1
    s.k, s.v = _pool(s.lay, case["layers"], pages, gen)
    s.table, s.refs = _ints(table), _ints(refs)
    parent = np.repeat(np.arange(p), c)
    child = p + np.arange(p * c)
    held = ctx[parent]
    s.forks = _ints(np.stack([parent, child, held], 1))
    s.grown = _ints(np.stack([child, held, held + case["grow"]], 1))
    s.whole = _ints(np.stack([child, 0 * held, held + case["grow"]], 1))
    _fork(s.k, s.v, s.table, s.refs, s.forks)  # the last step's children
    _extend(s.table, s.refs, s.grown)


def _prepare_compact(s, case, gen, rs, seed):
    refs, rows = _scattered(case, seed)
    stride = max(len(r) for r in rows) + 1
    table = np.full((len(rows), stride), -1, np.int64)
    for i, r in enumerate(rows):
        table[i, :len(r)] = r
    s.k, s.v = _pool(s.lay, case["layers"], case["pages"], gen)
    s.table0, s.refs0 = _ints(table), _ints(refs)
    s.table, s.refs = s.table0.clone(), s.refs0.clone()
    s.live = torch.zeros(1, dtype=torch.int32, device="cuda")


def _prepare_copy(s, case, gen, rs, seed):
    at = rs.permutation(case["pages"])[:2 * case["n"]]
    s.k, s.v = _pool(s.lay, case["layers"], case["pages"], gen)
    s.src, s.dst = _ints(at[:case["n"]]), _ints(at[case["n"]:])
    s.table = _ints(np.zeros((1, 1)))


def _prepare_attend(s, case, gen, rs, seed):
    hq, hkv, d, _, _ = LAYOUTS[s.lay]
    start, prefix, ctx = _attend_lens(case)
    group = np.repeat(np.arange(len(prefix)), np.diff(start))
    shared = prefix // PAGE  # whole pages of the prefix; its last part is in pages of each request's own
    n = _ceil_all(ctx)
    pages = int(shared.sum() + (n - shared[group]).sum()) + 3
    perm = rs.permutation(pages)
    stride = int(n.max()) + 1
    table = np.full((len(ctx), stride), -1, np.int64)
    at = 0
    first = []
    for g in shared:
        first.append(perm[at:at + g])
        at += g
    for r, g in enumerate(group):
        k = int(n[r] - shared[g])
        table[r, :shared[g]] = first[g]
        table[r, shared[g]:n[r]] = perm[at:at + k]
        at += k
    s.k, s.v = _pool(s.lay, 2, pages, gen)
    s.layer = 1
    tail = np.flatnonzero(prefix[group] % PAGE)  # the prefix's last part is the same in every request
    src = np.concatenate([table[start[group[r]], shared[group[r]]] * PAGE + np.arange(prefix[group[r]] % PAGE) for r in tail] or [np.zeros(0)])
    dst = np.concatenate([table[r, shared[group[r]]] * PAGE + np.arange(prefix[group[r]] % PAGE) for r in tail] or [np.zeros(0)])
    src, dst = _ints(src, torch.int64), _ints(dst, torch.int64)
    for x in (s.k, s.v):
        if x is not None:
            x[:, dst] = x[:, src]
    s.table = _ints(table)
    s.start, s.prefix, s.ctx = _ints(start), _ints(prefix), _ints(ctx)
    dk, dv = (d, d) if hkv else (LATENT + PE, LATENT)
    s.q = (1.5 * torch.randn(len(ctx), hq, dk, generator=gen, device="cuda")).to(torch.bfloat16)
    s.scale = 1 / math.sqrt(d if hkv else 192)
    s.out = torch.empty(len(ctx), hq, dv, dtype=torch.bfloat16, device="cuda")
    s.lse = torch.empty(len(ctx), hq, dtype=torch.float32, device="cuda")
    # what the scheduler knows of the batch, for the plain form's padded arrays
    s.sizes = (int(np.diff(start).max()), int(prefix.max()), int((ctx - prefix[group]).max()))
    s.group = _ints(group, torch.int64)


# ---------------------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------------------

def run(s):
    return {"append": _run_append, "beam": _run_beam, "compact": _run_compact,
            "copy": _run_copy, "attend": _run_attend}[s.case["op"]](s)


def _pools(s):
    return {"k": s.k} if s.v is None else {"k": s.k, "v": s.v}


def _run_append(s):
    if own:
        s.km.kamera_append(s.handle, s.pool, s.layer, s.q, s.kn, s.vn, s.qw, s.kw, s.pos, s.req, s.tok, EPS, s.out, s.status)
        return {"q": s.out, **_pools(s)}
    hq, hkv, d, theta, sec = LAYOUTS[s.lay]
    q, k = s.q.float(), s.kn.float()
    if hkv:
        q, k = _norm(q, s.qw), _norm(k, s.kw)
        q, k = _rotate(q, s.pos, theta, sec), _rotate(k, s.pos, theta, sec)
    else:
        q = torch.cat([q[..., :LATENT], _rotate(q[..., LATENT:], s.pos, theta, sec)], -1)
        k = torch.cat([_norm(k[..., :LATENT], s.kw), _rotate(k[..., LATENT:], s.pos, theta, sec)], -1)
    slots = s.table[s.req.long(), s.tok.long() // PAGE].long() * PAGE + s.tok.long() % PAGE
    s.k[s.layer].index_copy_(0, slots, k.flatten(1).to(torch.bfloat16))
    if hkv:
        s.v[s.layer].index_copy_(0, slots, s.vn.flatten(1))
    return {"q": q.to(torch.bfloat16), **_pools(s)}


def _norm(x, w):
    return x * torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS) * w.float()


def _rotate(x, pos, theta, sec):
    """Pairs half a head apart turned by position times frequency, the angles in 64 bits."""
    half = x.shape[-1] // 2
    freq = theta ** (-torch.arange(half, dtype=torch.float64, device=x.device) / half)
    if sum(sec):
        axis = torch.repeat_interleave(torch.arange(3, device=x.device), torch.tensor(sec, device=x.device), output_size=half)
        angle = pos[:, axis].double() * freq
    else:
        angle = pos[:, None].double() * freq
    c, n = angle.cos().float()[:, None], angle.sin().float()[:, None]
    a, b = x[..., :half], x[..., half:]
    return torch.cat([a * c - b * n, b * c + a * n], -1)


def _run_beam(s):
    if own:
        s.km.kamera_free(s.handle, s.pool, s.whole, s.refs, s.status)
        s.km.kamera_fork(s.handle, s.pool, s.forks, s.refs, s.work, s.status)
        s.km.kamera_extend(s.handle, s.pool, s.grown, s.refs, s.work, s.status)
    else:
        _free(s.table, s.refs, s.whole)
        _fork(s.k, s.v, s.table, s.refs, s.forks)
        _extend(s.table, s.refs, s.grown)
    return {"table": s.table, "refs": s.refs, **_pools(s)}


def _free_pages(refs):
    """Free pages, the lowest first (then the others)."""
    n = refs.numel()
    return torch.sort(torch.arange(n, device=refs.device) + n * (refs != 0)).values % n


def _free(table, refs, spans):
    req, first, last = spans[:, 0].long(), -(-spans[:, 1:2] // PAGE), -(-spans[:, 2:3] // PAGE)
    col = torch.arange(table.shape[1], device=table.device)[None]
    held = (col >= first) & (col < last)
    rows = table[req]
    refs.index_add_(0, torch.where(held, rows, 0).flatten(), -held.flatten().int())
    table[req] = torch.where(held, -1, rows)


def _fork(k, v, table, refs, forks):
    parent, child, held = forks[:, 0].long(), forks[:, 1].long(), forks[:, 2].long()
    full, rest = held // PAGE, held % PAGE
    part = rest > 0
    page = _free_pages(refs)[(part.long().cumsum(0) - 1).clamp_min(0)]
    col = torch.arange(table.shape[1], device=table.device)[None]
    rows = table[parent]
    whole = col < full[:, None]
    refs.index_add_(0, torch.where(whole, rows, 0).flatten(), whole.flatten().int())
    refs.index_add_(0, torch.where(part, page, 0), part.int())
    last = rows.gather(1, full[:, None].clamp_max(table.shape[1] - 1)).long()
    table[child] = torch.where(whole, rows, torch.where((col == full[:, None]) & part[:, None], page[:, None].int(), table[child]))
    off = torch.arange(PAGE, device=table.device)[None]
    held = off < rest[:, None]
    src, dst = (last * PAGE + off)[held], (page[:, None] * PAGE + off)[held]
    for x in (k, v):
        if x is not None:
            x.index_copy_(1, dst, x.index_select(1, src))


def _extend(table, refs, spans):
    req, first, last = spans[:, 0].long(), -(-spans[:, 1] // PAGE), -(-spans[:, 2] // PAGE)
    n = last - first
    at = n.cumsum(0) - n
    col = torch.arange(table.shape[1], device=table.device)[None]
    new = (col >= first[:, None]) & (col < last[:, None])
    pages = _free_pages(refs)
    page = pages[torch.where(new, at[:, None] + col - first[:, None], 0)]
    refs.index_add_(0, torch.where(new, page, 0).flatten(), new.flatten().int())
    table[req] = torch.where(new, page.int(), table[req])


def _run_compact(s):
    s.table.copy_(s.table0)  # a fragmented pool again: the pages' rows are where they were
    s.refs.copy_(s.refs0)
    if own:
        s.km.kamera_compact(s.handle, s.pool, s.refs, s.live, s.work, s.status)
        return {"table": s.table, "refs": s.refs, "live": s.live, **_pools(s)}
    live = s.refs > 0
    n = live.sum()
    ids = torch.arange(s.refs.numel(), device="cuda")
    src = torch.nonzero(live & (ids >= n)).flatten()
    dst = torch.nonzero(~live & (ids < n)).flatten()
    to = ids.index_copy(0, src, dst).int()
    s.table.copy_(torch.where(s.table >= 0, to[s.table.clamp_min(0).long()], s.table))
    s.refs[dst] = s.refs[src]
    s.refs[src] = 0
    _copy_pages(s, src, dst)
    s.live.fill_(n)
    return {"table": s.table, "refs": s.refs, "live": s.live, **_pools(s)}


def _copy_pages(s, src, dst):
    for x in (s.k, s.v):
        if x is not None:
            y = x.view(x.shape[0], -1, PAGE * x.shape[2])
            y.index_copy_(1, dst, y.index_select(1, src))


def _run_copy(s):
    if own:
        s.km.kamera_copy_pages(s.handle, s.pool, s.src, s.dst, s.status)
    else:
        _copy_pages(s, s.src.long(), s.dst.long())
    return _pools(s)


def _run_attend(s):
    if own:
        s.km.kamera_prefix_attention(s.handle, s.pool, s.layer, s.q, s.start, s.prefix, s.ctx, s.scale, s.out, s.lse, s.work, s.status)
        return {"out": s.out, "lse": s.lse}
    hq, hkv, d, _, _ = LAYOUTS[s.lay]
    members, most, more = s.sizes
    dev = s.q.device
    R, G, H = s.q.shape[0], s.prefix.shape[0], max(hkv, 1)
    start, prefix, ctx = s.start.long(), s.prefix.long(), s.ctx.long()
    # the prefixes, once for each group: rows are the group's (request, query head) pairs
    t = torch.arange(most, device=dev)[None]
    have = t < prefix[:, None]
    slots = torch.where(have, s.table[start[:-1]].gather(1, (t // PAGE).expand(G, -1)).clamp_min(0) * PAGE + t % PAGE, 0)
    j = torch.arange(members, device=dev)[None]
    who = (start[:-1, None] + j).clamp_max(R - 1)
    q = s.q.float().view(R, H, hq // H, -1)
    one = _part(s, q[who].permute(0, 2, 1, 3, 4).flatten(2, 3), slots, have)
    at = torch.arange(R, device=dev) - start[s.group]
    o1, l1 = (x.unflatten(2, (members, hq // H)).permute(0, 2, 1, 3, *range(4, x.dim() + 1))[s.group, at] for x in one)
    # the rest of each request's context
    t = torch.arange(more, device=dev)[None] + prefix[s.group][:, None]
    have = t < ctx[:, None]
    slots = torch.where(have, s.table.gather(1, (t // PAGE).clamp_max(s.table.shape[1] - 1)).clamp_min(0) * PAGE + t % PAGE, 0)
    o2, l2 = _part(s, q, slots, have)
    top = torch.maximum(l1, l2)
    a, b = (l1 - top).exp(), (l2 - top).exp()
    out = (o1 * a[..., None] + o2 * b[..., None]) / (a + b)[..., None]
    return {"out": out.flatten(1, 2).to(torch.bfloat16), "lse": (top + (a + b).log()).flatten(1, 2)}


def _part(s, q, slots, have):
    """Attention of q [n][H][rows][dk] over the tokens at slots [n][t]: outputs and log-sum-exp."""
    hq, hkv, d, _, _ = LAYOUTS[s.lay]
    k = s.k[s.layer][slots].float().unflatten(2, (max(hkv, 1), -1)).transpose(1, 2)
    v = k[..., :LATENT] if s.v is None else s.v[s.layer][slots].float().unflatten(2, (hkv, -1)).transpose(1, 2)
    x = torch.matmul(q, k.transpose(2, 3)).mul_(s.scale).masked_fill_(~have[:, None, None], -math.inf)
    top = x.amax(-1, keepdim=True)
    p = x.sub_(top).exp_()
    total = p.sum(-1, keepdim=True)
    return torch.matmul(p, v) / total, (top + total.log()).squeeze(-1)


# ---------------------------------------------------------------------------------------
# the definitions in 64 bits
# ---------------------------------------------------------------------------------------

def exact(case, seed):
    if case["op"] not in ("append", "attend"):
        return None  # pages move whole: nothing is computed
    s = prepare(case, seed)
    hq, hkv, d, theta, sec = LAYOUTS[s.lay]
    if case["op"] == "append":
        band = d if hkv else PE
        i = torch.arange(band // 2, device="cuda")
        axis = (i >= sec[0]).long() + (i >= sec[0] + sec[1]).long() if sum(sec) else 0 * i
        where = s.pos if s.pos.dim() == 2 else s.pos[:, None]
        turn = torch.polar(torch.ones((), dtype=torch.float64, device="cuda"),
                           where.index_select(1, axis).double() / theta ** (2 * i.double() / band))

        def made(x, w, plain, normed):
            x = x.double().clone()
            if w is not None:
                y = x[..., :normed]
                x[..., :normed] = y / torch.sqrt((y * y).sum(-1, keepdim=True) / normed + EPS) * w.double()
            z = torch.complex(x[..., plain:plain + band // 2], x[..., plain + band // 2:]) * turn[:, None]
            return torch.cat([x[..., :plain], z.real, z.imag], -1)

        plain = 0 if hkv else LATENT
        q = made(s.q, s.qw, plain, d)
        pools = {n: x.double() for n, x in _pools(s).items()}
        req, tok = s.req.cpu().numpy(), s.tok.cpu().numpy()
        table = s.table.cpu().numpy()
        slot = torch.as_tensor(table[req, tok // PAGE].astype(np.int64) * PAGE + tok % PAGE).cuda()
        pools["k"][s.layer, slot] = made(s.kn, s.kw, plain, d if hkv else LATENT).reshape(len(req), -1)
        if hkv:
            pools["v"][s.layer, slot] = s.vn.double().reshape(len(req), -1)
        return {"q": q, **pools}
    start, prefix, ctx = _attend_lens(case)
    table = s.table.cpu().numpy().astype(np.int64)
    out, lse = [], []
    for r, n in enumerate(ctx):
        t = np.arange(n)
        slot = torch.as_tensor(table[r, t // PAGE] * PAGE + t % PAGE).cuda()
        k = s.k[s.layer].index_select(0, slot).double().view(int(n), max(hkv, 1), -1)
        v = k[..., :LATENT] if s.v is None else s.v[s.layer].index_select(0, slot).double().view(int(n), hkv, -1)
        q = s.q[r].double().view(max(hkv, 1), -1, s.q.shape[2])
        x = s.scale * torch.einsum("hgd,thd->hgt", q, k)
        z = torch.logsumexp(x, -1)
        out.append(torch.einsum("hgt,thd->hgd", torch.exp(x - z[..., None]), v).reshape(hq, -1))
        lse.append(z.reshape(hq))
    return {"out": torch.stack(out), "lse": torch.stack(lse)}
