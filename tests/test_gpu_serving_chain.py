"""Calls that write the page table followed at once, on the same stream, by the calls that read it:
the kernels start while those before them still run, and have to see what they wrote."""
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
    "gqa": wl.Layout(kind=wl.GQA, num_layers=1, page_size=5, num_kv_heads=2, head_dim=64,
                     rope_dim=64),
    "mla": wl.Layout(kind=wl.MLA, num_layers=1, page_size=16, latent_dim=512, rope_dim=64),
}


@pytest.mark.parametrize("captured", [False, True])
@pytest.mark.parametrize("tokens", [3, 350, 1400])
@pytest.mark.parametrize("name", sorted(LAYOUTS))
def test_rows_go_where_the_table_says_now(name, tokens, captured):
    # Each step releases the request of three steps before, gives the next one pages and appends its
    # tokens, with page ids that change from step to step; at last the live requests' rows are those
    # appended. Position 0 and no norm: a row is its input, bit for bit.
    lay, steps, R = LAYOUTS[name], 40, 7
    ps, rs = lay.page_size, np.random.RandomState(tokens)
    per = -(-tokens // ps) + 1
    lens = rs.randint(max(1, tokens - 40), tokens + 1, steps)
    pages = 4 * per
    g = torch.Generator().manual_seed(tokens)
    k = torch.zeros(1, pages * ps, lay.row_k, dtype=torch.bfloat16, device="cuda")
    gqa = lay.kind == wl.GQA
    v = torch.zeros(1, pages * ps, lay.row_v, dtype=torch.bfloat16, device="cuda") if gqa else None
    table = torch.full((R, per), -1, dtype=torch.int32, device="cuda")
    refs = torch.zeros(pages, dtype=torch.int32, device="cuda")
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    h, pool = km.create(lay), km.Pool(k, v, table)
    ws = torch.empty(km.kamera_page_workspace(h, pages * ps, 1), dtype=torch.uint8, device="cuda")
    H, dk = (lay.num_kv_heads, lay.head_dim) if gqa else (1, lay.row_k)
    i32 = lambda x: torch.as_tensor(np.array(x), dtype=torch.int32).cuda()  # noqa: E731
    todo = []
    for i, n in enumerate(lens):
        x = wl.normal_bf16((n, 2 * H, dk), 1.0, g, "cpu").cuda()
        todo.append(dict(x=x, span=i32([[i % R, 0, n]]), req=i32([i % R] * n), tok=i32(np.arange(n)),
                         pos=torch.zeros(n, dtype=torch.int64, device="cuda")))

    def chain():
        for i, d in enumerate(todo):
            if i >= 3:
                km.kamera_free(h, pool, todo[i - 3]["span"], refs, st)
            km.kamera_extend(h, pool, d["span"], refs, ws, st)
            km.kamera_append(h, pool, 0, None, d["x"][:, :H], d["x"][:, H:] if gqa else None, None,
                             None, d["pos"], d["req"], d["tok"], 0.0, None, st)

    torch.cuda.synchronize()
    if captured:
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            chain()
        graph.replay()
    else:
        chain()
    torch.cuda.synchronize()
    assert int(st.item()) == 0
    # the table by the calls' own definitions: the lowest free pages, in order
    count, want = np.zeros(pages, int), np.full((R, per), -1)
    for i, n in enumerate(lens):
        if i >= 3:
            row = want[(i - 3) % R]
            count[row[row >= 0]] -= 1
            row[:] = -1
        c = -(-int(n) // ps)
        pick = np.flatnonzero(count == 0)[:c]
        want[i % R, :c] = pick
        count[pick] += 1
    assert np.array_equal(table.cpu().numpy(), want)
    assert np.array_equal(refs.cpu().numpy(), count)
    kb, vb = wl.bf16_bits(k)[0], None if v is None else wl.bf16_bits(v)[0]
    for i in range(steps - 3, steps):
        t = np.arange(lens[i])
        slots = want[i % R, t // ps] * ps + t % ps
        x = wl.bf16_bits(todo[i]["x"])
        assert np.array_equal(kb[slots], x[:, :H].reshape(len(t), -1))
        if gqa:
            assert np.array_equal(vb[slots], x[:, H:].reshape(len(t), -1))
