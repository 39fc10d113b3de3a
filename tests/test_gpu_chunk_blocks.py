"""kamera_chunk_attention: workers that take several blocks one after another."""
import numpy as np
import pytest
import torch

from tests.chunk_checks import check_rows
from tests.chunk_testlib import Chunks

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _cuda(cuda_ok):
    return cuda_ok


def repeat(b, times):
    """The batch's call, `times` times: right, and the same bytes each time."""
    b.run()
    check_rows(b)
    out, lse = b.out.clone(), b.lse.clone()
    for _ in range(times - 1):
        b.out.fill_(-7)
        b.lse.fill_(-7)
        b.call()
        assert torch.equal(b.out, out) and torch.equal(b.lse, lse)
    assert int(b.st.item()) == 0


@pytest.mark.parametrize("name,reqs", [("gqa128-group7", 76), ("gqa64-group3", 152),
                                       ("mha64-page5", 152)])
@pytest.mark.parametrize("ctx", [256, 300, 500])
@pytest.mark.parametrize("sharp", [1.0, 6.0])
def test_blocks_whose_tiles_are_taken_in_turns(name, reqs, ctx, sharp):
    # requests that decode, as many blocks of one length for each of 152 workers: each takes two or
    # more whole ones, and its two query tiles join their sums at the end of each
    repeat(Chunks(name, [(1, ctx - 1)] * reqs, seed=20, sharp=sharp), 20)


@pytest.mark.parametrize("name,reqs", [("gqa128-group7", 400), ("gqa64-group3", 900),
                                       ("gqa128-group4-page64", 900), ("mha64-page5", 400)])
def test_blocks_of_one_tile(name, reqs):
    # a context of 128 is one whole tile: the other query tile has nothing to do but keep step, for
    # several blocks in a row and in the last
    repeat(Chunks(name, [(1, 127)] * reqs, seed=21), 40)


@pytest.mark.parametrize("name,many", [("gqa128-group7", 36), ("gqa64-group3", 84),
                                       ("gqa128-group4-page64", 60)])
@pytest.mark.parametrize("seed", [22, 23])
def test_blocks_of_one_tile_behind_others(name, many, seed):
    # behind blocks of two query tiles, of one tile of tokens and of more, and before them
    pattern = [(many, 128 - many), (1, 127), (1, 127), (many, 300), (1, 127), (1, 40), (1, 200)]
    rs = np.random.RandomState(seed)
    reqs = [pattern[k] for k in rs.randint(0, len(pattern), 300)]
    repeat(Chunks(name, reqs, seed=seed), 20)


def cut_in_two(b, least):
    """(request, first of its new tokens, new tokens) of the blocks of more than `least` query rows
    that the last call has cut between exactly two workers, by the records that it left in the
    workspace: 16 integers a worker (a cut block begins, parts that follow, its first row of q, its
    query rows, ...)."""
    skew = -b.ws.data_ptr() % 128
    rec = b.ws[skew:skew + 152 * 64].view(torch.int32).view(152, 16).cpu().numpy()
    found = []
    for head, more, row, rows in rec[:, :4]:
        if head == 1 and more == 1 and rows > least:
            r = int(np.searchsorted(b.start, row, "right")) - 1
            found.append((r, int(row - b.start[r]), int(rows) // (b.hq // b.H)))
    return found


def values_from(b, tokens, value):
    """The batch with V of the given (request, token of the context) not finite, and which rows of q
    see one of them."""
    me = np.arange(b.rows)
    sees = np.zeros(b.rows, bool)
    for r, u in tokens:
        x = b.pool.k if b.v is None else b.pool.v
        x[:, int(b.slots(r)[u])] = value
        at = me - b.start[r] + b.ctx[r] - b.new[r]
        mine = (me >= b.start[r]) & (me < b.start[r + 1])
        sees |= mine & (at >= u) & ((at - u < b.window) if b.window else True)
    return torch.as_tensor(sees).cuda()


@pytest.mark.parametrize("name,least", [("gqa128-group7", 128), ("gqa64-group3", 128),
                                        ("gqa128-group4-page64", 128), ("mla-16-heads", 64)])
@pytest.mark.parametrize("window", [0, 4, 64, 300])
@pytest.mark.parametrize("value", [float("nan"), float("inf")])
def test_values_not_seen_in_blocks_cut_in_two(name, least, window, value):
    # what the join has made not finite for a row that does not see it is taken again, and stays so
    b = Chunks(name, [(700, 0), (5, 60)], window=window, seed=24).run()
    check_rows(b)
    blocks = cut_in_two(b, least)
    assert blocks, "no block is cut in two: another batch is wanted"
    # the last token of each such block; without a window all that follow see it, so one block's
    sets = [[(r, int(b.ctx[r] - b.new[r]) + t + n - 1) for r, t, n in blocks]]
    if not window:
        sets = [[s] for s in sorted(set(sets[0]))[:6]]
    clean = (b.pool.k.clone(), None if b.v is None else b.pool.v.clone())
    for tokens in sets:
        b.pool.k.copy_(clean[0])
        if b.v is not None:
            b.pool.v.copy_(clean[1])
        sees = values_from(b, tokens, value)
        assert bool(sees.any()) and not bool(sees[:700].all())
        want = None
        for _ in range(20):
            b.out.fill_(-7)
            b.lse.fill_(-7)
            b.call()
            got = torch.cat([b.out.flatten(1).float(), b.lse], 1)
            if want is None:
                want = got
                check_rows(b, only=~sees)
            assert torch.equal(got.nan_to_num(9e9, 8e9, 7e9), want.nan_to_num(9e9, 8e9, 7e9))
