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
