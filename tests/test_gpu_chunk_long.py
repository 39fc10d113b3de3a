"""kamera_chunk_attention over long contexts, each output bounded by the values that it weighs: one tile
of V left out, or taken twice, is far outside of it."""
import types

import numpy as np
import pytest
import torch

from tests.chunk_checks import check_rows, exact
from tests.chunk_testlib import Chunks

gpu = pytest.mark.gpu


@pytest.fixture
def cuda(cuda_ok):
    return cuda_ok


@gpu
@pytest.mark.parametrize("name", ["gqa128-group7", "gqa128-group4-page64", "mha128-page1",
                                  "gqa64-group3", "mha64-page5", "gqa80", "gqa256", "mla-16-heads",
                                  "mla-130-heads-page3", "mla-narrow"])
@pytest.mark.parametrize("reqs,window", [
    ([(1, 5000)], 0), ([(1, 11999), (1, 6), (2, 4000)], 0), ([(257, 1300), (1, 2999)], 0),
    ([(40, 8000), (9, 0)], 3000), ([(130, 2500), (1, 2500)], 1000)])
def test_every_tile_of_values_counts(cuda, name, reqs, window):
    check_rows(Chunks(name, reqs, window=window, seed=40).run())


@gpu
@pytest.mark.parametrize("name", ["gqa128-group7", "gqa64-group3", "mla-16-heads", "gqa80"])
@pytest.mark.parametrize("sharp", [3.0, 8.0])
def test_sharp_scores(cuda, name, sharp):
    check_rows(Chunks(name, [(60, 3000), (1, 4000), (1, 100)], seed=41, sharp=sharp).run())


def test_the_bound_shows_a_tile_that_is_missing():
    # (of a model of a batch on the host: outputs without 128 of 5000 tokens of V)
    g = torch.Generator().manual_seed(42)
    c, dv = 5000, 128
    x = torch.randn(1, 1, c, generator=g).double()
    v = torch.randn(1, c, dv, generator=g).double()
    b = types.SimpleNamespace(H=1, new=np.array([1]), start=np.array([0, 1]),
                              st=torch.zeros(1), exact=lambda r: (x, torch.full((1, 1), 1e-6), v))
    o, size, lse, _ = exact(b, 0)
    b.lse = lse.float()
    b.out = o.bfloat16()
    check_rows(b)
    p = torch.softmax(x[0, 0], 0)
    for tile in (0, 17, 38):
        rows = slice(128 * tile, 128 * tile + 128)
        b.out = (o - torch.einsum("c,cd->d", p[rows], v[0, rows])).bfloat16()
        with pytest.raises(AssertionError):
            check_rows(b)
