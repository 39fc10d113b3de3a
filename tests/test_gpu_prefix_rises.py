"""Wide blocks of kamera_prefix_attention whose running maximum rises in every tile of tokens, so
that O is rescaled each time: both halves of O's columns have to be scaled before a product of the
next tile is added to any of them. The bounds are those of test_gpu_prefix_attention."""
import pytest
import torch

from tests.test_gpu_prefix_attention import Batch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _cuda(cuda_ok):
    return cuda_ok


def rising(name, prefix, size, seed, every=1):
    """A batch over one prefix. The first quarter of K's columns says which tile of 128 tokens a key
    is of, by a step that a query row of ones turns into 9 powers of two (more than the 8 that let a
    maximum stand); the others are random, so that a tile's weight is spread over all its tokens.
    The queries of every `every`-th request have the ones, those of the others zeros there."""
    b = Batch(name, [(prefix, [r % 4 for r in range(size)])], seed=seed)
    d = b.dk // 4
    b.scale = 1 / 16
    step = 9 * 0.6931 * 16 / d  # in K; 25 of them are rounded by half a unit at most
    b.k = b.k * 0.5
    H = b.k.shape[2] // b.dk
    for r in range(size):
        s = torch.as_tensor(b.slots(r))
        tile = torch.arange(len(s)) // 128
        assert int(tile.max()) <= 25
        for h in range(H):
            b.k[:, s, h * b.dk:h * b.dk + d] = (tile * step)[:, None].to(torch.bfloat16)
    b.q[..., :d] = 0
    b.q[::every, :, :d] = 1
    return b


@pytest.mark.parametrize("name,size", [
    ("gqa128-group7", 40), ("gqa128-group7", 15), ("gqa64-group3", 90), ("gqa64-group3", 30),
    ("gqa128-one-kv-head", 9), ("mla-16-heads", 20)])
@pytest.mark.parametrize("prefix", [1900, 3207])
def test_rises_in_every_tile(name, size, prefix):
    # two tiles of query rows and one; every row rises, and every third request's rows alone
    for every in (1, 3):
        b = rising(name, prefix, size, seed=size + prefix, every=every)
        assert b.run() == 0
        b.check(reqs=sorted({0, 1, 2, size // 2, size - 2, size - 1}))
        first, lse = b.out.clone(), b.lse.clone()
        for _ in range(20):
            b.out.fill_(-7)
            b.call()
            torch.cuda.synchronize()
            assert torch.equal(b.out.view(torch.int16), first.view(torch.int16))
            assert torch.equal(b.lse, lse)
