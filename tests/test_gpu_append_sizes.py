"""kamera_append on both sides of the borders between its kernels: a token a CTA, four, a warp a
token (multiples of the number of SMs, halved where the queries' latents are copied by CTAs of
their own)."""
import pytest

from tests import test_gpu_append as base

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _cuda(cuda_ok):
    return cuda_ok


MORE = {
    "mla-8-heads": (base.mla(512, 64), 8),       # copies by warps where many tokens come
    "gqa128-48-heads": (base.gqa(128, 8), 48),   # six warps fit
    "gqa128-56-heads": (base.gqa(128, 8), 56),   # five
}


@pytest.mark.parametrize("edge", [152, 304, 608, 1216])
@pytest.mark.parametrize("name", ["gqa128", "gqa64-page5", "mla", "mla-8-heads", "gqa128-48-heads",
                                  "gqa128-56-heads"])
def test_around_the_borders(monkeypatch, name, edge):
    if name in MORE:
        monkeypatch.setitem(base.LAYOUTS, name, MORE[name])
    for tokens in (edge - 1, edge, edge + 1):
        r = base.Run(name, [tokens // 3, tokens - tokens // 3], seed=tokens)
        assert r.call() == 0
        r.check(r.want())


@pytest.mark.parametrize("edge", [304, 1216])
def test_around_the_borders_in_place(edge):
    for tokens in (edge, edge + 1):
        r = base.Run("mla", [tokens], seed=tokens, apart=True)
        want = r.want()
        assert r.call(out=r.q) == 0
        r.check(want, out=r.q)
