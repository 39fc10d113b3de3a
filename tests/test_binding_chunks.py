"""What the Python binding checks of a batch of new tokens, of masses and of evictions (no GPU
needed): all of it before the C call, which here would be given addresses of CPU tensors."""
import types

import pytest
import torch

from position_independent_multimodal_gb300 import _binding as kb

CPU = -1  # the device index of CPU tensors
I32, F32, BF16 = torch.int32, torch.float32, torch.bfloat16
HANDLE = types.SimpleNamespace(_dk=16, _dv=16, _page=4, ptr=None)


class Called(Exception):
    pass


@pytest.fixture
def no_call(monkeypatch):
    """The pool is taken as it is, and a call that passes the checks ends here."""
    def call(*args):
        raise Called

    c = types.SimpleNamespace(kamera_chunk_attention=call, kamera_attention_mass=call,
                              kamera_evict=call)
    monkeypatch.setattr(kb, "_pool_c", lambda handle, pool: (kb.kamera_pool(), CPU))
    monkeypatch.setattr(kb, "_stream_on", lambda stream, dev: None)
    monkeypatch.setattr(kb, "lib", lambda: c)


def test_batches_that_are_taken():
    start, ctx = torch.zeros(4, dtype=I32), torch.zeros(3, dtype=I32)
    x = torch.zeros(5, 2 * 96 + 8, dtype=BF16)
    q = x[:, 96:192].unflatten(1, (6, 16))  # among other columns of a wider row
    assert kb._chunk(HANDLE, CPU, q, start, ctx) == \
        (q.data_ptr(), 200, 5, 6, start.data_ptr(), ctx.data_ptr(), 3)
    assert kb._chunk(HANDLE, CPU, q[:0], start[:1], ctx[:0])[2:4] == (0, 6)
    assert kb._chunk(HANDLE, CPU, q[1:2], start, ctx)[1] == 96  # of one token: any


@pytest.mark.parametrize("kw", [
    dict(q=torch.zeros(5, 96, dtype=BF16)), dict(q=torch.zeros(5, 6, 32, dtype=BF16)),
    dict(q=torch.zeros(5, 6, 16)), dict(q=torch.zeros(5, 6, 32, dtype=BF16)[..., ::2]),
    dict(q=torch.zeros(5, 12, 16, dtype=BF16)[:, ::2]),
    dict(q=torch.zeros(6, 5, 16, dtype=BF16).transpose(0, 1)), dict(start=torch.zeros(3, dtype=I32)),
    dict(start=torch.zeros(4, dtype=torch.int64)), dict(start=torch.zeros(8, dtype=I32)[::2]),
    dict(ctx=torch.zeros(4, dtype=I32)), dict(ctx=torch.zeros(3)),
    dict(ctx=torch.zeros(6, dtype=I32)[::2])])
def test_batches_that_are_refused(kw):
    args = dict(q=torch.zeros(5, 6, 16, dtype=BF16), start=torch.zeros(4, dtype=I32),
                ctx=torch.zeros(3, dtype=I32))
    args.update(kw)
    with pytest.raises(ValueError):
        kb._chunk(HANDLE, CPU, *args.values())


def _batch():
    return (torch.zeros(5, 6, 16, dtype=BF16), torch.zeros(4, dtype=I32), torch.zeros(3, dtype=I32))


@pytest.mark.parametrize("kw", [
    dict(), dict(out=torch.zeros(6, 6, 16, dtype=BF16)), dict(out=torch.zeros(5, 6, 32, dtype=BF16)),
    dict(out=torch.zeros(5, 6, 16)), dict(out=torch.zeros(5, 6, 32, dtype=BF16)[..., ::2]),
    dict(lse=torch.zeros(6, 5)), dict(lse=torch.zeros(5, 6, dtype=BF16)),
    dict(lse=torch.zeros(6, 5).t()), dict(ws=torch.zeros(64)[::2]), dict(status=torch.zeros(1))])
def test_chunk_attention(no_call, kw):
    args = dict(out=torch.zeros(5, 6, 16, dtype=BF16), lse=torch.zeros(5, 6),
                ws=torch.zeros(64, dtype=torch.uint8), status=torch.zeros(1, dtype=I32))
    args.update(kw)
    with pytest.raises(ValueError if kw else Called):
        kb.kamera_chunk_attention(HANDLE, None, 0, *_batch(), 1.0, *args.values())


@pytest.mark.parametrize("kw", [
    dict(), dict(lse=torch.zeros(5, 7)), dict(lse=torch.zeros(5, 6, dtype=torch.float64)),
    dict(mass=torch.zeros(4, 80)), dict(mass=torch.zeros(240)), dict(mass=torch.zeros(3, 80).half()),
    dict(mass=torch.zeros(3, 160)[:, :80]), dict(ws=torch.zeros(64)[::2]), dict(status=torch.zeros(1))])
def test_attention_mass(no_call, kw):
    args = dict(lse=torch.zeros(5, 6), decay=0.5, mass=torch.zeros(3, 80),
                ws=torch.zeros(64, dtype=torch.uint8), status=torch.zeros(1, dtype=I32))
    args.update(kw)
    with pytest.raises(ValueError if kw else Called):
        kb.kamera_attention_mass(HANDLE, None, 0, *_batch(), 1.0, *args.values())


@pytest.mark.parametrize("kw", [
    dict(), dict(items=torch.zeros(2, 4, dtype=I32)), dict(items=torch.zeros(10, dtype=I32)),
    dict(items=torch.zeros(2, 5)), dict(items=torch.zeros(2, 10, dtype=I32)[:, ::2]),
    dict(refs=torch.zeros(4, dtype=I32)), dict(refs=torch.zeros(5)), dict(mass=torch.zeros(2, 80)),
    dict(mass=torch.zeros(3, 80, dtype=torch.float64)), dict(mass=torch.zeros(3, 90)[:, :80]),
    dict(kept=torch.zeros(3, 60, dtype=I32)), dict(kept=torch.zeros(2, 60)),
    dict(kept=torch.zeros(120, dtype=I32)), dict(ws=torch.zeros(64)[::2]), dict(status=torch.zeros(1))])
def test_evict(no_call, kw):
    pool = types.SimpleNamespace(page_table=torch.zeros(3, 5, dtype=I32), num_slots=20)
    args = dict(items=torch.zeros(2, 5, dtype=I32), refs=torch.zeros(5, dtype=I32),
                mass=torch.zeros(3, 80), kept=torch.zeros(2, 60, dtype=I32),
                ws=torch.zeros(64, dtype=torch.uint8), status=torch.zeros(1, dtype=I32))
    args.update(kw)
    with pytest.raises(ValueError if kw else Called):
        kb.kamera_evict(HANDLE, pool, *args.values())
