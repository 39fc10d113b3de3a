"""What the Python binding checks of the serving calls' arguments (no GPU needed)."""
import types

import pytest
import torch

from position_independent_multimodal_gb300 import _binding as kb

CPU = -1  # the device index of CPU tensors


def test_page_table_of_whole_rows():
    t = torch.arange(35, dtype=torch.int32).reshape(5, 7)
    assert kb._table(t, CPU) == (t.data_ptr(), 5, 7)
    assert kb._table(t[1:4], CPU) == (t[1].data_ptr(), 3, 7)
    # of one row the stride says nothing
    for one in (t[2:3], t[2:3, 1:6], t[:, :1].contiguous().t(), t[1:2].expand(1, 7)):
        assert kb._table(one, CPU) == (one.data_ptr(), 1, one.shape[1])


@pytest.mark.parametrize("cut", [lambda t: t[:, 1:], lambda t: t[:, :6], lambda t: t[:, ::2],
                                 lambda t: t[::2], lambda t: t.t(), lambda t: t[0],
                                 lambda t: t[:1].expand(5, 7), lambda t: t.reshape(5, 7, 1),
                                 lambda t: t.long(), lambda t: t[:, 3:4]])
def test_other_page_tables_are_refused(cut):
    t = torch.arange(35, dtype=torch.int32).reshape(5, 7)
    with pytest.raises(ValueError):
        kb._table(cut(t), CPU)


def _handle(mrope):
    return types.SimpleNamespace(_positions=3 if mrope else 1)


@pytest.mark.parametrize("shape", [(3, 7), (21,), (1, 7, 3), (7, 1, 3), (7, 2), (6, 3), (7,)])
def test_mrope_positions_of_other_shapes_are_refused(shape):
    with pytest.raises(ValueError):
        kb._check_positions(_handle(True), torch.zeros(shape, dtype=torch.int64), 7)


def test_positions_that_are_taken():
    kb._check_positions(_handle(True), torch.zeros(7, 3, dtype=torch.int64), 7)
    kb._check_positions(_handle(True), torch.zeros(0, 3, dtype=torch.int64), 0)
    for shape in ((7,), (7, 1), (1, 7)):
        kb._check_positions(_handle(False), torch.zeros(shape, dtype=torch.int64), 7)
    for shape in ((6,), (7, 3), (21,)):
        with pytest.raises(ValueError):
            kb._check_positions(_handle(False), torch.zeros(shape, dtype=torch.int64), 7)


def test_token_strides():
    x = torch.zeros(5, 12 * 16 + 4, dtype=torch.bfloat16)[:, :192].unflatten(1, (12, 16))
    assert kb._heads("k", x[:, 4:8], CPU, 5, 4, 16) == 196
    for n in (0, 1):  # what the stride is does not matter
        assert kb._heads("k", x[:n, 4:8], CPU, n, 4, 16) == 64
    for bad in (x[:, ::2], x[:, :6], x[..., ::2], x.float(), x[:4]):
        with pytest.raises(ValueError):
            kb._heads("k", bad, CPU, 5, 12, 16)
