"""What the Python binding checks of the serving calls' arguments (no GPU needed)."""
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
