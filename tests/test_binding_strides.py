"""What the binding makes of its arguments (no GPU).  Row strides: torch gives a dimension of one element any stride,
which says nothing about where the rows lie."""

import pytest
import torch

import block_scaled_fp8_act_amd as ds


def test_matrix_row_stride():
    one_row = torch.zeros(64, 1).t()                    # [1, 64], strides (1, 1)
    assert one_row.stride() == (1, 1) and ds._ld(one_row) == 64 and ds._row(one_row, 64) == 64
    one_column = torch.zeros(1, 64).t()                 # [64, 1], strides (1, 64)
    assert one_column.stride() == (1, 64) and ds._ld(one_column) == 1 and ds._row(one_column, 1) == 1
    wide = torch.zeros(5, 100)[:, 3:40]
    assert ds._ld(wide) == 100 and ds._row(wide, 37) == 100
    assert ds._ld(wide[:, :0]) == 0 and ds._ld(wide[:0]) == 37
    assert ds._ld(torch.zeros(7, 3, 8)) == 8 and ds._ld(torch.zeros(7, 3, 9)[:, :, :8]) == 9


def test_stacked_row_stride():
    whole = torch.zeros(4, 3, 10)
    assert ds._expert_ld(whole, "w") == 10
    assert ds._expert_ld(whole[:, :, :8], "w") == 10
    assert ds._expert_ld(whole[:, :1], "w") == 30       # one row each: an expert's stride is its row's
    assert ds._expert_ld(whole[:, :1, :8], "w") == 30
    assert ds._expert_ld(whole[1:2, :2, :8], "w") == 10     # one expert: the next one's place does not matter
    assert ds._expert_ld(whole[:, :2, :0], "w") == 0 and ds._expert_ld(whole[:0], "w") == 10
    assert ds._expert_ld(torch.zeros(4, 10).as_strided((4, 1, 10), (10, 7, 1)), "w") == 10
    with pytest.raises(ds.Dsfp8Error):
        ds._expert_ld(whole[:, :2], "w")
    with pytest.raises(ds.Dsfp8Error):
        ds._expert_ld(whole[:, ::2], "w")


@pytest.mark.parametrize("bad", [64, [0] * 64, torch.zeros(64, dtype=torch.uint8)])
def test_workspace_that_is_no_device_tensor(bad):
    with pytest.raises(ds.Dsfp8Error):
        ds._workspace(bad, 16, torch.zeros(1))
