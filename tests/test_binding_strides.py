"""The row strides that the binding passes on, from torch's strides (no GPU): torch gives a dimension of one element
any stride, which says nothing about where the rows lie."""

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
