"""Teacher lists as views: strides that no element takes are not looked at."""

import pytest
import torch

import sampling_support_b200 as vsb


def refusal(x, ids, lp):
    with pytest.raises(ValueError) as e:
        vsb.distill_fwd(x, ids, lp)
    return str(e.value)


def test_strides_of_one_row_and_of_one_column():
    """Lists that are well formed get as far as the check of the device."""
    ids, lp = torch.zeros(3, 8, dtype=torch.int32), torch.zeros(3, 16)
    x = torch.zeros(3, 16)
    assert "CUDA" in refusal(x[:1], ids[:1, :5], lp[:1, :5])  # one row, of wider lists of two widths
    assert "CUDA" in refusal(x, ids[:, :0], lp[:, :0])
    assert "stride" in refusal(x[:2], ids[:2, :5], lp[:2, :5])
    assert "stride" in refusal(x[:1], ids[:1, ::2], lp[:1, :4])


def test_one_column_of_any_stride_within_the_row():
    ids, lp = torch.zeros(3, 4, dtype=torch.int32)[:, :1], torch.zeros(3, 4).as_strided((3, 1), (4, 7))
    assert "CUDA" in refusal(torch.zeros(3, 16), ids, lp)
