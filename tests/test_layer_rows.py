"""The rows that a call counts in a tensor: host side only, so they run without a GPU."""
import pytest
import torch

from trellis_row_decode_gb300 import layer


@pytest.mark.parametrize("lead", [(), (1,), (6,), (2, 3), (4, 1, 5), (0, 3), (3, 0), (2, 3, 0, 5)])
@pytest.mark.parametrize("d", [0, 1, 8])
def test_rows_are_the_leading_dimensions(lead, d):
    rows = 1
    for n in lead:
        rows *= n
    got = layer._rows(torch.empty(*lead, d, device="meta"), "x")
    assert got[:2] == (rows, d)
    assert rows <= 1 or got[2] == d


def test_rows_of_no_columns_of_a_view():
    """Leading dimensions that could not be merged hold nothing: there is nothing to refuse."""
    t = torch.empty(4, 3, 8).transpose(0, 1)
    with pytest.raises(ValueError, match="mergeable"):
        layer._rows(t, "x")
    assert layer._rows(t[..., :0], "x") == (12, 0, 0)
