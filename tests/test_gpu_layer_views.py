"""Views that the memory layer's calls take as they are: expanded rows, leading dimensions."""
import pytest
import torch

import trellis_row_decode_gb300 as cp

from layer_util import DTYPES, gen, randn

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("d", [16, 33, 1024])
def test_embed_of_an_expanded_row(d, dtype):
    """A table whose rows are one row (stride 0), as every input may be."""
    g = gen(d)
    row = randn(g, 1, d, dtype=dtype).cuda()
    ids = torch.tensor([0, 9, -1, 4, 10], device="cuda")
    got = cp.embed(row.expand(10, d), ids, 2.0)
    assert torch.equal(got, cp.embed(row.expand(10, d).contiguous(), ids, 2.0))
    assert torch.equal(got[1], 2 * row[0]) and not got[[2, 4]].any()
