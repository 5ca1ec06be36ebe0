"""Dropout of rows of almost 2^32 columns, the most that the library takes: the last octet is stored to
its end and no further."""
import numpy as np
import pytest
import torch

import trellis_row_decode_gb300 as cp

from linear_util import philox

pytestmark = pytest.mark.gpu


def kept(first, d, p, seed):
    """The mask of row 0 from column `first` (a multiple of 4) to d."""
    quad = np.arange(first // 4, (d + 3) // 4, dtype=np.uint64)
    z = np.zeros_like(quad)
    w = np.stack(philox(quad, z, z, z, seed, 0), -1).reshape(-1)[:d - first]
    return torch.from_numpy(w < np.uint64(int((1 - p) * 2.0 ** 32 + 0.5)))


@pytest.mark.parametrize("short", [1, 5, 8, 12])
@pytest.mark.parametrize("residual", [False, True])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_dropout_of_the_widest_row_stops_at_its_end(short, residual, dtype):
    d, p, seed = (1 << 32) - short, 0.5, 7
    x = torch.ones(1, d, dtype=dtype, device="cuda")
    out = torch.full((d + 64,), 3.0, dtype=dtype, device="cuda")
    got = out[:d][None]
    cp.dropout(x, p, seed, residual=x if residual else None, out=got)
    add = 1.0 if residual else 0.0
    for first in (0, d // 8 * 4, (d - 4096) // 4 * 4):
        n = min(d - first, 4096)
        want = 2.0 * kept(first, first + n, p, seed).double() + add
        assert torch.equal(got[0, first:first + n].cpu().double(), want)
    assert bool((out[d:] == 3.0).all())
