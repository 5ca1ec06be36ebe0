"""Dropout of more than 2^32 elements in each of its layouts, with the residual's addition and in
place: rows at the ends and around 2^32 elements against 64 bits."""
import numpy as np
import pytest
import torch

import trellis_row_decode_gb300 as cp

from layer_util import U32, assert_within, rounded
from linear_util import philox

pytestmark = pytest.mark.gpu


def kept(rows, d, p, seed):
    quad = np.arange((d + 3) // 4, dtype=np.uint64)[None, :]
    row = np.array(rows, dtype=np.uint64)[:, None]
    z = np.zeros((1, 1), dtype=np.uint64)
    w = np.stack(np.broadcast_arrays(*philox(quad + z, row + z, z, z, seed, 0)), -1)
    return torch.from_numpy(w.reshape(len(rows), -1)[:, :d] < int((1 - p) * 2.0 ** 32 + 0.5))


def check(got, x, keep, p, residual=None):
    drop = torch.where(keep, x.double() / (1 - p), 0.0)
    want = drop + (residual.double() if residual is not None else 0.0)
    assert_within(got, want, 3 * U32 * (drop.abs() + want.abs()) + rounded(want, x.dtype))


# one behind the other in whole octets, apart, and on any boundary
@pytest.mark.parametrize("d,pitch", [(65536, 65536), (65528, 65536), (65535, 65535), (65533, 65536)])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_dropout_past_32_bits_keeps_its_values(d, pitch, dtype):
    m, p = 66100, 0.25
    over = (1 << 32) // pitch
    rows = [0, 1, over - 1, over, over + 1, m - 2, m - 1]
    x = torch.zeros(m * pitch, dtype=dtype, device="cuda").as_strided((m, d), (pitch, 1))
    r = torch.zeros(m * pitch, dtype=dtype, device="cuda").as_strided((m, d), (pitch, 1))
    for i in rows:
        x[i].normal_()
        r[i].normal_()
    xs, rs, keep = x[rows].cpu(), r[rows].cpu(), kept(rows, d, p, 9)
    out = cp.dropout(x, p, 9, residual=r, out=torch.empty_like(x)[:, :d])
    check(out[rows], xs, keep, p, rs)
    del out
    assert cp.dropout(x, p, 9, residual=r, out=r) is r            # the stream is updated in place
    check(r[rows], xs, keep, p, rs)
    assert cp.dropout(x, p, 9, residual=x, out=x) is x             # the input is its own residual
    check(x[rows], xs, keep, p, xs)
    x.zero_()
    x[rows] = xs.cuda()
    assert cp.dropout(x, p, 9, out=x) is x
    check(x[rows], xs, keep, p)
