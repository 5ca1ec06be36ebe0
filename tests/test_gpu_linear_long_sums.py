"""What 16-bit outputs of long sums of positive products lose to one side: the tensor core cuts what it
adds, and up to an eighth of the outputs' own half step may go that way."""
import pytest
import torch

import trellis_row_decode_gb300 as cp

from layer_util import UNIT

pytestmark = pytest.mark.gpu


def positive(g, rows, k, most, dtype):
    """Rows of positive values, each row of a scale of its own, so that roundings do not line up."""
    scale = torch.rand(rows, 1, generator=g, device="cuda") * 0.5 + 0.5
    return (torch.rand(rows, k, generator=g, device="cuda") * scale * most).to(dtype)


def within(got, ref, dtype):
    """The mean of N roundings, evenly spread up to UNIT either way, deviates by UNIT over the root of 3 N:
    five of those, and the eighth."""
    off = ((got.double() - ref) / ref).mean().abs()
    return float(off) < UNIT[dtype] / 8 + 5 * UNIT[dtype] / (3 * got.numel()) ** 0.5


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("k", [4096, 16384, 24576, 65536])
def test_linear_long_sums(k, dtype):
    g = torch.Generator(device="cuda").manual_seed(k)
    x, w = positive(g, 2560, k, 1.0, dtype), positive(g, 2560, k, 0.5, dtype)
    for m in (2560, 40):
        ref = x[:m:8].double() @ w[::8].double().T
        assert within(cp.linear(x[:m], w)[::8, ::8], ref, dtype)
        if m > 128:                               # kept sums have the operands' type, whatever the outputs'
            other = torch.bfloat16 if dtype == torch.float16 else torch.float16
            out, pre = cp.linear(x[:m], w, dtype=other, pre=True)
            assert within(pre[::8, ::8], ref, dtype) and within(out[::8, ::8], ref, other)
    assert cp.linear_status() == cp.CP_OK


@pytest.mark.parametrize("m,n,k", [(20000, 2048, 2048), (400, 16000, 4096), (2048, 20000, 1024)])
def test_linear_grad_long_sums(m, n, k):
    dtype = torch.float16
    g = torch.Generator(device="cuda").manual_seed(m)
    dy, x, w = positive(g, m, n, 0.5, dtype), positive(g, m, k, 0.5, dtype), positive(g, n, k, 0.5, dtype)
    dx, dw, db = cp.linear_grad(dy, x, w, db_dtype=torch.float32)
    assert within(dx[::8, ::8], dy[::8].double() @ w[:, ::8].double(), dtype)
    assert within(dw[::8, ::8], dy[:, ::8].double().T @ x[:, ::8].double(), dtype)
    ref = dy.double().sum(0)
    assert float(((db.double() - ref) / ref).abs().max()) < (m / 8 + 64) * 2.0 ** -24
    assert cp.linear_status() == cp.CP_OK
