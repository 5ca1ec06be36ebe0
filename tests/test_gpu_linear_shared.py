"""Arrays of one call that share a buffer: columns beside one another are as good as buffers of their own,
outputs on what is read meanwhile are refused."""
import pytest
import torch

import trellis_row_decode_gb300 as cp

pytestmark = pytest.mark.gpu
BF = torch.bfloat16


@pytest.mark.parametrize("m", [1, 5, 128, 700])
def test_columns_of_one_array(m):
    n, k = 96, 160
    g = torch.Generator(device="cuda").manual_seed(m)
    wide = torch.randn(m, k + 3 * n, generator=g, device="cuda").to(BF)
    x, res, out, pre = wide.split([k, n, n, n], 1)
    w = torch.randn(n, k, generator=g, device="cuda").to(BF)
    dy = torch.randn(m, n, generator=g, device="cuda").to(BF)
    want = cp.linear(x.clone(), w, None, "silu", residual=res.clone(), pre=True)
    cp.linear(x, w, None, "silu", residual=res, out=out, pre=pre)
    assert torch.equal(out, want[0]) and torch.equal(pre, want[1])
    cp.linear(x, w, None, "silu", residual=res, out=res)               # the stream, in place
    assert torch.equal(res, want[0])
    want = cp.linear_grad(dy, x.clone(), w, "silu", pre.clone())
    out.copy_(dy)
    both = torch.empty(m, k + 64, dtype=BF, device="cuda")
    got = cp.linear_grad(out, x, w, "silu", pre, dx=both[:, :k])
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    want = cp.dropout(out.clone(), 0.3, 1, residual=res.clone())
    cp.dropout(out, 0.3, 1, residual=res, out=pre)
    assert torch.equal(pre, want)


@pytest.mark.parametrize("m", [3, 300])
def test_outputs_on_inputs_are_refused(m):
    n = 64
    x = torch.ones(m, n, dtype=BF, device="cuda")
    w = torch.ones(n, n, dtype=BF, device="cuda")
    y = torch.ones(m, n, dtype=BF, device="cuda")
    for call in [lambda: cp.linear(x, w, out=x), lambda: cp.linear(x, w, residual=x, out=x),
                 lambda: cp.linear(x, w, pre=x), lambda: cp.linear(x, w, residual=y, out=y, pre=y),
                 lambda: cp.linear_grad(y, x, w, dx=y), lambda: cp.linear_grad(y, x, w, dx=x),
                 lambda: cp.linear_grad(y, x, w, dw=w),
                 lambda: cp.dropout(x[1:], 0.5, out=x[:-1]),
                 lambda: cp.dropout(y[1:], 0.5, residual=x[:-1], out=x[1:])]:
        with pytest.raises(cp.CPError, match="lies on"):
            call()
    assert bool((x == 1).all()) and bool((w == 1).all()) and bool((y == 1).all())
    # dy that a pass of its own reads first may be written over, and a weight that is not read
    want = cp.linear_grad(y, x, w, p=0.5, seed=3)
    got = cp.linear_grad(y, x, w, p=0.5, seed=3, dx=y)
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    want = cp.linear_grad(y, x, w)[1]
    assert torch.equal(cp.linear_grad(y, x, w, need_dx=False, need_db=False, dw=w)[1], want)
