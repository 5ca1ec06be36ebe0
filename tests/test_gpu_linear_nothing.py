"""Products of no columns (k = 0) in every shape and in both forms of a call: the sums are zeros, one
for each row that the leading dimensions have."""
import pytest
import torch

import trellis_row_decode_gb300 as cp

from layer_util import randn, gen

pytestmark = pytest.mark.gpu
BF = torch.bfloat16
LEADS = [(), (7,), (2, 3), (300,), (5, 1, 60), (0, 4), (4, 0)]


@pytest.mark.parametrize("lead", LEADS)
@pytest.mark.parametrize("form", ["common", "stream", "out"])
def test_linear_of_no_columns(lead, form):
    bias = randn(gen(1), 70).cuda()
    x, w = torch.empty(*lead, 0, dtype=BF, device="cuda"), torch.empty(70, 0, dtype=BF, device="cuda")
    out = torch.full((*lead, 70), float("nan"), device="cuda")
    pre = torch.full((*lead, 70), float("nan"), dtype=BF, device="cuda")
    s = torch.cuda.current_stream()
    kw = {"common": dict(dtype=torch.float32, pre=True),
          "stream": dict(dtype=torch.float32, pre=True, stream=s),
          "out": dict(out=out, pre=pre)}[form]
    out, pre = cp.linear(x, w, bias, "relu", **kw)
    assert out.shape == pre.shape == (*lead, 70)
    assert torch.equal(out, bias.clamp(min=0).expand(*lead, 70))
    assert torch.equal(pre, bias.to(BF).expand(*lead, 70))


@pytest.mark.parametrize("lead", LEADS)
@pytest.mark.parametrize("form", ["common", "stream", "given"])
def test_linear_grad_of_no_columns(lead, form):
    dy = torch.ones(*lead, 40, dtype=BF, device="cuda")
    x, w = torch.empty(*lead, 0, dtype=BF, device="cuda"), torch.empty(40, 0, dtype=BF, device="cuda")
    db = torch.full((40,), float("nan"), device="cuda")
    kw = {"common": dict(db_dtype=torch.float32),
          "stream": dict(db_dtype=torch.float32, stream=torch.cuda.current_stream()),
          "given": dict(db=db, dx=torch.empty_like(x), dw=torch.empty_like(w))}[form]
    dx, dw, db = cp.linear_grad(dy, x, w, **kw)
    assert dx.shape == x.shape and dw.shape == w.shape
    rows = dy[..., 0].numel()
    assert torch.equal(db, torch.full((40,), float(rows), device="cuda"))


@pytest.mark.parametrize("lead", [(7,), (2, 3), (5, 1, 60), (4, 0)])
def test_matmul_fp8_of_no_columns(lead):
    a = torch.empty(*lead, 0, device="cuda").to(torch.float8_e4m3fn)
    w = torch.empty(70, 0, device="cuda").to(torch.float8_e4m3fn)
    out = torch.full((*lead, 70), float("nan"), device="cuda")
    cp.matmul_fp8(a, torch.empty(*lead, 0, device="cuda"), w, torch.empty(1, 0, device="cuda"),
                  out=out)
    assert bool((out == 0).all())
