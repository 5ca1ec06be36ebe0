"""The norm's gradient on rows so small that their mean square is a subnormal number, with eps = 0.

Bounds: as in test_gpu_layer_norm.py (KG of the magnitudes), and for the sum of squares: each of its
d terms and its mean round to multiples of 2^-149, so the mean is off by at most 2 * 2^-150 beyond
the ordinary roundings, a share e = 2^-149 / mean(h^2) of it.  r carries half of that, r n mean(t n)
three halves.
"""
import pytest
import torch

import trellis_row_decode_gb300 as cp

from layer_util import U32, assert_within, gen, norm_grad64, randn, rounded

pytestmark = pytest.mark.gpu
KG = 160 * U32


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("size", [4.5e-20, 1e-20])
@pytest.mark.parametrize("m,d", [(5, 96), (7, 257), (3, 2048), (2, 4001), (2, 9000), (300, 1024)])
def test_gradient_of_tiny_rows(m, d, size, dtype):
    g = gen(m + d)
    h = (torch.sign(randn(g, m, d)) * size * (1 + 0.1 * torch.rand(m, d, generator=g))).to(dtype)
    dy, dres, w = randn(g, m, d, dtype=dtype), randn(g, m, d, dtype=dtype), randn(g, d)
    dx, dw = cp.rms_norm_grad(dy.cuda(), h.cuda(), w.cuda(), 0.0, dres=dres.cuda())
    rx, rx_mag, rw, rw_mag = norm_grad64(dy, h, w, 0.0, dres)
    e = 2.0 ** -149 / h.double().square().mean(-1, keepdim=True)
    assert torch.isfinite(dx).all() and torch.isfinite(dw).all()
    assert_within(dx, rx, rx_mag * (KG + 2 * e) + rounded(rx, dtype), "dx")
    assert_within(dw, rw, rw_mag * ((min(m, 400) + 80) * U32 + float(e.max())) +
                  rounded(rw, torch.float32), "dw")
