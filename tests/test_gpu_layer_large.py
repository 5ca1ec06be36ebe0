"""The memory layer's operators where an index passes 32 bits: many groups, long rows, far rows."""
import pytest
import torch

import trellis_row_decode_gb300 as cp

from layer_util import E4M3, U32, assert_within, scales64

pytestmark = pytest.mark.gpu


def test_quantize_past_2_30_groups():
    """2^30 + 100 rows of one column: a group each, and 256 threads for 64 of them, so a thread's
    own index passes 2^32.  Every group is written: the buffers start as NaN."""
    rows = (1 << 30) + 100
    x = torch.empty(rows, 1, dtype=torch.bfloat16, device="cuda")
    slab = 1 << 27
    for lo in range(0, rows, slab):
        i = torch.arange(lo, min(lo + slab, rows), device="cuda")
        x[lo:lo + slab, 0] = ((i * 2654435761 >> 9) % 255 - 127).to(torch.bfloat16)
    q = torch.full((rows, 1), 0x7F, dtype=torch.uint8, device="cuda").view(E4M3)
    scales = torch.full((rows, 1), float("nan"), device="cuda")
    cp.quantize_fp8(x, 1, out=q, scales=scales)
    for lo in range(0, rows, slab):
        v = x[lo:lo + slab, 0].float()
        # one rounded division; |v| / scale is 448 up to two roundings, and 448 is the nearest value
        ref = v.abs().clamp(min=1e-30) / 448.0
        assert bool(((scales[lo:lo + slab, 0] - ref).abs() <= 4 * U32 * ref).all()), lo
        assert torch.equal(q[lo:lo + slab, 0].float(), 448.0 * torch.sign(v)), lo


@pytest.mark.parametrize("block", [1, 128])
def test_quantize_a_row_of_almost_2_32_columns(block):
    """The last octet of the row is part full and its end lies past 2^32: nothing is written
    behind the row, and the last groups are what their own columns say."""
    d = (1 << 32) - 3
    x = torch.empty(1, d, dtype=torch.bfloat16, device="cuda")
    piece = torch.randn(1 << 24, generator=torch.Generator().manual_seed(block)).bfloat16().cuda()
    for lo in range(0, d, 1 << 24):
        n = min(1 << 24, d - lo)
        torch.mul(piece[:n], 1 + lo / d, out=x[0, lo:lo + n])
    buf = torch.full((d + 64,), 0x55, dtype=torch.uint8, device="cuda")
    groups = (d + 127) // 128
    scales = torch.full((1, groups), float("nan"), device="cuda")
    q = buf[:d].view(1, d).view(E4M3)
    cp.quantize_fp8(x, block, out=q, scales=scales)
    assert bool((buf[d:] == 0x55).all())
    assert bool(torch.isfinite(scales).all())
    for g0, g1 in ((0, 40), (groups // 2 - 20, groups // 2 + 20), (groups - 40, groups)):
        lo, hi = g0 * 128, min(g1 * 128, d)
        ref = x[:, lo:hi].cpu().double()
        sc, spread = scales64(ref, 1)
        assert_within(scales[:, g0:g1], sc, sc * 4 * U32, "scales")
        got = q[:, lo:hi].cpu().float().double() * spread
        step = torch.maximum(ref.abs() * 2.0 ** -4, spread * 2.0 ** -10)
        assert_within(got, ref, step * (1 + 1e-5) + ref.abs() * 8 * U32, "values")


def test_rows_of_2_32_columns_are_refused():
    """The library takes a row's length in 32 bits; a longer row is no row of length mod 2^32."""
    d = (1 << 32) + 128
    x = torch.empty(1, d, dtype=torch.bfloat16, device="cuda")
    w = torch.ones(128, device="cuda")
    ids = torch.zeros(1, dtype=torch.int64, device="cuda")
    for call in [lambda: cp.quantize_fp8(x), lambda: cp.quantize_fp8(x, 128),
                 lambda: cp.rms_norm(x, w), lambda: cp.rms_norm(x[0], w),
                 lambda: cp.rms_norm_fp8(x, w), lambda: cp.rms_norm_fp8(x.view(1, 1, d), w),
                 lambda: cp.rms_norm_grad(x, x, w), lambda: cp.embed(x, ids),
                 lambda: cp.embed_grad(x, ids, 1)]:
        with pytest.raises(ValueError):
            call()
