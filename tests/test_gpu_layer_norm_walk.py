"""The norms and their gradient where every team of threads walks over five rows and more: the next
rows' loads, the turns of the ring and of the sums' two halves, words shared between warps.  One
width for each team, on and off boundaries of eight elements; 64-bit forms, computed on the device.

Bounds: as in test_gpu_layer_norm.py (K and KG); the gradient by the weight adds at most 8 rows a
team, 64 teams a CTA, 16 parts a warp and 32 warps.
"""
import pytest
import torch

import trellis_row_decode_gb300 as cp

from layer_util import DTYPES, TINY, U32, UNIT, norm_grad64

pytestmark = pytest.mark.gpu
K, KG = 64 * U32, 160 * U32
SMS = 152
# (d on octet boundaries, d off them, teams that run at once in the forward pass)
WIDTHS = [(32, 29, 192), (64, 61, 96), (128, 125, 48), (256, 250, 24), (512, 505, 24),
          (1024, 1001, 12), (1536, 1531, 8), (2048, 2001, 6), (3000, 2999, 4), (4096, 4001, 3),
          (6144, 6001, 2), (8192, 8001, 1), (16384, 16001, 1)]
CASES = [(d, teams) for on, off, teams in WIDTHS for d in (on, off)]


def _within(got, ref, bound, what):
    off = (got.double() - ref).abs()
    assert bool((off <= bound).all()), (what, float((off / bound).max()))


def _rounded(ref, dtype):
    return ref.abs() * UNIT[dtype] + TINY[dtype]


def _inputs(m, d, dtype, seed, count):
    g = torch.Generator(device="cuda").manual_seed(seed)
    rows = torch.exp(torch.randn(m, 1, generator=g, device="cuda"))        # each row its own size
    return [(rows * torch.randn(m, d, generator=g, device="cuda")).to(dtype) for _ in range(count)] + [
        torch.randn(d, generator=g, device="cuda")]


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("d,teams", CASES)
def test_norm_of_many_rows(d, teams, dtype):
    m = 5 * SMS * teams + 3
    x, res, w = _inputs(m, d, dtype, d, 2)
    groups = -(-d // 128)
    for r in (res, None):
        s = x.double() + (r.double() if r is not None else 0.0)
        y = s / torch.sqrt(s.square().mean(-1, keepdim=True) + 1e-5) * w.double()
        got = cp.rms_norm(x, w, 1e-5, residual=r)
        got8 = cp.rms_norm_fp8(x, w, 1e-5, residual=r)
        if r is not None:
            for h in (got[1], got8[2]):
                _within(h, s, s.abs() * U32 + _rounded(s, dtype), "h")
            got = got[0]
        _within(got, y, y.abs() * K + _rounded(y, dtype), "y")
        pad = torch.nn.functional.pad(y, (0, groups * 128 - d)).view(m, groups, 128)
        scales = pad.abs().amax(-1).clamp(min=1e-30) / 448.0
        _within(got8[1], scales, scales * (K + 2 * U32), "scales")
        spread = scales.repeat_interleave(128, 1)[:, :d]
        back = got8[0].double() * got8[1].double().repeat_interleave(128, 1)[:, :d]
        step = torch.maximum(y.abs() * 2.0 ** -4, spread * 2.0 ** -10)
        _within(back, y, step * (1 + 1e-5) + y.abs() * (K + 4 * U32) * 1.1, "e4m3")


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("d,teams", CASES)
def test_norm_grad_of_many_rows(d, teams, dtype):
    m = 5 * SMS * teams + 3
    h, dy, dres, w = _inputs(m, d, dtype, d + 1, 3)
    for r in (dres, None):
        dx, dw = cp.rms_norm_grad(dy, h, w, 1e-5, dres=r)
        rx, rx_mag, rw, rw_mag = norm_grad64(dy, h, w, 1e-5, r)
        _within(dx, rx, rx_mag * KG + _rounded(rx, dtype), "dx")
        _within(dw, rw, rw_mag * (8 + 64 + 16 + 32 + 44) * U32 + _rounded(rw, torch.float32), "dw")
