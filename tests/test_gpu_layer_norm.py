"""rms_norm, rms_norm_fp8, rms_norm_grad and quantize_fp8 against plain 64-bit forms.

Bounds: the kernels sum a row in fp32 through at most 48 terms a thread, 5 shuffles and
32 warps, so mean(s^2) is off by at most 88 U32, r by 44 U32 and some roundings, y by
K = 64 U32 relative; the gradient's sums pass twice through such a tree (K = 160 U32 of
the magnitudes they add).
"""
import pytest
import torch

import trellis_row_decode_gb300 as cp

from layer_util import (DTYPES, E4M3, TINY, U32, UNIT, assert_within, gen, norm64, norm_grad64,
                        randn, rounded, scales64)

pytestmark = pytest.mark.gpu
K = 64 * U32
KG = 160 * U32
SHAPES = [(1, 1), (3, 7), (5, 64), (1, 128), (9, 129), (2, 1000), (33, 1024), (4, 1025), (3, 2048),
          (17, 4096), (3, 4104), (2, 8192), (2, 9000), (3, 16384), (2, 24576), (1, 49152)]


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("m,d", SHAPES)
def test_norm_matches(m, d, dtype):
    g = gen(m * d)
    x, res = randn(g, m, d, dtype=dtype), randn(g, m, d, dtype=dtype, std=3.0)
    if m > 2:
        x[1] = 0
        res[1] = 0                                     # a row of zeros: r = 1 / sqrt(eps)
    w = randn(g, d)
    y, h = cp.rms_norm(x.cuda(), w.cuda(), 1e-5, residual=res.cuda())
    ry, rs = norm64(x, w, 1e-5, res)
    cancel = (x.double().abs() + res.double().abs()) * U32       # of the sum itself
    assert_within(h, rs, cancel * 0 + rs.abs() * U32 + rounded(rs, dtype))
    assert_within(y, ry, ry.abs() * K + rounded(ry, dtype))
    y2 = cp.rms_norm(x.cuda(), w.cuda(), 1e-5)
    ry2, _ = norm64(x, w, 1e-5)
    assert_within(y2, ry2, ry2.abs() * K + rounded(ry2, dtype))


def _check_q(q, scales, ref, block=1, rel=K):
    sc, spread = scales64(ref, block)
    assert q.dtype == E4M3 and scales.shape == sc.shape
    assert_within(scales, sc, sc * (rel + 2 * U32), "scales")
    got = q.cpu().float().double() * scales.cpu().double().repeat_interleave(block, 0)[
        :ref.shape[0]].repeat_interleave(128, 1)[:, :ref.shape[1]]
    # half a step of e4m3: 2^-4 of a normal value, 2^-10 of the scale below; y itself and
    # the multiplication by the rounded reciprocal (2 U32) add their own errors
    step = torch.maximum(ref.abs() * 2.0 ** -4, spread * 2.0 ** -10)
    assert_within(got, ref, step * (1 + 1e-5) + ref.abs() * (rel + 4 * U32) * 1.1, "values")


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("m,d", SHAPES)
def test_norm_fp8_matches(m, d, dtype):
    g = gen(m + d)
    x, res = randn(g, m, d, dtype=dtype), randn(g, m, d, dtype=dtype)
    res[:, ::97] *= 30                                  # a few strong channels
    if m > 2:
        x[1] = 0
        res[1] = 0
    w = 1 + randn(g, d, dtype=torch.bfloat16, std=0.3)
    q, sc, h = cp.rms_norm_fp8(x.cuda(), w.cuda(), 1e-6, residual=res.cuda())
    ry, rs = norm64(x, w, 1e-6, res)
    _check_q(q, sc, ry)
    assert_within(h, rs, rs.abs() * U32 + rounded(rs, dtype))
    q2, sc2 = cp.rms_norm_fp8(x.cuda(), w.cuda(), 1e-6)
    _check_q(q2, sc2, norm64(x, w, 1e-6)[0])


def test_norm_in_place_strides_and_shapes():
    g = gen(4)
    for d in (512, 77, 20000):
        wide = randn(g, 6, d + 60, dtype=torch.bfloat16).cuda()
        x = wide[:, 8:8 + d]
        res = randn(g, 6, d, dtype=torch.bfloat16).cuda()
        w = randn(g, d, dtype=torch.float16).cuda()
        y, h = cp.rms_norm(x.contiguous(), w, residual=res.clone())
        stream = res.clone()
        y2, h2 = cp.rms_norm(x, w, residual=stream, residual_out=stream)
        assert h2 is stream and torch.equal(y, y2) and torch.equal(h, stream)
        xin = x.contiguous()
        y3, h3 = cp.rms_norm(xin, w, residual=res, out=xin)
        assert torch.equal(y3, y) and torch.equal(h3, h)
        row = res[:1].expand(6, d)                       # one row for all (stride 0)
        y4, h4 = cp.rms_norm(x, w, residual=row)
        y5, h5 = cp.rms_norm(x, w, residual=row.contiguous())
        assert torch.equal(y4, y5) and torch.equal(h4, h5)
        y6 = cp.rms_norm(res.view(2, 3, d), w)
        assert y6.shape == (2, 3, d) and torch.equal(y6.view(6, d), cp.rms_norm(res, w))
        q, sc = cp.rms_norm_fp8(res.view(2, 3, d), w)
        assert q.shape == (2, 3, d) and sc.shape == (2, 3, -(-d // 128))


def test_norm_not_finite():
    """NaN and infinity stay in their row, and in 8 bits poison what the formula says."""
    x = torch.ones(4, 300, device="cuda")
    x[1, 5] = float("nan")
    x[2, 200] = float("inf")
    w = torch.ones(300, device="cuda")
    y = cp.rms_norm(x, w)
    assert torch.isfinite(y[0]).all() and torch.isfinite(y[3]).all()
    assert torch.isnan(y[1]).all()
    assert torch.isnan(y[2, 200]) and not y[2, :200].any()     # inf * 0, 1 * 0
    q, sc = cp.rms_norm_fp8(x, w)
    assert torch.isnan(sc[1]).all() and torch.isnan(q[1].float()).all()
    assert torch.isnan(sc[2, 1]) and torch.isfinite(sc[2, 0])
    q, sc = cp.quantize_fp8(x)
    assert torch.isnan(sc[1, 0]) and torch.isfinite(sc[1, 1])
    assert torch.isinf(sc[2, 1]) and torch.isnan(q[2, 200].float())
    assert not q[2, 128:200].float().any()                     # 1 / inf


def test_norm_empty_and_eps():
    w = torch.ones(16, device="cuda")
    assert cp.rms_norm(torch.empty(0, 16, device="cuda"), w).shape == (0, 16)
    q, sc = cp.rms_norm_fp8(torch.empty(0, 16, device="cuda"), w)
    assert q.shape == (0, 16) and sc.shape == (0, 1)
    dx, dw = cp.rms_norm_grad(torch.empty(0, 16, device="cuda"),
                              torch.empty(0, 16, device="cuda"), w)
    assert dx.shape == (0, 16) and not dw.any()
    y = cp.rms_norm(torch.zeros(2, 16, device="cuda"), w, 0.0)
    assert torch.isnan(y).all()                                # 0 / 0, as the formula says


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("m,d", SHAPES + [(700, 96), (3000, 264), (1300, 2056), (400, 8200)])
def test_norm_grad_matches(m, d, dtype):
    g = gen(m * 3 + d)
    h, dy = randn(g, m, d, dtype=dtype, std=2.0), randn(g, m, d, dtype=dtype)
    dres = randn(g, m, d, dtype=dtype)
    w = randn(g, d)
    for res in (dres, None):
        dx, dw = cp.rms_norm_grad(dy.cuda(), h.cuda(), w.cuda(), 1e-5,
                                  dres=None if res is None else res.cuda())
        rx, rx_mag, rw, rw_mag = norm_grad64(dy, h, w, 1e-5, res)
        assert_within(dx, rx, rx_mag * KG + rounded(rx, dtype), "dx")
        # a CTA adds at most ceil(m / ctas) rows, 38 parts a warp, 32 warps: m terms bound them all
        assert_within(dw, rw, rw_mag * (min(m, 400) + 80) * U32 + rounded(rw, torch.float32), "dw")


def test_norm_grad_weight_types_strides_and_in_place():
    g = gen(11)
    for d in (256, 99, 9000):
        m = 37
        h = randn(g, m, d + 32, dtype=torch.bfloat16).cuda()[:, 16:16 + d]
        dy = randn(g, m, d, dtype=torch.bfloat16).cuda()
        dres = randn(g, m, d, dtype=torch.bfloat16).cuda()
        for wt in DTYPES:
            w = randn(g, d, dtype=wt)
            dx, dw = cp.rms_norm_grad(dy, h, w.cuda(), dres=dres)
            rx, rx_mag, rw, rw_mag = norm_grad64(dy.cpu(), h.cpu(), w, 1e-6, dres.cpu())
            assert dw.dtype == wt
            assert_within(dx, rx, rx_mag * KG + rounded(rx, torch.bfloat16))
            assert_within(dw, rw, rw_mag * (m + 80) * U32 + rounded(rw, wt))
            into = dres.clone()
            dx2, dw2 = cp.rms_norm_grad(dy, h, w.cuda(), dres=into, dx=into)
            assert torch.equal(dx2, dx) and torch.equal(dw2, dw)
            into = dy.clone()
            dx3, dw3 = cp.rms_norm_grad(into, h, w.cuda(), dres=dres, dx=into)
            assert torch.equal(dx3, dx) and torch.equal(dw3, dw)
        one = dy[:1].expand(m, d)
        dx4, dw4 = cp.rms_norm_grad(one, h, w.cuda())
        dx5, dw5 = cp.rms_norm_grad(one.contiguous(), h, w.cuda())
        assert torch.equal(dx4, dx5) and torch.equal(dw4, dw5)


def test_norm_grad_against_differences():
    """Directional derivatives of the 64-bit forward, by central differences."""
    g = gen(21)
    m, d, eps, t = 6, 160, 1e-3, 1e-4
    h, w, dy = randn(g, m, d), randn(g, d), randn(g, m, d)
    dx, dw = cp.rms_norm_grad(dy.cuda(), h.cuda(), w.cuda(), eps)

    def value(hh, ww):
        r = 1.0 / torch.sqrt(hh.square().mean(-1, keepdim=True) + eps)
        return (dy.double() * hh * r * ww).sum()

    for _ in range(4):
        vh, vw = randn(g, m, d).double(), randn(g, d).double()
        along = (value(h.double() + t * vh, w.double()) - value(h.double() - t * vh, w.double()))
        ref = float(along) / (2 * t)
        got = float((dx.cpu().double() * vh).sum())
        # truncation t^2 times third derivatives of order one per element; fp32 gradients
        assert abs(got - ref) <= m * d * (10 * t * t + 20 * U32)
        along = (value(h.double(), w.double() + t * vw) - value(h.double(), w.double() - t * vw))
        ref = float(along) / (2 * t)
        got = float((dw.cpu().double() * vw).sum())
        assert abs(got - ref) <= m * d * 40 * U32


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("block", [1, 128])
@pytest.mark.parametrize("m,k", [(1, 1), (1, 128), (3, 130), (127, 256), (128, 128), (129, 1000),
                                 (300, 2304), (5, 24576), (1000, 77)])
def test_quantize_matches(m, k, block, dtype):
    g = gen(m * k + block)
    x = randn(g, m, k, dtype=dtype)
    x[:, : k // 3] *= 0.01
    if m > 2:
        x[2] = 0
    q, sc = cp.quantize_fp8(x.cuda(), block)
    _check_q(q, sc, x.double(), block, rel=0)


@pytest.mark.parametrize("d", [7, 130, 265])
def test_e4m3_rows_that_start_on_any_byte(d):
    """Rows of odd length put the 8-bit output on every byte boundary; an output buffer of the
    caller's is written to its last byte and no further."""
    g = gen(d)
    m = 41
    x = randn(g, m, d)
    for offset in range(9):
        buf = torch.full((m * d + 16,), 0x7F, dtype=torch.uint8, device="cuda")
        out = buf[offset:offset + m * d].view(m, d).view(E4M3)
        q, sc = cp.quantize_fp8(x.cuda(), 1, out=out)
        _check_q(q, sc, x.double(), rel=0)
        assert bool((buf[:offset] == 0x7F).all()) and bool((buf[offset + m * d:] == 0x7F).all())
        q, sc = cp.quantize_fp8(x.cuda(), 128, out=out)
        _check_q(q, sc, x.double(), 128, rel=0)
        assert bool((buf[:offset] == 0x7F).all()) and bool((buf[offset + m * d:] == 0x7F).all())


def test_quantize_extremes_and_views():
    x = torch.zeros(4, 256)
    x[0, :128] = 1e-38                                  # below the smallest amax: zeros
    x[1, 0], x[1, 1] = 3e38, -3e38                      # the type's largest
    x[2, :2] = torch.tensor([448.0, 464.0])
    q, sc = cp.quantize_fp8(x.cuda())
    assert not q[0].float().any() and float(sc[0, 0]) == pytest.approx(1e-30 / 448, rel=1e-6)
    assert q[1, :2].float().tolist() == [448, -448]
    assert torch.isfinite(q.float()).all() and torch.isfinite(sc).all()
    wide = torch.randn(300, 500, device="cuda").to(torch.float16)
    for lo, hi in [(0, 256), (8, 136), (5, 300)]:
        for block in (1, 128):
            a, b = cp.quantize_fp8(wide[:, lo:hi], block), cp.quantize_fp8(
                wide[:, lo:hi].contiguous(), block)
            assert torch.equal(a[0].view(torch.uint8), b[0].view(torch.uint8))
            assert torch.equal(a[1], b[1])
    q, sc = cp.quantize_fp8(torch.empty(0, 5, device="cuda"), 128)
    assert q.shape == (0, 5) and sc.shape == (0, 1)


def test_norm_on_another_stream_and_in_a_graph():
    g = gen(31)
    x, res = randn(g, 300, 2048, dtype=torch.bfloat16).cuda(), randn(
        g, 300, 2048, dtype=torch.bfloat16).cuda()
    w = randn(g, 2048).cuda()
    torch.cuda.synchronize()
    ref = cp.rms_norm_fp8(x, w, residual=res)
    rgrad = cp.rms_norm_grad(res, x, w, dres=x)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    got = cp.rms_norm_fp8(x, w, residual=res, stream=s)
    grad = cp.rms_norm_grad(res, x, w, dres=x, stream=s)
    s.synchronize()
    for a, b in zip(ref + rgrad, got + grad):
        assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))
    q, sc, h = (torch.zeros_like(t) for t in ref)
    dx, dw = (torch.zeros_like(t) for t in rgrad)
    ws = cp.rms_norm_grad_workspace(300, 2048)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        cp.rms_norm_fp8(x, w, residual=res, out=q, scales=sc, residual_out=h)
        cp.rms_norm_grad(res, x, w, dres=x, dx=dx, dw=dw, workspace=ws)
    graph.replay()
    torch.cuda.synchronize()
    for a, b in zip(ref + rgrad, (q, sc, h, dx, dw)):
        assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))


def test_norm_refusals():
    x = torch.zeros(4, 64, device="cuda")
    w = torch.ones(64, device="cuda")
    for call in [
        lambda: cp.rms_norm(x.double(), w),
        lambda: cp.rms_norm(x, w[:63]),
        lambda: cp.rms_norm(x, w.double()),
        lambda: cp.rms_norm(x.t(), torch.ones(4, device="cuda")),
        lambda: cp.rms_norm(x, w, residual=x.bfloat16()),
        lambda: cp.rms_norm(x, w, residual=x[:3]),
        lambda: cp.rms_norm(x, w, residual_out=x),
        lambda: cp.rms_norm(x, w, out=x.bfloat16()),
        lambda: cp.rms_norm(x.cpu(), w),
        lambda: cp.rms_norm_fp8(x, w, out=torch.zeros(4, 64, device="cuda")),
        lambda: cp.rms_norm_fp8(x, w, scales=torch.zeros(4, 2, device="cuda")),
        lambda: cp.rms_norm_grad(x, x[:3], w),
        lambda: cp.rms_norm_grad(x, x, w, dres=x.bfloat16()),
        lambda: cp.rms_norm_grad(x, x, w, workspace=torch.zeros(1, dtype=torch.uint8,
                                                                device="cuda")),
        lambda: cp.quantize_fp8(x, 64),
        lambda: cp.quantize_fp8(x[0]),
    ]:
        with pytest.raises(ValueError):
            call()
    wide = torch.zeros(1, 50000, device="cuda")
    for call in [lambda: cp.rms_norm(wide, wide[0]), lambda: cp.rms_norm(x, w, -1.0),
                 lambda: cp.rms_norm(x, w, float("nan")),
                 lambda: cp.rms_norm_grad_workspace(4, 50000)]:
        with pytest.raises(cp.CPError):
            call()
