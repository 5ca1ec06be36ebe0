"""linear against a plain 64-bit form: one row to many, odd sizes and strides, each activation,
bias, dropout and residual, kept sums, graphs, streams, refusals."""
import pytest
import torch

import trellis_row_decode_gb300 as cp

from layer_util import DTYPES, U32, assert_within, gen, randn, rounded
from linear_util import ACTS, linear64, out_bound, sum_bound

pytestmark = pytest.mark.gpu
HALF = [torch.bfloat16, torch.float16]


def _case(m, n, k, dtype, seed=0):
    g = gen(seed + m * n + k)
    return randn(g, m, k, dtype=dtype), randn(g, n, k, dtype=dtype, std=max(k, 1) ** -0.5), g


def _check(got, x, w, dtype, **kw):
    out, z, mag = linear64(x, w, **kw)
    assert_within(got, out, out_bound(out, z, mag, x.shape[1], dtype, kw.get("p", 0.0)))


SIZES = [(1, 1, 1), (1, 64, 64), (1, 4096, 1024), (1, 1000, 24576), (2, 77, 304), (3, 130, 2320),
         (8, 256, 512), (16, 512, 384), (17, 129, 1040), (32, 128, 256), (33, 257, 272),
         (48, 1024, 2048), (65, 1000, 1000), (128, 128, 128), (128, 130, 129), (129, 384, 2304),
         (200, 2050, 528), (256, 256, 1024), (257, 32, 8192), (333, 1001, 2321), (513, 770, 896),
         (1024, 1024, 512), (2000, 40, 64), (700, 4096, 32), (130, 5, 3), (129, 1, 1)]


@pytest.mark.parametrize("m,n,k", SIZES)
def test_linear_matches(m, n, k):
    x, w, _ = _case(m, n, k, torch.bfloat16)
    got = cp.linear(x.cuda(), w.cuda(), dtype=torch.float32)
    _check(got, x, w, torch.float32)
    assert torch.equal(got, cp.linear(x.cuda(), w.cuda(), dtype=torch.float32))   # the same bits
    assert cp.linear_status() == cp.CP_OK


@pytest.mark.parametrize("dtype", HALF)
@pytest.mark.parametrize("out", DTYPES)
@pytest.mark.parametrize("m,n,k", [(1, 300, 512), (20, 200, 256), (150, 390, 400), (300, 288, 96),
                                   (70, 33, 77), (260, 64, 3000)])
def test_linear_types(m, n, k, dtype, out):
    x, w, _ = _case(m, n, k, dtype)
    _check(cp.linear(x.cuda(), w.cuda(), dtype=out), x, w, out)


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("p", [0.0, 0.3])
@pytest.mark.parametrize("m,n,k", [(5, 260, 320), (140, 192, 256), (300, 205, 64), (160, 96, 4000)])
def test_linear_epilogue(m, n, k, act, p):
    """Everything at once, the sums kept, for each kernel and both ways to store."""
    x, w, g = _case(m, n, k, torch.bfloat16)
    bias, res = randn(g, n, dtype=torch.bfloat16), randn(g, m, n, dtype=torch.bfloat16)
    seed, offset = 0x1234567890ABCDEF, (7 << 40) + 3
    got, pre = cp.linear(x.cuda(), w.cuda(), bias.cuda(), act, residual=res.cuda(), p=p, seed=seed,
                         offset=offset, pre=True)
    out, z, mag = linear64(x, w, bias, act, res, p, seed, offset)
    assert_within(got, out, out_bound(out, z, mag, k, torch.bfloat16, p))
    assert_within(pre, z, sum_bound(mag, k) + rounded(z, torch.bfloat16))
    # in 32 bits, without the sums, in place of the residual
    stream = res.float().cuda()
    assert cp.linear(x.cuda(), w.cuda(), bias.float().cuda(), act, residual=stream, p=p, seed=seed,
                     offset=offset, out=stream) is stream
    assert_within(stream, out, out_bound(out, z, mag, k, torch.float32, p))


@pytest.mark.parametrize("act", ACTS)
def test_activations_over_their_range(act):
    """z itself through a product with one: values from the smallest to where they saturate."""
    z = torch.cat([torch.linspace(-100, 100, 2001), torch.linspace(-1, 1, 1001),
                   torch.tensor([0.0, 1e-30, -1e-30, 65504.0, -65504.0])]).bfloat16()
    x, one = z[:, None].contiguous(), torch.ones(1, 1, dtype=torch.bfloat16)
    got = cp.linear(x.cuda(), one.cuda(), None, act, dtype=torch.float32)
    _check(got, x, one, torch.float32, act=act)


@pytest.mark.parametrize("m", [3, 200])
def test_linear_strides_and_boundaries(m):
    """Rows apart, off 16-byte boundaries, repeated (stride 0), NaN around them."""
    n, k = 130, 200
    g = gen(m)

    def rows(count, width, pitch, offset, dtype=torch.bfloat16):
        buf = torch.full((count * pitch + 64,), float("nan"), dtype=dtype, device="cuda")
        view = torch.as_strided(buf, (count, width), (pitch, 1), offset)
        view.copy_(randn(g, count, width, dtype=dtype))
        return view
    for px, ox, pw, ow, po, oo in [(208, 0, 216, 8, 160, 16), (201, 1, 200, 0, 131, 1),
                                   (200, 0, 203, 5, 144, 3), (205, 3, 201, 7, 130, 0)]:
        x, w = rows(m, k, px, ox), rows(n, k, pw, ow)
        res = rows(m, n, po + 2, oo)
        buf = torch.full((m * po + 64,), 7.0, dtype=torch.bfloat16, device="cuda")
        keep = torch.full((m * po + 64,), 7.0, dtype=torch.bfloat16, device="cuda")
        out = torch.as_strided(buf, (m, n), (po, 1), oo)
        pre = torch.as_strided(keep, (m, n), (po, 1), oo)
        ws = cp.linear_workspace(x, w)
        cp.linear(x, w, None, "silu", residual=res, out=out, pre=pre, workspace=ws)
        ref, z, mag = linear64(x.cpu(), w.cpu(), None, "silu", res.cpu())
        assert_within(out, ref, out_bound(ref, z, mag, k, torch.bfloat16))
        assert_within(pre, z, sum_bound(mag, k) + rounded(z, torch.bfloat16))
        out.fill_(7.0)
        pre.fill_(7.0)
        assert bool((buf == 7).all()) and bool((keep == 7).all())
    x, w = randn(g, 1, k, dtype=torch.float16), randn(g, 1, k, dtype=torch.float16)
    res = randn(g, 1, n, dtype=torch.float16)
    got = cp.linear(x.cuda().expand(m, k), w.cuda().expand(n, k), residual=res.cuda().expand(m, n))
    _check(got, x.expand(m, k), w.expand(n, k), torch.float16, residual=res.expand(m, n))


@pytest.mark.parametrize("m", [3, 300])
@pytest.mark.parametrize("n", [121, 124, 126, 128, 130, 132, 136, 200])
def test_linear_writes_its_columns_alone(m, n):
    """Rows on 16-byte boundaries whose ends are not: what lies behind them stays, in each type, with
    the residual and the kept sums on such rows too."""
    x, w, g = _case(m, n, 72, torch.bfloat16)
    for dtype in DTYPES:
        buf = torch.full((m + 1, 208), 7.0, dtype=dtype, device="cuda")
        keep = torch.full((m + 1, 208), 7.0, dtype=torch.bfloat16, device="cuda")
        wide = torch.full((m, 208), float("nan"), dtype=dtype, device="cuda")
        res = wide[:, :n]
        res.copy_(randn(g, m, n, dtype=dtype))
        for r in (None, res):
            cp.linear(x.cuda(), w.cuda(), None, "relu", residual=r, out=buf[:m, :n],
                      pre=keep[:m, :n])
            out, z, mag = linear64(x, w, None, "relu", None if r is None else r.cpu())
            assert_within(buf[:m, :n], out, out_bound(out, z, mag, 72, dtype))
            assert_within(keep[:m, :n], z, sum_bound(mag, 72) + rounded(z, torch.bfloat16))
            for t in (buf, keep):
                assert bool((t[:, n:] == 7).all()) and bool((t[m] == 7).all())


@pytest.mark.parametrize("m", [3, 300])
@pytest.mark.parametrize("k", [1, 63, 65, 130, 201, 204, 519])
def test_linear_reads_its_columns_alone(m, k):
    """Rows on 16-byte boundaries with NaN behind their ends, for either operand."""
    g = gen(m + k)
    n, ld = 140, -(-k // 8) * 8 + 16
    x = torch.full((m, ld), float("nan"), dtype=torch.float16)
    w = torch.full((n, ld), float("nan"), dtype=torch.float16)
    x[:, :k], w[:, :k] = randn(g, m, k, dtype=torch.float16), randn(g, n, k, dtype=torch.float16)
    got = cp.linear(x.cuda()[:, :k], w.cuda()[:, :k], dtype=torch.float32)
    _check(got, x[:, :k], w[:, :k], torch.float32)
    dy = randn(g, m, n, dtype=torch.float16)
    dx, dw, _ = cp.linear_grad(dy.cuda(), x.cuda()[:, :k], w.cuda()[:, :k])
    X, W, D = x[:, :k].double(), w[:, :k].double(), dy.double()
    assert_within(dx, D @ W, sum_bound(D.abs() @ W.abs(), n) + rounded(D @ W, torch.float16))
    assert_within(dw, D.T @ X, sum_bound(D.abs().T @ X.abs(), m) + rounded(D.T @ X, torch.float16))


@pytest.mark.parametrize("m", [1, 128, 129, 1000])
def test_linear_sums_of_nothing(m):
    bias = torch.randn(70)
    x, w = torch.empty(m, 0, dtype=torch.bfloat16), torch.empty(70, 0, dtype=torch.bfloat16)
    got = cp.linear(x.cuda(), w.cuda(), bias.cuda(), "silu", dtype=torch.float32)
    _check(got, x, w, torch.float32, bias=bias, act="silu")
    assert cp.linear(x.cuda(), w[:0].cuda()).shape == (m, 0)
    assert cp.linear(x[:0].cuda(), w.cuda()).shape == (0, 70)


@pytest.mark.parametrize("m", [2, 200])
def test_linear_special_values(m):
    """An infinity or NaN stays in its row or column; one that dropout drops leaves no trace."""
    n, k = 100, 96
    x, w, _ = _case(m, n, k, torch.bfloat16)
    x[1, 5], w[7, 9], w[7, 5] = float("nan"), float("inf"), 1.0
    got = cp.linear(x.cuda(), w.cuda(), dtype=torch.float32, p=0.5, seed=3)
    keep = torch.from_numpy(__import__("linear_util").mask64(m, n, 0.5, 3, 0).numpy())
    got = got.cpu()
    assert bool((got[~keep] == 0).all())
    assert bool(torch.isnan(got[1][keep[1]]).all())
    assert not bool(torch.isfinite(got[:, 7][keep[:, 7]]).any())
    rest = keep.clone()
    rest[1], rest[:, 7] = False, False
    assert bool(torch.isfinite(got[rest]).all())
    gone = cp.linear(x.cuda(), w.cuda(), dtype=torch.float32, p=1.0)
    assert bool((gone == 0).all())


def test_linear_shapes_and_dtypes_of_arguments():
    x, w, g = _case(6, 40, 48, torch.bfloat16)
    res = randn(g, 2, 3, 40)
    got = cp.linear(x.cuda().view(2, 3, 48), w.cuda(), residual=res.cuda(), dtype=torch.float32)
    assert got.shape == (2, 3, 40)
    _check(got.view(6, 40), x, w, torch.float32, residual=res.view(6, 40))
    one = cp.linear(x[0].cuda(), w.cuda(), dtype=torch.float32)
    assert one.shape == (40,)
    _check(one[None], x[:1], w, torch.float32)


@pytest.mark.parametrize("m", [4, 300])
def test_linear_in_a_graph_on_another_stream(m):
    """Captured with a seed on the device, replayed with others: the masks follow."""
    n, k = 128, 2000
    x, w, _ = _case(m, n, k, torch.bfloat16)
    xc, wc = x.cuda(), w.cuda()
    rng = torch.tensor([5, 10], dtype=torch.int64, device="cuda")
    out = torch.empty(m, n, device="cuda")
    ws = cp.linear_workspace(xc, wc)
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    cp.linear(xc, wc, p=0.4, rng=rng, offset=2, out=out, workspace=ws, stream=s)
    s.synchronize()
    _check(out, x, w, torch.float32, p=0.4, seed=5, offset=12)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        cp.linear(xc, wc, p=0.4, rng=rng, offset=2, out=out, workspace=ws)
    for seed, offset in [(5, 10), (6, 10), ((1 << 62) + 9, (1 << 33) + 1)]:
        rng.copy_(torch.tensor([seed, offset]))
        out.fill_(-1.0)
        graph.replay()
        torch.cuda.synchronize()
        _check(out, x, w, torch.float32, p=0.4, seed=seed, offset=offset + 2)


def test_linear_refusals():
    x, w, _ = _case(4, 40, 48, torch.bfloat16)
    x, w = x.cuda(), w.cuda()
    f = torch.empty(4, 40, device="cuda")
    for call in [lambda: cp.linear(x.float(), w.float()), lambda: cp.linear(x, w.half()),
                 lambda: cp.linear(x, w[0]), lambda: cp.linear(x, w[:, :40]),
                 lambda: cp.linear(x, w, activation="tanh"), lambda: cp.linear(x, w, out=f[:, :39]),
                 lambda: cp.linear(x, w, out=f, dtype=torch.float16),
                 lambda: cp.linear(x, w, residual=f), lambda: cp.linear(x, w, f[0, :39]),
                 lambda: cp.linear(x, w, pre=f), lambda: cp.linear(x, w, seed=-1),
                 lambda: cp.linear(x, w, offset=1 << 64), lambda: cp.linear(x.cpu(), w),
                 lambda: cp.linear(x, w.cpu()), lambda: cp.linear(x.T, w),
                 lambda: cp.linear(x, w, p=0.1, rng=torch.zeros(2, device="cuda")),
                 lambda: cp.linear(x, w, p=0.1, rng=torch.zeros(2, dtype=torch.int64)),
                 lambda: cp.linear(x, w, out=f[:1].expand(4, 40))]:
        with pytest.raises(ValueError):
            call()
    for p in (-0.1, 1.5, float("nan")):
        with pytest.raises(cp.CPError):
            cp.linear(x, w, p=p)
    wide = torch.zeros(130, 50, dtype=torch.bfloat16, device="cuda")[:, :49]
    with pytest.raises(ValueError):
        cp.linear(wide, wide, workspace=torch.empty(8, dtype=torch.uint8, device="cuda"))
