"""dropout against a plain 64-bit form: types, odd rows, strides, the mask's use again, graphs,
refusals."""
import pytest
import torch

import trellis_row_decode_gb300 as cp

from layer_util import DTYPES, U32, assert_within, gen, randn, rounded
from linear_util import drop64, mask64

pytestmark = pytest.mark.gpu


def _check(got, x, p, seed, offset, residual=None):
    """The scale is rounded once, the product once, the addition once."""
    drop = drop64(x.double(), p, seed, offset)
    want = drop + (residual.double() if residual is not None else 0.0)
    assert_within(got, want, 3 * U32 * (drop.abs() + want.abs()) + rounded(want, x.dtype))


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("rows,d", [(1, 1), (1, 7), (1, 100003), (3, 8), (5, 1000), (129, 33),
                                    (700, 1024), (2049, 26), (4, 65536)])
def test_dropout_matches(rows, d, dtype):
    g = gen(rows + d)
    x, res = randn(g, rows, d, dtype=dtype), randn(g, rows, d, dtype=dtype)
    for p, seed, offset in [(0.1, 1, 0), (0.5, (1 << 64) - 1, (1 << 64) - 1), (0.93, 1 << 40, 1 << 33)]:
        _check(cp.dropout(x.cuda(), p, seed, offset), x, p, seed, offset)
        _check(cp.dropout(x.cuda(), p, seed, offset, residual=res.cuda()), x, p, seed, offset, res)


def test_dropout_at_its_ends():
    """p = 0 keeps every bit, p = 1 and a p within 2^-33 of it keep nothing, one close to 0 all;
    dropped infinities and NaN leave zeros."""
    x = torch.randn(40, 100)
    x[3, 4], x[5, 6], x[7, 8] = float("inf"), float("nan"), -float("inf")
    c = x.cuda()
    assert torch.equal(cp.dropout(c, 0.0).view(torch.int32), c.view(torch.int32))
    assert bool((cp.dropout(c, 1.0) == 0).all()) and bool((cp.dropout(c, 1 - 2.0 ** -34) == 0).all())
    got = cp.dropout(c, 2.0 ** -40, 4)
    assert_within(got, x.double(), 2 * U32 * x.double().abs().nan_to_num(0, 0, 0))
    got, keep = cp.dropout(c, 0.5, 11).cpu(), mask64(40, 100, 0.5, 11, 0)
    assert bool((got[~keep] == 0).all())
    _check(got, x, 0.5, 11, 0)
    res = torch.ones(40, 100, device="cuda")
    assert torch.equal(cp.dropout(c, 1.0, residual=res), res)


def test_dropout_keeps_the_share_it_should():
    """1 - p of 4 million, within six standard deviations; neighbours and other offsets unlike."""
    x = torch.ones(2048, 2048, device="cuda")
    for p in (0.1, 0.5):
        a = cp.dropout(x, p, 7, 0) != 0
        sd = (p * (1 - p) / a.numel()) ** 0.5
        assert abs(float(a.double().mean()) - (1 - p)) < 6 * sd
        both = (1 - p) ** 2 + p ** 2                 # two independent draws agree this often
        sd = (both * (1 - both) / a.numel()) ** 0.5
        for b in (cp.dropout(x, p, 7, 1) != 0, cp.dropout(x, p, 8, 0) != 0, a.roll(1, 0),
                  a.roll(1, 1), a.roll(4, 1)):
            assert abs(float((a == b).double().mean()) - both) < 6 * sd


def test_dropout_mask_is_that_of_linear():
    """linear's dropout is dropout of its rows, whichever kernel runs."""
    for m in (3, 200):
        x, w = torch.ones(m, 64, device="cuda").bfloat16(), torch.ones(77, 64, device="cuda").bfloat16()
        got = cp.linear(x, w, p=0.3, seed=21, offset=5, dtype=torch.float32)
        want = cp.dropout(torch.full((m, 77), 64.0, device="cuda"), 0.3, 21, 5)
        assert torch.equal(got, want)


@pytest.mark.parametrize("dtype", DTYPES)
def test_dropout_strides_and_in_place(dtype):
    g = gen(8)
    for d, pitch, at in [(96, 128, 0), (96, 97, 3), (51, 60, 1), (64, 64, 8)]:
        buf = torch.full((33 * pitch + 64,), 7.0, dtype=dtype, device="cuda")
        x = torch.as_strided(buf, (33, d), (pitch, 1), at)
        x.copy_(randn(g, 33, d, dtype=dtype))
        x0 = x.cpu()
        res = randn(g, 1, d, dtype=dtype)
        got = cp.dropout(x, 0.4, 5, 6, residual=res.cuda().expand(33, d))
        _check(got, x0, 0.4, 5, 6, res.expand(33, d))
        assert cp.dropout(x, 0.4, 5, 6, out=x) is x
        _check(x, x0, 0.4, 5, 6)
        x.fill_(7.0)
        assert bool((buf == 7).all())
    x, res = randn(g, 50, 40, dtype=dtype), randn(g, 50, 40, dtype=dtype)
    stream = res.cuda()
    cp.dropout(x.cuda(), 0.2, 1, residual=stream, out=stream)
    _check(stream, x, 0.2, 1, 0, res)


def test_dropout_shapes():
    x = torch.randn(4, 5, 12)
    _check(cp.dropout(x.cuda(), 0.3, 2).view(20, 12), x.view(20, 12), 0.3, 2, 0)
    _check(cp.dropout(x[0, 0].cuda(), 0.3, 2)[None], x[0, 0][None], 0.3, 2, 0)
    assert cp.dropout(torch.empty(0, 12, device="cuda"), 0.3).shape == (0, 12)
    assert cp.dropout(torch.empty(3, 0, device="cuda"), 0.3).shape == (3, 0)


def test_dropout_grad_is_the_mask():
    dy = torch.randn(60, 200)
    _check(cp.dropout_grad(dy.cuda(), 0.35, 9, 10), dy, 0.35, 9, 10)
    rng = torch.tensor([9, 4], dtype=torch.int64, device="cuda")
    assert torch.equal(cp.dropout_grad(dy.cuda(), 0.35, rng=rng, offset=6),
                       cp.dropout_grad(dy.cuda(), 0.35, 9, 10))


def test_dropout_in_a_graph_and_on_another_stream():
    x = torch.randn(100, 64)
    c, out = x.cuda(), torch.empty(100, 64, device="cuda")
    rng = torch.tensor([1, 2], dtype=torch.int64, device="cuda")
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    got = cp.dropout(c, 0.5, rng=rng, stream=s)
    s.synchronize()
    _check(got, x, 0.5, 1, 2)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        cp.dropout(c, 0.5, rng=rng, out=out)
        rng[1] += 1                                   # the next replay draws another mask
    for i in range(3):
        graph.replay()
        torch.cuda.synchronize()
        _check(out, x, 0.5, 1, 2 + i)


def test_dropout_refusals():
    x = torch.zeros(4, 8, device="cuda")
    for call in [lambda: cp.dropout(x.int(), 0.1), lambda: cp.dropout(x.cpu(), 0.1),
                 lambda: cp.dropout(x.T, 0.1), lambda: cp.dropout(x, 0.1, seed=-1),
                 lambda: cp.dropout(x, 0.1, offset=1 << 64), lambda: cp.dropout(x, 0.1, residual=x.half()),
                 lambda: cp.dropout(x, 0.1, residual=x[:2]), lambda: cp.dropout(x, 0.1, out=x.half()),
                 lambda: cp.dropout(x, 0.1, out=x[:1].expand(4, 8)),
                 lambda: cp.dropout(x, 0.1, rng=torch.zeros(3, dtype=torch.int64, device="cuda")),
                 lambda: cp.dropout(torch.zeros((), device="cuda"), 0.1)]:
        with pytest.raises(ValueError):
            call()
    for p in (-0.01, 1.01, float("nan"), float("inf")):
        with pytest.raises(cp.CPError):
            cp.dropout(x, p)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("d", [1, 7, 13, 63, 96, 101, 250])
def test_dropout_keeps_to_its_columns(d, dtype):
    """NaN behind the rows of the input and the residual stays out, what lies behind those of the
    output stays; rows one behind the other too, where the next row follows at once."""
    g = gen(d)
    x, r = randn(g, 300, d, dtype=dtype), randn(g, 300, d, dtype=dtype)
    wide = [torch.full((300, 256), float("nan"), dtype=dtype, device="cuda") for _ in range(2)]
    wide[0][:, :d], wide[1][:, :d] = x.cuda(), r.cuda()
    for residual in (None, wide[1][:, :d]):
        out = torch.full((301, 256), 7.0, dtype=dtype, device="cuda")
        cp.dropout(wide[0][:, :d], 0.3, 5, out=out[:300, :d], residual=residual)
        _check(out[:300, :d], x, 0.3, 5, 0, None if residual is None else r)
        assert bool((out[:, d:] == 7).all()) and bool((out[300] == 7).all())
        flat = torch.full((302 * d,), 7.0, dtype=dtype, device="cuda")
        cp.dropout(x.cuda(), 0.3, 5, out=flat[d:301 * d].view(300, d),
                   residual=None if residual is None else r.cuda())
        _check(flat[d:301 * d].view(300, d), x, 0.3, 5, 0, None if residual is None else r)
        assert bool((flat[:d] == 7).all()) and bool((flat[301 * d:] == 7).all())
