"""embed and embed_grad against plain 64-bit forms: types, odd and strided rows, ids out
of range, hot rows, empty calls, accumulation, other streams, graphs, refusals."""
import pytest
import torch

import trellis_row_decode_gb300 as cp

from layer_util import (DTYPES, TINY, U32, UNIT, assert_within, embed64, embed_grad64, gen, randn,
                        rounded)

pytestmark = pytest.mark.gpu


def _ids(g, n, n_rows, kind):
    if kind == "same":
        return torch.full((n,), n_rows // 2, dtype=torch.int64)
    if kind == "sorted":
        return torch.sort(torch.randint(0, n_rows, (n,), generator=g)).values
    if kind == "hot":                       # half of the lookups on one row, the rest spread
        ids = torch.randint(0, n_rows, (n,), generator=g)
        return torch.where(torch.rand(n, generator=g) < 0.5, torch.tensor(n_rows - 1), ids)
    if kind == "low":                       # rows at the table's end are never met
        return torch.randint(0, max(1, n_rows // 50), (n,), generator=g)
    ids = torch.randint(0, n_rows, (n,), generator=g)
    if kind == "holes":                     # ids outside the table among them
        bad = torch.tensor([-1, n_rows, n_rows + 7, 1 << 40, -(1 << 62)])
        at = torch.rand(n, generator=g) < 0.3
        ids = torch.where(at, bad[torch.randint(0, 5, (n,), generator=g)], ids)
    return ids


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("n_rows,d,n", [(7, 1, 5), (100, 8, 33), (50, 13, 200), (300, 256, 1000),
                                        (40, 1000, 77), (64, 1024, 257), (9, 4096, 3),
                                        (5, 5003, 11)])
def test_embed_matches(n_rows, d, n, dtype):
    g = gen(n_rows * d + n)
    w = randn(g, n_rows, d, dtype=dtype)
    ids = _ids(g, n, n_rows, "holes")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = cp.embed(w.cuda(), ids.cuda(), 3.7, status=status)
    ref = embed64(w, ids, torch.tensor(3.7, dtype=torch.float32).item())
    # one fp32 product, one rounding to the type
    assert_within(out, ref, ref.abs() * U32 + rounded(ref * (1 + U32), dtype))
    bad = (ids < 0) | (ids >= n_rows)
    assert not out.cpu()[bad].any()
    assert int(status.item()) == (1 if bad.any() else 0)


def test_embed_strided_views_and_shapes():
    g = gen(2)
    wide = randn(g, 60, 100, dtype=torch.bfloat16).cuda()
    for lo, hi in [(0, 64), (8, 72), (3, 50), (99, 100)]:
        w = wide[:, lo:hi]
        ids = torch.randint(0, 60, (4, 9), generator=g).cuda()
        buf = torch.full((4 * 9, 128), 5.0, dtype=torch.bfloat16, device="cuda")
        got = cp.embed(w, ids)
        assert got.shape == (4, 9, hi - lo)
        assert torch.equal(got, w[ids])
        view = buf[:, 8:8 + hi - lo]
        cp.embed(w, ids.view(-1), out=view)
        assert torch.equal(view, w[ids.view(-1)])
        assert bool((buf[:, :8] == 5).all()) and bool((buf[:, 8 + hi - lo:] == 5).all())


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("d", [9, 40, 129])
def test_rows_that_start_on_any_element(d, dtype):
    """Every offset of a row's start from a 16-byte boundary, and NaN all around the rows: in
    embed, and as the rows of dy and of the gradient."""
    g = gen(d)
    n_rows, n, pitch = 24, 50, d + 37
    ids = torch.randint(0, n_rows, (n,), generator=g).cuda()
    for offset in range(17):
        def rows(count, seed):
            buf = torch.full((count * pitch + 32,), float("nan"), dtype=dtype, device="cuda")
            view = torch.as_strided(buf, (count, d), (pitch, 1), offset)
            view.copy_(randn(gen(seed), count, d, dtype=dtype))
            return buf, view
        _, w = rows(n_rows, offset)
        buf, out = rows(n, 100)
        cp.embed(w, ids, out=out)
        assert torch.equal(out, w[ids])
        assert int(torch.isnan(buf).sum()) == buf.numel() - n * d      # nothing else written
        _, dy = rows(n, 200 + offset)
        gbuf, grad = rows(n_rows, 300)
        cp.embed_grad(dy, ids, n_rows, out=grad)
        ref, mags, count = embed_grad64(dy.cpu(), ids.cpu(), n_rows, 1.0)
        assert_within(grad, ref, (count[:, None] + 2) * U32 * mags + rounded(ref, dtype))
        assert int(torch.isnan(gbuf).sum()) == gbuf.numel() - n_rows * d


def test_embed_special_values_and_empty():
    w = torch.tensor([[float("inf"), float("nan"), -0.0, 1e38]], device="cuda")
    out = cp.embed(w, torch.zeros(2, dtype=torch.int64, device="cuda"), 10.0)
    assert torch.isinf(out[:, 0]).all() and torch.isnan(out[:, 1]).all()
    assert torch.isinf(out[:, 3]).all()
    none = torch.empty(0, dtype=torch.int64, device="cuda")
    assert cp.embed(w, none).shape == (0, 4)
    empty = torch.empty(0, 4, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = cp.embed(empty, torch.zeros(3, dtype=torch.int64, device="cuda"), float("inf"),
                   status=status)
    assert not out.any() and int(status.item()) == 1


def test_embed_offsets_past_32_bits():
    """Rows whose byte and element offsets pass 2^32 (5.1e9 elements, 10.2 GB)."""
    n_rows, d = 5_000_000, 1024
    w = torch.empty(n_rows, d, dtype=torch.bfloat16, device="cuda")
    ids = torch.tensor([n_rows - 1, 4_194_304, 4_194_303, 0, 2_097_152], device="cuda")
    mark = torch.arange(5 * d, device="cuda").view(5, d).to(torch.bfloat16)
    w[ids] = mark
    assert torch.equal(cp.embed(w, ids), mark)


def _check_grad(dy, ids, n_rows, scale, out_dtype, **kw):
    got = cp.embed_grad(dy.cuda(), ids.cuda(), n_rows, scale, dtype=out_dtype, **kw)
    ref, mags, count = embed_grad64(dy.cpu(), ids.cpu(), n_rows, scale)
    bound = (count[:, None] + 2) * U32 * mags + rounded(ref, out_dtype)
    assert_within(got, ref, bound)
    assert not got.cpu()[count == 0].any()
    again = cp.embed_grad(dy.cuda(), ids.cuda(), n_rows, scale, dtype=out_dtype, **kw)
    assert torch.equal(got.view(torch.uint8), again.view(torch.uint8))     # the same bits
    return got


@pytest.mark.parametrize("kind", ["uniform", "same", "sorted", "hot", "low", "holes"])
@pytest.mark.parametrize("n_rows,d,n", [(1, 8, 1), (1, 16, 5000), (37, 24, 100), (400, 256, 4095),
                                        (400, 264, 4096), (5000, 64, 4097), (3, 1000, 9000),
                                        (100_000, 40, 30_000), (70_000, 8, 20)])
def test_embed_grad_matches(n_rows, d, n, kind):
    g = gen(n_rows + d + n)
    _check_grad(randn(g, n, d), _ids(g, n, n_rows, kind), n_rows, 0.75, torch.float32)


@pytest.mark.parametrize("din", DTYPES)
@pytest.mark.parametrize("dout", DTYPES)
@pytest.mark.parametrize("d", [7, 1024])
def test_embed_grad_types(din, dout, d):
    g = gen(d)
    ids = _ids(g, 700, 90, "holes")
    _check_grad(randn(g, 700, d, dtype=din, std=0.1), ids, 90, 2.0, dout)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("d,gap", [(1, 0), (25, 0), (25, 3), (200, 8), (255, 0), (256, 0),
                                   (257, 0), (601, 0), (601, 5), (520, 1)])
def test_embed_grad_clears_the_rows_that_no_id_names(d, gap, dtype):
    """Narrow and wide rows, with and without a gap, on any boundary; nothing around them."""
    g = gen(d + gap)
    n_rows, ids = 700, torch.tensor([5, 698, 5, 300, 301, -1])
    dy = randn(g, 6, d, dtype=dtype)
    ref, mags, count = embed_grad64(dy, ids, n_rows, 1.0)
    bound = (count[:, None] + 2) * U32 * mags + rounded(ref, dtype)
    for offset in (0, 1, 8, 15):
        buf = torch.full((n_rows * (d + gap) + 32,), float("nan"), dtype=dtype, device="cuda")
        out = torch.as_strided(buf, (n_rows, d), (d + gap, 1), offset)
        cp.embed_grad(dy.cuda(), ids.cuda(), n_rows, out=out)
        assert_within(out, ref, bound)
        assert int(torch.isnan(buf).sum()) == buf.numel() - n_rows * d


def test_embed_grad_many_tiles():
    """More ids than one sub-tile per sort tile (2.2e6), and keys of four digits."""
    g = gen(5)
    n, n_rows = 2_200_000, (1 << 27) + 3
    ids = torch.randint(0, n_rows, (n,), generator=g)
    ids[::3] = torch.randint(0, 5, (ids[::3].numel(),), generator=g) * (n_rows // 5)
    dy = randn(g, n, 8).cuda()
    got = cp.embed_grad(dy, ids.cuda(), n_rows)
    order = torch.sort(ids.cuda(), stable=True)
    uniq, counts = torch.unique_consecutive(order.values, return_counts=True)
    sums = torch.zeros(uniq.numel(), 8, dtype=torch.float64, device="cuda")
    mags = torch.zeros_like(sums)
    where = torch.repeat_interleave(torch.arange(uniq.numel(), device="cuda"), counts)
    sums.index_add_(0, where, dy[order.indices].double())
    mags.index_add_(0, where, dy[order.indices].double().abs())
    bound = (counts[:, None] + 2) * U32 * mags + sums.abs() * U32
    assert bool(((got[uniq].double() - sums).abs() <= bound).all())
    got[uniq] = 0
    assert not got.any()


def test_embed_grad_strides_and_expanded_rows():
    g = gen(8)
    n, n_rows, d = 900, 60, 72
    ids = _ids(g, n, n_rows, "hot").cuda()
    wide = randn(g, n, 100).cuda()
    buf = torch.full((n_rows, 90), 3.0, device="cuda")
    view = buf[:, 8:8 + d]
    dy = wide[:, 16:16 + d]
    cp.embed_grad(dy, ids, n_rows, out=view)
    ref, mags, count = embed_grad64(dy.cpu(), ids.cpu(), n_rows, 1.0)
    assert_within(view, ref, (count[:, None] + 2) * U32 * mags + rounded(ref, torch.float32))
    assert bool((buf[:, :8] == 3).all()) and bool((buf[:, 8 + d:] == 3).all())
    one = wide[:1, :d].expand(n, d)                     # the gradient of a sum: one row, stride 0
    got = cp.embed_grad(one, ids, n_rows)
    ref, mags, count = embed_grad64(one.cpu(), ids.cpu(), n_rows, 1.0)
    assert_within(got, ref, (count[:, None] + 2) * U32 * mags + rounded(ref, torch.float32))


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("n_rows,d,n,kind", [(500, 64, 300, "uniform"), (9, 33, 6000, "hot"),
                                             (200_000, 256, 9000, "holes"), (40, 16, 1, "same")])
def test_embed_grad_accumulate(n_rows, d, n, kind, dtype):
    g = gen(n_rows + n)
    ids = _ids(g, n, n_rows, kind)
    dy = randn(g, n, d, dtype=dtype)
    base = randn(g, n_rows, d, dtype=dtype)
    out = base.cuda()
    cp.embed_grad(dy.cuda(), ids.cuda(), n_rows, -0.125, out=out, accumulate=True)
    ref, mags, count = embed_grad64(dy, ids, n_rows, -0.125)
    full = ref + base.double()
    assert_within(out, full, (count[:, None] + 2) * U32 * mags + rounded(full, dtype) * (1 + 1e-6))
    same = count == 0
    assert torch.equal(out.cpu()[same], base[same])


@pytest.mark.parametrize("group,d", [(2, 64), (24, 256), (7, 33)])
def test_embed_grad_of_groups(group, d):
    """The gradient of sums over groups of lookups: one row of dy per group, as if repeated."""
    g = gen(group)
    t, n_rows = 300, 500
    ids = _ids(g, t * group, n_rows, "holes").view(t, group)
    dy = randn(g, t, d, dtype=torch.bfloat16)
    got = cp.embed_grad(dy.cuda(), ids.cuda(), n_rows, 0.5, dtype=torch.float32, group=group)
    whole = dy.repeat_interleave(group, 0)
    same = cp.embed_grad(whole.cuda(), ids.view(-1).cuda(), n_rows, 0.5, dtype=torch.float32)
    assert torch.equal(got, same)
    ref, mags, count = embed_grad64(whole, ids.view(-1), n_rows, 0.5)
    assert_within(got, ref, (count[:, None] + 2) * U32 * mags + rounded(ref, torch.float32))


def test_embed_grad_empty_and_status():
    out = torch.full((5, 8), 2.0, device="cuda")
    none = torch.empty(0, dtype=torch.int64, device="cuda")
    dy0 = torch.empty(0, 8, device="cuda")
    cp.embed_grad(dy0, none, 5, out=out, accumulate=True)
    assert bool((out == 2).all())
    cp.embed_grad(dy0, none, 5, out=out)
    assert not out.any()
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    dy = torch.ones(3, 8, device="cuda")
    cp.embed_grad(dy, torch.tensor([0, 4, 4], device="cuda"), 5, out=out, status=status)
    assert int(status.item()) == 0 and out[:, 0].tolist() == [1, 0, 0, 0, 2]
    cp.embed_grad(dy, torch.tensor([0, 5, -1], device="cuda"), 5, out=out, status=status)
    assert int(status.item()) == 1 and out[:, 0].tolist() == [1, 0, 0, 0, 0]
    # rows that no id names are zeros whatever the scale
    cp.embed_grad(dy, torch.tensor([0, 0, 0], device="cuda"), 5, float("nan"), out=out)
    assert not out[1:].any()


def test_embed_grad_not_finite_rows_stay_apart():
    """An infinity or a NaN in one lookup reaches its own row only."""
    dy = torch.ones(200, 16, device="cuda")
    ids = torch.arange(200, device="cuda") % 10
    dy[17, 3] = float("inf")
    dy[28, 5] = float("nan")
    out = cp.embed_grad(dy, ids, 10)
    bad = ~torch.isfinite(out)
    assert bad.nonzero().tolist() == [[7, 3], [8, 5]]


def test_embed_grad_is_the_lookups_derivative():
    """<dy, embed(W + t V) - embed(W - t V)> / 2t = <embed_grad(dy), V> (embed is linear)."""
    g = gen(3)
    n_rows, d, n = 50, 32, 400
    w, v = randn(g, n_rows, d), randn(g, n_rows, d)
    ids = _ids(g, n, n_rows, "holes").cuda()
    dy = randn(g, n, d).cuda()
    t = 0.5
    up = cp.embed((w + t * v).cuda(), ids, 1.5).double()
    down = cp.embed((w - t * v).cuda(), ids, 1.5).double()
    left = (dy.double() * (up - down)).sum() / (2 * t)
    grad = cp.embed_grad(dy, ids, n_rows, 1.5).double()
    right = (grad * v.cuda().double()).sum()
    # each of n * d terms is off by a few U32 of values of size ~10
    assert abs(float(left - right)) <= n * d * 40 * U32


def test_embed_on_another_stream_and_in_a_graph():
    g = gen(9)
    n_rows, d, n = 3000, 128, 20_000
    w = randn(g, n_rows, d).cuda()
    ids = _ids(g, n, n_rows, "hot").cuda()
    torch.cuda.synchronize()
    ref = cp.embed(w, ids, 2.0)
    ref_grad = cp.embed_grad(ref, ids, n_rows, 0.5)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    outs = [(cp.embed(w, ids, 2.0, stream=s)) for _ in range(3)]
    grads = [cp.embed_grad(o, ids, n_rows, 0.5, stream=s) for o in outs]
    s.synchronize()
    for o, gr in zip(outs, grads):
        assert torch.equal(o, ref) and torch.equal(gr, ref_grad)
    out, grad = torch.zeros_like(ref), torch.zeros_like(ref_grad)
    ws = cp.embed_grad_workspace(n, n_rows, d)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        cp.embed(w, ids, 2.0, out=out)
        cp.embed_grad(out, ids, n_rows, 0.5, out=grad, workspace=ws)
    ids.copy_(torch.flip(ids, (0,)))
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, w[ids] * 2)
    assert torch.allclose(grad, ref_grad, rtol=1e-4, atol=1e-3)   # the same terms, another order


def test_embed_refusals():
    w = torch.zeros(10, 16, device="cuda")
    ids = torch.zeros(4, dtype=torch.int64, device="cuda")
    dy = torch.zeros(4, 16, device="cuda")
    for call in [
        lambda: cp.embed(w.double(), ids),
        lambda: cp.embed(w.t(), ids),
        lambda: cp.embed(w, ids.int()),
        lambda: cp.embed(w, torch.zeros(8, dtype=torch.int64, device="cuda")[::2]),
        lambda: cp.embed(w, ids.cpu()),
        lambda: cp.embed(w, ids, out=torch.zeros(4, 15, device="cuda")),
        lambda: cp.embed(w, ids, out=torch.zeros(4, 16, device="cuda", dtype=torch.bfloat16)),
        lambda: cp.embed(w, ids, out=torch.zeros(1, 16, device="cuda").expand(4, 16)),
        lambda: cp.embed(w, ids, status=torch.zeros(1, device="cuda")),
        lambda: cp.embed_grad(dy[:3], ids, 10),
        lambda: cp.embed_grad(dy, ids, 10, group=2),
        lambda: cp.embed_grad(dy, ids, 10, group=0),
        lambda: cp.embed_grad(dy, ids, 10, accumulate=True),
        lambda: cp.embed_grad(dy, ids, 10, dtype=torch.float64),
        lambda: cp.embed_grad(dy, ids, 10, out=torch.zeros(9, 16, device="cuda")),
        lambda: cp.embed_grad(dy, ids, 10, workspace=torch.zeros(8, dtype=torch.uint8,
                                                                 device="cuda")),
    ]:
        with pytest.raises(ValueError):
            call()
    with pytest.raises(cp.CPError):
        cp.embed_grad_workspace(4, 1 << 31, 16)
