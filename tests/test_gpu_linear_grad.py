"""linear_grad against the formula in 64 bits and against differences of linear: each
activation and dropout, types, odd sizes, strides, accumulation, graphs, refusals."""
import pytest
import torch

import trellis_row_decode_gb300 as cp

from layer_util import TINY, U32, UNIT, assert_within, gen, randn, rounded
from linear_util import ACTS, drop64, linear64, slope64, sum_bound

pytestmark = pytest.mark.gpu
HALF = [torch.bfloat16, torch.float16]


def _reference(dy, x, w, act="none", pre=None, p=0.0, seed=0, offset=0):
    """(dx, dw, db) in 64 bits, each with a bound without its last rounding."""
    dtype = x.dtype
    scale = 1.0 / (1.0 - p) if p < 1 else 0.0
    dz = drop64(dy.double(), p, seed, offset)
    own = torch.zeros_like(dz)                # error of dz in fp32: slope, scale, products
    if act != "none":
        # a slope's arithmetic: 16 roundings relative to |z| + 1
        own = 16 * U32 * (pre.double().abs() + 1) * dz.abs()
        dz = dz * slope64(pre, act)
    own = own + 4 * U32 * dz.abs() + (TINY[torch.float32] if act != "none" or p else 0)
    cut = own
    if act != "none" or p or dy.dtype != dtype:
        cut = own * 1.01 + dz.abs() * UNIT[dtype] + TINY[dtype]
    X, W = x.double(), w.double()
    m, n = dz.shape
    dx, dw, db = dz @ W, dz.T @ X, dz.sum(0)
    return ((dx, cut @ W.abs() + sum_bound((dz.abs() + cut) @ W.abs(), n)),
            (dw, cut.T @ X.abs() + sum_bound((dz.abs() + cut).T @ X.abs(), m)),
            (db, own.sum(0) + (m + 64) * U32 * (dz.abs() + own).sum(0)))


def _check(got, ref, dtypes):
    for value, (want, bound), dtype in zip(got, ref, dtypes):
        assert value.dtype == dtype
        assert_within(value, want, bound + rounded(want, dtype))


def _case(m, n, k, dtype, act="none", dy_dtype=None):
    g = gen(m * n + k)
    x, w = randn(g, m, k, dtype=dtype), randn(g, n, k, dtype=dtype, std=max(k, 1) ** -0.5)
    dy = randn(g, m, n, dtype=dy_dtype or dtype)
    return dy, x, w, randn(g, m, n, dtype=dtype, std=2.0) if act != "none" else None


def _cuda(*ts):
    return [None if t is None else t.cuda() for t in ts]


SIZES = [(1, 1, 1), (1, 64, 64), (3, 130, 2320), (64, 64, 64), (129, 384, 257), (200, 333, 101),
         (256, 256, 256), (512, 384, 256), (1000, 72, 1000), (4096, 64, 96), (33, 2050, 40),
         (5000, 8, 8), (130, 1, 5)]


@pytest.mark.parametrize("m,n,k", SIZES)
def test_linear_grad_matches(m, n, k):
    dy, x, w, _ = _case(m, n, k, torch.bfloat16)
    a = _cuda(dy, x, w)
    got = cp.linear_grad(*a, dw_dtype=torch.float32, db_dtype=torch.float32)
    _check(got, _reference(dy, x, w), (torch.bfloat16, torch.float32, torch.float32))
    again = cp.linear_grad(*a, dw_dtype=torch.float32, db_dtype=torch.float32)
    assert all(torch.equal(u, v) for u, v in zip(got, again))
    assert cp.linear_status() == cp.CP_OK


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("p", [0.0, 0.3])
@pytest.mark.parametrize("m,n,k", [(300, 256, 128), (77, 205, 93)])
def test_linear_grad_epilogue(m, n, k, act, p):
    dy, x, w, pre = _case(m, n, k, torch.bfloat16, act)
    kw = dict(p=p, seed=(1 << 63) + 11, offset=1 << 40)
    got = cp.linear_grad(*_cuda(dy, x, w), act, *_cuda(pre), **kw, db_dtype=torch.float32)
    _check(got, _reference(dy, x, w, act, pre, **kw),
           (torch.bfloat16, torch.bfloat16, torch.float32))


@pytest.mark.parametrize("dtype", HALF)
@pytest.mark.parametrize("dy32", [False, True])
@pytest.mark.parametrize("n", [96, 61])
def test_linear_grad_types(dtype, dy32, n):
    dy, x, w, pre = _case(150, n, 72, dtype, "gelu", torch.float32 if dy32 else None)
    got = cp.linear_grad(*_cuda(dy, x, w), "gelu", pre.cuda())
    _check(got, _reference(dy, x, w, "gelu", pre), (dtype, dtype, dtype))
    got = cp.linear_grad(*_cuda(dy, x, w), dw_dtype=torch.float32, db_dtype=torch.float32)
    _check(got, _reference(dy, x, w), (dtype, torch.float32, torch.float32))


@pytest.mark.parametrize("act", ["silu", "gelu", "gelu_tanh"])
def test_linear_grad_is_the_slope_of_linear(act):
    """Central differences in 64 bits of the forward formula, along random directions of x, w
    and bias, against the products of the gradients with them (dz in 16 bits: 2^-8 of the terms'
    magnitudes)."""
    g = gen(4)
    m, n, k, p, seed = 24, 40, 32, 0.25, 9
    x, w = randn(g, m, k, dtype=torch.bfloat16), randn(g, n, k, dtype=torch.bfloat16, std=0.2)
    b, dy = randn(g, n, std=0.3), randn(g, m, n, dtype=torch.bfloat16)
    _, pre = cp.linear(*_cuda(x, w, b), act, p=p, seed=seed, pre=True)
    dx, dw, db = cp.linear_grad(*_cuda(dy, x, w), act, pre, p=p, seed=seed,
                                dw_dtype=torch.float32, db_dtype=torch.float32)
    ux, uw, ub = (randn(g, *t.shape).double() for t in (x, w, b))
    h = 1e-5

    def loss(s):
        out, _, _ = linear64(x.double() + s * ux, w.double() + s * uw, b.double() + s * ub, act, p=p,
                             seed=seed)
        return float((out * dy.double()).sum())
    slope = (loss(h) - loss(-h)) / (2 * h)
    got = float((dx.cpu().double() * ux).sum() + (dw.cpu().double() * uw).sum()
                + (db.cpu().double() * ub).sum())
    # dz's rounding and that of pre (2^-8 |z| of slopes that change by at most 1 a unit), dx's
    dz = drop64(dy.double(), p, seed, 0).abs() * 1.13
    off = 2.0 ** -8 * (1 + pre.cpu().double().abs()) * dz
    bound = float((off * (ux.abs() @ w.double().abs().T + x.double().abs() @ uw.abs().T
                          + ub.abs())).sum()) + 2.0 ** -8 * float((dx.cpu().double() * ux).abs().sum())
    assert abs(got - slope) <= bound and bound < 0.2 * float((dz * 20).sum())


@pytest.mark.parametrize("m,n,k", [(40, 48, 64), (300, 130, 71)])
def test_linear_grad_accumulates(m, n, k):
    dy, x, w, _ = _case(m, n, k, torch.bfloat16)
    g = gen(1)
    for dw_dtype in (torch.float32, torch.bfloat16):
        dw0, db0 = randn(g, n, k, dtype=dw_dtype), randn(g, n)
        dw, db = dw0.cuda(), db0.cuda()
        out = cp.linear_grad(*_cuda(dy, x, w), accumulate=True, dw=dw, db=db)
        assert out[1] is dw and out[2] is db
        ref = _reference(dy, x, w)
        want, bound = ref[1][0] + dw0.double(), ref[1][1] + 2 * U32 * (ref[1][0].abs() + dw0.double().abs())
        assert_within(dw, want, bound + rounded(want, dw_dtype))
        want, bound = ref[2][0] + db0.double(), ref[2][1] + 2 * U32 * (ref[2][0].abs() + db0.double().abs())
        assert_within(db, want, bound + rounded(want, torch.float32))
        # a batch without rows adds nothing
        kept = dw.clone(), db.clone()
        cp.linear_grad(dy[:0].cuda(), x[:0].cuda(), w.cuda(), accumulate=True, dw=dw, db=db)
        assert torch.equal(dw, kept[0]) and torch.equal(db, kept[1])


def test_linear_grad_of_nothing():
    bf = torch.bfloat16
    dx, dw, db = cp.linear_grad(torch.empty(0, 40, dtype=bf, device="cuda"),
                                torch.empty(0, 24, dtype=bf, device="cuda"),
                                torch.ones(40, 24, dtype=bf, device="cuda"))
    assert dx.shape == (0, 24) and bool((dw == 0).all()) and bool((db == 0).all())
    dx, dw, db = cp.linear_grad(torch.empty(30, 0, dtype=bf, device="cuda"),
                                torch.ones(30, 24, dtype=bf, device="cuda"),
                                torch.empty(0, 24, dtype=bf, device="cuda"))
    assert bool((dx == 0).all()) and dx.shape == (30, 24) and dw.shape == (0, 24) and db.numel() == 0
    dx, dw, db = cp.linear_grad(torch.ones(30, 40, dtype=bf, device="cuda"),
                                torch.empty(30, 0, dtype=bf, device="cuda"),
                                torch.empty(40, 0, dtype=bf, device="cuda"))
    assert dx.shape == (30, 0) and dw.shape == (40, 0) and bool((db == 30).all())


@pytest.mark.parametrize("need", [(1, 0, 0), (0, 1, 0), (0, 0, 1), (1, 1, 0), (1, 0, 1), (0, 1, 1),
                                  (0, 0, 0)])
def test_linear_grad_parts(need):
    dy, x, w, pre = _case(200, 96, 80, torch.bfloat16, "silu")
    a = _cuda(dy, x, w) + ["silu", pre.cuda()]
    want = cp.linear_grad(*a, p=0.2, seed=5)
    got = cp.linear_grad(*a, p=0.2, seed=5, need_dx=bool(need[0]), need_dw=bool(need[1]),
                         need_db=bool(need[2]))
    for g, v, n in zip(got, want, need):
        assert torch.equal(g, v) if n else g is None


def test_linear_grad_strides_and_boundaries():
    """Rows apart, off 16-byte boundaries or repeated, NaN around them; outputs in wider arrays."""
    g = gen(2)
    m, n, k = 140, 72, 104

    def rows(count, width, pitch, offset, dtype=torch.bfloat16):
        buf = torch.full((count * pitch + 64,), float("nan"), dtype=dtype, device="cuda")
        view = torch.as_strided(buf, (count, width), (pitch, 1), offset)
        view.copy_(randn(g, count, width, dtype=dtype))
        return view
    for pd, od, px, ox, pw, ow in [(80, 0, 112, 8, 104, 0), (73, 1, 104, 0, 104, 0),
                                   (72, 0, 105, 3, 104, 0), (72, 0, 104, 0, 109, 7),
                                   (75, 2, 107, 1, 111, 5)]:
        dy, x, w = rows(m, n, pd, od), rows(m, k, px, ox), rows(n, k, pw, ow)
        buf = torch.full((m * 150,), 7.0, dtype=torch.bfloat16, device="cuda")
        dx = torch.as_strided(buf, (m, k), (150, 1), 11)
        ws = cp.linear_grad_workspace(m, n, k)
        got = cp.linear_grad(dy, x, w, dx=dx, workspace=ws, db_dtype=torch.float32)
        _check(got, _reference(dy.cpu(), x.cpu(), w.cpu()),
               (torch.bfloat16, torch.bfloat16, torch.float32))
        dx.fill_(7.0)
        assert bool((buf == 7).all())
    dy = randn(g, 1, n, dtype=torch.bfloat16).cuda().expand(m, n)
    x = randn(g, 1, k, dtype=torch.bfloat16).cuda().expand(m, k)
    got = cp.linear_grad(dy, x, w, db_dtype=torch.float32)
    _check(got, _reference(dy.cpu(), x.cpu(), w.cpu()),
           (torch.bfloat16, torch.bfloat16, torch.float32))


def test_linear_grad_in_a_graph():
    dy, x, w, pre = _case(260, 128, 96, torch.bfloat16, "gelu_tanh")
    rng = torch.tensor([3, 4], dtype=torch.int64, device="cuda")
    a = _cuda(dy, x, w) + ["gelu_tanh", pre.cuda()]
    ws = cp.linear_grad_workspace(260, 128, 96)
    outs = [torch.empty_like(a[1]), torch.empty_like(a[2]), torch.empty(128, device="cuda")]

    def call():
        cp.linear_grad(*a, p=0.5, rng=rng, offset=1, dx=outs[0], dw=outs[1], db=outs[2],
                       workspace=ws)
    call()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    for seed in (3, 8):
        rng[0] = seed
        for o in outs:
            o.fill_(5.0)
        graph.replay()
        torch.cuda.synchronize()
        _check(outs, _reference(dy, x, w, "gelu_tanh", pre, 0.5, seed, 5),
               (torch.bfloat16, torch.bfloat16, torch.float32))


def test_linear_grad_refusals():
    dy, x, w, pre = _cuda(*_case(20, 24, 32, torch.bfloat16, "silu"))
    f = torch.zeros(24, device="cuda")
    for call in [lambda: cp.linear_grad(dy.half(), x, w), lambda: cp.linear_grad(dy[:, :20], x, w),
                 lambda: cp.linear_grad(dy[:10], x, w), lambda: cp.linear_grad(dy, x, w, "silu"),
                 lambda: cp.linear_grad(dy, x, w, pre=pre),
                 lambda: cp.linear_grad(dy, x, w, "silu", pre.float()),
                 lambda: cp.linear_grad(dy, x, w, accumulate=True),
                 lambda: cp.linear_grad(dy, x, w, accumulate=True, need_dw=False),
                 lambda: cp.linear_grad(dy, x, w, dx=x[:10]),
                 lambda: cp.linear_grad(dy, x, w, need_dx=False, dx=torch.empty_like(x)),
                 lambda: cp.linear_grad(dy, x, w, need_db=False, db=f),
                 lambda: cp.linear_grad(dy, x, w, dw=w.float(), dw_dtype=torch.bfloat16),
                 lambda: cp.linear_grad(dy, x, w, db=f, db_dtype=torch.bfloat16),
                 lambda: cp.linear_grad(dy, x, w, db=torch.zeros(48, device="cuda")[::2]),
                 lambda: cp.linear_grad(dy.cpu(), x, w), lambda: cp.linear_grad(dy, x, w.float()),
                 lambda: cp.linear_grad(dy, x, w, "silu", pre,
                                        workspace=torch.empty(9, dtype=torch.uint8, device="cuda"))]:
        with pytest.raises(ValueError):
            call()
    with pytest.raises(cp.CPError):
        cp.linear_grad(dy, x, w, p=2.0)
    with pytest.raises(cp.CPError):
        cp.linear_grad_workspace(1 << 30, 4, 4)


@pytest.mark.parametrize("act", ["none", "silu"])
@pytest.mark.parametrize("m", [5, 300])
@pytest.mark.parametrize("n,k", [(121, 126), (130, 124), (77, 136), (136, 201)])
def test_linear_grad_keeps_to_its_columns(m, n, k, act):
    """Every array on 16-byte boundaries with rows that end inside 16 bytes: NaN behind the rows of
    inputs stay out, what lies behind those of outputs stays."""
    g = gen(m + n + k)

    def rows(count, width):
        t = torch.full((count, 216), float("nan"), dtype=torch.bfloat16, device="cuda")
        t[:, :width] = randn(g, count, width, dtype=torch.bfloat16).cuda()
        return t[:, :width]
    dy, x, w, pre = rows(m, n), rows(m, k), rows(n, k), rows(m, n)
    kw = {} if act == "none" else {"activation": act, "pre": pre}
    ref = _reference(dy.cpu(), x.cpu(), w.cpu(), act, pre.cpu())
    for dtype in (torch.bfloat16, torch.float32):
        dx = torch.full((m + 1, 216), 7.0, dtype=torch.bfloat16, device="cuda")
        dw = torch.full((n + 1, 216), 7.0, dtype=dtype, device="cuda")
        db = torch.full((n + 1,), 7.0, device="cuda")
        cp.linear_grad(dy, x, w, **kw, dx=dx[:m, :k], dw=dw[:n, :k], db=db[:n])
        _check((dx[:m, :k], dw[:n, :k], db[:n]), ref, (torch.bfloat16, dtype, torch.float32))
        assert bool((dx[:, k:] == 7).all()) and bool((dx[m] == 7).all())
        assert bool((dw[:, k:] == 7).all()) and bool((dw[n] == 7).all()) and float(db[n]) == 7
        dw.fill_(7.0)
        cp.linear_grad(dy, x, w, **kw, need_dx=False, need_db=False, dw=dw[:n, :k], accumulate=True)
        want = ref[1][0] + 7.0
        assert_within(dw[:n, :k], want, ref[1][1] + 2 * U32 * (ref[1][0].abs() + 7)
                      + rounded(want, dtype))
        assert bool((dw[:, k:] == 7).all()) and bool((dw[n] == 7).all())
