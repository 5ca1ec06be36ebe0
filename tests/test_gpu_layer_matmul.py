"""matmul_fp8 against a plain 64-bit product: one token to many, odd sizes and strides,
special values, other streams, graphs, refusals.

Bound: the products of e4m3 values are exact in fp32; a group of 128 is summed, scaled
and added to the running sum, so at most 128 + ceil(k / 128) + 10 additions (10: a split
along k and the scale's own roundings) lie over any term.  2 U32 each: the tensor core
may cut instead of round.
"""
import pytest
import torch

import trellis_row_decode_gb300 as cp

from layer_util import DTYPES, E4M3, U32, assert_within, gen, matmul64, randn, rounded

pytestmark = pytest.mark.gpu


def _operands(g, m, n, k, lda=None, ldw=None, offset=0):
    def e4m3(rows, ld):
        ld = k if ld is None else ld
        flat = (torch.randn(rows * ld + offset, generator=g) * 60).clamp(-448, 448).to(E4M3)
        return flat.cuda()[offset:].view(rows, ld)[:, :k] if rows * ld else flat.cuda().view(rows, ld)
    kb = -(-k // 128)
    sa = torch.exp(randn(g, m, kb)) * 0.01
    sw = torch.exp(randn(g, -(-n // 128), kb)) * 0.01
    return e4m3(m, lda), sa.cuda(), e4m3(n, ldw), sw.cuda()


def _check(a, sa, w, sw, dtype, got):
    ref, mag = matmul64(a.cpu(), sa.cpu(), w.cpu(), sw.cpu())
    terms = 128 + -(-a.shape[1] // 128) + 10
    assert_within(got, ref, mag * terms * 2 * U32 + rounded(ref, dtype))


SIZES = [(1, 1, 1), (1, 128, 128), (1, 4096, 1024), (1, 1000, 24576), (2, 77, 300), (3, 130, 2320),
         (8, 256, 512), (9, 300, 640), (16, 512, 384), (17, 129, 1040), (31, 640, 4096),
         (32, 128, 256), (33, 257, 272), (48, 1024, 2048), (64, 64, 64), (65, 1000, 1000),
         (100, 300, 129), (128, 128, 128), (129, 384, 2304), (200, 2050, 528), (256, 256, 1024),
         (333, 1000, 2320), (513, 770, 896), (1024, 1024, 512)]


@pytest.mark.parametrize("m,n,k", SIZES)
def test_matmul_matches(m, n, k):
    g = gen(m * n + k)
    a, sa, w, sw = _operands(g, m, n, k)
    got = cp.matmul_fp8(a, sa, w, sw, dtype=torch.float32)
    _check(a, sa, w, sw, torch.float32, got)
    again = cp.matmul_fp8(a, sa, w, sw, dtype=torch.float32)
    assert torch.equal(got, again)                       # the same bits


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("m,n,k", [(1, 300, 512), (20, 200, 256), (150, 390, 400), (70, 33, 77)])
def test_matmul_types(m, n, k, dtype):
    g = gen(m + n + k)
    a, sa, w, sw = _operands(g, m, n, k)
    _check(a, sa, w, sw, dtype, cp.matmul_fp8(a, sa, w, sw, dtype=dtype))


@pytest.mark.parametrize("m", [1, 5, 40, 140])
@pytest.mark.parametrize("lda,ldw,offset", [(640, 1024, 0), (528, 512, 16), (513, 700, 0),
                                            (512, 512, 1), (516, 600, 4), (512, 516, 0)])
def test_matmul_strides_and_boundaries(m, lda, ldw, offset):
    g = gen(m + lda)
    n, k = 260, 512
    a, sa, w, sw = _operands(g, m, n, k, lda, ldw, offset)
    buf = torch.full((m, 300), 7.0, device="cuda")
    out = buf[:, 3:3 + n]
    cp.matmul_fp8(a, sa, w, sw, out=out)
    _check(a, sa, w, sw, torch.float32, out)
    assert bool((buf[:, :3] == 7).all()) and bool((buf[:, 3 + n:] == 7).all())


@pytest.mark.parametrize("m", [1, 9, 40, 140, 300])
@pytest.mark.parametrize("k", [1, 250, 385, 500])
def test_matmul_ignores_what_lies_behind_the_rows(m, k):
    """Padded rows: the bytes between a row's end and the next row are NaN and stay out."""
    g = gen(m + k)
    n, ld = 300, -(-k // 16) * 16 + 32
    a, sa, w, sw = _operands(g, m, n, k, ld, ld)
    for t, rows in ((a, m), (w, n)):
        whole = torch.as_strided(t.view(torch.uint8), (rows, ld), (ld, 1))
        whole[:, k:] = 0x7F
    _check(a, sa, w, sw, torch.float32, cp.matmul_fp8(a, sa, w, sw, dtype=torch.float32))


@pytest.mark.parametrize("m", [17, 130])
@pytest.mark.parametrize("k", [15, 33, 600, 2049, 4100])
def test_matmul_rows_on_any_byte(m, k):
    """Every offset of the rows from a 16-byte boundary, for either operand, NaN around them."""
    g = gen(m + k)
    n, kb = 70, -(-k // 128)
    sa, sw = torch.exp(randn(g, m, kb)).cuda() * 0.01, torch.exp(randn(g, 1, kb)).cuda() * 0.01

    def rows(count, ld, offset):
        buf = torch.full((count * ld + 32,), 0x7F, dtype=torch.uint8, device="cuda").view(E4M3)
        view = torch.as_strided(buf, (count, k), (ld, 1), offset)
        view.copy_((randn(g, count, k) * 60).clamp(-448, 448).to(E4M3))
        return view
    even = -(-k // 16) * 16
    for offset in range(16):
        pitch = k + 3 * offset + 1
        for a, w in ((rows(m, pitch, offset), rows(n, even, 0)),
                     (rows(m, even, 0), rows(n, pitch, offset)),
                     (rows(m, even + 16, offset), rows(n, pitch, 15 - offset))):
            ws = cp.matmul_fp8_workspace(a, w)
            got = cp.matmul_fp8(a, sa, w, sw, dtype=torch.float32, workspace=ws)
            _check(a, sa, w, sw, torch.float32, got)
            assert torch.equal(got, cp.matmul_fp8(a, sa, w, sw, dtype=torch.float32))


def test_matmul_rows_on_any_byte_in_a_graph_and_refusals():
    g = gen(5)
    a, sa, w, sw = _operands(g, 50, 300, 1001)
    need = (50 + 300) * 1008
    ws = cp.matmul_fp8_workspace(a, w)
    assert ws.numel() == need
    assert cp.matmul_fp8_workspace(a[:, :1], w[:, :1]).numel() == 350 * 16
    ref = cp.matmul_fp8(a, sa, w, sw)
    for bad in (ws[1:], ws.view(torch.int8), ws.cpu()):
        with pytest.raises(ValueError):
            cp.matmul_fp8(a, sa, w, sw, workspace=bad)
    with pytest.raises(cp.CPError):                      # not on a 16-byte boundary
        cp.matmul_fp8(a, sa, w, sw, workspace=torch.empty(need + 8, dtype=torch.uint8,
                                                          device="cuda")[8:])
    with pytest.raises(ValueError):
        cp.matmul_fp8_workspace(a, w[:, :7])
    out = torch.zeros_like(ref)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        cp.matmul_fp8(a, sa, w, sw, out=out)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(ref, out)


@pytest.mark.parametrize("m", [1, 20, 300])
def test_matmul_of_no_columns(m):
    """k = 0: zeros, and only where the output's rows are."""
    buf = torch.full((m, 12), 7.0, device="cuda")
    a, w = torch.empty(m, 0, device="cuda").to(E4M3), torch.empty(5, 0, device="cuda").to(E4M3)
    cp.matmul_fp8(a, torch.empty(m, 0, device="cuda"), w, torch.empty(1, 0, device="cuda"),
                  out=buf[:, 3:8])
    assert not buf[:, 3:8].any() and bool((buf[:, :3] == 7).all()) and bool((buf[:, 8:] == 7).all())


@pytest.mark.parametrize("m", [1, 40, 300])
def test_matmul_broadcast_rows(m):
    """One activation row for all (stride 0)."""
    g = gen(m)
    a, sa, w, sw = _operands(g, 1, 200, 256)
    many = cp.matmul_fp8(a.expand(m, 256), sa.expand(m, 2).contiguous(), w, sw,
                         dtype=torch.float32)
    _check(a.expand(m, 256), sa.expand(m, 2), w, sw, torch.float32, many)


@pytest.mark.parametrize("m", [1, 30, 200])
@pytest.mark.parametrize("k", [256, 250])
def test_matmul_special_values(m, k):
    """A NaN operand reaches its own row or column only, a zero, NaN or infinite scale acts
    as a factor of its group."""
    g = gen(m)
    n = 300
    a, sa, w, sw = _operands(g, m, n, k)
    w.view(torch.uint8)[7, 3] = 0x7F                     # NaN
    if m > 1:
        a.view(torch.uint8)[1, 200] = 0xFF
        sa[2:5, 1] = torch.tensor([0.0, float("inf"), float("nan")], device="cuda")
    got = cp.matmul_fp8(a, sa, w, sw, dtype=torch.float32).cpu()
    assert torch.isnan(got[:, 7]).all()
    if m > 1:
        assert torch.isnan(got[1]).all() and torch.isnan(got[4]).all()
        assert not torch.isfinite(got[3]).any()
    rows = [i for i in range(m) if not (m > 1 and i in (1, 3, 4))]
    cols = [j for j in range(n) if j != 7]
    ref, mag = matmul64(a[rows].cpu(), sa[rows].cpu(), w[cols[:7]].cpu(), sw[:1].cpu())
    assert_within(got[rows][:, :7], ref, mag * 140 * 2 * U32 + rounded(ref, torch.float32))
    assert torch.isfinite(got[rows][:, cols]).all()


def test_matmul_overflow_and_empty():
    a = torch.full((3, 128), 448.0, device="cuda").to(E4M3)
    w = torch.full((5, 128), 448.0, device="cuda").to(E4M3)
    one = torch.ones(3, 1, device="cuda")
    got = cp.matmul_fp8(a, one, w, torch.full((1, 1), 1.0, device="cuda"), dtype=torch.float16)
    assert torch.isinf(got).all()                        # 2.6e7 rounds past the type's largest
    none = torch.empty(0, 128, device="cuda").to(E4M3)
    assert cp.matmul_fp8(none, one[:0], w, one[:1]).shape == (0, 5)
    thin = torch.empty(3, 0, device="cuda").to(E4M3)
    wthin = torch.empty(5, 0, device="cuda").to(E4M3)
    out = torch.ones(3, 5, device="cuda")
    cp.matmul_fp8(thin, torch.empty(3, 0, device="cuda"), wthin, torch.empty(1, 0, device="cuda"),
                  out=out)
    assert not out.any()                                 # the sum over no columns


def test_matmul_takes_what_the_norm_and_the_quantiser_leave():
    g = gen(77)
    m, n, d = 50, 700, 1024
    x, res = randn(g, m, d, dtype=torch.bfloat16).cuda(), randn(g, m, d,
                                                                dtype=torch.bfloat16).cuda()
    gain, proj = randn(g, d).cuda(), randn(g, n, d, dtype=torch.bfloat16, std=0.03).cuda()
    q, sc, h = cp.rms_norm_fp8(x, gain, residual=res)
    w, sw = cp.quantize_fp8(proj, 128)
    got = cp.matmul_fp8(q, sc, w, sw, dtype=torch.float32)
    _check(q, sc, w, sw, torch.float32, got)
    # and the whole is the unquantised projection up to two e4m3 roundings (2^-4 each, at
    # random over 1024 terms: well inside 2^-4 of the norm)
    y = cp.rms_norm(x, gain, residual=res)[0].double() @ proj.double().T
    assert float((got.double() - y).norm() / y.norm()) < 2.0 ** -4


def test_matmul_on_another_stream_and_in_a_graph():
    g = gen(78)
    for m in (1, 40, 300):
        a, sa, w, sw = _operands(g, m, 520, 1024)
        torch.cuda.synchronize()
        ref = cp.matmul_fp8(a, sa, w, sw)
        torch.cuda.synchronize()
        s = torch.cuda.Stream()
        got = cp.matmul_fp8(a, sa, w, sw, stream=s)
        s.synchronize()
        assert torch.equal(ref, got)
        out = torch.zeros_like(ref)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            cp.matmul_fp8(a, sa, w, sw, out=out)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(ref, out)


def test_matmul_status_is_clear():
    assert cp.matmul_fp8_status() == cp.CP_OK


def test_matmul_refusals():
    g = gen(1)
    a, sa, w, sw = _operands(g, 4, 200, 256)
    for call in [
        lambda: cp.matmul_fp8(a.float(), sa, w, sw),
        lambda: cp.matmul_fp8(a, sa[:, :1], w, sw),
        lambda: cp.matmul_fp8(a, sa, w, sw[:1]),
        lambda: cp.matmul_fp8(a, sa.double(), w, sw),
        lambda: cp.matmul_fp8(a[:, :128], sa[:, :1].contiguous(), w, sw),
        lambda: cp.matmul_fp8(a, sa, w.t(), sw),
        lambda: cp.matmul_fp8(a, sa, w, sw, dtype=torch.float64),
        lambda: cp.matmul_fp8(a, sa, w, sw, out=torch.zeros(4, 199, device="cuda")),
        lambda: cp.matmul_fp8(a, sa, w, sw, out=torch.zeros(1, 200, device="cuda").expand(4, 200)),
        lambda: cp.matmul_fp8(a.cpu(), sa, w, sw),
        lambda: cp.matmul_fp8(a, sa.cpu(), w, sw),
    ]:
        with pytest.raises(ValueError):
            call()
