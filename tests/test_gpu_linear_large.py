"""The projection and dropout where offsets pass 32 bits: outputs, kept sums and gradients of more
than 2^32 elements, rows far apart; rows at the ends and around 2^32 elements are checked."""
import pytest
import torch

import trellis_row_decode_gb300 as cp

from layer_util import U32, assert_within, gen, randn, rounded
from linear_util import drop64, linear64, out_bound, philox, slope64, sum_bound

pytestmark = pytest.mark.gpu
M, N, K = 70001, 65536, 8
ROWS = [0, 1, 65535, 65536, 65537, 70000]       # 65536 * 65536 = 2^32


def _mask_rows(rows, d, p, seed):
    import numpy as np
    quad = np.arange(d // 4, dtype=np.uint64)[None, :]
    row = np.array(rows, dtype=np.uint64)[:, None]
    z = np.zeros((1, 1), dtype=np.uint64)
    w = np.stack(np.broadcast_arrays(*philox(quad + z, row + z, z, z, seed, 0)), -1)
    return torch.from_numpy(w.reshape(len(rows), d) < int((1 - p) * 2.0 ** 32 + 0.5))


def test_dropout_past_32_bits():
    x = torch.empty(M, N, dtype=torch.bfloat16, device="cuda")
    x.view(-1)[:1 << 20].normal_()
    for r in ROWS:
        x[r].normal_()
    out = cp.dropout(x, 0.25, 9, residual=x, out=x)
    assert out is x
    y = torch.empty(M, N, dtype=torch.bfloat16, device="cuda").fill_(1.0)
    out = cp.dropout(y, 0.25, 9)
    keep = _mask_rows(ROWS, N, 0.25, 9)
    got = out[ROWS].float().cpu()
    want = keep.float() * torch.tensor(1 / 0.75).bfloat16().float()
    assert torch.equal(got, want)


def test_linear_and_its_gradient_past_32_bits():
    g = gen(0)
    x, w = randn(g, M, K, dtype=torch.bfloat16), randn(g, N, K, dtype=torch.bfloat16, std=0.3)
    xc, wc = x.cuda(), w.cuda()
    out, pre = cp.linear(xc, wc, None, "silu", pre=True)
    ref, z, mag = linear64(x[ROWS], w, None, "silu")
    assert_within(out[ROWS], ref, out_bound(ref, z, mag, K, torch.bfloat16))
    assert_within(pre[ROWS], z, sum_bound(mag, K) + rounded(z, torch.bfloat16))
    out.zero_()                                  # a gradient whose rows are mostly zeros
    out[ROWS] = randn(g, len(ROWS), N, dtype=torch.bfloat16).cuda()
    dy = out[ROWS].cpu().double()
    dx, dw, db = cp.linear_grad(out, xc, wc, "silu", pre, db_dtype=torch.float32)
    zs = pre[ROWS].cpu().double()
    own = 16 * U32 * (zs.abs() + 1) * dy.abs()
    dz = dy * slope64(zs, "silu")
    cut = own * 1.01 + dz.abs() * (2.0 ** -8 + 4 * U32) + 2.0 ** -130
    X, W = x[ROWS].double(), w.double()
    assert_within(dx[ROWS], dz @ W, cut @ W.abs() + sum_bound((dz.abs() + cut) @ W.abs(), N)
                  + rounded(dz @ W, torch.bfloat16))
    assert_within(dw, dz.T @ X, cut.T @ X.abs() + sum_bound((dz.abs() + cut).T @ X.abs(), M)
                  + rounded(dz.T @ X, torch.bfloat16))
    assert_within(db, dz.sum(0), (own + 4 * U32 * dz.abs()).sum(0)
                  + (M + 64) * U32 * (dz.abs() + own).sum(0) + rounded(dz.sum(0), torch.float32))
    assert cp.linear_status() == cp.CP_OK


@pytest.mark.parametrize("m", [12, 200])
def test_linear_rows_far_apart(m):
    """Row strides of 2^28 and more elements: 12 rows span 6 GB, 200 rows 4 GB a side."""
    g = gen(m)
    n, k = 48, 64
    pitch = (1 << 28) + 8 if m == 12 else (1 << 23) + 8
    x = torch.empty(m * pitch, dtype=torch.bfloat16, device="cuda").as_strided((m, k), (pitch, 1))
    out = torch.empty(m * pitch, dtype=torch.bfloat16, device="cuda").as_strided((m, n), (pitch, 1))
    xs, w = randn(g, m, k, dtype=torch.bfloat16), randn(g, n, k, dtype=torch.bfloat16, std=0.125)
    x.copy_(xs)
    cp.linear(x, w.cuda(), None, "relu", out=out)
    ref, z, mag = linear64(xs, w, None, "relu")
    assert_within(out, ref, out_bound(ref, z, mag, k, torch.bfloat16))
    cp.dropout(x[:, :n], 0.5, 3, out=out)
    want = drop64(xs[:, :n].double(), 0.5, 3, 0)
    assert_within(out, want, 2 * U32 * want.abs() + rounded(want, torch.bfloat16))


def test_linear_sums_a_long_k():
    """131,072 positive products a sum: what the sums lose to one side shows in the outputs' mean
    error, where their own roundings cancel."""
    m, n, k = 2560, 2560, 1 << 17
    at = torch.Generator(device="cuda").manual_seed(5)
    x = torch.rand(m, k, generator=at, device="cuda", dtype=torch.float16)
    w = torch.rand(n, k, generator=at, device="cuda", dtype=torch.float16)
    w *= (torch.rand(n, 1, generator=at, device="cuda") * 0.25 + 0.25).half()
    out = cp.linear(x, w)
    ref, z, mag = linear64(x[::20].cpu(), w[::20].cpu())
    got = out[::20, ::20].cpu().double()
    assert_within(got, ref, out_bound(ref, z, mag, k, torch.float16))
    # 16,384 roundings of up to 2^-11 each have a mean of 2.2e-6 (one deviation); sums of 512 cut at
    # each addition, joined by additions that round, lose up to 5.5e-7 + 256 U32
    assert ((got - ref) / ref).mean().abs() < 5 * 2.2e-6 + 5.5e-7 + 256 * U32
    assert cp.linear_status() == cp.CP_OK


@pytest.mark.parametrize("m,n,k", [(8192, 2048, 200), (16384, 1024, 520), (4096, 1000, 1100)])
def test_dropout_changes_no_sum(m, n, k):
    """Dropout may choose another tile: what it keeps is what the product without it has, bit by bit."""
    at = torch.Generator(device="cuda").manual_seed(m)
    x = torch.randn(m, k, generator=at, device="cuda").half()
    w = torch.randn(n, k, generator=at, device="cuda").half()
    r = torch.randn(m, n, generator=at, device="cuda")
    z = cp.linear(x, w, dtype=torch.float32)
    out = cp.linear(x, w, residual=r, p=0.25, seed=3, offset=4, dtype=torch.float32)
    assert torch.equal(out, cp.dropout(z, 0.25, 3, 4, residual=r))
    assert cp.linear_status() == cp.CP_OK
