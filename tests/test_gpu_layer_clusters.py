"""Kernels whose CTAs meet at a barrier of their cluster while lanes of a warp come from branches of
their own: ids outside the table beside valid ones, outputs that end inside a warp's share."""
import pytest
import torch

import trellis_row_decode_gb300 as cp

from layer_util import E4M3, U32, assert_within, embed_grad64, gen, matmul64, randn, rounded

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("every", [2, 7, 33, 5000])
@pytest.mark.parametrize("n", [4097, 9000, 70_001])
def test_embed_grad_reports_scattered_ids_outside(n, every):
    """One id in `every` lies outside (none, where there are fewer ids): the lanes that meet it set the status word, the others do
    not, and both count on."""
    g = gen(n + every)
    n_rows, d = 600, 40
    ids = torch.randint(0, n_rows, (n,), generator=g)
    ids[every - 1::every] = torch.tensor(-1) if every % 2 else torch.tensor(n_rows)
    dy = randn(g, n, d)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    got = cp.embed_grad(dy.cuda(), ids.cuda(), n_rows, status=status)
    ref, mags, count = embed_grad64(dy, ids, n_rows, 1.0)
    assert_within(got, ref, (count[:, None] + 2) * U32 * mags + rounded(ref, torch.float32))
    assert int(status.item()) == int(n >= every)


# rows of w that are shared by 2, 4 and 8 CTAs (few rows of a, at most 8 MB of w), ends inside the
# CTA's 16 rows of w and its 8 or 16 rows of a, rows on any byte
@pytest.mark.parametrize("m,n,k", [(1, 2000, 4096), (3, 1001, 8192), (8, 333, 24576), (9, 90, 65536),
                                   (16, 17, 40000), (5, 1001, 8191), (13, 333, 24575), (16, 1, 99999)])
def test_matmul_of_shared_rows(m, n, k):
    g = gen(m * n + k)
    kb = -(-k // 128)
    a = (randn(g, m, k) * 60).clamp(-448, 448).to(E4M3)
    w = (randn(g, n, k) * 60).clamp(-448, 448).to(E4M3)
    sa, sw = torch.exp(randn(g, m, kb)) * 0.01, torch.exp(randn(g, -(-n // 128), kb)) * 0.01
    buf = torch.full((m, n + 9), 7.0, device="cuda")
    cp.matmul_fp8(a.cuda(), sa.cuda(), w.cuda(), sw.cuda(), out=buf[:, 4:4 + n])
    ref, mag = matmul64(a, sa, w, sw)
    # 128 products of a group, the groups, and the parts of 8 warps and 8 CTAs lie over a term
    assert_within(buf[:, 4:4 + n], ref, mag * (128 + kb + 16) * 2 * U32 + rounded(ref, torch.float32))
    assert bool((buf[:, :4] == 7).all()) and bool((buf[:, 4 + n:] == 7).all())
