"""linear and linear_grad on small whole numbers: every product and every partial sum stays below
2^24 and is exact in fp32 however it is split, cut or joined, so the outputs have to be the exact
sums' bits.  One size for each width of a tile, each split of k and each kernel; and the segments
that long sums of fp32 outputs are joined from."""
import pytest
import torch

import trellis_row_decode_gb300 as cp

from layer_util import gen

pytestmark = pytest.mark.gpu


def whole(g, *shape, most=3, dtype=torch.bfloat16):
    return torch.randint(-most, most + 1, shape, generator=g).to(dtype)


def product(a, b):
    """a @ b in 64 bits."""
    return (a.cuda().double() @ b.cuda().double())


# m, n, k: columns of a tile 32, 64, 96, 128, 160, 192, 224, 256; then units that share a tile's k 2, 3, 4,
# 6, 8, 12, 16, 24, 32; rows that end inside a tile and inside 16 bytes among them
WIDTHS = [(130, 32, 200), (130, 2500, 200), (300, 2500, 72), (300, 4000, 200), (777, 2500, 520),
          (5000, 500, 200), (777, 4000, 72), (5000, 700, 200)]
SPLITS = [(300, 4000, 16384), (5000, 32, 4096), (4096, 32, 4096), (130, 333, 3000), (130, 32, 3000),
          (300, 96, 4096), (130, 32, 4096), (130, 96, 8192), (130, 32, 8192)]
# the kernel for few rows, each of its widths, and long k on both sides of its limit
LONG = [(1, 1000, 24576), (16, 130, 8193), (32, 257, 2321), (48, 1024, 24576), (64, 200, 24576),
        (96, 77, 8193), (128, 130, 24576), (129, 130, 24576), (300, 513, 8193), (700, 1000, 2321),
        (1000, 2050, 24576)]


@pytest.mark.parametrize("m,n,k", WIDTHS + SPLITS + LONG)
def test_linear_sums_are_exact(m, n, k):
    g = gen(m + n + k)
    x, w = whole(g, m, k), whole(g, n, k)
    bias, res = whole(g, n, most=9), whole(g, m, n, most=99, dtype=torch.float32)
    z = product(x, w.T) + bias.cuda().double()
    a = x.cuda(), w.cuda(), bias.cuda()
    assert torch.equal(cp.linear(*a, dtype=torch.float32), z.float())
    out, pre = cp.linear(*a, "relu", residual=res.cuda(), dtype=torch.float32, pre=True)
    assert torch.equal(out, (z.clamp(min=0) + res.cuda().double()).float())
    assert torch.equal(pre, z.float().bfloat16())
    assert torch.equal(cp.linear(*a), pre)
    assert cp.linear_status() == cp.CP_OK


# columns of dx's tiles 32 to 256 and of dw's, and both products with their k shared (dw's by 3, 4, 6, 8,
# 12 and 16 units, dx's by 3, 4, 6, 8, 12 and 16)
GRADS = [(130, 90, 300), (130, 30, 304), (300, 30, 300), (300, 30, 1500), (500, 30, 304),
         (500, 30, 2049), (777, 90, 304), (777, 30, 300), (130, 30, 2049), (130, 500, 304),
         (200, 700, 300), (130, 700, 304), (200, 900, 304), (130, 900, 304), (130, 1340, 300),
         (5000, 30, 2600), (5000, 30, 1500), (4090, 30, 1000), (3000, 30, 304), (5000, 30, 520),
         (4090, 30, 304), (5000, 2500, 64), (300, 4000, 200), (130, 4000, 768), (130, 2500, 64),
         (130, 4000, 64), (130, 4096, 64), (4096, 4096, 64), (4096, 4096, 520)]


@pytest.mark.parametrize("m,n,k", GRADS)
def test_linear_grad_sums_are_exact(m, n, k):
    g = gen(m + n + k)
    dy, x, w = whole(g, m, n), whole(g, m, k), whole(g, n, k)
    a = dy.cuda(), x.cuda(), w.cuda()
    dx, dw, db = product(dy, w), product(dy.T, x), dy.cuda().double().sum(0)
    got = cp.linear_grad(*a, dw_dtype=torch.float32, db_dtype=torch.float32)
    assert torch.equal(got[0], dx.float().bfloat16())
    assert torch.equal(got[1], dw.float()) and torch.equal(got[2], db.float())
    got = cp.linear_grad(*a)
    assert torch.equal(got[0], dx.float().bfloat16())
    assert torch.equal(got[1], dw.float().bfloat16()) and torch.equal(got[2], db.float().bfloat16())
    # relu's slope is 0 or 1: dz is exact in 16 bits; one gradient alone, and added to
    pre = whole(g, m, n)
    dz = torch.where(pre > 0, dy, torch.zeros_like(dy))
    dw = product(dz.T, x)
    have = whole(g, n, k, most=99, dtype=torch.float32).cuda()
    want = (dw + have.double()).float()
    cp.linear_grad(*a, "relu", pre.cuda(), need_dx=False, need_db=False, dw=have, accumulate=True)
    assert torch.equal(have, want)
    dx = cp.linear_grad(*a, "relu", pre.cuda(), need_dw=False, need_db=False)[0]
    assert torch.equal(dx, product(dz, w).float().bfloat16())
    assert cp.linear_status() == cp.CP_OK


def joined(parts):
    """Sums added up in order, each addition rounded to fp32."""
    total = torch.zeros_like(parts[0])
    for part in parts:
        total = total + part
    return total


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("m,n,k", [(5000, 2560, 4096), (2560, 5000, 24576), (3000, 4000, 2321),
                                   (48, 20000, 4096), (1, 20000, 24576), (100, 40000, 1000)])
def test_fp32_sums_are_those_of_segments(m, n, k, dtype):
    """The tensor core adds 512 of k alone; what it makes of them is joined by fp32 additions: the bits
    of the products of 512 of k each, added up in order.  (Sizes whose k is not shared by several
    units, for many rows and for few.)"""
    g = torch.Generator(device="cuda").manual_seed(k)
    x = torch.randn(m, -(-k // 8) * 8, generator=g, device="cuda").to(dtype)[:, :k]
    w = torch.randn(n, -(-k // 8) * 8, generator=g, device="cuda").to(dtype)[:, :k]
    parts = [cp.linear(x[:, i:i + 512], w[:, i:i + 512], dtype=torch.float32)
             for i in range(0, k, 512)]
    assert torch.equal(cp.linear(x, w, dtype=torch.float32), joined(parts))


@pytest.mark.parametrize("m,n,k", [(4096, 4096, 2048), (1300, 5000, 2560)])
def test_fp32_gradients_are_those_of_segments(m, n, k):
    g = torch.Generator(device="cuda").manual_seed(m)
    dy, x, w = (torch.randn(*s, generator=g, device="cuda").bfloat16() for s in ((m, n), (m, k), (n, k)))
    parts = [cp.linear_grad(dy[i:i + 512], x[i:i + 512], w, dw_dtype=torch.float32)[1]
             for i in range(0, m, 512)]
    assert torch.equal(cp.linear_grad(dy, x, w, dw_dtype=torch.float32)[1], joined(parts))
