"""Shared by the memory layer's GPU tests: element types, their rounding units, and
plain 64-bit forms of the operators (CPU, float64).

Error bounds used by the tests, from the formulas and the way the kernels sum:
U32 = 2^-24 is the unit of an fp32 rounding; a sum of n terms in any fixed order is off
by at most (n - 1) U32 times the sum of magnitudes, and the one rounding to the output's
type adds UNIT[type] times the result (TINY[type] where it is subnormal).
"""
import torch

DTYPES = [torch.float32, torch.float16, torch.bfloat16]
U32 = 2.0 ** -24
UNIT = {torch.float32: 2.0 ** -24, torch.float16: 2.0 ** -11, torch.bfloat16: 2.0 ** -8}
TINY = {torch.float32: 2.0 ** -149, torch.float16: 2.0 ** -25, torch.bfloat16: 2.0 ** -133}
E4M3 = torch.float8_e4m3fn


def gen(seed):
    return torch.Generator().manual_seed(seed)


def randn(g, *shape, dtype=torch.float32, std=1.0):
    return (torch.randn(shape, generator=g) * std).to(dtype)


def assert_within(got, ref, bound, what=""):
    """Every element of got within bound of ref; non-finite ones equal in kind."""
    got, ref = got.detach().cpu().double(), ref.double()
    assert got.shape == ref.shape, what
    fine = torch.isfinite(ref)
    assert torch.equal(torch.isnan(got), torch.isnan(ref)), what
    inf = torch.isinf(ref)
    assert torch.equal(got[inf], ref[inf]), what
    off = (got - ref).abs()[fine]
    bound = torch.as_tensor(bound, dtype=torch.float64).expand(ref.shape)[fine]
    bad = ~(off <= bound)
    assert not bad.any(), (f"{what}: {int(bad.sum())} of {off.numel()} off, worst "
                           f"{float((off / bound.clamp(min=1e-300)).max()):.3g} times the bound")


def rounded(ref, dtype):
    """The last rounding's share of a bound."""
    return ref.abs() * UNIT[dtype] + TINY[dtype]


# ------------------------------------------------------------------ 64-bit forms

def embed64(weight, ids, scale):
    out = torch.zeros(ids.numel(), weight.shape[1], dtype=torch.float64)
    for j, i in enumerate(ids.tolist()):
        if 0 <= i < weight.shape[0]:
            out[j] = weight[i].double() * scale
    return out


def embed_grad64(dy, ids, n_rows, scale):
    """(gradient, sum of magnitudes, lookups of each row)."""
    grad = torch.zeros(n_rows, dy.shape[1], dtype=torch.float64)
    mags = torch.zeros_like(grad)
    count = torch.zeros(n_rows, dtype=torch.int64)
    ok = (ids >= 0) & (ids < n_rows)
    at, rows = ids[ok], dy[ok].double() * scale
    grad.index_add_(0, at, rows)
    mags.index_add_(0, at, rows.abs())
    count.index_add_(0, at, torch.ones_like(at))
    return grad, mags, count


def norm64(x, weight, eps, residual=None):
    s = x.double() + (residual.double() if residual is not None else 0.0)
    r = 1.0 / torch.sqrt(s.square().mean(-1, keepdim=True) + eps)
    return s * r * weight.double(), s


def scales64(y, block=1):
    """amax / 448 of every block of `block` x 128, and spread over the elements."""
    m, k = y.shape
    mb, kb = -(-m // block), -(-k // 128)
    pad = torch.zeros(mb * block, kb * 128, dtype=torch.float64)
    pad[:m, :k] = y
    amax = pad.abs().view(mb, block, kb, 128).amax((1, 3))
    scales = amax.clamp(min=1e-30) / 448.0
    return scales, scales.repeat_interleave(block, 0)[:m].repeat_interleave(128, 1)[:, :k]


def norm_grad64(dy, h, weight, eps, dres=None):
    """(dx, dw) and the magnitudes that their sums pass through."""
    h, dy, w = h.double(), dy.double(), weight.double()
    d = h.shape[-1]
    r = 1.0 / torch.sqrt(h.square().mean(-1, keepdim=True) + eps)
    n, t = h * r, dy * w
    res = dres.double() if dres is not None else torch.zeros_like(h)
    dx = res + r * (t - n * (t * n).mean(-1, keepdim=True))
    dx_mag = res.abs() + r * (t.abs() + n.abs() * (t * n).abs().mean(-1, keepdim=True))
    return dx, dx_mag, (dy * n).sum(0), (dy * n).abs().sum(0)


def matmul64(a, sa, w, sw):
    """(product, sum of magnitudes) from the values that the e4m3 bytes stand for."""
    m, k = a.shape
    n = w.shape[0]
    A = a.float().double() * sa.double().repeat_interleave(128, 1)[:, :k]
    W = w.float().double() * sw.double().repeat_interleave(128, 0)[:n].repeat_interleave(
        128, 1)[:, :k]
    return A @ W.T, A.abs() @ W.abs().T
