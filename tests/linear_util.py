"""Shared by the tests of the 16-bit projection and of dropout: the generator, the mask and
the operators in plain 64-bit forms (CPU), and the bounds that go with them.

The generator is written from its publication (Salmon, Moraes, Dror and Shaw, "Parallel random
numbers: as easy as 1, 2, 3", 2011); its known answers are in test_linear_args.py.
"""
import math

import numpy as np
import torch

from layer_util import U32, rounded

ACTS = ["none", "relu", "silu", "gelu", "gelu_tanh"]


def philox(c0, c1, c2, c3, k0, k1):
    """Philox4x32-10 on uint64 arrays that hold 32-bit words."""
    low = np.uint64(0xFFFFFFFF)
    c = [np.asarray(v, dtype=np.uint64) for v in (c0, c1, c2, c3)]
    k = [np.uint64(k0), np.uint64(k1)]
    for _ in range(10):
        a, b = c[0] * np.uint64(0xD2511F53), c[2] * np.uint64(0xCD9E8D57)
        c = [(b >> np.uint64(32)) ^ c[1] ^ k[0], b & low, (a >> np.uint64(32)) ^ c[3] ^ k[1],
             a & low]
        k = [(k[0] + np.uint64(0x9E3779B9)) & low, (k[1] + np.uint64(0xBB67AE85)) & low]
    return c


def mask64(rows, d, p, seed, offset):
    """True where an element of [rows, d] is kept."""
    quad = np.arange((d + 3) // 4, dtype=np.uint64)[None, :]
    row = np.arange(rows, dtype=np.uint64)[:, None]
    z = np.zeros((1, 1), dtype=np.uint64)
    words = philox(quad + z, row + z, z + np.uint64(offset & 0xFFFFFFFF),
                   z + np.uint64(offset >> 32), seed & 0xFFFFFFFF, seed >> 32)
    words = np.stack(np.broadcast_arrays(*words), -1).reshape(rows, -1)[:, :d]
    return torch.from_numpy(words < np.uint64(int((1.0 - p) * 2.0 ** 32 + 0.5)))


def drop64(v, p, seed, offset):
    if p == 0:
        return v
    keep = mask64(*v.shape, p, seed, offset)
    return torch.where(keep, v / (1.0 - p) if p < 1 else v, torch.zeros_like(v))


def act64(z, act):
    if act == "relu":
        return torch.where(z < 0, torch.zeros_like(z), z)
    if act == "silu":
        return z * torch.special.expit(z)
    if act == "gelu":
        return z * torch.special.ndtr(z)
    if act == "gelu_tanh":
        return 0.5 * z * (1 + torch.tanh(math.sqrt(2 / math.pi) * (z + 0.044715 * z ** 3)))
    return z


def slope64(z, act):
    z = z.double().requires_grad_()
    return torch.autograd.grad(act64(z, act).sum(), z)[0] if act != "none" else torch.ones_like(z)


def linear64(x, w, bias=None, act="none", residual=None, p=0.0, seed=0, offset=0):
    """(out, pre, magnitude of the sums)."""
    x, w = x.double(), w.double()
    z, mag = x @ w.T, x.abs() @ w.abs().T
    if bias is not None:
        z, mag = z + bias.double(), mag + bias.double().abs()
    out = drop64(act64(z, act), p, seed, offset)
    if residual is not None:
        out = out + residual.double()
    return out, z, mag


def sum_bound(mag, terms):
    """fp32 sums of `terms` exact products, split and joined in any way: 2 U32 an addition, since
    the tensor core may cut instead of round."""
    return mag * (terms + 40) * 2 * U32


def out_bound(out, z, mag, k, dtype, p=0.0):
    """The sums' error through an activation (no slope exceeds 1.13), 16 roundings of the
    activation's own arithmetic relative to |z| + 1, dropout's scale (once rounded, one product)
    and the residual's addition, and the last rounding."""
    scale = 1.0 / (1.0 - p) if p < 1 else 0.0
    return (1.13 * sum_bound(mag, k) + 16 * U32 * (z.abs() + 1)) * scale * 1.01 \
        + 2 * U32 * (out.abs() + scale * z.abs()) + rounded(out, dtype)
