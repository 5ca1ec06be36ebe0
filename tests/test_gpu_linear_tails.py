"""Activations and their slopes against 64 bits, relative to their own values: where silu and both
forms of gelu fade out towards minus infinity too.

Bounds, in units U32 of an fp32 rounding.  An exponential takes the rounding errors of its argument a as
a relative error: two roundings and a constant's for silu's a = |z| (2.5 |a|) and gelu's a = z^2 / 2
(2.5 a), seven for the tanh form's a (7.5 |a|); everything behind it (the two approximate
instructions, at most 4 and 2, additions, products, the polynomial's 3) makes fewer than 20.  Below
2^-126 the exponential is zero."""
import math

import pytest
import torch

import trellis_row_decode_gb300 as cp

from layer_util import U32, assert_within

pytestmark = pytest.mark.gpu


def values():
    z = torch.cat([torch.linspace(-16, 16, 6001), torch.linspace(-100, 30, 1301),
                   torch.linspace(-1e-3, 1e-3, 101), torch.tensor([0.0, -1e-30, 1e-30])])
    return z.bfloat16().unique()


def cdf64(z):
    """Phi(z) by the complementary error function (torch.special.ndtr cancels below -1)."""
    return 0.5 * torch.special.erfc(-z * math.sqrt(0.5))


def value64(z, act):
    if act == "gelu":
        return z * cdf64(z)
    return z * torch.special.expit(
        z if act == "silu" else 2 * math.sqrt(2 / math.pi) * (z + 0.044715 * z ** 3))


def argument(z, act):
    """Units of the exponential's relative error."""
    if act == "silu":
        return 2.5 * z.abs()
    if act == "gelu":
        return 1.25 * z.square()
    return 7.5 * 2 * math.sqrt(2 / math.pi) * (z + 0.044715 * z ** 3).abs()


@pytest.mark.parametrize("act", ["silu", "gelu", "gelu_tanh"])
@pytest.mark.parametrize("few", [False, True])
def test_activations_relative_to_their_values(act, few):
    z = values()
    one = torch.ones(1, 1, dtype=torch.bfloat16, device="cuda")
    if few:
        got = cp.linear(one, z.cuda()[:, None].contiguous(), None, act, dtype=torch.float32)[0]
    else:
        got = cp.linear(z.cuda()[:, None].contiguous(), one, None, act, dtype=torch.float32)[:, 0]
    z = z.double()
    want = value64(z, act)
    # where the exponential overflows the sigmoid is 0: below |z| 2^-125
    assert_within(got, want, (20 + argument(z, act)) * U32 * want.abs() + z.abs() * 2.0 ** -125)


def test_gelu_slope_relative_to_its_terms():
    """db of a single row of ones is the slope itself: Phi(z) + z times the bell."""
    z = values()
    pre, dy = z.cuda()[None], torch.ones(1, z.numel(), dtype=torch.bfloat16, device="cuda")
    x = torch.ones(1, 8, dtype=torch.bfloat16, device="cuda")
    w = torch.zeros(z.numel(), 8, dtype=torch.bfloat16, device="cuda")
    db = cp.linear_grad(dy, x, w, "gelu", pre, db_dtype=torch.float32)[2]
    z = z.double()
    low, high = cdf64(z), z * torch.exp(-z.square() / 2) / math.sqrt(2 * math.pi)
    assert_within(db, low + high, (20 + argument(z, "gelu")) * U32 * (low + high.abs())
                  + (1 + z.abs()) * 2.0 ** -125)
