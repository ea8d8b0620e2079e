"""The stated bounds of the gated block's activations, on a million fp32 gates each, against 64 bits.

In u = 2^-24, relative to the terms of act = g p and of its slope p + g p q v' (p the logistic or the normal
distribution function of v, q = 1 - p): 16 of silu and gelu, 16 + 5 |v| of gelu_tanh, whose v = 2 sqrt(2 / pi)
(g + 0.044715 g^3) is five times rounded (the cubic's constant 0.58 u and its two products 2, their sum 1,
2 sqrt(2 / pi) 0.48 and its product 1: 5.06 |v|, and |v| < 90 where anything is left above 2^-126); and 20
of the forward pass's silu where |g| <= 16, whose exponential's argument is rounded and not corrected (at
most 2^-20 of an argument up to 23.1 to the base 2, ln 2 of that 11.1 u, and 1 / ln 2 0.32 |g| u = 5.1).
What is below 2^-126 may count as 0."""
import math

import pytest
import torch

import gradient_compression_amd as gca
from tests.gpu_helpers import log

pytestmark = pytest.mark.gpu

U, LOW = 2.0 ** -24, 2.0 ** -126


def gates():
    gen = torch.Generator("cuda").manual_seed(17)
    rand = lambda n: torch.rand(n, generator=gen, device="cuda", dtype=torch.float64)  # noqa: E731
    far = torch.cat([60 * rand(400000) - 30, 16.0 + 80 * rand(100000), -16.0 - 80 * rand(100000),
                     40.0 * (rand(200000) - 0.5) ** 3, 10.0 ** (14 * rand(248576) - 12)])
    return far.float()


def terms(act, g):
    """(act, slope, and what their bounds are relative to, the slope's two terms; v) in 64 bits."""
    if act == "gelu":
        p = 0.5 * torch.special.erfc(g / -math.sqrt(2.0))
        d = g * torch.exp(-0.5 * g * g) / math.sqrt(2.0 * math.pi)
        return g * p, p + d, p + d.abs(), torch.zeros_like(g)
    if act == "silu":
        v, dv = g, torch.ones_like(g)
    else:
        k = 2.0 * math.sqrt(2.0 / math.pi)
        v, dv = k * (g + 0.044715 * g ** 3), k * (1.0 + 3 * 0.044715 * g * g)
    p, q = torch.sigmoid(v), torch.sigmoid(-v)
    t = g * p * q * dv
    return g * p, p + t, p + t.abs(), v


def within(got, want, bound, what):
    worst = ((got.double() - want).abs() / (bound + LOW)).max().item()
    log(f"[gated] {what}: worst {worst:.3f} of the bound")
    assert worst <= 1.0, f"{what}: {worst} of the bound"


@pytest.mark.parametrize("act", ["silu", "gelu", "gelu_tanh"])
def test_the_stated_bounds(act):
    g = gates()
    a, s, around, v = terms(act, g.double())
    units = 16.0 + (5.0 * v.abs().clamp(max=90.0) if act == "gelu_tanh" else 0.0)
    g = g.view(-1, 64)
    one, dgate, dup = torch.ones_like(g), torch.empty_like(g), torch.empty_like(g)
    gca.gated_linear_backward(one, g, one, dgate, dup, activation=act)
    within(dup.view(-1), a, U * units * a.abs(), f"{act}, backward")
    within(dgate.view(-1), s, U * units * around, f"{act}'s slope")
    # forward, through an identity and a weight of the ones
    x = torch.cat((g, torch.ones(g.shape[0], 8, device="cuda")), 1)
    wg, wu = torch.zeros(64, 72, device="cuda"), torch.zeros(64, 72, device="cuda")
    wg[:, :64], wu[:, 64] = torch.eye(64), 1.0
    h, gate = torch.empty_like(g), torch.empty_like(g)
    gca.gated_linear(x, wg, wu, h, gate=gate, activation=act)
    assert torch.equal(gate, g)
    if act == "silu":
        units = torch.where(g.view(-1).abs() <= 16.0, 20.0, 16.0)
    within(h.view(-1), a, U * units * a.abs(), f"{act}, forward")
