"""The feed-forward layers' formulas in 64 bits, written from their definitions, and
the error bounds that the tests derive from the types."""
from __future__ import annotations

import math

import torch

TYPES = {"bf16": torch.bfloat16, "f16": torch.float16}
ACTS = ("none", "relu", "gelu", "gelu_tanh", "silu")


def act(name, z):
    """act(z) and act'(z) of a float64 tensor."""
    if name == "none":
        return z, torch.ones_like(z)
    if name == "relu":
        return torch.where(z > 0, z, 0.0), (z > 0).double()
    if name == "gelu":
        phi = 0.5 * torch.erfc(-z * math.sqrt(0.5))   # (1 + erf) would lose the lower tail
        return z * phi, phi + z * torch.exp(-z * z / 2) / math.sqrt(2 * math.pi)
    if name == "silu":
        s = torch.sigmoid(z)
        return z * s, s * (1 + z * torch.sigmoid(-z))
    c = math.sqrt(2 / math.pi)
    s = torch.sigmoid(2 * c * (z + 0.044715 * z ** 3))
    r = torch.sigmoid(-2 * c * (z + 0.044715 * z ** 3))
    return z * s, s + z * s * r * 2 * c * (1 + 3 * 0.044715 * z ** 2)


# Lipschitz constants of act and of act' (their largest slopes: relu 1, gelu 1.13 and 0.8,
# silu 1.1 and 0.5), rounded up, and the largest |act'|.
SLOPE = 1.13
CURVE = 0.82


def linear(name, x, w, b=None, r=None):
    z = x @ w.T + (0 if b is None else b)
    y = act(name, z)[0]
    return y + (0 if r is None else r), z


def gated(name, x, wg, wu, bg=None, bu=None):
    g = x @ wg.T + (0 if bg is None else bg)
    u = x @ wu.T + (0 if bu is None else bu)
    return act(name, g)[0] * u, g, u


def linear_backward(name, x, w, z, dy):
    dz = dy * act(name, z)[1] if name != "none" else dy
    return dz @ w, dz.T @ x, dz.sum(0), dz


def gated_backward(name, x, wg, wu, g, u, dh):
    a, s = act(name, g)
    dg, du = dh * u * s, dh * a
    return dg @ wg + du @ wu, dg.T @ x, du.T @ x, dg.sum(0), du.sum(0), dg, du


def half_step(t):
    """The largest relative error of one rounding to the type."""
    return torch.finfo(t).eps / 2


def tiny(t):
    """Half a step below the smallest normal number: the rounding's absolute error there."""
    return torch.finfo(t).tiny * torch.finfo(t).eps / 2
