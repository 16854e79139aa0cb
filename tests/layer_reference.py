"""The layers' formulas in 64 bits, for the tests of the layer kernels."""
import math

import torch


def act_value(act, z):
    if act == "none":
        return z
    if act == "relu":
        return z.clamp(min=0)
    if act == "gelu":
        return 0.5 * z * (1 + torch.erf(z / math.sqrt(2)))
    if act == "silu":
        return z * torch.sigmoid(z)
    return 0.5 * z * (1 + torch.tanh(math.sqrt(2 / math.pi) * (z + 0.044715 * z ** 3)))


def act_slope(act, z):
    if act == "none":
        return torch.ones_like(z)
    if act == "relu":
        return (z > 0).to(z.dtype)
    if act == "gelu":
        return 0.5 * (1 + torch.erf(z / math.sqrt(2))) + z * torch.exp(-z * z / 2) / math.sqrt(2 * math.pi)
    if act == "silu":
        s = torch.sigmoid(z)
        return s * (1 + z * (1 - s))
    t = torch.tanh(math.sqrt(2 / math.pi) * (z + 0.044715 * z ** 3))
    return 0.5 * (1 + t) + 0.5 * z * (1 - t * t) * math.sqrt(2 / math.pi) * (1 + 3 * 0.044715 * z * z)


def linear_grads(act, dy, x, w, z):
    dz = dy * act_slope(act, z)
    return dz @ w.t(), x.t() @ dz, dz.sum(0)


def gated_grads(act, dh, x, wg, wu, g, u):
    dg, du = dh * u * act_slope(act, g), dh * act_value(act, g)
    return dg @ wg.t() + du @ wu.t(), x.t() @ dg, x.t() @ du


def layer_norm_grads(dy, x, w, mean, rstd):
    h = (x - mean[:, None]) * rstd[:, None]
    t = dy if w is None else dy * w
    dx = rstd[:, None] * (t - t.mean(1, keepdim=True) - h * (t * h).mean(1, keepdim=True))
    return dx, (dy * h).sum(0), dy.sum(0)
