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


# ------------------------------------------------ gradients by differences --

def derivative_bounds(act):
    """The largest magnitude of an activation's second and third derivatives."""
    z = torch.linspace(-12, 12, 200001, dtype=torch.float64, requires_grad=True)
    d, found = act_value(act, z).sum(), []
    for _ in range(3):
        d, = torch.autograd.grad(d.sum(), z, create_graph=True)
        found.append(float(d.detach().abs().max()))
    return found[1], found[2]


def difference_bound(act, dy, z, q, h, sums, step):
    """How far <gradient, v> may be from the central difference of <dy, act(z)>
    with the step h, where z moves by q along v: the third derivative's h^2 / 6
    q^3; the errors of two evaluations, `sums` each and 4e-7 |act(z)| with the
    activation's, over 2 h; and the slope at z rounded to 16 bits, half a step
    `step` of it."""
    second, third = derivative_bounds(act)
    wide = z.abs() + h * q.abs()
    each = h * h / 6 * third * q.abs() ** 3 + (1.13 * sums + 4e-7 * wide) / h + second * step * z.abs() * q.abs()
    return float((dy.abs() * each).sum())
