"""Plain 64-bit forms of row quantisation and of the 8-bit integer product, and the product's bounds."""
import torch

from tests._train_ref import HALF, TINY, U, act64, gate_err

LEAST = 2.0 ** -126


def codes64(x):
    """(codes int8, scales fp32) of x's rows by the definition.  In 64 bits a quotient of two fp32 values cannot round to
    the middle between two integers unless it lies there: x - (n + 1/2) s is a multiple of s 2^-24 / 2."""
    x = x.detach().cpu().double()
    amax = x.abs().amax(1)
    bad = ~torch.isfinite(x).all(1)
    scale = (amax / 127).float().clamp(min=LEAST)
    q = torch.round(torch.where(bad[:, None], torch.zeros_like(x), x) / scale.double().where(~bad, torch.ones(()).double())[:, None])
    scale[bad] = float("nan")
    return q.to(torch.int8), scale


def q8_64(qx, sx, w, sw, bias, act, residual):
    z = (qx.double() @ w.double().t()) * sx.double()[:, None] * sw.double()
    if bias is not None:
        z = z + bias.double()
    y = act64(act, z)
    return (y if residual is None else y + residual.double()), z


def q8_bound(qx, sx, w, sw, bias, act, residual, y_dtype):
    """Bound of y: the exact sum is rounded once to fp32, each scale's product and the bias's sum once more (first order
    4 u of what they act on, 5 u counted), then the activation as in the fp32 product, the residual's sum and y's type."""
    z0 = ((qx.double() @ w.double().t()) * sx.double()[:, None] * sw.double()).abs()
    ez = 5 * U * (z0 + (0 if bias is None else bias.double().abs()))
    y, z = q8_64(qx, sx, w, sw, bias, act, None)
    if act == "swiglu":
        g, u = z.chunk(2, 1)
        eg, eu = ez.chunk(2, 1)
        s = g * torch.sigmoid(g)  # silu's slope is below 1.1
        ey = 1.1 * eg * (u.abs() + eu) + (s.abs() + 1.1 * eg) * eu + y.abs() * gate_err("silu", g)
    elif act == "none":
        ey = ez
    else:  # GELU's slope is below 1.13
        ey = 1.13 * ez + y.abs() * gate_err(act, z)
    if residual is not None:
        y = y + residual.double()
        ey = ey + 2 * U * (y.abs() + residual.double().abs())
    h = HALF[y_dtype]
    return ey * (1 + h) + h * y.abs() + TINY
