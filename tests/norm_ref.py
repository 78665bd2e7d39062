"""RMS norm with residual and 8-bit rows, and its gradients, stated plainly in 64 bits.
Each function gives values and the magnitudes that their errors are relative to."""
import torch


def add(x, residual):
    """The row as the residual stream holds it: one fp32 sum, rounded to the rows' type."""
    return x if residual is None else (x.float() + residual.float()).to(x.dtype)


def norm(s, weight, eps):
    s = s.double()
    r = 1 / torch.sqrt((s * s).mean(-1, keepdim=True) + eps)
    return s * r * weight.double()


def scales(y):
    top = y.abs().amax(-1)
    return torch.where(top > 0, top / 448, torch.ones_like(top))


def grads(d_y, s, weight, eps, d_s=None):
    """(d_x, its magnitude, d_weight, its magnitude)"""
    d_y, s, w = d_y.double(), s.double(), weight.double()
    r = 1 / torch.sqrt((s * s).mean(-1, keepdim=True) + eps)
    h, g = s * r, d_y * w
    mean = (g * h).mean(-1, keepdim=True)
    d_x = r * (g - h * mean)
    size = r * (g.abs() + h.abs() * (g * h).abs().mean(-1, keepdim=True))
    if d_s is not None:
        d_x, size = d_x + d_s.double(), size + d_s.double().abs()
    return d_x, size, (d_y * h).sum(0), (d_y * h).abs().sum(0)
