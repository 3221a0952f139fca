"""Plain float64 form of the layer norm and its gradient, and the bounds on the library's errors (see ffn_ref.py for u,
step and CHAIN).

The mean is a sum of fp32 sums of up to 64 values a thread, joined with their rounding errors: within 2^-18 of the mean
magnitude.  Its error reaches y through rstd gamma; everything else is the fp32 chain of a row."""

import torch

import ffn_ref as R

MEAN = 2.0 ** -18


def layer_norm(x, residual, gamma, beta, eps):
    """s, y, mean, rstd and the bound on y's error before its rounding."""
    s = x.double() + (residual.double() if residual is not None else 0.0)
    mean = s.mean(1)
    d = s - mean[:, None]
    rstd = 1.0 / torch.sqrt((d * d).mean(1) + eps)
    q = d * rstd[:, None] * gamma.double()
    y = q + (beta.double() if beta is not None else 0.0)
    em = MEAN * s.abs().mean(1)
    # rstd's own error from the mean's: (em rstd)^2 / 2 relative
    rel = R.CHAIN + (em * rstd) ** 2
    ey = rel[:, None] * q.abs() + (em * rstd)[:, None] * gamma.double().abs() + 2.0 ** -23 * y.abs()
    return {"s": s, "y": y, "mean": mean, "rstd": rstd, "em": em, "rel": rel, "ey": ey}


def layer_norm_backward(dy, dh, h, gamma, mean, rstd):
    dy, h, gamma, mean, rstd = (t.double() for t in (dy, h, gamma, mean, rstd))
    a, n = dy * gamma, (h - mean[:, None]) * rstd[:, None]
    dx = rstd[:, None] * (a - a.mean(1, keepdim=True) - n * (a * n).mean(1, keepdim=True))
    if dh is not None:
        dx = dx + dh.double()
    return dx, (dy * n).sum(0), dy.sum(0)


def gradient_bounds(dy, h, gamma, mean, rstd, dx):
    """Bounds on dx's error before its rounding, and dgamma's and dbeta's (rows added one after another)."""
    rows = dy.shape[0]
    dy, h, gamma, mean, rstd = (t.double() for t in (dy, h, gamma, mean, rstd))
    a = (dy * gamma).abs()
    n = ((h - mean[:, None]) * rstd[:, None]).abs()
    # h - mean is rounded once, relative to itself
    ex = R.CHAIN * rstd[:, None] * (a + a.mean(1, keepdim=True) + n * (a * n).mean(1, keepdim=True)) + 2.0 ** -23 * dx.abs()
    lim = (rows + 64) * 2.0 ** -24
    return ex, lim * (dy.abs() * n).sum(0) + 1e-30, lim * dy.abs().sum(0) + 1e-30
