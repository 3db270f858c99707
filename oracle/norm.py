"""Layer norm in float64: the plain definition.

mean = sum x / D, var = sum (x - mean)^2 / D, rstd = 1 / sqrt(var + eps),
h = (x - mean) rstd, y = h w + b (w, b None: ones, zeros);
dx = rstd (u - mean(u) - h mean(u h)) + dresidual with u = dy w,
dw = sum_n dy h, db = sum_n dy.
"""

import numpy as np

from .mlp import as_f64


def _h(x, eps):
    mean = x.mean(axis=1, keepdims=True)
    rstd = 1.0 / np.sqrt(((x - mean) ** 2).mean(axis=1, keepdims=True) + eps)
    return (x - mean) * rstd, mean, rstd


def layernorm(x, w, b, eps):
    h, mean, rstd = _h(as_f64(x), eps)
    y = h * (1.0 if w is None else as_f64(w)) + (0.0 if b is None else as_f64(b))
    return {"y": y, "mean": mean[:, 0], "rstd": rstd[:, 0]}


def layernorm_backward(dy, x, w, eps, dresidual=None):
    dy = as_f64(dy)
    h, _, rstd = _h(as_f64(x), eps)
    u = dy * (1.0 if w is None else as_f64(w))
    dx = rstd * (u - u.mean(axis=1, keepdims=True) - h * (u * h).mean(axis=1, keepdims=True))
    if dresidual is not None:
        dx = dx + as_f64(dresidual)
    return {"dx": dx, "dw": (dy * h).sum(axis=0), "db": dy.sum(axis=0)}
