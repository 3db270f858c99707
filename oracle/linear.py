"""One linear layer in float64, unsharded: Z = X W + b, Y = act(Z) + R, and its
gradients dZ = dY act'(Z), dX = dZ W^T, dW = X^T dZ, db = sum_n dZ (the residual's
is dY). act None: act(z) = z."""

import numpy as np

from .mlp import act as activation, act_grad, as_f64


def forward(X, W, b=None, act=None, R=None):
    Z = as_f64(X) @ as_f64(W)
    if b is not None:
        Z = Z + as_f64(b)
    Y = activation(Z, act) if act else Z
    if R is not None:
        Y = Y + as_f64(R)
    return {"Z": Z, "Y": Y}


def backward(X, W, dY, Z=None, act=None):
    dZ = as_f64(dY)
    if act:
        dZ = dZ * act_grad(as_f64(Z), act)
    return {"dX": dZ @ as_f64(W).T, "dW": as_f64(X).T @ dZ, "db": np.sum(dZ, axis=0)}
