"""dZ of a column layer with rows in turn (many tokens): every activation, pitches of
dY and Z that differ, panels that do not come out even. Bounds as in the split linear
layers' tests."""

import numpy as np
import pytest
import torch

import oracle
import tensor_transformer_mlp_columnparallel_gb300 as tp
from tests.test_split_linear_gpu import ACTS, acc, dev, f64, layer, matrix, within

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    import __graft_entry__
    __graft_entry__.build()
    torch.cuda.set_device(0)
    yield
    assert tp.tpmlp_check_device_error() == 0


@pytest.mark.parametrize("act", ACTS[1:])
@pytest.mark.parametrize("dt,N,D,F,T,pads", [("bf16", 2600, 64, 8192, 1, (0, 0)), ("f32", 5003, 32, 2040, 2, (0, 0)),
                                             ("bf16", 1501, 64, 24568, 1, (8, 24)), ("bf16", 5000, 64, 2056, 1, (0, 40)),
                                             ("f32", 1300, 16, 8200, 2, (12, 0))])
def test_every_activation(dt, N, D, F, T, pads, act):
    X, W, full, _, _, _, _ = layer("column", N, D, F, T, dt, 3)
    g = torch.Generator().manual_seed(8)
    dY, Z = matrix(g, N, F, dt, pads[0]), matrix(g, N, F, dt, pads[1], 1.5)
    assert N * F >= 8 * 152 * 8192
    dX, dW, db = tp.column_linear_backward(X, W, dY, Z=Z, act=act, bias_grads=True)
    o = oracle.linear.backward(X, full, dY, Z, act)
    a = np.abs(f64(dY) * oracle.mlp.act_grad(f64(Z), act))
    slope = np.abs(f64(dY)) * (2.0 ** -18 + 4e-6)
    u = 0.0 if dt == "f32" else 2.0 ** -8
    Wa, Xa = np.abs(f64(full)), np.abs(f64(X))
    within(dX, o["dX"], (acc(F, dt) + u) * (a @ Wa.T) + slope @ Wa.T, "dX")
    within(torch.cat(dW, 1), o["dW"], (acc(N, dt) + u) * (Xa.T @ a) + Xa.T @ slope, "dW")
    within(torch.cat(db), o["db"], (N / 8 + 64) * 2.0 ** -24 * a.sum(0) + slope.sum(0), "db")
