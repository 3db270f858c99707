"""A NaN passes ReLU and its derivative, as it passes the other activations: one in X
reaches its row of the output, one in Z its row of dX and its column of dW and db."""

import pytest
import torch

import tensor_transformer_mlp_columnparallel_gb300 as tp
from tests.test_split_linear_gpu import ACTS, dev, layer

pytestmark = pytest.mark.gpu
NAN = float("nan")


@pytest.fixture(scope="module", autouse=True)
def _built():
    import __graft_entry__
    __graft_entry__.build()
    torch.cuda.set_device(0)
    yield
    assert tp.tpmlp_check_device_error() == 0


@pytest.mark.parametrize("act", ACTS[1:])
@pytest.mark.parametrize("N,dt", [(7, "bf16"), (100, "bf16"), (300, "bf16"), (40, "f32")])
def test_forward(N, dt, act):
    X, W, _, _, bs, _, _ = layer("column", N, 128, 256, 2, dt, 4)
    want, _ = tp.column_linear(X, W, bs, act=act, save_z=True)
    X[3, 5] = NAN
    Y, Z = tp.column_linear(X, W, bs, act=act, save_z=True)
    assert torch.isnan(Z[3]).all() and torch.isnan(Y[3]).all()
    rest = [n for n in range(N) if n != 3]
    assert torch.equal(Y[rest], want[rest])


# dZ by columns and with rows in turn
@pytest.mark.parametrize("act", ACTS[1:])
@pytest.mark.parametrize("N,D,F,dt", [(7, 64, 256, "bf16"), (150, 64, 256, "bf16"), (2600, 64, 8192, "bf16"),
                                      (40, 48, 96, "f32"), (5003, 32, 2040, "f32")])
def test_gradient(N, D, F, dt, act):
    X, W, _, _, _, _, dY = layer("column", N, D, F, 1, dt, 5)
    Z = dY.clone()
    Z[5, 9] = NAN
    dX, dW, db = tp.column_linear_backward(X, W, dY, Z=Z, act=act, bias_grads=True)
    assert torch.isnan(dX[5]).all() and torch.isnan(dW[0][:, 9]).all() and torch.isnan(db[0][9])
    assert torch.isfinite(dX[[0, 4, 6]]).all() and torch.isfinite(dW[0][:, :9]).all() and torch.isfinite(db[0][10:]).all()


@pytest.mark.parametrize("N,dt", [(7, "bf16"), (128, "bf16"), (512, "bf16"), (40, "f32")])
def test_block(N, dt):
    X, W1, _, _, _, _, _ = layer("column", N, 128, 256, 2, dt, 6)
    _, W2, _, _, _, _, dY = layer("row", N, 128, 256, 2, dt, 7)
    _, H, Z = tp.mlp_forward(X, W1, W2, act="relu")
    Z[1][5, 9] = NAN
    dX, dW1, dW2, _, _ = tp.mlp_backward(X, W1, W2, H, Z, dY, act="relu")
    assert torch.isnan(dX[5]).all() and torch.isnan(dW1[1][:, 9]).all()
    assert torch.isfinite(dX[[0, 4, 6]]).all() and torch.isfinite(dW1[0]).all() and torch.isfinite(dW1[1][:, :9]).all()
    X[3, 5] = NAN
    Y, H, _ = tp.mlp_forward(X, W1, W2, act="relu")
    assert torch.isnan(H[0][3]).all() and torch.isnan(Y[3]).all() and torch.isfinite(Y[[0, 2, 4]]).all()
