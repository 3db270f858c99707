"""Split linear layers on matrices whose rows lie so far apart that element offsets
pass 32 bits, and two calls at once on two streams: the bits of the same calls on
close rows with the same scratch, one after the other."""

import pytest
import torch

import tensor_transformer_mlp_columnparallel_gb300 as tp
from tensor_transformer_mlp_columnparallel_gb300 import _binding
from tests.test_split_linear_gpu import TYPES, dev, layer

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    import __graft_entry__
    __graft_entry__.build()
    torch.cuda.set_device(0)
    yield
    assert tp.tpmlp_check_device_error() == 0
    torch.cuda.empty_cache()


@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_rows_beyond_32_bit_offsets(dt):
    N, D, F, T, pitch = 2200, 64, 128, 2, 1 << 20
    def apart(t):
        far = torch.empty((N - 1) * pitch + t.shape[1], dtype=TYPES[dt], device=dev()).as_strided(t.shape, (pitch, 1))
        far.copy_(t)
        return far
    def scratch(op):   # as the calls of the package take it
        n = tp.tpmlp_workspace_bytes_balanced(op, TYPES[dt], N, D, F, T, "splitk")
        return torch.empty(n, dtype=torch.uint8, device=dev()) if n else None
    X, W, _, _, bs, R, dY = layer("column", N, D, F, T, dt, 1)
    Y, Z = tp.column_linear(X, W, bs, act="gelu_tanh", residual=R, save_z=True)
    fX, fR, fY, fZ = apart(X), apart(R), apart(torch.zeros_like(Y)), apart(torch.zeros_like(Z))
    tp.tpmlp_column_linear(fX, W, bs, "gelu_tanh", fR, fY, fZ, scratch(_binding.OP_LINEAR))
    assert torch.equal(fY, Y) and torch.equal(fZ, Z)
    dX, dW, db = tp.column_linear_backward(X, W, dY, Z=Z, act="gelu_tanh", bias_grads=True)
    fY.copy_(dY)
    del fR
    gX, gW, gb = tp.column_linear_backward(fX, W, fY, Z=fZ, act="gelu_tanh", bias_grads=True)
    for a, b in zip([dX, *dW, *db], [gX, *gW, *gb]):
        assert torch.equal(a, b)
    del fX, fY, fZ
    X, W, _, _, b, R, dY = layer("row", N, D, F, T, dt, 2)
    Y = tp.row_linear(X, W, b, residual=R)
    fX, fY = apart(X), apart(R)
    tp.tpmlp_row_linear(fX, W, b, fY, fY, scratch(_binding.OP_LINEAR))   # in place onto the residual
    assert torch.equal(fY, Y)
    dX, dW, db = tp.row_linear_backward(X, W, dY, bias_grads=True)
    fY.copy_(dY)
    far = apart(torch.zeros_like(dX))
    gW, gb = [torch.empty_like(w) for w in dW], torch.empty_like(db)
    tp.tpmlp_row_linear_backward(fX, W, fY, far, gW, gb, scratch(_binding.OP_LINEAR_BACKWARD))
    for p, q in zip([dX, *dW, db], [far, *gW, gb]):
        assert torch.equal(p, q)


@pytest.mark.parametrize("N", [7, 300])
def test_two_calls_at_once(N):
    X, W, _, _, bs, R, dY = layer("column", N, 256, 512, 4, "bf16", 3)
    def step(k):
        Y, Z = tp.column_linear(X, W, bs, act="gelu_sigmoid", residual=R, save_z=True)
        dX, dW, db = tp.column_linear_backward(X, W, dY, Z=Z, act="gelu_sigmoid", bias_grads=True)
        y, mean, rstd = tp.layernorm(Y)
        return [Y, Z, dX, *dW, *db, y, *tp.layernorm_backward(dY, Y, None, mean, rstd)]
    want = step(0)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = [[], []]
    for _ in range(8):
        for k, s in enumerate(streams):
            with torch.cuda.stream(s):
                got[k].append(step(k))
    torch.cuda.synchronize()
    for run in got[0] + got[1]:
        for a, b in zip(want, run):
            assert torch.equal(a, b)
