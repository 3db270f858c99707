"""Activations of pre-activations far from zero, down to and up to the type's
last finite value, in every kernel form that applies one.

Bounds. Below -9.7 (tanh form) and -47 (sigmoid form) act and act' are below 1e-33
whatever z is, beyond the same numbers above act' is 1: a kernel may hold z there.
Where the definition gives less than 1e-30, so must the kernel; elsewhere act is off
by 2^-20 of z and 3e-6, act' by 2^-18 and 4e-6, and a bf16 output by 2^-8 of itself.
The gradients' bounds are those of the split linear layers' tests."""

import numpy as np
import pytest
import torch

import oracle
import tensor_transformer_mlp_columnparallel_gb300 as tp
from tests.test_split_linear_gpu import TYPES, acc, dev, f64, layer, within

pytestmark = [pytest.mark.gpu, pytest.mark.filterwarnings("ignore:overflow encountered")]
ACTS = ["relu", "gelu_erf", "gelu_sigmoid", "gelu_tanh"]


@pytest.fixture(scope="module", autouse=True)
def _built():
    import __graft_entry__
    __graft_entry__.build()
    torch.cuda.set_device(0)
    yield
    assert tp.tpmlp_check_device_error() == 0


def far(dt):
    f = torch.finfo(TYPES[dt])
    near = [0.0, -0.5, 0.75, -1.5, 2.0, -3.0, 4.0, -6.0, -9.5, 9.5, -9.75, 9.75, -12.0, -46.0, 46.0, -48.0, 48.0]
    wide = [100.0, 3600.0, 3616.0, 4000.0, 1e5, 1e11, 1e12, 1.5e13, 2e13, 1e18, 2e19, 1e25, 1e30, 1e36, 1.5e38, 2.5e38]
    z = near + wide + [-v for v in wide] + [f.min, f.max]
    return torch.tensor(z, dtype=torch.float64).to(TYPES[dt])


def spread_over(N, F, dt, seed):
    """[N, F] of the values above, every one beside every other."""
    z = far(dt)
    return z[torch.randint(0, len(z), (N, F), generator=torch.Generator().manual_seed(seed))]


def act_of(z, act):
    return oracle.mlp.act(f64(z), act)


def slope_of(z, act):
    return oracle.mlp.act_grad(f64(z), act)


def with_limits(z, act, f):
    """f(z, act), at infinities its limits: of the numbers 1e30 on their side (for act
    above zero, infinity)."""
    held = z.double().clamp(-1e30, 1e30)
    out = f(held, act)
    return np.where(f64(z) == np.inf, np.inf, out) if f is act_of else out


def close(got, ref, lim, what):
    tiny = np.abs(ref) < 1e-30
    within(got, np.where(tiny, 0.0, ref), np.where(tiny, 1e-30, lim), what)


# the few-token launch, single-CTA tiles, staged pair tiles; CUDA cores
@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("N,D,F,T,dt", [(7, 64, 256, 2, "bf16"), (100, 64, 256, 2, "bf16"), (300, 128, 512, 2, "bf16"),
                                        (40, 48, 96, 2, "f32")])
def test_layer(N, D, F, T, dt, act):
    X = torch.zeros(N, D, dtype=TYPES[dt], device=dev())
    W = [torch.ones(D, F // T, dtype=TYPES[dt], device=dev()) for _ in range(T)]
    z = spread_over(1, F, dt, 1)[0]
    Y, Z = tp.column_linear(X, W, [b.clone().to(dev()) for b in z.chunk(T)], act=act, save_z=True)
    assert torch.equal(Z, z.to(dev()).expand(N, F))
    ref = np.broadcast_to(act_of(z, act), (N, F))
    close(Y, ref, 2.0 ** -20 * np.abs(f64(z)) + 3e-6, f"{act}(z)")


# dZ by columns (both parts of few tokens, and one), with rows in turn
@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("N,D,F,T,dt", [(7, 64, 256, 2, "bf16"), (40, 64, 256, 2, "bf16"), (150, 64, 192, 3, "bf16"),
                                        (2600, 64, 8192, 1, "bf16"), (40, 48, 95, 1, "f32"), (5003, 32, 2040, 2, "f32")])
def test_layer_gradient(N, D, F, T, dt, act):
    X, W, full, _, _, _, dY = layer("column", N, D, F, T, dt, 5)
    Z = spread_over(N, F, dt, 6)
    dX, dW, db = tp.column_linear_backward(X, W, dY, Z=Z.to(dev()), act=act, bias_grads=True)
    s = slope_of(Z, act)
    dZ, a = f64(dY) * s, np.abs(f64(dY) * s)
    slope = np.abs(f64(dY)) * (2.0 ** -18 + 4e-6)
    u = lambda few: (0.0 if dt == "f32" else 2.0 ** -16 if N <= few else 2.0 ** -8)
    Wa, Xa = np.abs(f64(full)), np.abs(f64(X))
    within(dX, dZ @ f64(full).T, (acc(F, dt) + u(16)) * (a @ Wa.T) + slope @ Wa.T, "dX")
    within(torch.cat(dW, 1), f64(X).T @ dZ, (acc(N, dt) + u(64)) * (Xa.T @ a) + Xa.T @ slope, "dW")
    within(torch.cat(db), dZ.sum(0), (N / 8 + 64) * 2.0 ** -24 * a.sum(0) + slope.sum(0), "db")


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("mode", ["splitk", "partials"])
@pytest.mark.parametrize("N,T,dt", [(16, 2, "bf16"), (128, 2, "bf16"), (512, 4, "bf16"), (40, 2, "f32")])
def test_block(N, T, dt, mode, act):
    """X = I, so Z = W1; W2 = 0 but for a column of ones, dY = e_0, so dZ = act'(Z)
    and dW1 = dZ."""
    st, F = TYPES[dt], 256
    X, W1 = torch.eye(N, dtype=st, device=dev()), spread_over(N, F, dt, 7)
    W2, dY = torch.zeros(F, N, dtype=st, device=dev()), torch.zeros(N, N, dtype=st, device=dev())
    W2[:, 0], dY[:, 0] = 1.0, 1.0
    shards = [w.contiguous().to(dev()) for w in W1.chunk(T, dim=1)], [w.contiguous() for w in W2.chunk(T, dim=0)]
    _, H, Z = tp.mlp_forward(X, *shards, act=act, mode=mode)
    assert torch.equal(torch.cat(Z, 1), W1.to(dev()))
    close(torch.cat(H, 1), act_of(W1, act), 2.0 ** -20 * np.abs(f64(W1)) + 3e-6, f"{act}(z)")
    _, dW1, _, _, _ = tp.mlp_backward(X, *shards, H, Z, dY, act=act, mode=mode)
    close(torch.cat(dW1, 1), slope_of(W1, act), 2.0 ** -18 + 4e-6, f"{act}'(z)")


INF = float("inf")


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("N,D,F,T,dt", [(7, 64, 256, 2, "bf16"), (100, 64, 256, 2, "bf16"), (300, 128, 512, 2, "bf16"),
                                        (40, 48, 96, 2, "f32")])
def test_layer_infinities(N, D, F, T, dt, act):
    """A unit that its bias masks: 0, and no gradient; the limits on the other side."""
    X = torch.zeros(N, D, dtype=TYPES[dt], device=dev())
    W = [torch.ones(D, F // T, dtype=TYPES[dt], device=dev()) for _ in range(T)]
    z = torch.tensor([-INF, 1.0, INF, -2.0], dtype=TYPES[dt]).repeat(F // 4)
    Y, Z = tp.column_linear(X, W, [b.clone().to(dev()) for b in z.chunk(T)], act=act, save_z=True)
    assert torch.equal(Z, z.to(dev()).expand(N, F)) and (Y[:, 2::4] == INF).all()
    rest = [f for f in range(F) if f % 4 != 2]
    close(Y[:, rest], np.broadcast_to(with_limits(z, act, act_of)[rest], (N, len(rest))), 2.0 ** -18 + 3e-6, f"{act}(z)")
    _, W, full, _, _, _, dY = layer("column", N, D, F, T, dt, 5)
    X = dY[:, :D].contiguous()
    dX, dW, db = tp.column_linear_backward(X, W, dY, Z=Z, act=act, bias_grads=True)
    s = with_limits(z, act, slope_of)
    dZ, a = f64(dY) * s, np.abs(f64(dY) * s)
    slope = np.abs(f64(dY)) * (2.0 ** -18 + 4e-6)
    u = 0.0 if dt == "f32" else 2.0 ** -8
    Wa, Xa = np.abs(f64(full)), np.abs(f64(X))
    within(dX, dZ @ f64(full).T, (acc(F, dt) + u) * (a @ Wa.T) + slope @ Wa.T, "dX")
    within(torch.cat(dW, 1), f64(X).T @ dZ, (acc(N, dt) + u) * (Xa.T @ a) + Xa.T @ slope, "dW")
    within(torch.cat(db), dZ.sum(0), (N / 8 + 64) * 2.0 ** -24 * a.sum(0) + slope.sum(0), "db")


@pytest.mark.parametrize("N,dt", [(7, "bf16"), (300, "bf16"), (40, "f32")])
def test_block_and_gated_block_infinities(N, dt):
    st, F = TYPES[dt], 64
    z = torch.tensor([-INF, 1.0, 0.5, -2.0], dtype=st).repeat(F // 4)
    X, W1, W2 = (torch.zeros(r, c, dtype=st, device=dev()) for r, c in ((N, 64), (64, F), (F, 64)))
    dY = torch.ones(N, 64, dtype=st, device=dev())
    W2[:, 0] = 1.0
    for act in ACTS:
        _, H, Z = tp.mlp_forward(X, [W1], [W2], [z.to(dev())], None, act=act)
        close(H[0], np.broadcast_to(with_limits(z, act, act_of), (N, F)), 2.0 ** -18 + 3e-6, f"{act}(z)")
        _, _, _, db1, _ = tp.mlp_backward(X, [W1], [W2], H, Z, dY, act=act, bias_grads=True)
        close(db1[0], N * with_limits(z, act, slope_of), N * (2.0 ** -18 + 4e-6 + u_of(dt)), f"{act}'(z)")
    X[:, 0], W1[0] = 1.0, z.to(dev())
    W1[1:] = 0.0
    U = torch.full((64, F), 0.25, dtype=st, device=dev())
    X[:, 1:] = 0.0
    _, H, G, _ = tp.swiglu_forward(X, [W1], [U], [W2], save_gate_up=True)
    assert torch.equal(G[0], z.to(dev()).expand(N, F))
    held = z.double().clamp(-1e30, 1e30).numpy()
    close(H[0], np.broadcast_to(0.25 * oracle.mlp.silu(held), (N, F)), 2.0 ** -20, "H")


def u_of(dt):   # dZ rounded before its columns are added
    return 0.0 if dt == "f32" else 2.0 ** -8
