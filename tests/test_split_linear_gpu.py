"""Column- and row-split linear layers on the GPU against the float64 definition.

Tolerances, element by element. fp32: K products added one after the other are off
by K 2^-24 of the sum of magnitudes S = |X||W|. bf16: the tensor core adds 16
products at a time, (K / 16 + 2) 2^-23 S; an output is rounded once, 2^-8 of itself;
an activation's slope is at most 1.13, its form in the epilogue off by 2^-20 and
2e-6. A gradient made from a rounded dZ (bf16, with an activation, more than 64
tokens for dW, 16 for dX) is off by 2^-8 of |dZ||W| (|X||dZ|) too, with fewer tokens
by 2^-16 of it, and by the slope's error (2^-18 of |dY| + 4e-6)."""

import numpy as np
import pytest
import torch

import oracle
import tensor_transformer_mlp_columnparallel_gb300 as tp
from tensor_transformer_mlp_columnparallel_gb300 import _binding

pytestmark = pytest.mark.gpu
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
ACTS = [None, "relu", "gelu_tanh", "gelu_erf", "gelu_sigmoid"]


@pytest.fixture(scope="module", autouse=True)
def _built():
    import __graft_entry__
    __graft_entry__.build()
    torch.cuda.set_device(0)
    yield
    assert tp.tpmlp_check_device_error() == 0


def dev():
    return torch.device("cuda:0")


def f64(t):
    return t.double().cpu().numpy()


def matrix(g, N, C, dt, pad=0, std=1.0, whole=None):
    """[N, C] in rows of C + pad; whole: sparse numbers in {-1, 0, 1} instead."""
    z = torch.full((N, C + pad), 1000.0)
    r = torch.randn(N, C, generator=g)
    z[:, :C] = r * std if whole is None else (r.sign() * (torch.rand(N, C, generator=g) < whole))
    return z.to(TYPES[dt]).to(dev())[:, :C]


def within(got, ref, tol, what):
    g = f64(got)
    if got.dtype == torch.bfloat16:
        tol = tol + 2.0 ** -8 * np.abs(ref)
    assert g.shape == ref.shape, what
    bad = np.abs(g - ref) - tol
    assert not np.isnan(bad).any() and bad.max(initial=-1.0) <= 0, f"{what}: over by {np.nanmax(bad):.2e}"


def acc(K, dt):
    return K * 2.0 ** -24 if dt == "f32" else (K / 16 + 2) * 2.0 ** -23


def layer(split, N, D, F, T, dt, seed, pad=0, whole=None):
    """X, W shards, the whole W, bias (shards or not), residual, dY."""
    g = torch.Generator().manual_seed(seed)
    column = split == "column"
    n_in, n_out = (D, F) if column else (F, D)
    X = matrix(g, N, n_in, dt, pad, whole=whole)
    W = [matrix(g, *((D, F // T) if column else (F // T, D)), dt, 0, 0.05, whole) for _ in range(T)]
    b = matrix(g, 1, n_out, dt, 0, 1.0, whole)[0].contiguous()
    R, dY = matrix(g, N, n_out, dt, pad, whole=whole), matrix(g, N, n_out, dt, pad, whole=whole)
    full = torch.cat(W, dim=1 if column else 0)
    return X, W, full, b, ([x.clone() for x in b.chunk(T)] if column else b), R, dY


def forward(split, X, W, b, act=None, R=None, save_z=False):
    if split == "row":
        return tp.row_linear(X, W, b, residual=R), None
    return tp.column_linear(X, W, b, act=act, residual=R, save_z=save_z)


def check_forward(split, N, D, F, T, dt, act=None, pad=0, seed=0):
    X, W, full, b, bs, R, _ = layer(split, N, D, F, T, dt, seed, pad)
    S = np.abs(f64(X)) @ np.abs(f64(full))
    lim = acc(X.shape[1], dt) * S + 2.0 ** -22 * np.abs(f64(b))
    for bias, res in ((True, True), (False, False), (True, False), (False, True)):
        o = oracle.linear.forward(X, full, b if bias else None, act, R if res else None)
        save = act is not None and bias
        Y, Z = forward(split, X, W, bs if bias else None, act, R if res else None, save)
        extra = (1.13 - 1) * lim + 2.0 ** -20 * np.abs(o["Z"]) + 3e-6 if act else 0.0
        within(Y, o["Y"], lim + extra + 2.0 ** -22 * np.abs(f64(R)), f"Y {bias} {res}")
        if save:
            within(Z, o["Z"], lim, "Z")
        else:
            assert Z is None


def check_backward(split, N, D, F, T, dt, act=None, pad=0, seed=0, bias=True):
    X, W, full, _, _, _, dY = layer(split, N, D, F, T, dt, seed, pad)
    Z = None
    if act:
        g = torch.Generator().manual_seed(seed + 9)
        Z = matrix(g, N, F, dt, pad, 1.5)
    if split == "row":
        dX, dW, db = tp.row_linear_backward(X, W, dY, bias_grads=bias)
    else:
        dX, dW, db = tp.column_linear_backward(X, W, dY, Z=Z, act=act, bias_grads=bias)
    o = oracle.linear.backward(X, full, dY, Z, act)
    a = np.abs(f64(dY))
    if act:
        a = a * np.abs(oracle.mlp.act_grad(f64(Z), act))
    slope = np.abs(f64(dY)) * 2.0 ** -18 + 4e-6 * np.abs(f64(dY)) if act else 0.0 * a
    u = lambda few: (0.0 if not act or dt == "f32" else 2.0 ** -16 if N <= few else 2.0 ** -8)
    Wa, Xa = np.abs(f64(full)), np.abs(f64(X))
    within(dX, o["dX"], (acc(a.shape[1], dt) + u(16)) * (a @ Wa.T) + slope @ Wa.T, "dX")
    got = torch.cat(dW, dim=1 if split == "column" else 0)
    within(got, o["dW"], (acc(N, dt) + u(64)) * (Xa.T @ a) + Xa.T @ slope, "dW")
    if bias:
        got = torch.cat(db) if split == "column" else db
        within(got, o["db"], (N / 8 + 64) * 2.0 ** -24 * a.sum(0) + slope.sum(0), "db")
    else:
        assert db is None


BF16 = [(1, 8, 8, 1), (1, 64, 256, 2), (3, 72, 40, 5), (5, 256, 512, 4), (16, 264, 1040, 2), (17, 512, 128, 1),
        (33, 128, 2048, 8), (64, 520, 768, 3), (65, 256, 256, 2), (129, 1024, 512, 4), (200, 136, 264, 3),
        (400, 512, 1024, 2), (769, 264, 520, 1), (1030, 512, 4096, 16)]


@pytest.mark.parametrize("split", ["column", "row"])
@pytest.mark.parametrize("N,D,F,T", BF16)
def test_bf16_shapes(split, N, D, F, T):
    act = ACTS[(N + T) % 5] if split == "column" else None
    pad = 8 * (N % 3)
    check_forward(split, N, D, F, T, "bf16", act, pad, seed=N)
    check_backward(split, N, D, F, T, "bf16", act, pad, seed=N + 1, bias=N % 2 == 1)


@pytest.mark.parametrize("split", ["column", "row"])
@pytest.mark.parametrize("N,D,F,T", [(1, 1, 1, 1), (2, 3, 5, 5), (7, 33, 66, 2), (64, 256, 1024, 2), (65, 30, 21, 3),
                                     (130, 128, 96, 4)])
def test_f32_shapes(split, N, D, F, T):
    act = ACTS[(N + T + 1) % 5] if split == "column" else None
    check_forward(split, N, D, F, T, "f32", act, N % 4, seed=N)
    check_backward(split, N, D, F, T, "f32", act, N % 4, seed=N + 1)


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("N", [8, 150])
def test_every_activation(N, act, dt):
    check_forward("column", N, 128, 192, 3, dt, act, seed=5)
    check_backward("column", N, 128, 192, 3, dt, act, seed=6)


# dZ with rows in turn: panels of every group width, whole and not, in one panel and several
@pytest.mark.parametrize("dt,N,D,F,T", [("bf16", 2600, 64, 8192, 1), ("bf16", 2300, 64, 16384, 4),
                                        ("bf16", 4999, 64, 4096, 2), ("bf16", 10007, 64, 1992, 3),
                                        ("bf16", 1501, 64, 24568, 1), ("f32", 5003, 32, 2040, 2),
                                        ("f32", 20011, 16, 1000, 2)])
def test_many_tokens_with_activation(dt, N, D, F, T):
    check_backward("column", N, D, F, T, dt, "gelu_tanh", seed=3)


# every launch form adds the residual: whole numbers, so the bits are the definition's
@pytest.mark.parametrize("split", ["column", "row"])
@pytest.mark.parametrize("N,D,F,T", [(1, 128, 2048, 4), (4, 2048, 256, 2), (16, 512, 4096, 8), (40, 1024, 1024, 1),
                                     (64, 4096, 512, 2), (70, 256, 1536, 2), (128, 512, 512, 4), (130, 384, 640, 1),
                                     (300, 1024, 2048, 2), (513, 264, 4104, 3), (1200, 2048, 2048, 4)])
def test_whole_numbers_bit_for_bit(split, N, D, F, T):
    K = D if split == "column" else F
    X, W, full, b, bs, R, dY = layer(split, N, D, F, T, "bf16", N + D, pad=8, whole=min(0.3, 9 / K ** 0.5))
    o = oracle.linear.forward(X, full, b, "relu" if split == "column" else None, R)
    assert np.abs(o["Z"]).max() <= 255
    Y, Z = forward(split, X, W, bs, "relu" if split == "column" else None, R, split == "column")
    assert np.array_equal(f64(Y), o["Y"])
    if Z is not None:
        assert np.array_equal(f64(Z), o["Z"])
        Y2, _ = forward(split, X, W, bs, "relu", R)
        assert torch.equal(Y, Y2)
    # without the scratch, in place onto the residual
    buf = torch.zeros(N, Y.shape[1] + 16, dtype=torch.bfloat16, device=dev())
    into = buf[:, :Y.shape[1]]
    into.copy_(R)
    if split == "column":
        tp.tpmlp_column_linear(X, W, bs, "relu", into, into, None)
    else:
        tp.tpmlp_row_linear(X, W, bs, into, into)
    assert torch.equal(into, Y) and not buf[:, Y.shape[1]:].any()
    g = oracle.linear.backward(X, full, dY)
    if np.abs(g["dX"]).max() <= 256 and np.abs(g["dW"]).max() <= 256:
        call = tp.row_linear_backward if split == "row" else tp.column_linear_backward
        dX, dW, _ = call(X, W, dY)
        assert np.array_equal(f64(dX), g["dX"])
        assert np.array_equal(f64(torch.cat(dW, dim=1 if split == "column" else 0)), g["dW"])


def test_matches_the_block():
    """Up, then down onto nothing: the block of the same weights."""
    N, D, F, T = 150, 256, 512, 4
    X, W1, _, _, b1, _, _ = layer("column", N, D, F, T, "bf16", 1)
    _, W2, _, b2, _, _, _ = layer("row", N, D, F, T, "bf16", 2)
    Y, H, Z = tp.mlp_forward(X, W1, W2, b1, b2, act="gelu_tanh")
    h, z = tp.column_linear(X, W1, b1, act="gelu_tanh", save_z=True)
    assert torch.equal(h, torch.cat(H, 1)) and torch.equal(z, torch.cat(Z, 1))
    assert torch.equal(tp.row_linear(h, W2, b2), Y)


def test_empty_batch():
    X, W, _, _, bs, R, dY = layer("column", 0, 64, 128, 2, "bf16", 1)
    Y, Z = tp.column_linear(X, W, bs, act="relu", residual=R, save_z=True)
    assert Y.shape == Z.shape == (0, 128)
    dX, dW, db = tp.column_linear_backward(X, W, dY, Z=Z, act="relu", bias_grads=True)
    assert dX.shape == (0, 64) and not any(t.any() for t in dW + db)
    X, W, _, _, b, R, dY = layer("row", 0, 64, 128, 2, "f32", 1)
    assert tp.row_linear(X, W, b, residual=R).shape == (0, 64)
    dX, dW, db = tp.row_linear_backward(X, W, dY, bias_grads=True)
    assert dX.shape == (0, 128) and not db.any() and not any(t.any() for t in dW)


@pytest.mark.parametrize("N", [7, 300])
def test_repeat_other_stream_and_graph(N):
    X, W, _, _, bs, R, dY = layer("column", N, 256, 512, 4, "bf16", 3)
    def step():
        Y, Z = tp.column_linear(X, W, bs, act="gelu_erf", residual=R, save_z=True)
        dX, dW, db = tp.column_linear_backward(X, W, dY, Z=Z, act="gelu_erf", bias_grads=True)
        return [Y, Z, dX, *dW, *db]
    want = step()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        got = step()
    s.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        held = step()
    for t in held:
        t.zero_()
    g.replay()
    g.replay()
    torch.cuda.synchronize()
    for a, b, c in zip(want, got, held):
        assert torch.equal(a, b) and torch.equal(a, c)


def test_nan_stays_in_its_row():
    X, W, _, _, bs, R, _ = layer("column", 40, 128, 256, 2, "bf16", 4)
    Y, _ = tp.column_linear(X, W, bs, residual=R)
    X[3, 5], R[7, 200] = float("nan"), float("inf")
    Y2, _ = tp.column_linear(X, W, bs, residual=R)
    assert torch.isnan(Y2[3]).all() and torch.isinf(Y2[7, 200])
    rest = [n for n in range(40) if n not in (3, 7)]
    assert torch.equal(Y[rest], Y2[rest]) and torch.equal(Y[7, :200], Y2[7, :200])


def test_refusals_on_the_device():
    X, W, _, _, bs, R, dY = layer("column", 4, 64, 128, 2, "bf16", 1)
    with pytest.raises(KeyError):
        tp.column_linear(X, W, act="tanh")
    with pytest.raises(tp.TpmlpError):
        tp.column_linear(X, W, save_z=True)                 # Z is of no use without an activation
    with pytest.raises(ValueError):
        tp.column_linear(X, W[:1], bs)
    with pytest.raises(ValueError):
        tp.column_linear(X, W, residual=R[:, :64])
    with pytest.raises(ValueError):
        tp.row_linear(X, W)
    with pytest.raises(TypeError):
        tp.column_linear(X, W, residual=R.float())
    with pytest.raises(tp.TpmlpError) as e:
        tp.column_linear_backward(X, W, dY, act="relu")     # no Z
    assert e.value.status == _binding.ERR_ARG
    with pytest.raises(tp.TpmlpError) as e:
        tp.column_linear_backward(X, W, dY, Z=dY, act="relu", workspace=torch.empty(64, dtype=torch.uint8, device=dev()))
    assert e.value.status == _binding.ERR_WORKSPACE
    with pytest.raises(tp.TpmlpError) as e:
        tp.column_linear(X, [w[:, :60].contiguous() for w in W])
    assert e.value.status == _binding.ERR_ALIGN
