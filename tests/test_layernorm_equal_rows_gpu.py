"""Layer norm of finite rows whose elements are equal, or equal but for an ulp, far
from zero, up to the type's last value: the variance is 0 (or the ulp's), the output
the bias, whatever the fp32 mean's rounding, and rstd is 1 / sqrt(eps).

Bounds. The mean of equal elements is the element; rstd and y - bias of such rows have
nothing to be rounded but the result. Rows with one element an ulp u away: with
s = steps 2^-24 (the sums' error, see the layer norm's tests), mean off by s |mean| is
taken back to s^2 |mean| by the next look at the row's distances from it; what remains
is the rounding of that correction, 2^-24 s |mean|, as a fraction of the spread, and the
sums over the distances, s."""

import numpy as np
import pytest
import torch

import oracle
import tensor_transformer_mlp_columnparallel_gb300 as tp
from tests.test_layernorm_gpu import EPS, TYPES, U, dev, f64, rows, s_of, vector, within

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    import __graft_entry__
    __graft_entry__.build()
    torch.cuda.set_device(0)
    yield
    assert tp.tpmlp_check_device_error() == 0


VALUES = [1e37, -1e38, 1e6, -1e9, 1e10, 1e20, 3e30, None, -2.0 ** 120]   # None: the last finite one


# rows of a group of lanes, of a CTA, taken in turn (bf16 with fp32 parameters), read three times;
# few rows and many; whole 16-byte accesses and not
@pytest.mark.parametrize("N,D,pad", [(12, 48, 0), (12, 64, 0), (400, 200, 8), (333, 515, 0), (12, 1000, 0), (700, 4096, 0),
                                     (14, 4099, 0), (2600, 8192, 0), (2500, 7992, 8), (12, 12288, 0), (10, 40000, 8), (9, 70001, 0)])
@pytest.mark.parametrize("dt,wdt", [("bf16", "bf16"), ("bf16", "f32"), ("f32", "f32")])
@pytest.mark.parametrize("eps", [EPS, 1e-12])
def test_equal_rows_beside_others(N, D, pad, dt, wdt, eps):
    x, dy = rows(N, D, dt, 1, pad), rows(N, D, dt, 2, pad)
    w, b = vector(D, wdt, 1, 1.0), vector(D, wdt, 2, 0.0)
    want = tp.layernorm(x, w, b, eps=eps)
    at = torch.arange(N)[:: max(1, N // 9)][:len(VALUES)]
    for n, v in zip(at, VALUES):
        x[n] = torch.finfo(TYPES[dt]).max if v is None else v
    y, mean, rstd = tp.layernorm(x, w, b, eps=eps)
    rest = torch.ones(N, dtype=torch.bool)
    rest[at] = False
    rest = rest.to(dev())
    for got, ref in zip((y, mean, rstd), want):
        assert torch.equal(got[rest], ref[rest])
    assert torch.equal(y[at], b.to(y.dtype).expand(len(at), D))
    assert torch.equal(mean[at], x[at, 0].float())
    root = float(np.float32(eps)) ** -0.5   # two roundings from it: the root's, the quotient's
    within(rstd[at], np.full(len(at), root), 2.001 * U * root, "rstd")
    # the gradient: h = 0, dx = rstd (u - mean(u))
    dx, dw, db = tp.layernorm_backward(dy, x, w, mean, rstd)
    u = f64(dy[at]) * f64(w)
    ref = (u - u.mean(1, keepdims=True)) * root
    lim = 4 * s_of(D) * root * np.abs(u).max(1, keepdims=True)
    within(dx[at], ref, lim, "dx")
    none = dy.clone()
    none[at] = 0.0
    assert torch.equal(dw, tp.layernorm_backward(none, x, w, mean, rstd)[1])   # rows with h = 0 add nothing
    assert torch.isfinite(db.float()).all()


@pytest.mark.parametrize("N,D", [(9, 300), (400, 1030), (2600, 8192), (9, 40000)])
@pytest.mark.parametrize("at", [1e10, -1e10, 1e20, 1e37])
def test_one_ulp_in_a_row(N, D, at):
    x, w, b = rows(N, D, "f32", 1), vector(D, "f32", 1, 1.0), vector(D, "f32", 2, 0.0)
    x[3] = at
    x[3, D // 2] = float(np.nextafter(np.float32(at), np.float32(0)))
    y, mean, rstd = tp.layernorm(x, w, b)
    o, s = oracle.norm.layernorm(x[3:4], w, b, EPS), s_of(D)
    off = s * (1 + np.abs(at) * U * o["rstd"])
    h = np.abs((f64(x[3:4]) - o["mean"][:, None]) * o["rstd"][:, None])
    within(rstd[3:4], o["rstd"], 4 * off * o["rstd"], "rstd")
    within(y[3:4], o["y"], 4 * off[:, None] * np.abs(f64(w)) * (1 + h) + 2 * U * np.abs(f64(b)), "y")
    within(mean[3:4], o["mean"], 2 * U * np.abs(o["mean"]), "mean")


def test_equal_rows_without_eps():
    """Nothing to divide by: no finite result, in that row alone."""
    x = rows(4, 4099, "f32", 1)
    want = tp.layernorm(x, eps=0.0)[0]
    x[1], x[2] = 1e10, 1e37
    y, mean, rstd = tp.layernorm(x, eps=0.0)
    assert torch.isnan(y[1:3]).all() and torch.isinf(rstd[1:3]).all()
    assert torch.equal(mean[1:3], x[1:3, 0]) and torch.equal(y[[0, 3]], want[[0, 3]])
