"""Layer norm and its gradients on the GPU against the float64 definition.

Tolerances, element by element. A sum of D fp32 numbers is taken by threads of at
most `steps` additions in a row (64, or D / 1024, and a dozen that join them), so
it is off by steps 2^-24 of the sum of magnitudes; a mean of such a row's m by
that of mean|x|, which a far row's d takes back. With s = steps 2^-24:
  rstd         s of itself
  h            s (1 + |h|)  (and 2^-22 where a gradient takes h from a rounded mean)
  y            s |w| (1 + |h|) + 2^-23 |b|
  dx           4 s rstd (1 + max|h|)^2 max|u| + 2^-23 |dresidual|
  dw, db       (N / 152 + 64) 2^-24 sum_n |dy| (1 + |h|): the rows of one thread, then
               the CTAs' sums; and h's own error
A bf16 output is rounded once more: 2^-8 of itself."""

import time

import numpy as np
import pytest
import torch

import oracle
import tensor_transformer_mlp_columnparallel_gb300 as tp
from tensor_transformer_mlp_columnparallel_gb300 import _binding

pytestmark = pytest.mark.gpu
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
EPS = 1e-5
U = 2.0 ** -24


@pytest.fixture(scope="module", autouse=True)
def _built():
    import __graft_entry__
    __graft_entry__.build()
    torch.cuda.set_device(0)
    yield
    assert tp.tpmlp_check_device_error() == 0


def dev():
    return torch.device("cuda:0")


def rows(N, D, dt, seed, pad=0, std=1.0, offset=0.0, fill=1000.0):
    g = torch.Generator().manual_seed(seed)
    z = torch.full((N, D + pad), fill, dtype=TYPES[dt])
    z[:, :D] = (torch.randn(N, D, generator=g) * std + offset).to(TYPES[dt])
    return z.to(dev())[:, :D]


def vector(D, dt, seed, base):
    g = torch.Generator().manual_seed(seed)
    return (base + 0.2 * torch.randn(D, generator=g)).to(TYPES[dt]).to(dev())


def f64(t):
    return None if t is None else t.double().cpu().numpy()


def within(got, ref, tol, what):
    g = f64(got)
    if got.dtype == torch.bfloat16:
        tol = tol + 2.0 ** -8 * np.abs(ref)
    assert g.shape == ref.shape, what
    bad = np.abs(g - ref) - tol
    assert not np.isnan(bad).any() and bad.max(initial=-1.0) <= 0, f"{what}: over by {np.nanmax(bad):.2e}"


def s_of(D):
    return (max(64, D / 1024) + 16) * U


def check_forward(x, w, b, eps=EPS):
    keep = x.clone()
    y, mean, rstd = tp.layernorm(x, w, b, eps=eps)
    assert torch.equal(x, keep)
    o, s = oracle.norm.layernorm(x, w, b, eps), s_of(x.shape[1])
    h = np.abs((f64(x) - o["mean"][:, None]) * o["rstd"][:, None])
    wn, bn = np.abs(1.0 if w is None else f64(w)), np.abs(0.0 if b is None else f64(b))
    within(rstd, o["rstd"], 2 * s * o["rstd"], "rstd")
    spread = np.sqrt(np.mean(f64(x) ** 2, axis=1))
    within(mean, o["mean"], np.minimum(s * spread, s / o["rstd"]) + 2 * U * np.abs(o["mean"]), "mean")
    within(y, o["y"], 2 * s * wn * (1 + h) + 2 * U * bn, "y")
    return y, mean, rstd


def check_backward(x, w, dy, res=None, params=True, eps=EPS):
    _, mean, rstd = tp.layernorm(x, w, None, eps=eps)
    dx, dw, db = tp.layernorm_backward(dy, x, w, mean, rstd, dresidual=res, param_grads=params)
    o, (N, D) = oracle.norm.layernorm_backward(dy, x, w, eps, res), x.shape
    f = oracle.norm.layernorm(x, None, None, eps)
    h, s = np.abs(f["y"]), s_of(D) + 2.0 ** -22
    u = np.abs(f64(dy) * (1.0 if w is None else f64(w)))
    lim = 4 * s * f["rstd"][:, None] * (1 + h.max(1, initial=0.0, keepdims=True)) ** 2 * u.max(1, initial=0.0, keepdims=True)
    within(dx, o["dx"], lim + (0.0 if res is None else 2 * U * np.abs(f64(res))), "dx")
    if params:
        a = np.abs(f64(dy))
        many = (N / 152 + 64) * U
        within(dw, o["dw"], (many + s) * (a * (1 + h)).sum(0), "dw")
        within(db, o["db"], many * a.sum(0), "db")
    else:
        assert dw is None and db is None
    return dx, dw, db


SHAPES = [(1, 1, 0), (3, 7, 0), (1, 8, 0), (5, 64, 8), (2, 129, 0), (4, 130, 1), (9, 256, 8), (33, 512, 0), (7, 520, 16),
          (64, 1000, 24), (6, 1030, 7), (3, 2048, 0), (2, 2056, 8), (5, 4104, 8), (4, 8192, 0), (3, 8200, 0),
          (2, 12288, 0), (2, 12289, 3), (1, 16384, 0), (2, 33000, 0), (1, 70001, 0)]


@pytest.mark.parametrize("N,D,pad", SHAPES)
@pytest.mark.parametrize("dt,wdt", [("bf16", "bf16"), ("bf16", "f32"), ("f32", "f32")])
def test_shapes(N, D, pad, dt, wdt):
    x = rows(N, D, dt, D, pad, std=2.0)
    w, b = vector(D, wdt, 1, 1.0), vector(D, wdt, 2, 0.0)
    check_forward(x, w, b)
    dy = rows(N, D, dt, D + 1, pad)
    check_backward(x, w, dy)
    check_backward(x, w, dy, rows(N, D, dt, D + 2, pad))


# many rows: the forms that take rows in turn, full and partly filled groups of each width
@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("N,D,pad", [(20001, 1024, 0), (40003, 96, 8), (9000, 2000, 8), (5001, 4096, 0), (5003, 4088, 8),
                                     (2500, 8192, 0), (2503, 8008, 8), (3001, 515, 0), (2999, 2050, 2)])
def test_many_rows(N, D, pad, dt):
    x, w, b = rows(N, D, dt, 3, pad), vector(D, "f32", 1, 1.0), vector(D, "f32", 2, 0.0)
    check_forward(x, w, b)
    check_backward(x, w, rows(N, D, dt, 4, pad), rows(N, D, dt, 5, pad) if D % 16 else None)


# every number of threads to a row and of accesses to a thread, at its limits, for
# few rows (which have forms of their own) and for more
@pytest.mark.parametrize("N", [5, 203, 1301])
@pytest.mark.parametrize("D", [4, 60, 64, 68, 128, 132, 192, 196, 256, 260, 384, 388, 512, 516, 768, 1024, 1032, 1536, 2048,
                               2060, 4096, 4100, 6144, 6152, 8208, 12292, 16388, 24576, 24584, 32768, 32772])
@pytest.mark.parametrize("dt,wdt", [("bf16", "bf16"), ("bf16", "f32"), ("f32", "f32")])
def test_forward_widths(N, D, dt, wdt):
    if N > 1000 and D > 2100:
        N = 313
    pad = 4 if D % 8 else 0   # 8-byte rows of bf16
    check_forward(rows(N, D, dt, D, pad, std=3.0), vector(D, wdt, 1, 1.0), vector(D, wdt, 2, 0.0))


# rows longer than a CTA's columns: panels of them in turn, full and ragged
@pytest.mark.parametrize("N,D,pad", [(1000, 16384, 0), (1111, 9008, 8), (817, 12288, 0), (409, 24600, 8)])
@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_backward_of_many_long_rows(N, D, pad, dt):
    x, w = rows(N, D, dt, 3, pad, offset=30.0 if D == 12288 and dt == "f32" else 0.0), vector(D, "f32", 1, 1.0)
    dy = rows(N, D, dt, 4, pad)
    check_backward(x, w, dy, rows(N, D, dt, 5, pad))
    dx, _, _ = check_backward(x, w, dy)
    _, mean, rstd = tp.layernorm(x, w, None)
    assert torch.equal(tp.layernorm_backward(dy, x, w, mean, rstd, param_grads=False)[0], dx)
    dw, db = (torch.empty_like(w) for _ in range(2))
    ws = torch.empty(tp.tpmlp_layernorm_backward_workspace_bytes(N, D), dtype=torch.uint8, device=dev())
    tp.tpmlp_layernorm_backward(dy, x, w, mean, rstd, None, x, dw, db, ws)
    assert torch.equal(x, dx)


@pytest.mark.parametrize("D", [48, 256, 500, 2000, 7000])
@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_bad_rows_beside_good_ones(D, dt):
    """Rows that share a warp or a CTA: one overflows, one holds a NaN, the others
    are as they are alone."""
    x, w, b = rows(333, D, dt, 1), vector(D, "f32", 1, 1.0), vector(D, "f32", 2, 0.0)
    want, mean, rstd = tp.layernorm(x, w, b)
    far, bad = torch.arange(3, 333, 17), torch.arange(4, 333, 29)
    z = x.clone()
    z[far] *= 2.0 ** 80
    z[bad, D // 2] = float("nan")
    y, m, r = tp.layernorm(z, w, b)
    good = torch.ones(333, dtype=torch.bool)
    good[far] = good[bad] = False
    for got, ref in ((y, want), (m, mean), (r, rstd)):
        assert torch.equal(got[good.to(dev())], ref[good.to(dev())])
    assert torch.isnan(y[bad]).all()
    only = far[~torch.isin(far, bad)]
    o = oracle.norm.layernorm(z[only], w, b, EPS)
    h = np.abs(o["y"] - f64(b)) / np.abs(f64(w))
    within(y[only], o["y"], 8 * s_of(D) * np.abs(f64(w)) * (2 + h) + 4 * U, "overflowing rows")


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("N,D", [(3, 768), (2600, 8192)])
def test_without_parameters(N, D, dt):
    x, dy = rows(N, D, dt, 1), rows(N, D, dt, 2)
    w = vector(D, dt, 1, 1.0)
    check_forward(x, None, None)
    check_forward(x, w, None)
    check_forward(x, None, w)
    check_backward(x, None, dy)
    check_backward(x, None, dy, params=False)
    dx, dw, _ = check_backward(x, w, dy)
    assert dw.dtype == w.dtype


@pytest.mark.parametrize("N,D", [(4, 640), (5, 1001), (2600, 8192), (2, 20000)])
@pytest.mark.parametrize("offset", [5.0, 300.0, -20000.0])
def test_means_far_from_zero(N, D, offset):
    """The row's spread is small next to its mean: h has the spread's digits, not the mean's."""
    x = rows(N, D, "f32", 6, offset=offset)
    check_forward(x, vector(D, "f32", 1, 1.0), vector(D, "f32", 2, 0.0))
    check_backward(x, vector(D, "f32", 1, 1.0), rows(N, D, "f32", 7))


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("N,D", [(6, 300), (6, 8192), (2600, 8192), (6, 40000)])
def test_huge_tiny_and_bad_rows(N, D, dt):
    """Squares that overflow, rows of one value, infinities and NaN: each in its own row."""
    x = rows(N, D, dt, 8)
    x[1] *= 2.0 ** 100
    x[2] = 3.25
    x[3, 5] = float("nan")
    x[4, D - 1] = float("inf")
    x[5] = x[5].abs() * 1e-30
    w, b = vector(D, "f32", 1, 1.0), vector(D, "f32", 2, 0.0)
    y, mean, rstd = tp.layernorm(x, w, b)
    fine = [n for n in range(min(N, 40)) if n not in (1, 3, 4)]
    o = oracle.norm.layernorm(x[fine], w, b, EPS)
    s = s_of(D)
    within(y[fine], o["y"], 8 * s * np.abs(f64(w)) * (2 + np.abs(o["y"])) + 4 * U, "y")
    o = oracle.norm.layernorm(x[1:2], w, b, EPS)
    within(y[1:2], o["y"], 8 * s * np.abs(f64(w)) * (2 + np.abs(o["y"])), "huge row")
    within(mean[1:2], o["mean"], 4 * s * np.abs(f64(x[1])).mean() + 4 * U * np.abs(o["mean"]), "huge row's mean")
    within(rstd[1:2], o["rstd"], 4 * s * o["rstd"], "huge row's rstd")
    assert torch.isnan(y[3]).all() and torch.isnan(y[4]).all() and torch.isnan(mean[3]) and not torch.isfinite(rstd[4])
    assert torch.isfinite(y[[n for n in range(N) if n not in (3, 4)]]).all()
    # the gradient keeps a bad row's NaN out of the others' dx
    dx, _, _ = tp.layernorm_backward(rows(N, D, dt, 9), x, w, mean, rstd)
    assert torch.isnan(dx[3]).all() and torch.isfinite(dx[[n for n in range(N) if n not in (1, 3, 4)]]).all()


def test_eps_zero_and_constant_rows():
    x = rows(3, 100, "f32", 1)
    x[1] = 2.0
    y, mean, rstd = tp.layernorm(x, eps=0.0)
    assert torch.isnan(y[1]).all() and float(mean[1]) == 2.0
    check_forward(x[[0, 2]], None, None, eps=0.0)


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("N,D,pad", [(5, 300, 0), (5, 2049, 5), (2600, 8192, 0), (3, 9000, 0), (2, 40000, 8)])
def test_in_place(N, D, pad, dt):
    x, w, b = rows(N, D, dt, 1, pad), vector(D, "f32", 1, 1.0), vector(D, "f32", 2, 0.0)
    y, mean, rstd = tp.layernorm(x, w, b)
    z = rows(N, D, dt, 1, pad)
    tp.tpmlp_layernorm(z, w, b, EPS, z)
    assert torch.equal(z, y)
    dy, res = rows(N, D, dt, 2, pad), rows(N, D, dt, 3, pad)
    dx, dw, db = tp.layernorm_backward(dy, x, w, mean, rstd, dresidual=res)
    for which in range(3):
        bufs = [rows(N, D, dt, k, pad) for k in (2, 1, 3)]
        gw, gb = torch.empty_like(dw), torch.empty_like(db)
        ws = torch.empty(tp.tpmlp_layernorm_backward_workspace_bytes(N, D), dtype=torch.uint8, device=dev())
        tp.tpmlp_layernorm_backward(bufs[0], bufs[1], w, mean, rstd, bufs[2], bufs[which], gw, gb, ws)
        assert torch.equal(bufs[which], dx) and torch.equal(gw, dw) and torch.equal(gb, db)


def test_padding_is_left_alone():
    buf = torch.full((40, 80), 7.0, device=dev())
    x = rows(40, 64, "f32", 1)
    tp.tpmlp_layernorm(x, None, None, EPS, buf[:, :64])
    assert torch.equal(buf[:, 64:], torch.full((40, 16), 7.0, device=dev()))
    assert torch.equal(buf[:, :64], tp.layernorm(x)[0])


def test_gradients_against_differences_of_the_kernel():
    """The kernel's gradients against central differences of its own forward in
    fp32: step 2^-6 truncates at h^2/6 |f'''| <= 2e-3 for 24 elements of
    unit spread, and fp32 sums of 24 terms leave 2^-20 / h = 1e-4."""
    N, D, h = 1, 24, 2.0 ** -6
    x, dy, w, b = rows(N, D, "f32", 3), rows(N, D, "f32", 4), vector(D, "f32", 1, 1.0), vector(D, "f32", 2, 0.0)
    _, mean, rstd = tp.layernorm(x, w, b, eps=1e-2)
    dx, dw, db = tp.layernorm_backward(dy, x, w, mean, rstd)
    eye = h * torch.eye(D, device=dev())
    f = lambda q: (tp.layernorm(q, w, b, eps=1e-2)[0].double() * dy.double()).sum(1)
    num = (f(x + eye) - f(x - eye)) / (2 * h)
    assert float((num - dx[0].double()).abs().max()) <= 4e-3
    g = lambda k: (tp.layernorm(x, w + h * (torch.arange(D, device=dev()) == k), b, eps=1e-2)[0].double() * dy.double()).sum()
    base = (tp.layernorm(x, w, b, eps=1e-2)[0].double() * dy.double()).sum()
    for k in (0, 11, 23):
        assert abs(float((g(k) - base) / h - dw[k].double())) <= 2e-4
    assert torch.equal(db, dy[0])


def test_empty_batch():
    y, mean, rstd = tp.layernorm(rows(0, 64, "bf16", 1))
    assert y.shape == (0, 64) and mean.numel() == 0
    dx, dw, db = tp.layernorm_backward(rows(0, 64, "bf16", 1), rows(0, 64, "bf16", 1), vector(64, "f32", 1, 1.0), mean, rstd)
    assert dx.shape == (0, 64) and not dw.any() and not db.any() and dw.shape == (64,)


@pytest.mark.parametrize("N,D", [(3, 5000), (2600, 4096)])
def test_repeat_other_stream_and_graph(N, D):
    x, dy = rows(N, D, "bf16", 1), rows(N, D, "bf16", 2)
    w, b = vector(D, "f32", 1, 1.0), vector(D, "f32", 2, 0.0)
    def step():
        y, mean, rstd = tp.layernorm(x, w, b)
        return (y, mean, rstd, *tp.layernorm_backward(dy, x, w, mean, rstd, dresidual=y))
    want = step()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        got = step()
        again = step()
    s.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        held = step()
    for t in held:
        t.zero_()
    g.replay()
    g.replay()
    torch.cuda.synchronize()
    for a, b_, c, d in zip(want, got, again, held):
        assert torch.equal(a, b_) and torch.equal(a, c) and torch.equal(a, d)


def test_rows_beyond_32_bit_offsets():
    N, D, pitch = 3000, 64, 1 << 20
    buf = torch.zeros(N * pitch - pitch + D, dtype=torch.bfloat16, device=dev())
    x = buf.as_strided((N, D), (pitch, 1))
    part = rows(N, D, "bf16", 1)
    x.copy_(part)
    y, mean, rstd = tp.layernorm(x)
    want, mean2, _ = tp.layernorm(part)
    assert torch.equal(y, want) and torch.equal(mean, mean2)
    dy = rows(N, D, "bf16", 2)
    a, b = tp.layernorm_backward(dy, x, None, mean, rstd), tp.layernorm_backward(dy, part, None, mean, rstd)
    for p, q in zip(a, b):
        assert torch.equal(p, q)


LIMIT_NS, DEFAULT_NS = 20_000_000, 2_000_000_000


@pytest.mark.parametrize("D", [512, 8192])
def test_stalled_waits_run_out_and_the_next_call_is_right(D):
    """Rows in turn come by bulk copies under a bounded wait. A stalled call gives up, drains
    the copies that are on their way and says so; the next one is right."""
    N = 2600 * 8192 // D
    x, dy = rows(N, D, "bf16", 1), rows(N, D, "bf16", 2)
    weight = vector(D, "f32", 6, 1.0)
    y, mean, rstd = tp.layernorm(x, weight)
    want = tp.layernorm_backward(dy, x, None, mean, rstd)
    X, W = rows(16384, 64, "bf16", 3), [rows(64, 1024, "bf16", 4).contiguous()]
    dY = rows(16384, 1024, "bf16", 5)
    linear = lambda: tp.column_linear_backward(X, W, dY, Z=dY, act="relu", bias_grads=True)[2][0]
    db = linear()
    assert tp.tpmlp_check_device_error() == 0
    tp.tpmlp_set_wait_timeout_ns(LIMIT_NS)
    tp.tpmlp_selftest_row_stall(1)
    try:
        calls = [lambda: tp.layernorm(x, weight)] if D == 8192 else []   # rows that are taken in turn
        for call in (*calls, lambda: tp.layernorm_backward(dy, x, None, mean, rstd), linear):
            t0 = time.perf_counter()
            call()
            torch.cuda.synchronize()
            assert LIMIT_NS * 1e-9 <= time.perf_counter() - t0 < 5.0
            assert tp.tpmlp_check_device_error() == _binding.ERR_TIMEOUT
    finally:
        tp.tpmlp_selftest_row_stall(0)
        tp.tpmlp_set_wait_timeout_ns(DEFAULT_NS)
    assert torch.equal(tp.layernorm(x, weight)[0], y) and torch.equal(linear(), db)
    for a, b in zip(tp.layernorm_backward(dy, x, None, mean, rstd), want):
        assert torch.equal(a, b)


def test_refusals_on_the_device():
    x, w = rows(4, 64, "bf16", 1), vector(64, "f32", 1, 1.0)
    with pytest.raises(tp.TpmlpError) as e:
        tp.layernorm(x, eps=-1.0)
    assert e.value.status == _binding.ERR_ARG
    with pytest.raises(tp.TpmlpError) as e:
        tp.layernorm(x.float(), vector(64, "bf16", 1, 1.0))
    assert e.value.status == _binding.ERR_DTYPE
    with pytest.raises(TypeError):
        tp.layernorm(x, w, vector(64, "bf16", 1, 1.0))
    with pytest.raises(ValueError):
        tp.layernorm(x, w[:60])
    with pytest.raises(ValueError):
        tp.layernorm(x.t(), w)
    _, mean, rstd = tp.layernorm(x, w)
    with pytest.raises(ValueError):
        tp.layernorm_backward(x[:3], x, w, mean, rstd)
    with pytest.raises(ValueError):
        tp.layernorm_backward(x, x, w, mean[:3], rstd)
    with pytest.raises(tp.TpmlpError) as e:
        tp.layernorm_backward(x, x, w, mean, rstd, workspace=torch.empty(16, dtype=torch.uint8, device=dev()))
    assert e.value.status == _binding.ERR_WORKSPACE
