"""Distillation from a teacher's top tokens on the GPU against the float64
definition, loss and gradient, in one call and in two.

Tolerances. fp32 numbers: 1e-5 of the tensor's largest magnitude (sums of up to
128000 positive terms per row in fp32, as for the cross-entropy). A bf16
gradient is rounded once, 2^-9 of its own magnitude, after fp32 arithmetic:
elementwise 2^-8 |d| + 1e-5 max |d|."""

import numpy as np
import pytest
import torch

import oracle
import tensor_transformer_mlp_columnparallel_gb300 as tp
from tensor_transformer_mlp_columnparallel_gb300 import _binding

pytestmark = pytest.mark.gpu
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
INF = float("inf")


@pytest.fixture(scope="module", autouse=True)
def _built():
    import __graft_entry__
    __graft_entry__.build()
    torch.cuda.set_device(0)
    yield
    assert tp.tpmlp_check_device_error() == 0


def dev():
    return torch.device("cuda:0")


def make(N, V, K, dt, seed, ld=None):
    g = torch.Generator().manual_seed(seed)
    z = torch.full((N, ld or V), 1000.0, dtype=TYPES[dt])
    z[:, :V] = (torch.randn(N, V, generator=g) * 2).to(TYPES[dt])
    ids = torch.stack([torch.randperm(V, generator=g)[:K] if K <= V else
                       torch.randint(0, V, (K,), generator=g) for _ in range(max(N, 1))])[:N]
    tl = torch.randn(N, K, generator=g) * 2 + 5
    w = torch.rand(N, generator=g) + 0.5
    return (z.to(dev())[:, :V], ids.to(torch.int32).to(dev()), tl.to(dev()), w.to(dev()))


def close(got, ref, what):
    g, o = got.double().cpu().numpy(), np.asarray(ref, dtype=np.float64)
    assert g.shape == o.shape, what
    fin = np.isfinite(o)
    np.testing.assert_array_equal(g[~fin], o[~fin], err_msg=what)
    if not fin.any():
        return
    big = max(np.max(np.abs(o[fin])), 1e-30)
    lim = 1e-5 * big + (2.0 ** -8 * np.abs(o[fin]) if got.dtype == torch.bfloat16 else 0.0)
    bad = np.abs(g[fin] - o[fin]) - lim
    assert np.max(bad) <= 0, f"{what}: {np.max(np.abs(g[fin] - o[fin])) / big:.2e} of the largest"


def check(z, ids, tl, w, T, tau, scale=1.0):
    zc = z.clone()
    loss, mean, lse = tp.vocab_distill(z, ids, tl, T, temperature=tau)
    d = tp.vocab_distill_backward(z, ids, tl, T, lse, temperature=tau, grad_scale=scale, grad_tokens=w)
    loss2, mean2, lse2, d2 = tp.vocab_distill_with_grad(z, ids, tl, T, temperature=tau,
                                                        grad_scale=scale, grad_tokens=w)
    assert torch.equal(z, zc)
    N, V = z.shape
    buf = z.clone() if z.is_contiguous() else torch.cat([z, z], 1)[:, :V]
    tp.vocab_distill_backward(buf, ids, tl, T, lse, temperature=tau, grad_scale=scale, grad_tokens=w,
                              in_place=True)
    buf2 = z.clone()
    tp.vocab_distill_with_grad(buf2, ids, tl, T, temperature=tau, grad_scale=scale, grad_tokens=w,
                               in_place=True)
    torch.cuda.synchronize()
    f = oracle.vocab.distill(z, ids, tl, tau)
    g = scale * (1.0 if w is None else w.double().cpu().numpy())
    dref = oracle.vocab.distill_backward(z, ids, tl, tau, g)
    for a, b, c in ((loss, mean, lse), (loss2, mean2, lse2)):
        close(a, f["loss"], "loss")
        close(b, np.array([f["mean"]]), "mean")
        close(c, f["lse"], "lse")
    for x, what in ((d, "dlogits"), (d2, "dlogits, one call"), (buf, "in place"), (buf2, "one call in place")):
        close(x, dref, what)


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("N,V,T,K,ld,tau", [
    (1, 1, 1, 1, None, 1.0), (2, 7, 7, 7, None, 1.0), (3, 64, 2, 5, 65, 2.0), (5, 257, 1, 1, None, 0.5),
    (9, 1000, 8, 20, 1003, 1.5), (4, 4099, 1, 128, 4099, 4.0), (17, 9999, 9, 33, 10001, 1.0),
    (2, 50001, 7, 1024, 50016, 3.0), (1, 128000, 8, 64, None, 2.0), (40, 16384, 16, 3, None, 1.0),
    (2, 150001, 1, 40, None, 1.0), (320, 2048, 2, 10, None, 2.0), (600, 515, 5, 2, 517, 1.0),
    (1, 600064, 8, 9, None, 1.0)])
def test_shapes(N, V, T, K, ld, tau, dt):
    z, ids, tl, w = make(N, V, K, dt, N + V + K, ld)
    check(z, ids, tl, w, T, tau, scale=1.0 / N)


@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_teacher_lists(dt):
    """Empty slots, empty rows, repeated ids, slots of probability 0, a
    teacher that is certain, no weights."""
    z, ids, tl, _ = make(9, 3000, 12, dt, 5)
    ids[0, 3:] = -1
    ids[1] = -1
    tl[2] = -INF
    tl[3, ::2] = -INF
    ids[4] = ids[4, 0]
    ids[5, 6:] = ids[5, :6]
    tl[6] = -200.0
    tl[6, 4] = 200.0
    ids[7, :11] = -1
    z[1].fill_(float("nan"))          # the logits of a padding position are not read
    loss, _, _, d = tp.vocab_distill_with_grad(z, ids, tl, 3, temperature=2.0)
    assert loss[1] == 0 and not d[1].any()
    z[1].fill_(0.0)
    check(z, ids, tl, None, 3, 2.0)
    check(z, ids, tl, None, 1, 1.0, scale=0.125)


@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_masked_students(dt):
    """Student rows that a mask leaves with a few tokens, one, or none."""
    z, ids, tl, w = make(6, 2500, 8, dt, 6)
    keep = torch.zeros(2500, dtype=torch.bool, device=dev())
    keep[ids[0].long()] = True
    z[0].masked_fill_(~keep, -INF)                    # the teacher's tokens remain
    z[1].masked_fill_(keep, -INF)
    z[1, ids[1, 2].long()] = -INF                     # one of them masked: infinite loss
    z[2].fill_(-INF)
    z[3].masked_fill_(~keep, torch.finfo(z.dtype).min)
    z[3, ids[3].long()] = 0.5
    z[4].fill_(-INF)
    z[4, ids[4, 0].long()] = 2.0
    tl[4, 1:] = -INF
    check(z, ids, tl, w, 1, 1.0)


def test_nan_rows_and_bad_ids():
    z, ids, tl, w = make(6, 1200, 5, "f32", 8)
    z[1, 600] = float("nan")
    z[2, 600] = INF
    tl[3, 2] = float("nan")
    loss, _, lse, d = tp.vocab_distill_with_grad(z, ids, tl, 4, grad_tokens=w)
    assert tp.tpmlp_check_device_error() == 0
    for n in (1, 2, 3):
        assert torch.isnan(loss[n]) and torch.isnan(d[n]).any()
    ids[4, 1] = 1200
    ids[5, 0] = -2
    loss, _, lse, d = tp.vocab_distill_with_grad(z, ids, tl, 4, grad_tokens=w)
    assert tp.tpmlp_check_device_error() == _binding.ERR_ARG
    for n in (4, 5):
        assert torch.isnan(loss[n]) and torch.isnan(d[n]).all()
    assert torch.isfinite(d[0]).all() and torch.isfinite(loss[0])


def test_gradient_against_differences_of_the_loss():
    """The kernel's gradient against central differences of the kernel's own
    loss in fp32 (step 2^-6: truncation h^2/6 |f'''| <= 5e-5, rounding
    2^-23 |f| / h <= 2e-4 for losses below 30)."""
    z, ids, tl, w = make(1, 24, 4, "f32", 11)
    tau, h = 1.5, 2.0 ** -6
    _, _, lse = tp.vocab_distill(z, ids, tl, 1, temperature=tau)
    d = tp.vocab_distill_backward(z, ids, tl, 1, lse, temperature=tau)
    up = z.repeat(24, 1) + h * torch.eye(24, device=dev())
    dn = z.repeat(24, 1) - h * torch.eye(24, device=dev())
    f = lambda q: tp.vocab_distill(q, ids.repeat(24, 1), tl.repeat(24, 1), 1, temperature=tau)[0].double()
    num = (f(up) - f(dn)) / (2 * h)
    assert float((num - d[0].double()).abs().max()) <= 3e-4


def test_takes_the_list_that_logprobs_returns():
    """A teacher's top list and the same logits as a student of its own: with
    the whole vocabulary listed the divergence and the gradient vanish (to
    the cancellation of two lse's, 2^-22 of about 10)."""
    z, _, _, _ = make(5, 100, 3, "f32", 12)
    t = torch.zeros(5, dtype=torch.int64, device=dev())
    _, _, _, ids, top = tp.vocab_logprobs(z, t, 4, top_k=100)
    loss, _, _, d = tp.vocab_distill_with_grad(z, ids, top, 4)
    assert float(loss.abs().max()) <= 5e-6 and float(d.abs().max()) <= 5e-6


def test_rows_beyond_32_bit_offsets():
    N, V, K = 17000, 128000, 4
    z = torch.zeros(N, V, dtype=torch.bfloat16, device=dev())
    r = [0, 16776, 16778, N - 1]
    part, ids4, tl4, _ = make(len(r), V, K, "bf16", 13)
    z[r] = part
    ids = torch.full((N, K), -1, dtype=torch.int32, device=dev())
    tl = torch.zeros(N, K, device=dev())
    ids[r], tl[r] = ids4, tl4
    loss, _, _, d = tp.vocab_distill_with_grad(z, ids, tl, 8, in_place=True)
    assert d.data_ptr() == z.data_ptr()
    close(loss[r], oracle.vocab.distill(part, ids4, tl4, 1.0)["loss"], "loss")
    close(d[r], oracle.vocab.distill_backward(part, ids4, tl4, 1.0, 1.0), "dlogits")
    assert int((d != 0).any(dim=1).sum()) == len(r)


def test_empty_batch_repeat_and_other_stream():
    z, ids, tl, w = make(0, 64, 3, "f32", 2)
    loss, mean, lse, d = tp.vocab_distill_with_grad(z, ids, tl, 4, grad_tokens=w)
    assert loss.numel() == 0 and d.shape == (0, 64) and torch.isnan(mean).all()
    z, ids, tl, w = make(65, 7001, 9, "bf16", 4)
    ref = tp.vocab_distill_with_grad(z, ids, tl, 1, grad_tokens=w)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        got = tp.vocab_distill_with_grad(z, ids, tl, 1, grad_tokens=w)
    s.synchronize()
    for a, b in zip(ref, got):
        assert torch.equal(a, b)


def test_refusals_on_the_device():
    z, ids, tl, w = make(4, 12, 3, "f32", 2)
    for kw in (dict(temperature=0.0), dict(temperature=float("inf"))):
        with pytest.raises(tp.TpmlpError) as e:
            tp.vocab_distill(z, ids, tl, 4, **kw)
        assert e.value.status == _binding.ERR_ARG
    with pytest.raises(tp.TpmlpError):
        tp.vocab_distill(z, ids, tl, 5)
    with pytest.raises(TypeError):
        tp.vocab_distill(z, ids.long(), tl, 4)
    with pytest.raises(ValueError):
        tp.vocab_distill(z, ids, tl[:, :2].contiguous(), 4)
    with pytest.raises(ValueError):
        tp.tpmlp_vocab_distill_backward(z, ids, tl, 4, 1.0, w, None, 1.0, z[:2])


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("V,T,K,ld", [
    (3, 3, 1, 4), (515, 5, 40, 517), (1000, 8, 200, None), (4096, 1, 33, None),
    (8199, 3, 7, 8201), (12001, 1, 130, 12001), (16384, 2, 5, None), (16400, 4, 5, None)])
def test_many_short_rows(V, T, K, ld, dt):
    """More rows than the device holds CTAs at a time; masked tokens, empty
    slots, empty rows and repeated ids among them."""
    N = 650
    z, ids, tl, w = make(N, V, K, dt, V + K, ld)
    g = torch.Generator().manual_seed(V)
    z[::5].masked_fill_((torch.rand(V, generator=g) < 0.5).to(dev()), -INF)
    z.scatter_(1, ids.long(), 1.0)                       # the teacher's tokens are not masked
    ids[1::7, K // 2:] = -1
    ids[2::9] = -1
    ids[3::4, K - 1] = ids[3::4, 0]
    check(z, ids, tl, w, T, 1.5, scale=0.3)


def test_many_short_rows_with_nan_and_bad_ids():
    z, ids, tl, w = make(700, 900, 6, "bf16", 8)
    z[5, 17] = float("nan")
    z[6] = -INF
    ids[7, 2] = 900
    loss, _, lse, d = tp.vocab_distill_with_grad(z, ids, tl, 3, grad_tokens=w)
    assert tp.tpmlp_check_device_error() == _binding.ERR_ARG
    one = [tp.vocab_distill_with_grad(z[n:n + 1], ids[n:n + 1], tl[n:n + 1], 3, grad_tokens=w[n:n + 1])
           for n in (4, 6, 8)]
    assert torch.isnan(loss[[5, 7]]).all() and torch.isnan(lse[[5, 7]]).all()
    assert torch.isnan(d[5]).all() and torch.isnan(d[7]).all()
    for n, o in zip((4, 6, 8), one):
        close(loss[n:n + 1], o[0].double().cpu().numpy(), "loss")
        close(d[n:n + 1], o[3].double().cpu().numpy(), "dlogits")


@pytest.mark.parametrize("N", [3, 700])
@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_vocabulary_of_one_token(N, dt):
    # p = q = 1 whatever the logits, however many slots share the token
    z, ids, tl, w = make(N, 1, 2, dt, 3)
    d = tp.vocab_distill_with_grad(z, ids, tl, 1, temperature=1.5, grad_tokens=w)[3]
    assert torch.equal(d, torch.zeros_like(d))
