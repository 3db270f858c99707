"""Clipped policy loss with its KL term on the GPU against the float64
definition, loss and gradient, in one call and in two.

Tolerances. l is taken to more digits than fp32 holds; the row's sum of up to
600000 positive terms is off by 2^-18 at the most (2^-20 as a rule), which the
ratio takes over: loss and slope 1e-5 of |A| rho (+ kl (1 + e^|r|)) of the token; k
as well as its own e^r - 1 times that. The gradient's element is w p or w (1 - p):
1e-5 of the row's largest, and bf16's rounding 2^-8 of itself."""

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


def f64(t):
    return t.double().cpu().numpy()


def make(N, V, dt, seed, ld=None, tau=1.0, low=0.2, high=0.28):
    """Rows, some of them sure of one token; tokens likely and unlikely; older and
    reference log probabilities near theirs, no ratio within 1e-3 of a border."""
    g = torch.Generator().manual_seed(seed)
    z = torch.full((N, ld or V), 1000.0, dtype=TYPES[dt])
    z[:, :V] = (torch.randn(N, V, generator=g) * 2).to(TYPES[dt])
    t = torch.randint(0, V, (N,), generator=g)
    z[torch.arange(N)[::2], t[::2]] = (6.0 + 14 * torch.rand(len(t[::2]), generator=g)).to(TYPES[dt])
    q = z[:, :V].double() / tau
    lp = q.gather(1, t[:, None])[:, 0] - torch.logsumexp(q, 1)
    old = (lp + 0.3 * torch.randn(N, generator=g)).float()
    for border in (1 - low, 1 + high):
        near = (torch.exp(lp - old.double()) - border).abs() < 1e-3
        old = torch.where(near, old + 0.01, old)
    adv, ref = torch.randn(N, generator=g), (lp + 0.3 * torch.randn(N, generator=g)).float()
    w = torch.rand(N, generator=g) + 0.5
    return [x.to(dev()) for x in (z, t, old, adv, ref, w)]


def close(got, ref, lim, what):
    g = f64(got)
    fin = np.isfinite(ref)
    np.testing.assert_array_equal(g[~fin], ref[~fin], err_msg=what)
    if got.dtype == torch.bfloat16:
        lim = lim + 2.0 ** -8 * np.abs(np.where(fin, ref, 0))
    bad = np.where(fin, np.abs(np.where(fin, g - np.where(fin, ref, 0), 0)) - lim, -1)
    assert not np.isnan(bad).any() and bad.max(initial=-1) <= 0, f"{what}: over by {bad.max():.2e}"


def check(z, t, old, adv, ref, w, T, kl=0.05, low=0.2, high=0.28, tau=1.0, scale=1.0):
    V = z.shape[1]
    opt = dict(ref_logprobs=ref, kl_coef=kl, clip_low=low, clip_high=high, temperature=tau)
    g = dict(grad_scale=scale, grad_tokens=w)
    keep = z.clone()
    one = tp.vocab_policy_with_grad(z, t, old, adv, T, **opt, **g)
    two = tp.vocab_policy(z, t, old, adv, T, **opt)
    d = tp.vocab_policy_backward(z, t, old, adv, T, two[2], **opt, **g)
    assert torch.equal(z, keep)
    in1, in2 = z.clone(), torch.cat([z, z], 1)[:, :V]
    tp.vocab_policy_with_grad(in1, t, old, adv, T, **opt, **g, in_place=True)
    tp.vocab_policy_backward(in2, t, old, adv, T, two[2], **opt, **g, in_place=True)
    o = oracle.vocab.policy(z, t, old, adv, ref, kl, low, high, tau)
    scale_n = scale * (1.0 if w is None else f64(w))
    dref = oracle.vocab.policy_backward(z, t, old, adv, ref, kl, low, high, tau, scale_n)
    with np.errstate(over="ignore", invalid="ignore"):
        rho = np.exp(o["logprob"] - f64(old))
        er = np.exp(np.abs(f64(ref) - o["logprob"])) if ref is not None else 0.0
        part = np.where(f64(adv) != 0, np.abs(f64(adv)) * np.maximum(rho, 1), 0) + kl * (1 + er)
        lim = np.where(np.isfinite(part), 1e-5 * part, 0) + 1e-7
    for loss, mean, lp, k in (one[:4], two):
        close(lp, o["logprob"], 1e-6 * np.abs(np.where(np.isfinite(o["logprob"]), o["logprob"], 0)) + 2.0 ** -18, "logprob")
        close(loss, o["loss"], lim, "loss")
        if np.isfinite(o["loss"]).all():
            close(mean, np.array([o["mean"]]), np.array([lim.mean() + 1e-6 * np.abs(o["loss"]).mean()]), "mean")
        if ref is not None:
            with np.errstate(invalid="ignore"):
                near = np.where(np.isfinite(er), 1e-5 * (er - 1) + 1e-10 + 2e-7 * o["kl"], 0)
            close(k, o["kl"], np.where(np.isfinite(near), near, 0), "kl")
        else:
            assert k is None
    big = np.abs(dref).max(axis=1, initial=0.0, keepdims=True)
    weight = np.broadcast_to(np.abs(scale_n), (z.shape[0],))[:, None] / tau
    for x, what in ((one[4], "one call"), (d, "two calls"), (in1, "one call in place"), (in2, "two calls in place")):
        close(x, dref, np.where(np.isfinite(big), 1e-5 * big, 0) + np.where(big > 0, lim[:, None] * weight, 0), what)


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("N,V,T,ld,tau", [
    (1, 1, 1, None, 1.0), (2, 7, 7, None, 1.0), (3, 64, 2, 65, 0.7), (5, 257, 1, None, 1.5), (9, 1000, 8, 1003, 1.0),
    (4, 4099, 1, 4099, 1.0), (17, 9999, 9, 10001, 0.7), (2, 50001, 7, 50016, 1.3), (1, 128000, 8, None, 1.0),
    (40, 16384, 16, None, 1.0), (2, 150001, 1, None, 1.0), (320, 2048, 2, None, 0.9), (650, 515, 5, 517, 1.0),
    (640, 8199, 3, 8201, 1.1), (1, 600064, 8, None, 1.0)])
def test_shapes(N, V, T, ld, tau, dt):
    z, *rest = make(N, V, dt, N + V, ld, tau)
    check(z[:, :V], *rest, T, tau=tau, scale=1.0 / N)


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("N", [9, 640])
def test_positions_without_a_token(N, dt):
    z, t, old, adv, ref, w = make(N, 3000, dt, 5)
    t[1], t[4], t[-1] = -1, -100, -(1 << 40)
    z[1].fill_(float("nan"))          # not read
    none = [1, 4, N - 1]
    loss, _, lp, kl, d = tp.vocab_policy_with_grad(z, t, old, adv, 3, ref_logprobs=ref, kl_coef=0.1)
    assert not loss[none].any() and not lp[none].any() and not kl[none].any() and not d[none].any()
    d = tp.vocab_policy_backward(z, t, old, adv, 3, lp, ref_logprobs=ref, kl_coef=0.1)
    assert not d[none].any()
    z[1].fill_(0.0)
    check(z, t, old, adv, ref, None, 1)
    check(z, t, old, adv, None, w, 3, kl=0.0)


@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_clipping_and_advantages(dt):
    """Tokens on each side of each border, no advantage, no clip range, no borders."""
    z, t, old, adv, ref, w = make(12, 500, dt, 6)
    lp = tp.vocab_policy(z, t, old, adv, 1)[2]
    for n, (r, a) in enumerate(((0.5, 1.0), (0.5, -1.0), (2.0, 1.0), (2.0, -1.0), (1.0, 1.0), (1.0, -1.0), (1.0, 0.0))):
        old[n], adv[n] = lp[n] - float(np.log(r)), a
    old[7] = lp[7] - 3.0
    check(z, t, old, adv, ref, w, 1)
    check(z, t, old, adv, ref, w, 1, kl=0.0)
    check(z, t, old, adv, None, None, 1, kl=0.0, low=1.0, high=INF)
    d = tp.vocab_policy_with_grad(z, t, old, adv, 1, ref_logprobs=ref)[4]
    assert not d[[1, 2, 6]].any() and d[[0, 3, 4, 5]].any(dim=1).all()


@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_masked_rows(dt):
    """Rows that a mask leaves with the token, with a few, with others only, with none;
    masks of the type's lowest value."""
    z, t, old, adv, ref, w = make(8, 2500, dt, 7)
    adv[:] = torch.tensor([1.0, 1.0, 1.0, -1.0, 1.0, 0.7, 0.7, 1.0], device=dev())
    own = z.gather(1, t[:, None])[:, 0].clone()
    z[0].fill_(-INF)
    z[0, t[0]] = own[0]
    z[1, 100:].fill_(-INF)
    z[1, t[1]] = own[1]
    z[2, t[2]] = -INF                        # the token itself is masked
    z[3, t[3]] = -INF
    z[4].fill_(-INF)
    z[5].fill_(torch.finfo(z.dtype).min)
    z[5, t[5]] = 1.5
    z[6].fill_(torch.finfo(z.dtype).min)
    z[7, t[7]] = torch.finfo(z.dtype).min
    old[5] = old[0] = 0.05
    old[6] = -float(np.log(2500)) + 0.01
    check(z, t, old, adv, None, w, 1, kl=0.0)
    # with a KL term a masked token's loss is infinite, its gradient not finite
    loss, _, lp, kl, d = tp.vocab_policy_with_grad(z, t, old, adv, 1, ref_logprobs=ref, kl_coef=0.1)
    assert torch.isinf(loss[[2, 3, 4, 7]]).all() and torch.isinf(kl[2]) and lp[2] == -INF
    assert torch.isfinite(loss[[0, 1, 5, 6]]).all() and torch.isfinite(d[[0, 1, 5]]).all()


@pytest.mark.parametrize("N", [6, 700])
def test_nan_rows_and_bad_targets(N):
    z, t, old, adv, ref, w = make(N, 1200, "f32", 8)
    z[1, 600], z[2, 600] = float("nan"), INF
    old[3] = float("nan")
    loss, _, lp, kl, d = tp.vocab_policy_with_grad(z, t, old, adv, 4, ref_logprobs=ref, kl_coef=0.1, grad_tokens=w)
    d2 = tp.vocab_policy_backward(z, t, old, adv, 4, lp, ref_logprobs=ref, kl_coef=0.1, grad_tokens=w)
    assert tp.tpmlp_check_device_error() == 0
    for n in (1, 2, 3):
        assert torch.isnan(loss[n]) and torch.isnan(d[n]).any() and torch.isnan(d2[n]).any()
    t[4], t[5] = 1200, 1 << 40
    loss, _, lp, kl, d = tp.vocab_policy_with_grad(z, t, old, adv, 4, ref_logprobs=ref, kl_coef=0.1, grad_tokens=w)
    assert tp.tpmlp_check_device_error() == _binding.ERR_ARG
    d2 = tp.vocab_policy_backward(z, t, old, adv, 4, lp, ref_logprobs=ref, kl_coef=0.1, grad_tokens=w)
    assert tp.tpmlp_check_device_error() == _binding.ERR_ARG
    for n in (4, 5):
        assert torch.isnan(loss[n]) and torch.isnan(lp[n]) and torch.isnan(d[n]).all() and torch.isnan(d2[n]).all()
    rest = [n for n in range(N) if not 1 <= n <= 5]
    assert torch.isfinite(d[rest]).all() and torch.isfinite(loss[rest]).all() and torch.isfinite(d2[rest]).all()


@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_unlikely_and_certain_tokens(dt):
    """Log probabilities far below those a later gradient takes from one number,
    and tokens whose 1 - p is a few ulps."""
    z, t, old, adv, ref, w = make(6, 4000, dt, 9)
    for n, up in enumerate((40.0, 300.0, 700.0)):
        z[n, (t[n] + 1) % 4000] = up
        old[n] = float(torch.log_softmax(z[n].double(), 0)[t[n]]) - 0.1
    for n, up in ((3, 15.0), (4, 22.0), (5, 60.0)):
        z[n, t[n]] = up
        old[n] = 0.05
    check(z, t, old, adv, None, w, 1, kl=0.0)


def test_gradient_against_differences_of_the_loss():
    """The kernel's gradient against central differences of its own loss in fp32
    (step 2^-6: truncation h^2/6 |f'''| <= 1e-4, rounding 2^-22 |f| / h <= 1e-4)."""
    z, t, old, adv, ref, w = make(1, 24, "f32", 11, tau=1.2)
    opt = dict(ref_logprobs=None, clip_low=1.0, clip_high=INF, temperature=1.2)
    d = tp.vocab_policy_with_grad(z, t, old, adv, 1, **{**opt, "ref_logprobs": ref}, kl_coef=0.3)[4]
    h = 2.0 ** -6
    eye = h * torch.eye(24, device=dev())
    rep = lambda x: x.repeat(24)
    f = lambda q: tp.vocab_policy(q, rep(t), rep(old), rep(adv), 1, **{**opt, "ref_logprobs": rep(ref)}, kl_coef=0.3)[0].double()
    num = (f(z + eye) - f(z - eye)) / (2 * h)
    assert float((num - d[0].double()).abs().max()) <= 4e-4


def test_rows_beyond_32_bit_offsets():
    N, V = 17000, 128000
    z = torch.zeros(N, V, dtype=torch.bfloat16, device=dev())
    r = [0, 16776, 16778, N - 1]
    part, *rest = make(len(r), V, "bf16", 13)
    z[r] = part
    t = torch.full((N,), -1, dtype=torch.int64, device=dev())
    vecs = [torch.zeros(N, device=dev()) for _ in range(3)]
    t[r] = rest[0]
    for v, x in zip(vecs, rest[1:4]):
        v[r] = x
    loss, _, _, _, d = tp.vocab_policy_with_grad(z, t, *vecs[:2], 8, ref_logprobs=vecs[2], kl_coef=0.1, in_place=True)
    want = tp.vocab_policy_with_grad(part, *rest[:3], 8, ref_logprobs=rest[3], kl_coef=0.1)
    assert d.data_ptr() == z.data_ptr()
    torch.testing.assert_close(loss[r], want[0], rtol=1e-5, atol=1e-6)
    torch.testing.assert_close(d[r].float(), want[4].float(), rtol=2.0 ** -7, atol=1e-8)
    assert int((d != 0).any(dim=1).sum()) == len(r)


def test_empty_batch_repeat_other_stream_and_graph():
    z, t, old, adv, ref, w = make(0, 64, "f32", 2)
    loss, mean, lp, kl, d = tp.vocab_policy_with_grad(z, t, old, adv, 4, ref_logprobs=ref, grad_tokens=w)
    assert loss.numel() == 0 and d.shape == (0, 64) and torch.isnan(mean).all()
    z, t, old, adv, ref, w = make(65, 7001, "bf16", 4)
    step = lambda: tp.vocab_policy_with_grad(z, t, old, adv, 1, ref_logprobs=ref, kl_coef=0.1, grad_tokens=w)
    want = step()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        got = step()
    s.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        held = step()
    for x in held:
        x.zero_()
    g.replay()
    torch.cuda.synchronize()
    for a, b, c in zip(want, got, held):
        assert torch.equal(a, b) and torch.equal(a, c)


def test_refusals_on_the_device():
    z, t, old, adv, ref, w = make(4, 12, "f32", 2)
    for kw in (dict(temperature=0.0), dict(kl_coef=0.1), dict(clip_low=1.5), dict(clip_high=-1.0)):
        with pytest.raises(tp.TpmlpError) as e:
            tp.vocab_policy(z, t, old, adv, 4, **kw)
        assert e.value.status == _binding.ERR_ARG
    with pytest.raises(tp.TpmlpError):
        tp.vocab_policy(z, t, old, adv, 5)
    with pytest.raises(TypeError):
        tp.vocab_policy(z, t.int(), old, adv, 4)
    with pytest.raises(ValueError):
        tp.vocab_policy(z, t, old[:3], adv, 4)
    with pytest.raises(ValueError):
        tp.tpmlp_vocab_policy_backward(z, t, old, adv, None, 4, 0.0, 0.2, 0.2, 1.0, old, None, 1.0, z[:2])
