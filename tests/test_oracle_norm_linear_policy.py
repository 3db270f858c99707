"""The float64 definitions of layer norm, the linear layer and the policy loss,
against central differences and torch in float64."""

import numpy as np
import pytest
import torch

import oracle


def differences(f, x, h=1e-6):
    """Central differences of the number f(x) over every element of x."""
    x = np.array(x, dtype=np.float64)
    g = np.zeros_like(x)
    for i in np.ndindex(*x.shape):
        keep = x[i]
        x[i] = keep + h
        up = f(x)
        x[i] = keep - h
        g[i] = (up - f(x)) / (2 * h)
        x[i] = keep
    return g


@pytest.mark.parametrize("affine", [True, False])
def test_layernorm_against_torch_and_differences(affine):
    rng = np.random.default_rng(1)
    x, dy, res = rng.normal(size=(4, 7)) + 2.0, rng.normal(size=(4, 7)), rng.normal(size=(4, 7))
    w, b = (rng.normal(size=7), rng.normal(size=7)) if affine else (None, None)
    o = oracle.norm.layernorm(x, w, b, 1e-3)
    t = lambda a: None if a is None else torch.tensor(a)
    ref = torch.nn.functional.layer_norm(t(x), (7,), t(w), t(b), 1e-3)
    np.testing.assert_allclose(o["y"], ref.numpy(), rtol=1e-12, atol=1e-13)
    g = oracle.norm.layernorm_backward(dy, x, w, 1e-3, res)
    f = lambda **k: float(np.sum(dy * oracle.norm.layernorm(**{**dict(x=x, w=w, b=b, eps=1e-3), **k})["y"]))
    np.testing.assert_allclose(g["dx"] - res, differences(lambda q: f(x=q), x), atol=1e-8)
    if affine:
        np.testing.assert_allclose(g["dw"], differences(lambda q: f(w=q), w), atol=1e-8)
        np.testing.assert_allclose(g["db"], differences(lambda q: f(b=q), b), atol=1e-8)


@pytest.mark.parametrize("act", [None, "relu", "gelu_tanh", "gelu_erf", "gelu_sigmoid"])
def test_linear_against_differences(act):
    rng = np.random.default_rng(2)
    X, W, b = rng.normal(size=(3, 5)), rng.normal(size=(5, 4)), rng.normal(size=4)
    R, dY = rng.normal(size=(3, 4)), rng.normal(size=(3, 4))
    o = oracle.linear.forward(X, W, b, act, R)
    g = oracle.linear.backward(X, W, dY, o["Z"], act)
    y = lambda **k: float(np.sum(dY * oracle.linear.forward(**{**dict(X=X, W=W, b=b, act=act, R=R), **k})["Y"]))
    for name, at in (("X", X), ("W", W), ("b", b)):
        np.testing.assert_allclose(g["d" + name], differences(lambda q: y(**{name: q}), at), atol=2e-8, err_msg=name)
    np.testing.assert_allclose(dY, differences(lambda q: y(R=q), R), atol=1e-8)


POLICY = dict(kl=0.1, low=0.2, high=0.3, tau=1.4)


def tokens(rng, N, V):
    """Logits, targets (one of them none) and neighbours of the tokens' log
    probabilities, on every side of the clip range."""
    z, t = rng.normal(size=(N, V)) * 2, rng.integers(0, V, N)
    t[1] = -1
    lp = np.log(np.exp(z / 1.4) / np.exp(z / 1.4).sum(1, keepdims=True))[np.arange(N), t]
    old = lp + np.linspace(-0.7, 0.7, N)
    return z, t, old, np.where(np.arange(N) % 3 == 0, -1.5, 0.8), lp + rng.normal(size=N) * 0.4


def test_policy_gradient_against_differences():
    rng = np.random.default_rng(3)
    z, t, old, adv, ref = tokens(rng, 9, 8)
    adv[4] = 0.0
    g = rng.normal(size=9)
    f = lambda q: float(np.sum(g * oracle.vocab.policy(q, t, old, adv, ref, **POLICY)["loss"]))
    num = differences(f, z)
    np.testing.assert_allclose(oracle.vocab.policy_backward(z, t, old, adv, ref, **POLICY, grad=g), num, atol=3e-8)
    assert not num[1].any()
    held = oracle.vocab.policy_backward(z, t, old, adv, None, **{**POLICY, "kl": 0.0}, grad=g)
    assert 0 < np.sum(~held.any(axis=1)) < 9       # some tokens are clipped, not all


def test_policy_matches_the_formula_in_torch():
    rng = np.random.default_rng(4)
    z, t, old, adv, ref = (torch.tensor(a) for a in tokens(rng, 12, 11))
    o = oracle.vocab.policy(z, t, old, adv, ref, **POLICY)
    live = t >= 0
    lp = torch.log_softmax(z / 1.4, 1).gather(1, t.clamp(min=0)[:, None])[:, 0]
    r = torch.exp(lp - old)
    loss = -torch.minimum(r * adv, r.clamp(0.8, 1.3) * adv) + 0.1 * (torch.exp(ref - lp) - (ref - lp) - 1)
    np.testing.assert_allclose(o["loss"], torch.where(live, loss, 0.0).numpy(), rtol=1e-11, atol=1e-13)
    np.testing.assert_allclose(o["logprob"], torch.where(live, lp, 0.0).numpy(), rtol=1e-11)


def test_policy_of_a_masked_token():
    z = np.array([[0.0, 1.0, -np.inf]])
    o = oracle.vocab.policy(z, [2], [-1.0], [1.0], None, 0.0, 0.2, 0.2, 1.0)
    assert o["logprob"][0] == -np.inf and o["loss"][0] == 0
    o = oracle.vocab.policy(z, [2], [-1.0], [-2.0], None, 0.0, 0.2, 0.2, 1.0)
    assert o["loss"][0] == pytest.approx(1.6)
    assert oracle.vocab.policy(z, [2], [-1.0], [1.0], [-1.0], 0.1, 0.2, 0.2, 1.0)["loss"][0] == np.inf
