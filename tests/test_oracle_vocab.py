"""The float64 definitions of the vocabulary-side operators and of the gated
block's gradients, against central differences and torch in float64."""

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


@pytest.mark.parametrize("tau", [1.0, 2.5])
def test_distill_gradient_against_differences(tau):
    rng = np.random.default_rng(3)
    z = rng.normal(size=(4, 11))
    ids = np.array([[2, 7, 0], [5, -1, -1], [-1, -1, -1], [4, 4, 9]])   # short, empty, repeated
    tl = rng.normal(size=(4, 3)) * 2
    tl[0, 1] = -np.inf
    g = rng.normal(size=4)
    num = differences(lambda q: float(np.sum(g * oracle.vocab.distill(q, ids, tl, tau)["loss"])), z)
    np.testing.assert_allclose(oracle.vocab.distill_backward(z, ids, tl, tau, g), num, atol=2e-8)
    assert not num[2].any()


def test_distill_matches_torch_kl():
    rng = np.random.default_rng(4)
    z, tau = rng.normal(size=(5, 9)), 1.7
    ids = np.stack([rng.permutation(9)[:4] for _ in range(5)])
    tl = rng.normal(size=(5, 4))
    lp = torch.log_softmax(torch.tensor(z) / tau, 1).gather(1, torch.tensor(ids))
    lq = torch.log_softmax(torch.tensor(tl) / tau, 1)
    ref = tau ** 2 * torch.nn.functional.kl_div(lp, lq, reduction="none", log_target=True).sum(1)
    np.testing.assert_allclose(oracle.vocab.distill(z, ids, tl, tau)["loss"], ref.numpy(), rtol=1e-12)


def test_logprobs_against_torch_and_by_hand():
    rng = np.random.default_rng(5)
    z = rng.normal(size=(6, 13)) * 3
    t = rng.integers(0, 13, 6)
    o = oracle.vocab.logprobs(z, t, 4)
    ref = torch.log_softmax(torch.tensor(z), 1)
    np.testing.assert_allclose(o["logprob"], ref.gather(1, torch.tensor(t)[:, None])[:, 0], rtol=1e-12)
    np.testing.assert_allclose(o["entropy"], torch.distributions.Categorical(logits=torch.tensor(z)).entropy(),
                               rtol=1e-12)
    np.testing.assert_array_equal(o["top_ids"], torch.topk(torch.tensor(z), 4).indices)
    # ties go to the lowest index; masked tokens have probability 0
    o = oracle.vocab.logprobs(np.array([[1.0, 2.0, 2.0, -np.inf, 1.0]]), [4], 5)
    assert list(o["top_ids"][0]) == [1, 2, 0, 4, 3] and o["rank"][0] == 4
    assert o["top_logprobs"][0, 4] == -np.inf
    # a row that the mask leaves empty
    o = oracle.vocab.logprobs(np.full((1, 4), -np.inf), [2], 2)
    assert o["lse"][0] == -np.inf and o["logprob"][0] == -np.inf and o["entropy"][0] == 0.0
    assert list(o["top_ids"][0]) == [0, 1] and o["rank"][0] == 3


def test_embedding_gradient_against_differences():
    rng = np.random.default_rng(6)
    E, dout = rng.normal(size=(5, 3)), rng.normal(size=(7, 3))
    ids = np.array([4, 0, 4, 4, 9, 2, -1])
    f = lambda q: float(np.sum(dout * 1.5 * oracle.embedding.vocab_embedding(ids, q)))
    np.testing.assert_allclose(oracle.vocab.embedding_backward(ids, dout, 5, 1.5), differences(f, E),
                               atol=1e-8)


def test_gated_gradients_against_differences():
    rng = np.random.default_rng(7)
    X, dY = rng.normal(size=(3, 4)), rng.normal(size=(3, 4))
    Wg, Wu, Wd = rng.normal(size=(4, 6)), rng.normal(size=(4, 6)), rng.normal(size=(6, 4))
    f = oracle.mlp.swiglu_forward(X, Wg, Wu, Wd)
    g = oracle.mlp.swiglu_backward(X, Wg, Wu, Wd, f["H"], f["G"], f["U"], dY)
    y = lambda **k: float(np.sum(dY * oracle.mlp.swiglu_forward(**{**dict(X=X, Wg=Wg, Wu=Wu, Wd=Wd), **k})["Y"]))
    for name in ("X", "Wg", "Wu", "Wd"):
        num = differences(lambda q: y(**{name: q}), dict(X=X, Wg=Wg, Wu=Wu, Wd=Wd)[name])
        np.testing.assert_allclose(g["d" + name], num, atol=3e-8, err_msg=name)
