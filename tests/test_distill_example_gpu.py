"""The distillation example: its loss falls, and one step's gradients agree
with torch autograd of the same model in float64 (bf16 storage and products:
the block's normwise bound of 2e-2, doubled for the two bf16 roundings of the
head's products in front of it)."""

import os
import sys

import numpy as np
import pytest
import torch

import tensor_transformer_mlp_columnparallel_gb300 as tp
from tests.tolerance import normwise_rel_err

pytestmark = pytest.mark.gpu
sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))


@pytest.fixture(scope="module", autouse=True)
def _built():
    import __graft_entry__
    __graft_entry__.build()
    torch.cuda.set_device(0)
    yield
    assert tp.tpmlp_check_device_error() == 0


def test_the_loss_falls():
    import distill_gated_block as ex
    losses, before, after = ex.distil(steps=30, tokens=256)
    assert all(np.isfinite(losses))
    thirds = [np.mean(losses[i:i + 10]) for i in (0, 10, 20)]
    assert thirds[0] > thirds[1] > thirds[2]
    assert after[0] > before[0]      # the teacher's answers became likelier


def test_one_step_against_autograd():
    import distill_gated_block as ex
    V, D, F, T, N, K, tau = 1024, 64, 256, 4, 96, 12, 1.5
    m = ex.BlockLM(V, D, F, T, 3)
    g = torch.Generator(device="cuda").manual_seed(4)
    ids = torch.randint(0, V, (N,), generator=g, device="cuda")
    top = torch.stack([torch.randperm(V, generator=g, device="cuda")[:K] for _ in range(N)]).to(torch.int32)
    tl = torch.randn(N, K, generator=g, device="cuda")
    logits, saved = m.forward(ids)
    loss, mean, _, dlogits = tp.vocab_distill_with_grad(logits, top, tl, T, temperature=tau, grad_scale=1.0 / N)
    dE, dWg, dWu, dWd = m.backward(dlogits, saved)

    P = [t.double().requires_grad_() for t in (m.E, torch.cat(m.Wg, 1), torch.cat(m.Wu, 1), torch.cat(m.Wd, 0))]
    E, Wg, Wu, Wd = P
    x = E[ids] * m.scale
    h = x + (torch.nn.functional.silu(x @ Wg) * (x @ Wu)) @ Wd
    lp = torch.log_softmax(h @ E.t() / tau, 1).gather(1, top.long())
    lq = torch.log_softmax(tl.double() / tau, 1)
    ref = (tau ** 2 * (lq.exp() * (lq - lp)).sum(1)).mean()
    ref.backward()
    ref = float(ref.detach())
    assert abs(float(mean) - ref) <= 2e-2 * abs(ref)
    for got, want, name in ((dE, E, "dE"), (torch.cat(dWg, 1), Wg, "dWg"), (torch.cat(dWu, 1), Wu, "dWu"),
                            (torch.cat(dWd, 0), Wd, "dWd")):
        err = normwise_rel_err(got, want.grad.cpu().numpy())
        assert err <= 4e-2, (name, err)
