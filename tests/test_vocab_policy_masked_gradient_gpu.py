"""The policy loss's gradient of masked tokens with a KL term: where the loss is
infinite, no gradient of the row is finite, in one call and in two, in place and
not; without a KL term it is 0 or as the definition has it, and rows beside are as
they are alone."""

import pytest
import torch

import tensor_transformer_mlp_columnparallel_gb300 as tp
from tests.test_vocab_policy_gpu import INF, dev, make

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    import __graft_entry__
    __graft_entry__.build()
    torch.cuda.set_device(0)
    yield
    assert tp.tpmlp_check_device_error() == 0


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("N,V", [(8, 2500), (8, 1), (9, 7), (640, 2048), (8, 50001)])
def test_rows_with_an_infinite_loss(N, V, dt):
    z, t, old, adv, ref, w = make(N, V, dt, 7)
    kw = dict(ref_logprobs=ref, kl_coef=0.1, grad_tokens=w)
    clean = tp.vocab_policy_with_grad(z, t, old, adv, 1, **kw)
    masked = [2, 4, 5]
    adv[masked] = torch.tensor([1.0, -1.0, 0.0], device=dev())
    z[2, t[2]] = -INF                 # the token alone (V = 1: the row)
    z[4].fill_(-INF)                  # everything
    z[5].fill_(-INF)                  # everything, no advantage
    keep = z.clone()
    loss, _, lp, kl, d = tp.vocab_policy_with_grad(z, t, old, adv, 1, **kw)
    d2 = tp.vocab_policy_backward(z, t, old, adv, 1, lp, **kw)
    assert torch.equal(z.view(torch.uint8), keep.view(torch.uint8))
    in1, in2 = z.clone(), z.clone()
    tp.vocab_policy_with_grad(in1, t, old, adv, 1, **kw, in_place=True)
    tp.vocab_policy_backward(in2, t, old, adv, 1, lp, **kw, in_place=True)
    assert (loss[masked] == INF).all() and (kl[masked] == INF).all() and (lp[masked] == -INF).all()
    for got in (d, d2, in1, in2):
        assert not torch.isfinite(got[masked]).any()
    rest = [n for n in range(N) if n not in masked]
    assert torch.equal(d[rest], clean[4][rest]) and torch.equal(in1[rest], clean[4][rest])
    assert torch.isfinite(d2[rest]).all() and torch.isfinite(in2[rest]).all()
    # nothing infinite without the KL term: these rows have no slope
    kw = dict(ref_logprobs=ref, kl_coef=0.0, grad_tokens=w)
    loss, _, lp, _, d = tp.vocab_policy_with_grad(z, t, old, adv, 1, **kw)
    d2 = tp.vocab_policy_backward(z, t, old, adv, 1, lp, **kw)
    assert torch.isfinite(loss).all() and not d[masked].any() and not d2[masked].any()
