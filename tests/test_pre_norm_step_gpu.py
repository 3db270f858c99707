"""One training step through the operators together, as they are used: layer norm,
the block's two halves onto the residual path, a last norm, the vocabulary head and
the policy loss, and the same way back; against the step in float64 by autograd.

Tolerance: every matrix in between is rounded to bf16 (2^-8 of itself) on the way
forward and back, eleven roundings deep, each on top of the others' propagated
errors: 16 2^-8 of a gradient's norm; fp32: the products' 1e-5."""

import numpy as np
import pytest
import torch

import tensor_transformer_mlp_columnparallel_gb300 as tp

pytestmark = pytest.mark.gpu
N, D, F, V, T = 96, 256, 512, 992, 4
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


@pytest.fixture(scope="module", autouse=True)
def _built():
    import __graft_entry__
    __graft_entry__.build()
    torch.cuda.set_device(0)
    yield
    assert tp.tpmlp_check_device_error() == 0


def parameters(dt):
    g = torch.Generator().manual_seed(1)
    r = lambda *s, std=1.0, base=0.0: (base + torch.randn(*s, generator=g) * std).to(TYPES[dt]).cuda()
    return dict(x=r(N, D), n1w=r(D, std=0.1, base=1.0), n1b=r(D, std=0.1), up=r(D, F, std=D ** -0.5),
                ub=r(F, std=0.1), down=r(F, D, std=F ** -0.5), db=r(D, std=0.1), n2w=r(D, std=0.1, base=1.0),
                n2b=r(D, std=0.1), head=r(D, V, std=2 * D ** -0.5))


def shards(w, dim):
    return [s.contiguous() for s in w.chunk(T, dim=dim)]


def step(p, t, old, adv, ref):
    up, down, head, ub = shards(p["up"], 1), shards(p["down"], 0), shards(p["head"], 1), shards(p["ub"], 0)
    h1, m1, r1 = tp.layernorm(p["x"], p["n1w"], p["n1b"])
    a, z = tp.column_linear(h1, up, ub, act="gelu_tanh", save_z=True)
    x2 = tp.row_linear(a, down, p["db"], residual=p["x"])
    h2, m2, r2 = tp.layernorm(x2, p["n2w"], p["n2b"])
    logits, _ = tp.column_linear(h2, head)
    loss, mean, lp, kl, dz = tp.vocab_policy_with_grad(logits, t, old, adv, T, ref_logprobs=ref, kl_coef=0.1,
                                                       grad_scale=1.0 / N, in_place=True)
    dh2, dhead, _ = tp.column_linear_backward(h2, head, dz)
    dx2, dn2w, dn2b = tp.layernorm_backward(dh2, x2, p["n2w"], m2, r2)
    da, ddown, ddb = tp.row_linear_backward(a, down, dx2, bias_grads=True)
    dh1, dup, dub = tp.column_linear_backward(h1, up, da, Z=z, act="gelu_tanh", bias_grads=True)
    dx, dn1w, dn1b = tp.layernorm_backward(dh1, p["x"], p["n1w"], m1, r1, dresidual=dx2)
    return mean, lp, dict(x=dx, n1w=dn1w, n1b=dn1b, up=torch.cat(dup, 1), ub=torch.cat(dub), down=torch.cat(ddown, 0),
                          db=ddb, n2w=dn2w, n2b=dn2b, head=torch.cat(dhead, 1))


def in_64_bits(p, t, old, adv, ref):
    q = {k: v.double().requires_grad_() for k, v in p.items()}
    f = torch.nn.functional
    h1 = f.layer_norm(q["x"], (D,), q["n1w"], q["n1b"])
    x2 = f.gelu(h1 @ q["up"] + q["ub"], approximate="tanh") @ q["down"] + q["db"] + q["x"]
    z = f.layer_norm(x2, (D,), q["n2w"], q["n2b"]) @ q["head"]
    live = t >= 0
    lp = torch.log_softmax(z, 1).gather(1, t.clamp(min=0)[:, None])[:, 0]
    r, k = torch.exp(lp - old), ref.double() - lp
    each = -torch.minimum(r * adv, r.clamp(0.8, 1.2) * adv) + 0.1 * (torch.expm1(k) - k)
    mean = torch.where(live, each, 0.0).sum() / N
    return mean, torch.where(live, lp, 0.0), dict(zip(q, torch.autograd.grad(mean, list(q.values()))))


def tokens(p):
    g = torch.Generator().manual_seed(2)
    t = torch.randint(0, V, (N,), generator=g).cuda()
    t[::7] = -1
    zero = torch.zeros(N, device="cuda")
    lp = in_64_bits(p, t, zero, zero, zero)[1]
    # ratios of 1.0 and 1.5, well away from the borders
    move = torch.where(torch.arange(N, device="cuda") % 2 == 0, 0.0, -0.4)
    return t, (lp + move).float(), torch.randn(N, generator=g).cuda(), (lp + 0.3).float()


@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_step_against_autograd(dt):
    p = parameters(dt)
    data = tokens(p)
    mean, lp, grads = step(p, *data)
    want_mean, want_lp, want = in_64_bits(p, *data)
    lim = 16 * 2.0 ** -8 if dt == "bf16" else 1e-5
    assert abs(float(mean) - float(want_mean)) <= lim * (1 + abs(float(want_mean)))
    assert float((lp.double() - want_lp).abs().max()) <= lim * 8
    for k, g in grads.items():
        assert g.shape == p[k].shape and g.dtype == p[k].dtype
        off = float((g.double() - want[k]).norm() / want[k].norm())
        assert off <= lim, f"{k}: {off:.2e}"


def test_captured_step_beside_an_eager_one():
    """Two captured steps and an eager one, each with its own memory, replayed in turn."""
    p = parameters("bf16")
    data = tokens(p)
    want = step(p, *data)
    graphs = []
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            held = step(p, *data)
        graphs.append((g, held))
    for g, _ in graphs:
        g.replay()
    eager = step(p, *data)
    for g, _ in graphs:
        g.replay()
    torch.cuda.synchronize()
    for got in (eager, *(h for _, h in graphs)):
        assert torch.equal(got[0], want[0])
        for k in want[2]:
            assert torch.equal(got[2][k], want[2][k]), k


def test_two_streams_at_once():
    p = parameters("bf16")
    data = tokens(p)
    want = step(p, *data)
    streams = [torch.cuda.Stream() for _ in range(3)]
    torch.cuda.synchronize()
    got = []
    for _ in range(3):
        for s in streams:
            with torch.cuda.stream(s):
                got.append(step(p, *data))
    torch.cuda.synchronize()
    for g in got:
        for k in want[2]:
            assert torch.equal(g[2][k], want[2][k]), k
