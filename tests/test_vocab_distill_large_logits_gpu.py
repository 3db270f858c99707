"""Distillation of rows whose logits lie far from zero: a common offset, equal
tokens at the type's lowest value, masks beside them. Loss and gradient, in
one call and in two, against the float64 definition of the same logits.

Tolerances, row by row. Only differences of logits enter p, and those are
rounded once (2^-24 of the difference, which the softmax's exponent divides by
tau): 1e-5 of the row's largest magnitude as for any other row, and a bf16
gradient's own rounding of 2^-8 |d|. lse itself is one fp32 number, 2^-23 of
its magnitude at best: 1e-5 of it."""

import numpy as np
import pytest
import torch

import oracle
import tensor_transformer_mlp_columnparallel_gb300 as tp

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


def rows_of(V, K, dt, seed):
    """Logits [9, V], their teacher's lists, weights; the last four rows hold no
    value but the type's lowest, -1e9 and masks."""
    g = torch.Generator().manual_seed(seed)
    t = TYPES[dt]
    z = (torch.randn(9, V, generator=g) * 2).float()
    ids = torch.stack([torch.randperm(V, generator=g)[:K] for _ in range(9)])
    for n, offset in enumerate((300.0, 3000.0, -1.0e4, 30000.0, -3.0e4)):
        z[n] += offset
    lowest = torch.finfo(t).min
    z[5] = -1.0e9
    z[6] = lowest
    z[7] = lowest
    z[7, torch.randperm(V, generator=g)[:V // 2]] = -INF
    z[8] = -INF
    z[8, ids[8]] = lowest
    tl = torch.randn(9, K, generator=g) * 2 + 5
    w = torch.rand(9, generator=g) + 0.5
    live = ~torch.isinf(z.to(t)).gather(1, ids)         # a masked token is not the teacher's
    ids = torch.where(live, ids, torch.full_like(ids, -1))
    return [x.cuda() for x in (z.to(t), ids.to(torch.int32), tl, w)]


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("tau", [0.5, 1.0, 1.5])
# a few rows over clusters of CTAs, many rows of one CTA each, and rows longer
# than a cluster keeps on chip
@pytest.mark.parametrize("V,copies", [(2500, 1), (9000, 1), (2500, 80), (30011, 1), (300007, 1)])
def test_offsets_and_lowest_values(V, copies, tau, dt):
    z, ids, tl, w = rows_of(V, 12, dt, V)
    f = oracle.vocab.distill(z, ids, tl, tau)
    dref = oracle.vocab.distill_backward(z, ids, tl, tau, 0.25 * w.double().cpu().numpy())
    z, ids, tl, w = [torch.cat([x] * copies) for x in (z, ids, tl, w)]
    loss, _, lse = tp.vocab_distill(z, ids, tl, 1, temperature=tau)
    kw = dict(temperature=tau, grad_scale=0.25, grad_tokens=w)
    d = tp.vocab_distill_backward(z, ids, tl, 1, lse, **kw)
    loss1, _, lse1, d1 = tp.vocab_distill_with_grad(z, ids, tl, 1, **kw)
    held = z.clone()
    tp.vocab_distill_backward(held, ids, tl, 1, lse, in_place=True, **kw)
    own = 2.0 ** -8 if dt == "bf16" else 0.0
    for n in (*range(9), *range(9 * copies - 9, 9 * copies)):
        ref, at = dref[n % 9], f["loss"][n % 9]
        for x, what in ((d, "two calls"), (d1, "one call"), (held, "in place")):
            err = np.abs(x[n].double().cpu().numpy() - ref) - own * np.abs(ref)
            assert np.max(err) <= 1e-5 * np.max(np.abs(ref)), (what, n, np.max(err) / np.max(np.abs(ref)))
        for x in (loss, loss1):
            assert abs(float(x[n]) - at) <= 1e-5 * max(1.0, abs(at)), (n, float(x[n]), at)
        if abs(f["lse"][n % 9]) < 3.4e38:       # the lowest value over tau = 0.5 has no fp32 number
            for x in (lse, lse1):
                assert abs(float(x[n]) - f["lse"][n % 9]) <= 1e-5 * max(1.0, abs(f["lse"][n % 9]))
    assert torch.equal(held, d)


@pytest.mark.parametrize("dt,far", [("f32", 32.0), ("bf16", 512.0)])
@pytest.mark.parametrize("copies", [1, 160])
def test_both_sides_of_the_lse_that_is_taken_as_it_is(copies, dt, far):
    """Up to |lse| = 32 (fp32 logits; 512 for bf16) p comes from lse, whose
    rounding is 2^-24 |lse| of p at most: 2^-19 and 2^-15. Beyond, from the row.
    fp32 p to 2^-18 (its exponent, |ln p| <= 12, is rounded twice, 12 2^-23),
    bf16 d to 2^-8 |d| + 2^-14 max |d|."""
    V, tau = 6007, 1.25
    g = torch.Generator().manual_seed(17)
    z = torch.randn(4, V, generator=g) * 0.5
    lse = torch.logsumexp(z.double() / tau, 1)
    want = torch.tensor([0.97 * far, 1.03 * far, -0.97 * far, -1.03 * far]).double()
    z = (z + ((want - lse) * tau)[:, None]).to(TYPES[dt])
    ids = torch.stack([torch.randperm(V, generator=g)[:6] for _ in range(4)]).to(torch.int32)
    tl = torch.randn(4, 6, generator=g)
    dref = oracle.vocab.distill_backward(z, ids, tl, tau, 1.0)
    z, ids, tl = [torch.cat([x] * copies).cuda() for x in (z, ids, tl)]
    lse = tp.vocab_distill(z, ids, tl, 1, temperature=tau)[2]
    assert [bool(abs(float(x)) > far) for x in lse[:4]] == [False, True, False, True]
    d = tp.vocab_distill_backward(z, ids, tl, 1, lse, temperature=tau)
    for n in range(4):
        got = d[4 * copies - 4 + n].double().cpu().numpy()
        err, big = np.abs(got - dref[n]), np.max(np.abs(dref[n]))
        if dt == "f32":
            tok = np.ones(V, dtype=bool)
            tok[ids[n].cpu().numpy()] = False                 # p alone
            assert np.max(err[tok] / dref[n][tok]) <= 2.0 ** -18
            assert np.max(err) <= 2.0 ** -18 * big
        else:
            assert np.max(err - 2.0 ** -8 * np.abs(dref[n])) <= 2.0 ** -14 * big
