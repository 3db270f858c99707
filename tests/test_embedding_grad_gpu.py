"""Scaled embedding lookup and the table's gradient on the GPU against the
float64 definition.

Tolerances. The lookup rounds one fp32 product: 2^-24 (fp32) or 2^-24 + 2^-9
(bf16) of each element: 2^-23 and 2^-8. A gradient is a sum of n fp32 terms
(n the tokens of one id): at most n 2^-24 sum |terms|, elementwise, then
2^-9 of itself for bf16."""

import numpy as np
import pytest
import torch

import oracle
import tensor_transformer_mlp_columnparallel_gb300 as tp
from tensor_transformer_mlp_columnparallel_gb300 import _binding

pytestmark = pytest.mark.gpu
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


@pytest.fixture(scope="module", autouse=True)
def _built():
    import __graft_entry__
    __graft_entry__.build()
    torch.cuda.set_device(0)
    yield
    assert tp.tpmlp_check_device_error() == 0


def dev():
    return torch.device("cuda:0")


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("N,V,H,T", [(1, 4, 1, 1), (5, 12, 3, 3), (33, 100, 64, 4), (257, 1000, 1030, 8),
                                     (1000, 64, 8, 16), (16, 640, 8200, 2), (3000, 77, 127, 7)])
def test_scaled_lookup(N, V, H, T, dt):
    g = torch.Generator().manual_seed(N + H)
    E = torch.randn(V, H, generator=g).to(TYPES[dt])
    ids = torch.randint(0, V, (N,), generator=g)
    table = [s.contiguous().to(dev()) for s in E.chunk(T)]
    scale = 1.7
    out = tp.vocab_embedding_scaled(ids.to(dev()), table, scale)
    ref = np.float64(np.float32(scale)) * oracle.embedding.vocab_embedding(ids, E)
    err = np.abs(out.double().cpu().numpy() - ref) - np.abs(ref) * (2.0 ** -8 if dt == "bf16" else 2.0 ** -23)
    assert err.max() <= 0
    one = tp.vocab_embedding_scaled(ids.to(dev()), table, 1.0)
    assert torch.equal(one, tp.vocab_embedding(ids.to(dev()), table))


def test_scaled_lookup_bad_ids_views_and_empty():
    E = torch.randn(40, 24, device=dev())
    ids = torch.tensor([3, -1, 40, 39, 1 << 40], device=dev())
    out = tp.vocab_embedding_scaled(ids, [E[:20], E[20:]], 2.0)
    assert tp.tpmlp_check_device_error() == _binding.ERR_ARG
    np.testing.assert_array_equal(out[[1, 2, 4]].cpu(), np.zeros((3, 24)))
    assert torch.equal(out[0], 2 * E[3]) and torch.equal(out[3], 2 * E[39])
    assert tp.vocab_embedding_scaled(ids[:0], [E], 2.0).shape == (0, 24)
    # table shards that start off a 16-byte boundary
    flat = torch.randn(1 + 40 * 24, device=dev())
    odd = flat[1:].view(40, 24)
    assert torch.equal(tp.vocab_embedding_scaled(ids[:1], [odd], 0.5)[0], 0.5 * odd[3])


def tokens(N, V, kind, seed):
    g = torch.Generator().manual_seed(seed)
    if kind == "flat":
        return torch.randint(0, V, (N,), generator=g)
    if kind == "one":
        return torch.full((N,), V // 2)
    if kind == "last":
        return torch.where(torch.rand(N, generator=g) < 0.9, torch.full((N,), V - 1),
                           torch.randint(0, V, (N,), generator=g))
    if kind == "pair":     # two long runs and what lies between
        return torch.cat([torch.zeros(N // 2, dtype=torch.int64), torch.full((N - N // 2,), V - 1)])
    u = torch.rand(N, generator=g, dtype=torch.float64)
    return (torch.exp(u * np.log(V + 1.0)) - 1).long().clamp(max=V - 1)


def check(ids, dout, V, T, scale, gdt, into=None):
    base = None if into is None else torch.cat([t.double().cpu() for t in into]).numpy()
    d = tp.vocab_embedding_backward(ids.to(dev()), dout.to(dev()), V, T, scale=scale,
                                    grad_dtype=TYPES[gdt], accumulate_into=into)
    torch.cuda.synchronize()
    got = torch.cat([t.double().cpu() for t in d]).numpy()
    ref = oracle.vocab.embedding_backward(ids, dout, V, scale)
    mag = oracle.vocab.embedding_backward(ids, dout.abs(), V, abs(scale))
    n = np.bincount(ids[(ids >= 0) & (ids < V)].numpy(), minlength=V)[:, None]
    lim = (n + 2) * 2.0 ** -24 * mag
    if base is not None:
        ref = ref + base
        lim = lim + 2.0 ** -23 * np.abs(base)
        np.testing.assert_array_equal(got[n[:, 0] == 0], base[n[:, 0] == 0])
    else:
        assert not got[n[:, 0] == 0].any()
    if gdt == "bf16":
        lim = lim * 1.01 + 2.0 ** -8 * np.abs(ref)
    assert np.all(np.abs(got - ref) <= lim)


@pytest.mark.parametrize("dt,gdt", [("bf16", "f32"), ("bf16", "bf16"), ("f32", "f32"), ("f32", "bf16")])
@pytest.mark.parametrize("N,V,H,T,kind", [
    (1, 1, 1, 1, "flat"), (1, 9, 8, 3, "flat"), (2, 600, 16, 2, "one"), (31, 7, 33, 7, "flat"),
    (64, 4, 64, 2, "flat"), (65, 100, 8, 1, "one"), (257, 512, 1030, 8, "zipf"), (511, 511, 40, 7, "pair"),
    (1000, 513, 128, 9, "last"), (4096, 1000, 24, 8, "zipf"), (4097, 600, 72, 6, "one"),
    (9000, 128000, 16, 8, "zipf"), (20000, 300, 8, 3, "last"), (3000, 270000, 8, 2, "flat"),
    (129, 33, 5000, 3, "zipf"), (70000, 50, 16, 1, "zipf"), (300, 2, 2056, 2, "pair")])
def test_table_gradient(N, V, H, T, kind, dt, gdt):
    g = torch.Generator().manual_seed(N + V)
    check(tokens(N, V, kind, N), torch.randn(N, H, generator=g).to(TYPES[dt]), V, T, 1.5, gdt)


@pytest.mark.parametrize("gdt", ["f32", "bf16"])
def test_accumulate_and_repeat(gdt):
    N, V, H, T = 2000, 900, 136, 3
    ids = tokens(N, V, "last", 3)
    dout = torch.randn(N, H, generator=torch.Generator().manual_seed(1)).to(torch.bfloat16)
    start = [torch.randn(V // T, H, device=dev()).to(TYPES[gdt]) for _ in range(T)]
    check(ids, dout, V, T, 2.0, gdt, into=[s.clone() for s in start])
    a = tp.vocab_embedding_backward(ids.to(dev()), dout.to(dev()), V, T, accumulate_into=[s.clone() for s in start])
    b = tp.vocab_embedding_backward(ids.to(dev()), dout.to(dev()), V, T, accumulate_into=[s.clone() for s in start])
    for x, y in zip(a, b):
        assert torch.equal(x, y)      # the same bits on every run


def test_bad_ids_drop_out_and_are_reported():
    ids = torch.tensor([0, 5, -1, 6, 5, 1 << 33, 2])
    dout = torch.randn(7, 40)
    check(ids, dout, 6, 2, 1.0, "f32")
    assert tp.tpmlp_check_device_error() == _binding.ERR_ARG
    check(torch.tensor([-5, 6, 7]), dout[:3], 6, 2, 1.0, "f32")     # nothing but bad ids
    assert tp.tpmlp_check_device_error() == _binding.ERR_ARG


def test_no_tokens():
    ids, dout = torch.empty(0, dtype=torch.int64), torch.empty(0, 16)
    check(ids, dout, 10, 2, 1.0, "f32")
    start = [torch.randn(5, 16, device=dev()) for _ in range(2)]
    check(ids, dout, 10, 2, 1.0, "f32", into=start)


def test_nan_stays_in_its_row():
    ids = torch.tensor([1, 2, 1, 3])
    dout = torch.randn(4, 64)
    dout[2, 5] = float("nan")
    d = torch.cat(tp.vocab_embedding_backward(ids.to(dev()), dout.to(dev()), 4, 2))
    assert torch.isnan(d[1, 5]) and int(torch.isnan(d).sum()) == 1


def test_odd_alignment_and_other_stream():
    flat = torch.randn(1 + 50 * 24, device=dev())
    dout = flat[1:].view(50, 24)
    ids = tokens(50, 12, "flat", 1)
    check(ids, dout.cpu(), 12, 2, 1.0, "f32")
    ref = tp.vocab_embedding_backward(ids.to(dev()), dout, 12, 2)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        got = tp.vocab_embedding_backward(ids.to(dev()), dout, 12, 2)
    s.synchronize()
    for a, b in zip(ref, got):
        assert torch.equal(a, b)


def test_gradient_matches_the_lookup():
    """<dout, lookup(E)> is linear in E with gradient dE: its difference over a
    step D is <dE, D>, for whole numbers exactly."""
    V, H, T, N = 50, 40, 5, 300
    g = torch.Generator().manual_seed(2)
    E = torch.randint(-4, 5, (V, H), generator=g).float()
    D = torch.randint(-4, 5, (V, H), generator=g).float()
    ids = tokens(N, V, "zipf", 5).to(dev())
    dout = torch.randint(-4, 5, (N, H), generator=g).float().to(dev())
    sh = lambda M: [s.contiguous().to(dev()) for s in M.chunk(T)]
    f = lambda M: float((dout.double() * tp.vocab_embedding_scaled(ids, sh(M), 2.0).double()).sum())
    dE = torch.cat(tp.vocab_embedding_backward(ids, dout, V, T, scale=2.0)).cpu()
    assert f(E + D) - f(E) == float((dE.double() * D.double()).sum())


@pytest.mark.parametrize("dt,gdt", [("bf16", "f32"), ("f32", "bf16")])
@pytest.mark.parametrize("kind", ["zipf", "last", "one"])
def test_wide_rows_joined_by_few_ctas(kind, dt, gdt):
    # more columns than a block's joining CTAs take at a time
    N, V, H, T = 8300, 40, 1300, 2
    g = torch.Generator().manual_seed(5)
    check(tokens(N, V, kind, 5), torch.randn(N, H, generator=g).to(TYPES[dt]), V, T, 0.5, gdt)


def test_wrong_shards_are_refused():
    ids = torch.zeros(3, dtype=torch.int64, device=dev())
    E = [torch.zeros(4, 8, device=dev()), torch.zeros(3, 8, device=dev())]
    launches = tp.tpmlp_launch_count()
    with pytest.raises(ValueError):
        tp.vocab_embedding_scaled(ids, E, 1.0)
    with pytest.raises(ValueError):
        tp.vocab_embedding_backward(ids, torch.zeros(3, 8, device=dev()), 8, 2, accumulate_into=E)
    with pytest.raises(TypeError):
        tp.vocab_embedding_scaled(ids, [E[0], E[0].bfloat16()], 1.0)
    assert tp.tpmlp_launch_count() == launches


@pytest.mark.parametrize("dt,gdt", [("bf16", "f32"), ("f32", "bf16")])
@pytest.mark.parametrize("N,V,H,kind", [
    (2049, 9000, 2056, "zipf"), (8192, 9000, 2056, "last"), (4100, 33000, 1030, "flat"),
    (65536, 700, 8, "zipf"), (65537, 700, 8, "zipf"), (5000, 7, 3200, "one"), (65000, 270000, 8, "flat")])
def test_sorted_by_several_ctas(N, V, H, kind, dt, gdt):
    """Tables large enough for the sort over several CTAs at few tokens, and its
    two tile sizes."""
    g = torch.Generator().manual_seed(N)
    check(tokens(N, V, kind, N), torch.randn(N, H, generator=g).to(TYPES[dt]), V, 1, 1.5, gdt)
