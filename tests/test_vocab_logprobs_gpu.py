"""Token log probabilities, ranks, entropies and top tokens on the GPU against
the float64 definition.

Tolerances. Each number is a sum of at most V = 128000 positive fp32 terms,
taken per thread and then over threads (at most 2^10 roundings in a chain:
2^-14 at the very worst, under 2^-20 for roundings of either sign), one
logarithm and differences of numbers below 100: 1e-5 of the tensor's largest
finite magnitude (the bound of the fp32 paths here), whole numbers exactly."""

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


def close(got, ref, what):
    g, o = got.double().cpu().numpy(), np.asarray(ref, dtype=np.float64)
    assert g.shape == o.shape, what
    fin = np.isfinite(o)
    np.testing.assert_array_equal(g[~fin], o[~fin], err_msg=what)   # infinities and NaN in place
    if fin.any():
        err = np.max(np.abs(g[fin] - o[fin])) / max(np.max(np.abs(o[fin])), 1e-30)
        assert err <= 1e-5, f"{what}: {err:.2e}"


def check(z, t, T, K):
    lp, rank, ent, ids, top = tp.vocab_logprobs(z, t, T, top_k=K)
    lse = torch.empty(z.shape[0], device=dev())
    tp.tpmlp_vocab_logprobs(z, None, T, 0, lse=lse)
    torch.cuda.synchronize()
    o = oracle.vocab.logprobs(z, t, K)
    close(lp, o["logprob"], "logprob")
    close(ent, o["entropy"], "entropy")
    close(lse, o["lse"], "lse")
    np.testing.assert_array_equal(rank.cpu().numpy(), o["rank"])
    np.testing.assert_array_equal(ids.cpu().numpy(), o["top_ids"])
    if K:
        close(top, o["top_logprobs"], "top_logprobs")


def rows(N, V, dt, seed, ld=None, std=2.0):
    g = torch.Generator().manual_seed(seed)
    z = torch.zeros(N, ld or V, dtype=TYPES[dt])
    z[:, :V] = (torch.randn(N, V, generator=g) * std).to(TYPES[dt])
    z[:, V:] = 1000.0      # what stands between the rows must not matter
    t = torch.randint(0, V, (N,), generator=g)
    return z.to(dev())[:, :V], t.to(dev())


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("N,V,T,K,ld", [
    (1, 1, 1, 1, None), (3, 7, 7, 7, None), (1, 8, 2, 0, None), (5, 33, 3, 4, None), (2, 255, 1, 20, 256),
    (9, 1000, 8, 20, 1003), (4, 4099, 1, 128, 4099), (17, 9999, 9, 5, 10001), (3, 32000, 4, 1, 32001),
    (2, 50001, 7, 64, 50016), (1, 128000, 8, 20, None), (60, 16384, 16, 3, None), (2, 150001, 1, 40, None),
    (400, 2048, 2, 10, None), (1500, 515, 5, 2, 517), (1, 600064, 8, 33, None)])
def test_shapes(N, V, T, K, ld, dt):
    z, t = rows(N, V, dt, 100 + N + V, ld)
    check(z, t, T, K)


def test_result_does_not_depend_on_the_shards_or_the_batch():
    z, t = rows(6, 4096, "bf16", 7)
    a = tp.vocab_logprobs(z, t, 1, top_k=9)
    b = tp.vocab_logprobs(z, t, 8, top_k=9)
    for x, y in zip(a, b):
        assert torch.equal(x, y)
    big, tb = rows(700, 4096, "bf16", 8)
    big[11], tb[11] = z[3], t[3]
    c = tp.vocab_logprobs(big, tb, 8, top_k=9)
    np.testing.assert_array_equal(c[3][11].cpu(), a[3][3].cpu())
    assert c[1][11] == a[1][3]
    torch.testing.assert_close(c[0][11], a[0][3], rtol=2e-6, atol=2e-6)


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("V", [40, 3001, 64000])
def test_masks(V, dt):
    """Rows masked to a few tokens, to one, to none; masked by the type's
    lowest value; the target masked; every logit alike; rising and falling
    rows; large offsets."""
    K = 20
    z, t = rows(12, V, dt, V)
    keep = torch.zeros(V, dtype=torch.bool, device=dev())
    keep[[1, V // 2, V - 1]] = True
    z[0].masked_fill_(~keep, -INF)
    t[0] = V // 2
    z[1].fill_(-INF)
    z[1, V - 2] = -3.0
    t[1] = V - 2
    z[2].fill_(-INF)
    low = torch.finfo(TYPES[dt]).min
    z[3].masked_fill_(~keep, low)
    z[4].fill_(low)
    z[5, t[5]] = -INF
    z[6].fill_(1.25)
    z[7].copy_(torch.sort(z[7]).values)
    z[8].copy_(torch.sort(z[8], descending=True).values)
    z[9] = (z[9] + 3000.0).to(z.dtype)
    z[10, ::2] = 0.0
    z[10, 1::2] = -0.0       # equal: the index decides
    z[11].masked_fill_(torch.arange(V, device=dev()) % 97 != 5, -INF)
    check(z, t, 1, K)


@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_nan_and_positive_infinity_rows(dt):
    V = 5000
    z, t = rows(5, V, dt, 3)
    z[1, 77] = float("nan")
    z[2, 4000] = INF
    z[3].fill_(-INF)
    z[3, 5] = float("nan")
    lp, rank, ent, ids, top = tp.vocab_logprobs(z, t, 4, top_k=6)
    for n in (1, 2, 3):
        assert torch.isnan(lp[n]) and torch.isnan(ent[n]) and torch.isnan(top[n]).all()
        assert (ids[n] >= 0).all() and (ids[n] < V).all()
    o = oracle.vocab.logprobs(z[[0, 4]], t[[0, 4]], 6)
    close(lp[[0, 4]], o["logprob"], "logprob")
    np.testing.assert_array_equal(ids[[0, 4]].cpu(), o["top_ids"])
    assert tp.tpmlp_check_device_error() == 0


def test_bad_target_gives_nan_and_device_error():
    z, t = rows(4, 100, "bf16", 1)
    t[1], t[2] = 100, -1
    lp, rank, ent, ids, _ = tp.vocab_logprobs(z, t, 4, top_k=3)
    assert tp.tpmlp_check_device_error() == _binding.ERR_ARG
    assert torch.isnan(lp[1:3]).all() and (rank[1:3] == 0).all()
    o = oracle.vocab.logprobs(z, t, 3)
    close(ent, o["entropy"], "entropy")
    close(lp[[0, 3]], o["logprob"][[0, 3]], "logprob")
    np.testing.assert_array_equal(ids.cpu().numpy(), o["top_ids"])


def test_rows_beyond_32_bit_offsets():
    """2^31 elements and more in front of a row."""
    N, V = 17000, 128000
    z = torch.zeros(N, V, dtype=torch.bfloat16, device=dev())
    r = [0, 8000, 16776, 16778, N - 1]
    part, _ = rows(len(r), V, "bf16", 9)
    z[r] = part
    t = torch.arange(N, device=dev()) % V
    lp, rank, ent, ids, top = tp.vocab_logprobs(z, t, 8, top_k=4)
    o = oracle.vocab.logprobs(part, t[r], 4)
    close(lp[r], o["logprob"], "logprob")
    np.testing.assert_array_equal(ids[r].cpu().numpy(), o["top_ids"])
    np.testing.assert_array_equal(rank[r].cpu().numpy(), o["rank"])
    flat = torch.full((N,), -float(np.log(V)), device=dev())
    flat[r] = lp[r]
    torch.testing.assert_close(lp, flat, rtol=1e-5, atol=0)


def test_empty_batch_and_other_stream():
    z, t = rows(0, 64, "f32", 2)
    out = tp.vocab_logprobs(z, t, 4, top_k=3)
    assert out[0].numel() == 0 and out[3].shape == (0, 3)
    s = torch.cuda.Stream()
    z, t = rows(33, 7001, "f32", 4)
    ref = tp.vocab_logprobs(z, t, 1, top_k=5)
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        got = tp.vocab_logprobs(z, t, 1, top_k=5)
    s.synchronize()
    for a, b in zip(ref, got):
        assert torch.equal(a, b)


def test_refusals_on_the_device():
    z, t = rows(4, 12, "f32", 2)
    with pytest.raises(tp.TpmlpError) as e:
        tp.vocab_logprobs(z, t, 5)
    assert e.value.status == _binding.ERR_SHAPE
    with pytest.raises(tp.TpmlpError):
        tp.vocab_logprobs(z, t, 4, top_k=13)
    with pytest.raises(ValueError):
        tp.vocab_logprobs(z.t(), t, 4)
    with pytest.raises(ValueError):
        tp.vocab_logprobs(z, t[:2], 4)
    with pytest.raises(TypeError):
        tp.vocab_logprobs(z.half(), t, 4)
    with pytest.raises(TypeError):
        tp.vocab_logprobs(z, t.int(), 4)


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("V,T,ld,K", [
    (1, 1, None, 1), (5, 5, 7, 3), (40, 1, None, 20), (64, 2, None, 64), (515, 5, 517, 32), (1000, 8, None, 64),
    (1000, 8, 1001, 128), (4096, 1, None, 32), (8199, 3, 8201, 20), (8192, 2, None, 33), (16384, 4, None, 64),
    (16401, 3, None, 64), (20001, 3, 20004, 21), (20001, 3, None, 22), (40000, 8, None, 5), (33000, 8, None, 0)])
def test_many_rows(V, T, ld, K, dt):
    """More rows than the device holds CTAs at a time, of every size that has
    its own number of threads, with lists up to its limit; masks, equal logits
    and ordered rows among them."""
    N = 640
    z, t = rows(N, V, dt, V + K, ld)
    g = torch.Generator().manual_seed(V)
    some = (torch.rand(V, generator=g) < 0.7).to(dev())
    z[::6].masked_fill_(some, -INF)
    z[1::12] = -INF
    z[2::12] = 0.5
    z[3::12] = torch.finfo(TYPES[dt]).min
    z[4::12] = torch.sort(z[4::12], dim=1).values
    z[5::12] = torch.sort(z[5::12], dim=1, descending=True).values
    z[7::12, V // 2:] = -INF
    z[8::12] = (z[8::12] * 4).round()                 # many equal ones
    check(z, t, T, K)
