"""The less travelled paths of the vocabulary-side operators: lists whose
candidates crowd into few threads or one chunk, more equal or larger entries
than the candidate buffer holds, long teacher lists, CUDA graphs, and the
bounded waits of the weight-gradient launch."""

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
    tp.tpmlp_selftest_gemm_stall(0)
    tp.tpmlp_set_wait_timeout_ns(2_000_000_000)
    assert tp.tpmlp_check_device_error() == 0


def dev():
    return torch.device("cuda:0")


def exact_lists(z, K, rows):
    """ids of the first K by (logit down, index up) for some rows."""
    got = tp.vocab_logprobs(z, torch.zeros(z.shape[0], dtype=torch.int64, device=dev()), 1, top_k=K)
    o = oracle.vocab.logprobs(z[rows], torch.zeros(len(rows)), K)
    np.testing.assert_array_equal(got[3][rows].cpu().numpy(), o["top_ids"])
    fin = np.isfinite(o["top_logprobs"])
    g = got[4][rows].double().cpu().numpy()
    assert np.array_equal(np.isfinite(g), fin)
    if fin.any():
        assert np.max(np.abs(g[fin] - o["top_logprobs"][fin])) <= 1e-5 * max(1.0, np.max(np.abs(o["top_logprobs"][fin])))


# few rows go to clusters of CTAs, many to one CTA each: both splits
@pytest.mark.parametrize("N", [3, 620])
@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("K", [1, 20, 128])
def test_crowded_lists(N, dt, K):
    V = 40000
    g = torch.Generator().manual_seed(N + K)
    z = (torch.randn(N, V, generator=g) * 0.1 - 5).to(TYPES[dt])
    v = torch.arange(V)
    per = 8 if dt == "bf16" else 4                      # elements of a 16-byte vector
    z[0] = torch.where((v // per) % 256 < 100, z[0] + 9, z[0])   # 100 of a CTA's 256 threads hold what is large
    z[1] = torch.where((v // per) % 256 == 17, z[1] + 9, z[1])   # one of them, in every chunk
    z[2] = torch.where((v >= 20000) & (v < 20300), z[2] + 9, z[2])   # one stretch
    exact_lists(z.to(dev()), K, [0, 1, 2])


@pytest.mark.parametrize("N", [4, 620])
@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_more_equal_and_larger_entries_than_the_buffer(N, dt):
    V, K = 40000, 128
    g = torch.Generator().manual_seed(N)
    z = torch.randn(N, V, generator=g).to(TYPES[dt])
    z[0] = 3.0                                          # every entry equal
    z[1] = 1.0
    z[1, torch.randperm(V, generator=g)[:K - 5]] = 2.0  # fewer larger ones than K, the rest equal
    z[2] = -INF
    z[2, torch.randperm(V, generator=g)[:7]] = 0.5      # a mask that leaves seven
    per = 8 if dt == "bf16" else 4
    v = torch.arange(V)
    hi = (v // per) % 256 < K - 1                       # K - 1 threads hold thousands of distinct large entries
    z[3] = torch.where(hi, 100 + torch.randint(0, 120, (V,), generator=g).float(), torch.tensor(-1.0)).to(TYPES[dt])
    exact_lists(z.to(dev()), K, [0, 1, 2, 3])


@pytest.mark.parametrize("N,K", [(3, 129), (3, 1000), (700, 300)])
def test_long_teacher_lists_in_place(N, K):
    V, tau = 9000, 2.0
    g = torch.Generator().manual_seed(K)
    z = torch.randn(N, V, generator=g).to(torch.bfloat16).to(dev())
    ids = torch.stack([torch.randperm(V, generator=g)[:K] for _ in range(N)]).to(torch.int32)
    ids[0, ::3] = -1
    ids[1, 5:] = ids[1, :K - 5].clone()                 # repeats across the list
    ids[2, :-1] = -1                                    # the one live slot comes last
    ids, tl = ids.to(dev()), (torch.randn(N, K, generator=g) * 2).to(dev())
    rows = [0, 1, 2, N - 1]
    f = oracle.vocab.distill(z[rows], ids[rows], tl[rows], tau)
    d = oracle.vocab.distill_backward(z[rows], ids[rows], tl[rows], tau, 0.5)
    loss, _, lse, dz = tp.vocab_distill_with_grad(z, ids, tl, 1, temperature=tau, grad_scale=0.5, in_place=True)
    assert np.max(np.abs(loss[rows].double().cpu().numpy() - f["loss"])) <= 1e-5 * np.max(np.abs(f["loss"]))
    err = np.abs(dz[rows].double().cpu().numpy() - d)
    assert np.all(err <= 2.0 ** -8 * np.abs(d) + 1e-5 * np.max(np.abs(d)))


def test_captured_into_a_graph():
    """One training-like step of all operators captured and replayed: the bits
    of the calls made eagerly (every kernel's order of additions is fixed)."""
    N, V, H, K, T = 96, 4096, 64, 16, 4
    gen = torch.Generator(device=dev()).manual_seed(1)
    r = lambda *s: torch.randn(*s, generator=gen, device=dev()).to(torch.bfloat16)
    table = list(r(V, H).view(T, V // T, H))
    ids = torch.randint(0, V, (N,), generator=gen, device=dev())
    z, dout = r(N, V), r(N, H)
    W = {k: [r(H, 128) for _ in range(2)] for k in ("g", "u")}
    Wd, act = [r(128, H) for _ in range(2)], [[r(N, 128) for _ in range(2)] for _ in range(3)]

    def step():
        x = tp.vocab_embedding_scaled(ids, table, 3.0)
        lp = tp.vocab_logprobs(z, ids, T, top_k=K)
        kd = tp.vocab_distill_with_grad(z, lp[3], lp[4], T, temperature=2.0)
        two = tp.vocab_distill(z, lp[3], lp[4], T)
        back = tp.vocab_distill_backward(z, lp[3], lp[4], T, two[2])
        dE = tp.vocab_embedding_backward(ids, dout, V, T)
        gg = tp.swiglu_backward(x, W["g"], W["u"], Wd, *act, dout)
        return [x, *lp, *kd, *two, back, *dE, gg[0], *gg[1], *gg[2], *gg[3]]

    want = [t.clone() for t in step()]
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        step()
    torch.cuda.current_stream().wait_stream(s)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step()
    for t in got:
        t.zero_()
    graph.replay()
    torch.cuda.synchronize()
    for a, b in zip(got, want):
        assert torch.equal(a, b)


@pytest.mark.parametrize("role", [1, 2, 3])
def test_weight_gradient_launch_times_out_and_recovers(role):
    """The bounded waits of the few-token weight gradients, as for the GEMM: a
    role that stalls runs into the limit, the error word says so, and the next
    call gives the bits it gave before."""
    N, D, Fs, T = 16, 256, 512, 2
    gen = torch.Generator(device=dev()).manual_seed(2)
    r = lambda *s: torch.randn(*s, generator=gen, device=dev()).to(torch.bfloat16)
    Wg, Wu, Wd = [r(D, Fs) for _ in range(T)], [r(D, Fs) for _ in range(T)], [r(Fs, D) for _ in range(T)]
    X, dY = r(N, D), r(N, D)
    act = [[r(N, Fs) for _ in range(T)] for _ in range(3)]
    call = lambda: tp.swiglu_backward(X, Wg, Wu, Wd, *act, dY)
    want = call()
    torch.cuda.synchronize()
    tp.tpmlp_set_wait_timeout_ns(20_000_000)
    tp.tpmlp_selftest_gemm_stall(role)
    call()
    assert tp.tpmlp_check_device_error() == _binding.ERR_TIMEOUT
    tp.tpmlp_selftest_gemm_stall(0)
    tp.tpmlp_set_wait_timeout_ns(2_000_000_000)
    got = call()
    assert tp.tpmlp_check_device_error() == 0
    assert torch.equal(got[0], want[0])
    for i in (1, 2, 3):
        for a, b in zip(got[i], want[i]):
            assert torch.equal(a, b)
