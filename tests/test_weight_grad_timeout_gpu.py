"""The bounded waits of the gated backward's few-token weight-gradient launch,
stalled by itself: the GEMMs before and after it run as ever, so the error
word's timeout is this launch's, and dX keeps its bits."""

import time

import pytest
import torch

import tensor_transformer_mlp_columnparallel_gb300 as tp
from tensor_transformer_mlp_columnparallel_gb300 import _binding

LIMIT_NS, DEFAULT_NS = 20_000_000, 2_000_000_000


@pytest.fixture(scope="module", autouse=True)
def _built():
    import __graft_entry__
    __graft_entry__.build()
    yield
    tp.tpmlp_selftest_weight_grad_stall(0)


def test_role_is_checked():
    lib = _binding.lib()
    assert lib.tpmlp_selftest_weight_grad_stall(4) == _binding.ERR_ARG
    assert lib.tpmlp_selftest_weight_grad_stall(-1) == _binding.ERR_ARG
    for role in (1, 2, 3, 0):
        assert lib.tpmlp_selftest_weight_grad_stall(role) == _binding.OK


# one k-block with what rounding left over, and several without
@pytest.mark.gpu
@pytest.mark.parametrize("N", [16, 200])
@pytest.mark.parametrize("role", [1, 2, 3])
def test_stalled_role_times_out_and_the_next_call_is_right(role, N):
    D, Fs, T = 256, 512, 2
    dev = torch.device("cuda:0")
    gen = torch.Generator(device=dev).manual_seed(2)
    r = lambda *s: torch.randn(*s, generator=gen, device=dev).to(torch.bfloat16)
    Wg, Wu, Wd = [r(D, Fs) for _ in range(T)], [r(D, Fs) for _ in range(T)], [r(Fs, D) for _ in range(T)]
    X, dY = r(N, D), r(N, D)
    act = [[r(N, Fs) for _ in range(T)] for _ in range(3)]
    call = lambda: tp.swiglu_backward(X, Wg, Wu, Wd, *act, dY)
    want = call()
    assert tp.tpmlp_check_device_error() == 0
    tp.tpmlp_set_wait_timeout_ns(LIMIT_NS)
    tp.tpmlp_selftest_weight_grad_stall(role)
    try:
        t0 = time.perf_counter()
        stalled = call()
        torch.cuda.synchronize()
        elapsed = time.perf_counter() - t0
    finally:
        tp.tpmlp_selftest_weight_grad_stall(0)
        tp.tpmlp_set_wait_timeout_ns(DEFAULT_NS)
    assert LIMIT_NS * 1e-9 <= elapsed < 5.0, elapsed
    assert tp.tpmlp_check_device_error() == _binding.ERR_TIMEOUT
    assert torch.equal(stalled[0], want[0])          # the products around it are not stalled
    got = call()
    assert tp.tpmlp_check_device_error() == 0
    assert torch.equal(got[0], want[0])
    for i in (1, 2, 3):
        for a, b in zip(got[i], want[i]):
            assert torch.equal(a, b)
