"""Temperatures that the distillation calls refuse: log2(e) / tau and tau^2,
which both enter, must be ordinary fp32 numbers (tau = 1e-39 gave NaN for every
row, 1e20 an infinite loss, 1e-30 a loss of 0)."""

import pytest

from tensor_transformer_mlp_columnparallel_gb300 import _binding as B

FAKE = 0x10000


@pytest.mark.parametrize("tau", [1e-39, 1e-30, 2.0 ** -61, 2.0 ** 61, 1e20, 3.4e38])
def test_refused(tau):
    import __graft_entry__
    __graft_entry__.build()
    lib = B.lib()
    before = lib.tpmlp_launch_count()
    rows = (0, 4, 12, 3, 2, FAKE, 12, FAKE, FAKE, tau)
    assert lib.tpmlp_vocab_distill(*rows, FAKE, None, None, None) == B.ERR_ARG
    assert lib.tpmlp_vocab_distill_backward(*rows, FAKE, None, 1.0, 2 * FAKE, 12, None) == B.ERR_ARG
    assert lib.tpmlp_vocab_distill_with_grad(*rows, FAKE, None, None, None, 1.0, 2 * FAKE, 12, None) == B.ERR_ARG
    assert lib.tpmlp_launch_count() == before
