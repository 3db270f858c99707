"""Memory of a distillation gradient: its own rows, whatever the pitch of the
logits' rows (the last position's logits of a batch of sequences have the
pitch of a whole sequence)."""

import pytest
import torch

import oracle
import tensor_transformer_mlp_columnparallel_gb300 as tp

LINE = 128   # bytes: rows keep their place within a cache line


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("V,ld", [(1000, 1000), (1000, 1003), (1000, 64000), (1001, 64063), (7, 1 << 20), (1, 5)])
def test_gradient_takes_its_own_rows(V, ld, dtype):
    N, es = 6, torch.empty((), dtype=dtype).element_size()
    logits = torch.empty(N * ld, dtype=dtype).as_strided((N, V), (ld, 1))
    d = tp._dlogits_like(logits, False)
    assert d.shape == logits.shape and d.dtype == dtype and d.stride(1) == 1
    assert d.untyped_storage().nbytes() <= N * (V * es + LINE)
    assert d.stride(0) >= V and (d.stride(0) - ld) * es % LINE == 0     # the same alignment, row by row
    assert tp._dlogits_like(logits, True) is logits
    one = tp._dlogits_like(logits[:1], False)
    assert one.shape == (1, V) and one.untyped_storage().nbytes() <= V * es + LINE


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_last_positions_of_a_batch(dtype):
    import __graft_entry__
    __graft_entry__.build()
    B, S, V, K, tau = 4, 300, 5003, 6, 1.5
    g = torch.Generator().manual_seed(3)
    z = (torch.randn(B, S, V, generator=g) * 2).to(dtype).cuda()[:, -1]
    ids = torch.stack([torch.randperm(V, generator=g)[:K] for _ in range(B)]).to(torch.int32).cuda()
    tl = torch.randn(B, K, generator=g).cuda()
    want = oracle.vocab.distill_backward(z, ids, tl, tau, 1.0)
    torch.cuda.synchronize()
    torch.cuda.reset_peak_memory_stats()
    before = torch.cuda.memory_allocated()
    d1 = tp.vocab_distill_with_grad(z, ids, tl, 1, temperature=tau)[3]
    lse = tp.vocab_distill(z, ids, tl, 1, temperature=tau)[2]
    d2 = tp.vocab_distill_backward(z, ids, tl, 1, lse, temperature=tau)
    assert torch.cuda.max_memory_allocated() - before < 4 << 20      # two gradients of 80 KB at most
    for d in (d1, d2):
        err = abs(d.double().cpu().numpy() - want)
        lim = 1e-5 * abs(want).max() + (2.0 ** -8 * abs(want) if dtype == torch.bfloat16 else 0.0)
        assert (err <= lim).all()
    assert tp.tpmlp_check_device_error() == 0
