"""Refusals of the vocabulary-side operators and of the gated backward, on the
host: the documented status, before anything reaches the device."""

import ctypes

import pytest
import torch

import tensor_transformer_mlp_columnparallel_gb300 as tp
from tensor_transformer_mlp_columnparallel_gb300 import _binding as B

FAKE = 0x10000   # 16-byte aligned, never dereferenced
PP = ctypes.POINTER(ctypes.c_void_p)


def ptrs(*vals):
    return ctypes.cast((ctypes.c_void_p * len(vals))(*vals), PP)


@pytest.fixture(scope="module")
def lib():
    import __graft_entry__
    __graft_entry__.build()
    return B.lib()


@pytest.fixture(autouse=True)
def no_launch(lib):
    before = lib.tpmlp_launch_count()
    yield
    assert lib.tpmlp_launch_count() == before


def logprobs(lib, dt=1, N=4, V=12, T=3, K=2, z=FAKE, ld=12, t=FAKE, lp=FAKE, rank=FAKE, ids=FAKE,
             top=FAKE):
    return lib.tpmlp_vocab_logprobs(dt, N, V, T, K, z, ld, t, lp, rank, None, None, ids, top, None)


def test_logprobs_refusals(lib):
    assert logprobs(lib, dt=2) == B.ERR_DTYPE
    assert logprobs(lib, N=-1) == B.ERR_ARG
    for bad in (dict(T=5), dict(T=0), dict(T=17, V=17, ld=17), dict(V=0, ld=0), dict(ld=11),
                dict(K=-1), dict(K=13), dict(V=300, ld=300, K=B.MAX_TOP + 1), dict(V=1 << 31, ld=1 << 31, T=1)):
        assert logprobs(lib, **bad) == B.ERR_SHAPE, bad
    for bad in (dict(z=None), dict(t=None), dict(t=None, lp=None), dict(ids=None), dict(top=None)):
        assert logprobs(lib, **bad) == B.ERR_ARG, bad
    assert logprobs(lib, z=FAKE + 1) == B.ERR_ALIGN
    assert logprobs(lib, dt=0, z=FAKE + 2) == B.ERR_ALIGN
    assert logprobs(lib, N=0, z=None, t=None, lp=None, rank=None, ids=None, top=None) == B.OK


def distill(lib, dt=1, N=4, V=12, T=3, K=2, z=FAKE, ld=12, ids=FAKE, tl=FAKE, tau=1.0, loss=FAKE):
    return lib.tpmlp_vocab_distill(dt, N, V, T, K, z, ld, ids, tl, tau, loss, None, None, None)


def distill_bwd(lib, dt=1, N=4, V=12, T=3, K=2, z=FAKE, ld=12, ids=FAKE, tl=FAKE, tau=1.0, lse=FAKE,
                d=2 * FAKE, ldd=12):
    return lib.tpmlp_vocab_distill_backward(dt, N, V, T, K, z, ld, ids, tl, tau, lse, None, 1.0, d,
                                            ldd, None)


def distill_both(lib, dt=1, N=4, V=12, T=3, K=2, z=FAKE, ld=12, ids=FAKE, tl=FAKE, tau=1.0,
                 loss=FAKE, d=2 * FAKE, ldd=12):
    return lib.tpmlp_vocab_distill_with_grad(dt, N, V, T, K, z, ld, ids, tl, tau, loss, None, None,
                                             None, 1.0, d, ldd, None)


@pytest.mark.parametrize("call", [distill, distill_bwd, distill_both])
def test_distill_refusals(lib, call):
    assert call(lib, dt=9) == B.ERR_DTYPE
    for bad in (dict(T=5), dict(V=0, ld=0, T=1), dict(ld=11), dict(K=0), dict(K=B.MAX_TEACHER + 1)):
        assert call(lib, **bad) == B.ERR_SHAPE, bad
    for bad in (dict(N=-2), dict(z=None), dict(ids=None), dict(tl=None), dict(tau=0.0), dict(tau=-1.0),
                dict(tau=float("nan")), dict(tau=float("inf"))):
        assert call(lib, **bad) == B.ERR_ARG, bad
    assert call(lib, z=FAKE + 1) == B.ERR_ALIGN
    if call is not distill_bwd:
        assert call(lib, loss=None) == B.ERR_ARG
    else:
        assert call(lib, lse=None) == B.ERR_ARG
    if call is not distill:
        assert call(lib, d=None) == B.ERR_ARG
        assert call(lib, ldd=11) == B.ERR_SHAPE
        assert call(lib, d=FAKE + 1) == B.ERR_ALIGN
        assert call(lib, d=FAKE, ldd=16) == B.ERR_ARG       # in place needs the same rows
    assert call(lib, N=0, z=None, ids=None, tl=None) == B.OK


def test_embedding_refusals(lib):
    def fwd(dt=1, N=4, V=12, H=8, T=2, ids=FAKE, table=ptrs(FAKE, FAKE), out=FAKE):
        return lib.tpmlp_vocab_embedding_scaled(dt, N, V, H, T, ids, table, 2.0, out, None)
    assert fwd(dt=5) == B.ERR_DTYPE
    assert fwd(N=-1) == B.ERR_ARG
    assert fwd(V=13) == B.ERR_SHAPE and fwd(H=0) == B.ERR_SHAPE and fwd(T=0) == B.ERR_SHAPE
    assert fwd(ids=None) == fwd(out=None) == fwd(table=None) == fwd(table=ptrs(FAKE, None)) == B.ERR_ARG
    assert fwd(N=0, ids=None, out=None) == B.OK

    size = lib.tpmlp_vocab_embedding_backward_workspace_bytes
    none = ctypes.c_size_t(-1).value
    assert size(-1, 12, 8) == size(4, 0, 8) == size(4, 12, 0) == size(4, 1 << 31, 8) == none
    need = size(4, 12, 8)

    def bwd(dt=1, gdt=0, N=4, V=12, H=8, T=2, ids=FAKE, dout=FAKE, tab=ptrs(FAKE, FAKE), ws=FAKE, n=need):
        return lib.tpmlp_vocab_embedding_backward(dt, gdt, N, V, H, T, ids, dout, 1.0, 0, tab, ws, n, None)
    assert bwd(dt=5) == bwd(gdt=5) == B.ERR_DTYPE
    assert bwd(N=-1) == B.ERR_ARG
    assert bwd(V=13) == bwd(H=0) == bwd(T=17, V=17) == bwd(N=1 << 31, n=1 << 60) == B.ERR_SHAPE
    assert bwd(ids=None) == bwd(dout=None) == bwd(tab=None) == bwd(tab=ptrs(None, FAKE)) == B.ERR_ARG
    assert bwd(ws=None) == bwd(n=need - 1) == B.ERR_WORKSPACE
    assert bwd(ws=FAKE + 4) == B.ERR_ALIGN


def test_gated_backward_refusals(lib):
    size = lib.tpmlp_workspace_bytes
    sh = lambda: ptrs(FAKE, FAKE)

    def bwd(dt=1, N=4, D=16, F=32, T=2, X=FAKE, Wg="ok", Wd="ok", G="ok", dY=FAKE, dX=FAKE, dWg="ok",
            mode=1, ws=FAKE, n=1 << 20):
        s = lambda v: sh() if v == "ok" else v
        return lib.tpmlp_swiglu_backward(dt, N, D, F, T, X, s(Wg), sh(), s(Wd), sh(), s(G), sh(), dY,
                                         dX, s(dWg), sh(), sh(), mode, ws, n, None)
    need = size(2, 1, 4, 16, 32, 2, 1)
    r256 = lambda x: (x + 255) // 256 * 256
    assert need == 2 * 2 * r256(2 * 4 * 16 * 2)      # dG, dU, each with what its rounding left over
    assert size(2, 1, 65, 16, 32, 2, 1) == 2 * 2 * r256(65 * 16 * 2)
    assert size(2, 1, 4, 16, 32, 2, 0) == need + 2 * r256(4 * 16 * 4)
    assert size(2, 0, 4, 16, 32, 2, 0) == 2 * 2 * r256(4 * 16 * 4) + 2 * r256(4 * 16 * 4)
    assert lib.tpmlp_workspace_bytes_balanced(2, 1, 4, 16, 32, 2, 1) == need     # no scratch for a few tokens
    assert lib.tpmlp_workspace_bytes_balanced(2, 1, 65, 16, 32, 2, 1) > size(2, 1, 65, 16, 32, 2, 1)
    assert bwd(dt=4) == B.ERR_DTYPE
    assert bwd(N=-1) == bwd(mode=3) == B.ERR_ARG
    assert bwd(F=33) == bwd(T=0) == bwd(D=0) == B.ERR_SHAPE
    assert bwd(D=12) == bwd(F=24) == bwd(X=FAKE + 8) == bwd(G=ptrs(FAKE, FAKE + 2)) == B.ERR_ALIGN
    assert bwd(X=None) == bwd(dY=None) == bwd(dX=None) == bwd(Wg=None) == B.ERR_ARG
    assert bwd(Wd=ptrs(FAKE, None)) == bwd(G=None) == bwd(dWg=None) == B.ERR_ARG
    assert bwd(ws=None) == bwd(n=need - 1) == B.ERR_WORKSPACE
    assert bwd(ws=FAKE + 8) == B.ERR_ALIGN


def test_binding_refuses_host_tensors_and_wrong_lists(lib):
    z = torch.zeros(3, 8)
    ids, tl = torch.zeros(3, 2, dtype=torch.int32), torch.zeros(3, 2)
    with pytest.raises(ValueError):
        tp.vocab_logprobs(z, torch.zeros(3, dtype=torch.int64), 2, top_k=2)
    with pytest.raises(ValueError):
        tp.vocab_distill(z, ids, tl, 2)
    with pytest.raises(ValueError):
        tp.vocab_embedding_scaled(torch.zeros(3, dtype=torch.int64), [torch.zeros(4, 8)], 1.0)
    with pytest.raises(ValueError):
        tp.vocab_embedding_backward(torch.zeros(3, dtype=torch.int64), torch.zeros(3, 8), 12, 2)
    with pytest.raises(tp.TpmlpError):
        tp.vocab_embedding_backward(torch.zeros(3, dtype=torch.int64), torch.zeros(3, 8), 13, 2)


def test_binding_refuses_wrong_shard_counts(lib):
    x = torch.zeros(3, 8)
    w, wd, h = [torch.zeros(8, 4)] * 2, [torch.zeros(4, 8)] * 2, [torch.zeros(3, 4)] * 2
    for bad in ({"Wu": w[:1]}, {"Wd": wd + wd}, {"H": []}, {"G": h[:1]}, {"U": h * 2}):
        a = dict({"Wg": w, "Wu": w, "Wd": wd, "H": h, "G": h, "U": h}, **bad)
        with pytest.raises(ValueError):
            tp.swiglu_backward(x, a["Wg"], a["Wu"], a["Wd"], a["H"], a["G"], a["U"], x, workspace=x)
