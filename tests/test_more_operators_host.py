"""Refusals of layer norm, the split linear layers and the policy loss, on the
host: the documented status, before anything reaches the device."""

import ctypes

import pytest
import torch

import tensor_transformer_mlp_columnparallel_gb300 as tp
from tensor_transformer_mlp_columnparallel_gb300 import _binding as B

FAKE = 0x10000   # 16-byte aligned, never dereferenced
PP = ctypes.POINTER(ctypes.c_void_p)
NONE = ctypes.c_size_t(-1).value
F32, BF16 = 0, 1


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


def norm(lib, dt=1, pdt=1, N=4, D=12, x=FAKE, ldx=12, w=FAKE, b=FAKE, eps=1e-5, y=2 * FAKE, ldy=12,
         mean=FAKE, rstd=FAKE):
    return lib.tpmlp_layernorm(dt, pdt, N, D, x, ldx, w, b, eps, y, ldy, mean, rstd, None)


def test_layernorm_refusals(lib):
    for bad in (dict(dt=2), dict(pdt=3), dict(dt=F32, pdt=BF16)):
        assert norm(lib, **bad) == B.ERR_DTYPE, bad
    for bad in (dict(N=-1), dict(x=None), dict(y=None), dict(eps=-1e-9), dict(eps=float("nan")),
                dict(eps=float("inf")), dict(y=FAKE, ldy=16)):
        assert norm(lib, **bad) == B.ERR_ARG, bad
    for bad in (dict(D=0), dict(ldx=11), dict(ldy=11), dict(D=1 << 31, ldx=1 << 31, ldy=1 << 31), dict(N=1 << 31),
                dict(ldx=1 << 41)):
        assert norm(lib, **bad) == B.ERR_SHAPE, bad
    for bad in (dict(x=FAKE + 1), dict(y=FAKE + 1), dict(w=FAKE + 1), dict(b=FAKE + 1), dict(pdt=F32, w=FAKE + 2),
                dict(mean=FAKE + 2), dict(rstd=FAKE + 1), dict(dt=F32, pdt=F32, x=FAKE + 2)):
        assert norm(lib, **bad) == B.ERR_ALIGN, bad
    assert norm(lib, N=0, x=None, y=None, mean=None, rstd=None) == B.OK


def norm_grad(lib, dt=1, pdt=1, N=4, D=12, dy=FAKE, lddy=12, x=2 * FAKE, ldx=12, w=FAKE, mean=FAKE, rstd=FAKE,
              res=3 * FAKE, lddres=12, dx=4 * FAKE, lddx=12, dw=FAKE, db=FAKE, ws=FAKE, n=1 << 30):
    return lib.tpmlp_layernorm_backward(dt, pdt, N, D, dy, lddy, x, ldx, w, mean, rstd, res, lddres, dx, lddx, dw, db,
                                        ws, n, None)


def test_layernorm_backward_refusals(lib):
    size = lib.tpmlp_layernorm_backward_workspace_bytes
    assert size(-1, 12) == size(4, 0) == size(1 << 31, 8) == size(4, 1 << 31) == NONE
    assert size(0, 12) == 0 and size(4, 12) > 0
    for bad in (dict(dt=2), dict(pdt=3), dict(dt=F32, pdt=BF16)):
        assert norm_grad(lib, **bad) == B.ERR_DTYPE, bad
    for bad in (dict(N=-1), dict(dy=None), dict(x=None), dict(dx=None), dict(mean=None), dict(rstd=None),
                dict(dw=None), dict(db=None), dict(dx=FAKE, lddx=16), dict(dx=2 * FAKE, lddx=16),
                dict(dx=3 * FAKE, lddx=16)):
        assert norm_grad(lib, **bad) == B.ERR_ARG, bad
    for bad in (dict(D=0), dict(lddy=11), dict(ldx=11), dict(lddx=11), dict(lddres=11)):
        assert norm_grad(lib, **bad) == B.ERR_SHAPE, bad
    for bad in (dict(dy=FAKE + 1), dict(x=FAKE + 1), dict(dx=FAKE + 1), dict(res=FAKE + 1), dict(w=FAKE + 1),
                dict(dw=FAKE + 1), dict(db=FAKE + 1), dict(mean=FAKE + 2), dict(rstd=FAKE + 2), dict(ws=FAKE + 8)):
        assert norm_grad(lib, **bad) == B.ERR_ALIGN, bad
    assert norm_grad(lib, ws=None) == norm_grad(lib, n=size(4, 12) - 1) == B.ERR_WORKSPACE
    assert norm_grad(lib, N=0, dw=None, db=None, ws=None, n=0) == B.OK


def column(lib, dt=1, N=4, D=16, F=32, T=2, act=1, X=FAKE, ldx=16, W="ok", b="ok", R=2 * FAKE, ldr=32, Y=3 * FAKE,
           ldy=32, Z=4 * FAKE, ldz=32, ws=None, n=0):
    s = lambda v: ptrs(FAKE, FAKE) if v == "ok" else v
    return lib.tpmlp_column_linear(dt, N, D, F, T, act, X, ldx, s(W), s(b), R, ldr, Y, ldy, Z, ldz, ws, n, None)


def row(lib, dt=1, N=4, D=16, F=32, T=2, X=FAKE, ldx=32, W="ok", b=FAKE, R=2 * FAKE, ldr=16, Y=3 * FAKE, ldy=16,
        ws=None, n=0):
    s = lambda v: ptrs(FAKE, FAKE) if v == "ok" else v
    return lib.tpmlp_row_linear(dt, N, D, F, T, X, ldx, s(W), b, R, ldr, Y, ldy, ws, n, None)


@pytest.mark.parametrize("call", [column, row])
def test_linear_refusals(lib, call):
    assert call(lib, dt=2) == B.ERR_DTYPE
    for bad in (dict(N=-1), dict(X=None), dict(Y=None), dict(W=None), dict(W=ptrs(FAKE, None)),
                dict(R=3 * FAKE, ldr=40)):
        assert call(lib, **bad) == B.ERR_ARG, bad
    for bad in (dict(T=3), dict(T=0), dict(T=17), dict(D=0), dict(F=33), dict(ldx=8), dict(ldy=8), dict(ldr=8),
                dict(ldx=1 << 39), dict(N=1 << 31)):
        assert call(lib, **bad) == B.ERR_SHAPE, bad
    for bad in (dict(D=12, ldr=16), dict(F=24, ldx=40), dict(X=FAKE + 8), dict(Y=FAKE + 8), dict(R=FAKE + 8),
                dict(ldx=36), dict(ldy=36), dict(ldr=36), dict(W=ptrs(FAKE, FAKE + 8)), dict(ws=FAKE + 8, n=64),
                dict(dt=F32, X=FAKE + 2), dict(dt=F32, Y=FAKE + 1)):
        assert call(lib, **bad) == B.ERR_ALIGN, bad
    assert call(lib, N=0, X=None, Y=None, R=None) == B.OK


def test_column_linear_refusals(lib):
    for bad in (dict(act=4), dict(act=-2), dict(act=-1), dict(b=ptrs(None, FAKE))):   # Z without an activation
        assert column(lib, **bad) == B.ERR_ARG, bad
    assert column(lib, ldz=24) == B.ERR_SHAPE and column(lib, Z=FAKE + 8) == column(lib, ldz=36) == B.ERR_ALIGN
    assert row(lib, b=FAKE + 4) == B.ERR_ALIGN


def column_grad(lib, dt=1, N=4, D=16, F=32, T=2, act=1, X=FAKE, ldx=16, W="ok", Z=FAKE, ldz=32, dY=FAKE, lddy=32,
                dX=FAKE, lddx=16, dW="ok", db="ok", ws=FAKE, n=1 << 30):
    s = lambda v: ptrs(FAKE, FAKE) if v == "ok" else v
    return lib.tpmlp_column_linear_backward(dt, N, D, F, T, act, X, ldx, s(W), Z, ldz, dY, lddy, dX, lddx, s(dW),
                                            s(db), ws, n, None)


def row_grad(lib, dt=1, N=4, D=16, F=32, T=2, X=FAKE, ldx=32, W="ok", dY=FAKE, lddy=16, dX=FAKE, lddx=32, dW="ok",
             db=FAKE, ws=None, n=0):
    s = lambda v: ptrs(FAKE, FAKE) if v == "ok" else v
    return lib.tpmlp_row_linear_backward(dt, N, D, F, T, X, ldx, s(W), dY, lddy, dX, lddx, s(dW), db, ws, n, None)


@pytest.mark.parametrize("call", [column_grad, row_grad])
def test_linear_backward_refusals(lib, call):
    assert call(lib, dt=2) == B.ERR_DTYPE
    for bad in (dict(N=-1), dict(X=None), dict(dY=None), dict(dX=None), dict(W=None), dict(dW=None),
                dict(dW=ptrs(FAKE, None))):
        assert call(lib, **bad) == B.ERR_ARG, bad
    for bad in (dict(T=3), dict(D=0), dict(F=33), dict(ldx=8), dict(lddy=8), dict(lddx=8)):
        assert call(lib, **bad) == B.ERR_SHAPE, bad
    for bad in (dict(X=FAKE + 8), dict(dY=FAKE + 2), dict(dX=FAKE + 4), dict(ldx=36), dict(lddy=36), dict(lddx=36),
                dict(dW=ptrs(FAKE + 8, FAKE))):
        assert call(lib, **bad) == B.ERR_ALIGN, bad


def test_column_linear_backward_workspace(lib):
    size, more = lib.tpmlp_workspace_bytes, lib.tpmlp_workspace_bytes_balanced
    assert size(B.OP_LINEAR, 1, 4, 16, 32, 2, 1) == size(B.OP_LINEAR_BACKWARD, 1, 4, 16, 32, 2, 1) == 0
    need = size(B.OP_LINEAR_BACKWARD_ACT, 1, 4, 16, 32, 2, 1)
    assert need >= 2 * 4 * 32 * 2                                     # dZ and what its rounding left over
    assert size(B.OP_LINEAR_BACKWARD_ACT, 1, 0, 16, 32, 2, 1) == 0
    assert more(B.OP_LINEAR, 1, 64, 16, 32, 2, 1) == 0                # no scratch for a few tokens
    assert more(B.OP_LINEAR, 1, 65, 16, 32, 2, 1) > 0 == more(B.OP_LINEAR, 0, 65, 16, 32, 2, 1)
    assert size(6, 1, 4, 16, 32, 2, 1) == size(B.OP_LINEAR, 1, 4, 16, 33, 2, 1) == NONE
    assert column_grad(lib, ws=None) == column_grad(lib, n=need - 1) == B.ERR_WORKSPACE
    assert column_grad(lib, ws=FAKE + 8) == B.ERR_ALIGN
    assert column_grad(lib, Z=None) == column_grad(lib, act=9) == column_grad(lib, db=ptrs(FAKE, None)) == B.ERR_ARG
    assert column_grad(lib, ldz=24) == B.ERR_SHAPE


def policy(lib, dt=1, N=4, V=12, T=3, z=FAKE, ld=12, t=FAKE, old=FAKE, adv=FAKE, ref=FAKE, kl=0.1, low=0.2, high=0.2,
           tau=1.0, loss=FAKE, lp=FAKE, k=FAKE):
    return lib.tpmlp_vocab_policy(dt, N, V, T, z, ld, t, old, adv, ref, kl, low, high, tau, loss, None, lp, k, None)


def policy_grad(lib, dt=1, N=4, V=12, T=3, z=FAKE, ld=12, t=FAKE, old=FAKE, adv=FAKE, ref=FAKE, kl=0.1, low=0.2,
                high=0.2, tau=1.0, lp=FAKE, w=FAKE, d=2 * FAKE, ldd=12):
    return lib.tpmlp_vocab_policy_backward(dt, N, V, T, z, ld, t, old, adv, ref, kl, low, high, tau, lp, w, 1.0, d,
                                           ldd, None)


def policy_both(lib, dt=1, N=4, V=12, T=3, z=FAKE, ld=12, t=FAKE, old=FAKE, adv=FAKE, ref=FAKE, kl=0.1, low=0.2,
                high=0.2, tau=1.0, loss=FAKE, lp=FAKE, k=FAKE, w=FAKE, d=2 * FAKE, ldd=12):
    return lib.tpmlp_vocab_policy_with_grad(dt, N, V, T, z, ld, t, old, adv, ref, kl, low, high, tau, loss, None, lp,
                                            k, w, 1.0, d, ldd, None)


@pytest.mark.parametrize("call", [policy, policy_grad, policy_both])
def test_policy_refusals(lib, call):
    nan, inf = float("nan"), float("inf")
    assert call(lib, dt=9) == B.ERR_DTYPE
    for bad in (dict(T=5), dict(T=0), dict(V=0, ld=0, T=1), dict(ld=11), dict(V=1 << 31, ld=1 << 31, T=1)):
        assert call(lib, **bad) == B.ERR_SHAPE, bad
    for bad in (dict(N=-2), dict(z=None), dict(t=None), dict(old=None), dict(adv=None), dict(ref=None),
                dict(kl=-0.1), dict(kl=nan), dict(kl=inf), dict(low=-0.1), dict(low=1.5), dict(low=nan),
                dict(high=-0.1), dict(high=nan), dict(tau=0.0), dict(tau=nan), dict(tau=inf), dict(tau=2.0 ** 61)):
        assert call(lib, **bad) == B.ERR_ARG, bad
    for bad in (dict(z=FAKE + 1), dict(t=FAKE + 4), dict(old=FAKE + 2), dict(adv=FAKE + 1), dict(ref=FAKE + 2),
                dict(lp=FAKE + 2)):
        assert call(lib, **bad) == B.ERR_ALIGN, bad
    if call is policy_grad:
        assert call(lib, lp=None) == B.ERR_ARG
    else:
        assert call(lib, loss=None) == call(lib, ref=None, kl=0.0) == B.ERR_ARG    # kl wanted without a reference
        assert call(lib, k=FAKE + 2) == B.ERR_ALIGN
    if call is not policy:
        assert call(lib, d=None) == call(lib, d=FAKE, ldd=16) == B.ERR_ARG
        assert call(lib, ldd=11) == B.ERR_SHAPE
        assert call(lib, d=FAKE + 1) == call(lib, w=FAKE + 2) == B.ERR_ALIGN
    assert call(lib, N=0, z=None, t=None, old=None, adv=None, ref=None) == B.OK


def test_binding_refuses_host_tensors(lib):
    x, v = torch.zeros(3, 8), torch.zeros(8)
    W, V = [torch.zeros(8, 4)] * 2, [torch.zeros(4, 8)] * 2
    n, t = torch.zeros(3), torch.zeros(3, dtype=torch.int64)
    for call in (lambda: tp.layernorm(x, v, v), lambda: tp.layernorm_backward(x, x, v, n, n),
                 lambda: tp.column_linear(x, W), lambda: tp.row_linear(x, V),
                 lambda: tp.column_linear_backward(x, W, x), lambda: tp.row_linear_backward(x, V, x),
                 lambda: tp.vocab_policy(x, t, n, n, 2), lambda: tp.vocab_policy_backward(x, t, n, n, 2, n),
                 lambda: tp.vocab_policy_with_grad(x, t, n, n, 2)):
        with pytest.raises(ValueError):
            call()
