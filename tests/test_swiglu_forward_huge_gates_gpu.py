"""Gates of the gated forward far below zero, down to the type's lowest value: SiLU
is 0 there (|g| exp(g) < 1e-32 from -80 down), whatever g's size; far above zero it
is g. Elsewhere it is off by 2^-20 of g, and H by that of |g u| and, in bf16, by 2^-8."""

import numpy as np
import pytest
import torch

import oracle
import tensor_transformer_mlp_columnparallel_gb300 as tp
from tests.test_split_linear_gpu import TYPES, dev, f64, within

pytestmark = [pytest.mark.gpu, pytest.mark.filterwarnings("ignore:overflow encountered")]


@pytest.fixture(scope="module", autouse=True)
def _built():
    import __graft_entry__
    __graft_entry__.build()
    torch.cuda.set_device(0)
    yield
    assert tp.tpmlp_check_device_error() == 0


# the few-token launch, single-CTA tiles, pair tiles; CUDA cores
@pytest.mark.parametrize("N,D,F,T,dt", [(7, 64, 256, 2, "bf16"), (100, 64, 256, 2, "bf16"), (300, 128, 512, 2, "bf16"),
                                        (40, 48, 96, 2, "f32")])
def test_gates_far_from_zero(N, D, F, T, dt):
    """X = e_0 in every row, so the gates are the first row of Wg and the ups that of Wu."""
    st, g = TYPES[dt], torch.Generator().manual_seed(3)
    at = torch.tensor([torch.finfo(st).min, -1e36, -1e20, -4000.0, -100.0, -81.0, -79.0, -20.0, -1.0, 0.0, 3.0, 90.0, 1e30],
                      dtype=torch.float64).to(st)
    gate = at[torch.randint(0, len(at), (F,), generator=g)]
    up = (torch.rand(F, generator=g) + 0.5).to(st)
    X, Wg, Wu = (torch.zeros(r, c, dtype=st) for r, c in ((N, D), (D, F), (D, F)))
    X[:, 0], Wg[0], Wu[0] = 1.0, gate, up
    Wd = torch.zeros(F, D, dtype=st)
    cols = lambda W: [w.contiguous().to(dev()) for w in W.chunk(T, dim=1)]
    _, H, G, U = tp.swiglu_forward(X.to(dev()), cols(Wg), cols(Wu), [w.contiguous().to(dev()) for w in Wd.chunk(T, dim=0)],
                                   save_gate_up=True)
    assert torch.equal(torch.cat(G, 1), gate.to(dev()).expand(N, F)) and torch.equal(torch.cat(U, 1), up.to(dev()).expand(N, F))
    ref = np.broadcast_to(oracle.mlp.silu(f64(gate)) * f64(up), (N, F))
    tiny = np.abs(ref) < 1e-30
    lim = 2.0 ** -20 * np.abs(f64(gate) * f64(up)) + 1e-30
    within(torch.cat(H, 1), np.where(tiny, 0.0, ref), np.where(tiny, 1e-30, lim), "H")
