"""Gates far below zero, down to the type's lowest value: SiLU and its
derivative are 0 there (|g| exp(g) < 1e-32 from -80 down), whatever g's size;
a NaN gate gives NaN. Bounds as for any other block."""

import pytest
import torch

import tensor_transformer_mlp_columnparallel_gb300 as tp
from tests.test_parity_swiglu_backward_gpu import check, dev, make, run

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    import __graft_entry__
    __graft_entry__.build()
    torch.cuda.set_device(0)
    yield
    assert tp.tpmlp_check_device_error() == 0


# the few-token launch, single-CTA tiles, staged pair tiles; CUDA cores
@pytest.mark.filterwarnings("ignore:overflow encountered in exp")
@pytest.mark.parametrize("N,D,F,T,dt", [(7, 64, 256, 2, "bf16"), (100, 64, 256, 2, "bf16"), (300, 128, 512, 2, "bf16"),
                                        (40, 48, 96, 2, "f32")])
def test_lowest_gates(N, D, F, T, dt):
    m, s = make(N, D, F, T, dt, N)
    lowest = torch.finfo(m["G"].dtype).min
    m["G"][:, ::4], m["G"][:, 1::4], m["G"][:, 2::8] = lowest, -1e36, -79.0
    m["H"][:, ::4] = m["H"][:, 1::4] = m["H"][:, 2::8] = 0.0
    for k in ("G", "H"):
        s[k] = [w.contiguous().to(dev()) for w in m[k].chunk(T, dim=1)]
    check(m, run(s, "splitk"), dt)


@pytest.mark.parametrize("N,dt", [(7, "bf16"), (300, "bf16"), (40, "f32")])
def test_nan_gate(N, dt):
    m, s = make(N, 64, 128, 2, dt, 3)
    s["G"][1][5, 9] = float("nan")
    dX, dWg, dWu, _ = run(s, "splitk")
    assert torch.isnan(dX[5]).all() and torch.isfinite(dX[[0, 4, 6]]).all()
    assert torch.isnan(dWg[1][:, 9]).all() and torch.isnan(dWu[1][:, 9]).all()
    assert torch.isfinite(dWg[0]).all() and torch.isfinite(dWg[1][:, :9]).all()
