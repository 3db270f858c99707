"""Gradients of the gated block on the GPU against the float64 chain rule
(normwise bounds of the block: 1e-5 in fp32, 2e-2 in bf16 with fp32
accumulation, where dG and dU are rounded to bf16 between the products)."""

import numpy as np
import pytest
import torch

import oracle
import tensor_transformer_mlp_columnparallel_gb300 as tp
from tensor_transformer_mlp_columnparallel_gb300 import _binding
from tests.tolerance import assert_close

pytestmark = pytest.mark.gpu
MODES = ["partials", "splitk"]
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


def make(N, D, F, T, dt, seed, whole=False):
    g = torch.Generator().manual_seed(seed)
    def t(r, c, std):
        if whole:
            return torch.randint(-2, 3, (r, c), generator=g).to(TYPES[dt])
        return (torch.randn(r, c, generator=g) * std).to(TYPES[dt])
    m = {"X": t(N, D, 1.0), "dY": t(N, D, 1.0), "Wg": t(D, F, D ** -0.5), "Wu": t(D, F, D ** -0.5),
         "Wd": t(F, D, F ** -0.5), "G": t(N, F, 1.0), "U": t(N, F, 1.0)}
    m["H"] = torch.from_numpy(oracle.mlp.silu(m["G"].double().numpy()) * m["U"].double().numpy()).to(TYPES[dt])
    Fs = F // T
    cols = lambda W: [W[:, r * Fs:(r + 1) * Fs].contiguous().to(dev()) for r in range(T)]
    s = {k: cols(m[k]) for k in ("Wg", "Wu", "H", "G", "U")}
    s["Wd"] = [m["Wd"][r * Fs:(r + 1) * Fs].contiguous().to(dev()) for r in range(T)]
    s["X"], s["dY"] = m["X"].to(dev()), m["dY"].to(dev())
    return m, s


def run(s, mode, workspace=None):
    return tp.swiglu_backward(s["X"], s["Wg"], s["Wu"], s["Wd"], s["H"], s["G"], s["U"], s["dY"],
                              mode=mode, workspace=workspace)


def check(m, out, dt):
    o = oracle.mlp.swiglu_backward(m["X"], m["Wg"], m["Wu"], m["Wd"], m["H"], m["G"], m["U"], m["dY"])
    dX, dWg, dWu, dWd = out
    torch.cuda.synchronize()
    assert_close(dX, o["dX"], dt, "dX")
    assert_close(torch.cat(dWg, 1), o["dWg"], dt, "dWg")
    assert_close(torch.cat(dWu, 1), o["dWu"], dt, "dWu")
    assert_close(torch.cat(dWd, 0), o["dWd"], dt, "dWd")


@pytest.mark.parametrize("mode", MODES)
@pytest.mark.parametrize("N,D,F,T,dt", [
    (1, 8, 8, 1, "bf16"), (1, 64, 128, 2, "bf16"), (7, 72, 3 * 40, 3, "bf16"), (16, 512, 2048, 4, "bf16"),
    (33, 264, 2 * 136, 2, "bf16"), (64, 256, 16 * 64, 16, "bf16"), (65, 200, 2 * 328, 2, "bf16"),
    (130, 136, 272, 2, "bf16"), (300, 520, 2 * 264, 2, "bf16"), (257, 384, 8 * 72, 8, "bf16"),
    (640, 1024, 4 * 768, 4, "bf16"), (768, 264, 2 * 200, 2, "bf16"), (800, 392, 3 * 136, 3, "bf16"), (1024, 512, 16 * 128, 16, "bf16"),
    (1, 3, 5, 1, "f32"), (5, 17, 3 * 7, 3, "f32"), (64, 256, 1024, 2, "f32"), (130, 70, 2 * 65, 2, "f32"),
    (200, 128, 16 * 12, 16, "f32")])
def test_shapes(N, D, F, T, dt, mode):
    m, s = make(N, D, F, T, dt, N + D)
    check(m, run(s, mode), dt)


@pytest.mark.parametrize("N", [16, 300])
def test_required_workspace_only(N):
    """Without the scratch of the balanced size: whole tiles, K split."""
    m, s = make(N, 512, 4 * 256, 4, "bf16", 3)
    ws = torch.empty(tp.tpmlp_workspace_bytes(_binding.OP_SWIGLU_BACKWARD, torch.bfloat16, N, 512, 1024,
                                              4, "splitk"), dtype=torch.uint8, device=dev())
    check(m, run(s, "splitk", ws), "bf16")


def test_shards_side_by_side_equal_one():
    """T shards are the same columns: dWg, dWu, dWd of T = 4 are the slices of
    T = 1, bit for bit where the sums are exact (whole numbers, SiLU aside:
    dWd = H^T dY only)."""
    m, s1 = make(192, 128, 512, 1, "bf16", 9, whole=True)
    m["H"] = torch.randint(-2, 3, m["H"].shape).to(torch.bfloat16)
    s1["H"] = [m["H"].to(dev())]
    s4 = {k: [w.contiguous() for w in s1[k][0].chunk(4, dim=1)] for k in ("Wg", "Wu", "H", "G", "U")}
    s4["Wd"] = [w.contiguous() for w in s1["Wd"][0].chunk(4, dim=0)]
    s4["X"], s4["dY"] = s1["X"], s1["dY"]
    a, b = run(s1, "splitk"), run(s4, "partials")
    assert torch.equal(a[3][0], torch.cat(b[3], 0))
    np.testing.assert_array_equal(a[3][0].double().cpu().numpy(), oracle.mlp.as_f64(m["H"]).T @ oracle.mlp.as_f64(m["dY"]))
    assert_close(a[0], b[0].double().cpu().numpy(), "bf16", "dX")


@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_extreme_gates(dt):
    """Saturated gates: SiLU and its derivative go to 0 (or u and 1), finite."""
    m, s = make(70, 64, 128, 2, dt, 4)
    m["G"][:, ::4], m["G"][:, 1::4], m["G"][3] = 3e4, -3e4, 0.0
    s["G"] = [w.contiguous().to(dev()) for w in m["G"].chunk(2, dim=1)]
    out = run(s, "splitk")
    assert all(torch.isfinite(t).all() for t in [out[0], *out[1], *out[2], *out[3]])
    check(m, out, dt)


def test_forward_then_backward_against_differences():
    """fp32 block: <dY, Y> differenced along a direction in the weights and in X
    against <gradient, direction> (step 2^-8; rounding 2^-22 |f| / h ~ 1e-4 |f|)."""
    m, s = make(40, 48, 96, 2, "f32", 6)
    _, H, G, U = tp.swiglu_forward(s["X"], s["Wg"], s["Wu"], s["Wd"], save_gate_up=True)
    s.update(H=H, G=G, U=U)
    dX, dWg, dWu, dWd = run(s, "splitk")
    f = lambda X, a, b, c: float((s["dY"].double() * tp.swiglu_forward(X, a, b, c)[0].double()).sum())
    h, g = 2.0 ** -8, torch.Generator().manual_seed(1)
    at = [s["X"], s["Wg"], s["Wu"], s["Wd"]]
    scale = float(s["dY"].norm() * tp.swiglu_forward(*at)[0].norm())
    for i, grad in enumerate((dX, dWg, dWu, dWd)):
        one = torch.is_tensor(grad)
        dirs = [torch.randn(t.shape, generator=g).to(dev()) * 0.1 for t in ([grad] if one else grad)]
        def moved(sign):
            a = list(at)
            a[i] = at[i] + sign * h * dirs[0] if one else [w + sign * h * d for w, d in zip(at[i], dirs)]
            return f(*a)
        num = (moved(1) - moved(-1)) / (2 * h)
        ana = sum(float((x.double() * d.double()).sum()) for x, d in zip([grad] if one else grad, dirs))
        assert abs(num - ana) <= 1e-3 * scale, (i, num, ana)


def test_no_tokens_writes_zeros():
    _, s = make(0, 64, 128, 2, "bf16", 1)
    dX, dWg, dWu, dWd = run(s, "splitk")
    torch.cuda.synchronize()
    assert dX.shape == (0, 64)
    for t in [*dWg, *dWu, *dWd]:
        assert not t.any()


def test_same_bits_again_and_on_another_stream():
    _, s = make(48, 512, 2048, 4, "bf16", 2)
    ref = run(s, "splitk")
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(st):
        got = run(s, "splitk")
    st.synchronize()
    assert torch.equal(ref[0], got[0])
    for i in (1, 2, 3):
        for a, b in zip(ref[i], got[i]):
            assert torch.equal(a, b)


def rounded_once_excess(m, o, dWg, dWu):
    """How far dWg and dWu are beyond one rounding of the exact gradient, in
    units of what their computation may add (at most 1 where it is sound).
    A computed v = exact + d is rounded to a value no further from v than the
    exact value's own rounding is: the error is at most that rounding's + 2|d|.
    |d| is at most 2^-16 of the terms' sizes for a factor in two bf16 parts
    (2^-8 of 2^-8), and 2^-24 of them for each fp32 addition (D for dH, N
    here) and 2^-20 for the gate's factors."""
    a = {k: np.abs(oracle.mlp.as_f64(v)) for k, v in m.items()}
    N, D = a["X"].shape
    dH = a["dY"] @ a["Wd"].T
    gate = 1.1 * a["U"], a["G"]                 # |silu'| < 1.1, |silu(g)| <= |g|
    rel = 2.0 ** -16 + (D + N) * 2.0 ** -24 + 2.0 ** -20
    worst = []
    for got, ref, f in ((dWg, o["dWg"], gate[0]), (dWu, o["dWu"], gate[1])):
        own = np.abs(torch.from_numpy(ref).to(torch.bfloat16).double().numpy() - ref)
        worst.append(np.max((np.abs(got - ref) - own) / (2 * rel * (a["X"].T @ (dH * f)))))
    return max(worst)


@pytest.mark.parametrize("N", [1, 2, 3, 16, 64])
def test_weight_gradients_of_few_tokens_are_rounded_once(N):
    m, s = make(N, 264, 2 * 136, 2, "bf16", 70 + N)
    o = oracle.mlp.swiglu_backward(m["X"], m["Wg"], m["Wu"], m["Wd"], m["H"], m["G"], m["U"], m["dY"])
    _, dWg, dWu, _ = run(s, "splitk")
    f64 = lambda parts: torch.cat(parts, 1).double().cpu().numpy()
    assert rounded_once_excess(m, o, f64(dWg), f64(dWu)) <= 1


@pytest.mark.parametrize("mode", MODES)
@pytest.mark.parametrize("N,D,F,T", [(1, 264, 272, 2), (2, 64, 1024, 1), (3, 72, 2048, 8), (15, 520, 272, 2),
                                     (16, 264, 4096, 4), (16, 2056, 136, 1)])
def test_input_gradient_of_few_tokens_is_rounded_once(N, D, F, T, mode):
    """As for the weight gradients: up to 16 tokens dX takes dG and dU in two
    parts, its fp32 additions are D for dH and 4 F here (both parts of both
    pairs)."""
    m, s = make(N, D, F, T, "bf16", 90 + N)
    o = oracle.mlp.swiglu_backward(m["X"], m["Wg"], m["Wu"], m["Wd"], m["H"], m["G"], m["U"], m["dY"])
    ref = o["dX"]
    got = run(s, mode)[0].double().cpu().numpy()
    a = {k: np.abs(oracle.mlp.as_f64(v)) for k, v in m.items()}
    dH = a["dY"] @ a["Wd"].T
    terms = (1.1 * dH * a["U"]) @ a["Wg"].T + (dH * a["G"]) @ a["Wu"].T
    rel = 2.0 ** -16 + (D + 4 * F) * 2.0 ** -24 + 2.0 ** -20
    own = np.abs(torch.from_numpy(ref).to(torch.bfloat16).double().numpy() - ref)
    assert np.all(np.abs(got - ref) <= own + 2 * rel * terms)
    # and well below it on the whole: the rounding's own error, to a tenth
    assert np.linalg.norm(got - ref) <= 1.1 * np.linalg.norm(own)


def test_wrong_shapes_and_lists_are_refused():
    m, s = make(8, 64, 2 * 32, 2, "bf16", 1)
    run(s, "splitk")
    other = {"X": s["X"][:, :32].contiguous(), "dY": s["dY"][:4], "H": s["H"][:1], "G": [s["G"][0]] * 3,
             "U": [s["U"][0], s["U"][1][:4]], "Wu": [s["Wu"][0], s["Wu"][1].t().contiguous()],
             "Wd": [s["Wd"][0], s["Wd"][1].t().contiguous()], "Wg": [s["Wg"][0], s["Wg"][1][:, :16].contiguous()]}
    launches = tp.tpmlp_launch_count()
    for name, value in other.items():
        with pytest.raises(ValueError):
            run(dict(s, **{name: value}), "splitk")
    with pytest.raises(TypeError):
        run(dict(s, H=[h.float() for h in s["H"]]), "splitk")
    with pytest.raises(ValueError):
        run(dict(s, U=[u.t().contiguous().t() for u in s["U"]]), "splitk")
    assert tp.tpmlp_launch_count() == launches
