"""Every pointer of the vocabulary-side calls has the alignment of its element,
or the call says TPMLP_ERR_ALIGN before anything reaches the device."""

import ctypes

import pytest

from tensor_transformer_mlp_columnparallel_gb300 import _binding as B

FAKE = 0x10000   # 16-byte aligned, never dereferenced
PP = ctypes.POINTER(ctypes.c_void_p)
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


# argument -> a byte offset that its element's size does not allow
LOGPROBS = {"z": 2, "t": 4, "lp": 2, "rank": 1, "ent": 2, "lse": 3, "ids": 2, "top": 2}
LOSS = {"z": 2, "ids": 2, "tl": 1, "loss": 2, "mean": 2, "lse": 2}
GRAD = {"z": 2, "ids": 2, "tl": 2, "lse": 1, "w": 2, "d": 2}
BOTH = {**LOSS, "w": 3, "d": 1}


@pytest.mark.parametrize("name", LOGPROBS)
def test_logprobs(lib, name):
    p = {k: FAKE for k in LOGPROBS}
    p[name] += LOGPROBS[name]
    assert lib.tpmlp_vocab_logprobs(F32, 4, 12, 3, 2, p["z"], 12, p["t"], p["lp"], p["rank"], p["ent"],
                                    p["lse"], p["ids"], p["top"], None) == B.ERR_ALIGN


@pytest.mark.parametrize("name", LOSS)
def test_distill(lib, name):
    p = {k: FAKE for k in LOSS}
    p[name] += LOSS[name]
    assert lib.tpmlp_vocab_distill(F32, 4, 12, 3, 2, p["z"], 12, p["ids"], p["tl"], 1.0, p["loss"],
                                   p["mean"], p["lse"], None) == B.ERR_ALIGN


@pytest.mark.parametrize("name", GRAD)
def test_distill_backward(lib, name):
    p = {k: FAKE * (2 if k == "d" else 1) for k in GRAD}
    p[name] += GRAD[name]
    assert lib.tpmlp_vocab_distill_backward(F32, 4, 12, 3, 2, p["z"], 12, p["ids"], p["tl"], 1.0, p["lse"],
                                            p["w"], 1.0, p["d"], 12, None) == B.ERR_ALIGN


@pytest.mark.parametrize("name", BOTH)
def test_distill_with_grad(lib, name):
    p = {k: FAKE * (2 if k == "d" else 1) for k in BOTH}
    p[name] += BOTH[name]
    assert lib.tpmlp_vocab_distill_with_grad(F32, 4, 12, 3, 2, p["z"], 12, p["ids"], p["tl"], 1.0, p["loss"],
                                             p["mean"], p["lse"], p["w"], 1.0, p["d"], 12, None) == B.ERR_ALIGN


@pytest.mark.parametrize("dt,off", [(F32, 2), (BF16, 1)])
@pytest.mark.parametrize("name", ["ids", "table", "out"])
def test_embedding_scaled(lib, name, dt, off):
    p = {"ids": FAKE, "table": FAKE, "out": FAKE}
    p[name] += 4 if name == "ids" else off
    assert lib.tpmlp_vocab_embedding_scaled(dt, 4, 12, 8, 2, p["ids"], ptrs(FAKE, p["table"]), 2.0, p["out"],
                                            None) == B.ERR_ALIGN


@pytest.mark.parametrize("dt,gdt", [(F32, F32), (F32, BF16), (BF16, F32), (BF16, BF16)])
@pytest.mark.parametrize("name", ["ids", "dout", "dtable"])
def test_embedding_backward(lib, name, dt, gdt):
    need = lib.tpmlp_vocab_embedding_backward_workspace_bytes(4, 12, 8)
    p = {"ids": FAKE, "dout": FAKE, "dtable": FAKE}
    p[name] += 4 if name == "ids" else (2 if (dt if name == "dout" else gdt) == F32 else 1)
    assert lib.tpmlp_vocab_embedding_backward(dt, gdt, 4, 12, 8, 2, p["ids"], p["dout"], 1.0, 0,
                                              ptrs(p["dtable"], FAKE), FAKE, need, None) == B.ERR_ALIGN


def test_a_table_without_tokens_is_checked_too(lib):
    need = lib.tpmlp_vocab_embedding_backward_workspace_bytes(0, 12, 8)
    assert lib.tpmlp_vocab_embedding_backward(F32, F32, 0, 12, 8, 1, None, None, 1.0, 0, ptrs(FAKE + 2), FAKE,
                                              need, None) == B.ERR_ALIGN


@pytest.mark.parametrize("H,off", [((1 << 31) - 2, 0), (16776961, 0), (4 * 16776960, 4)])
def test_rows_beyond_the_launch_are_refused_before_it(lib, H, off):
    """More accesses in a row than the grid has columns for: odd rows, rows whose
    pointers allow only single elements."""
    need = lib.tpmlp_vocab_embedding_backward_workspace_bytes(4, 12, H)
    assert lib.tpmlp_vocab_embedding_backward(F32, F32, 4, 12, H, 2, FAKE, FAKE + off, 1.0, 0, ptrs(FAKE, FAKE),
                                              FAKE, need, None) == B.ERR_SHAPE
