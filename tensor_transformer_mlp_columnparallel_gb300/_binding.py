"""ctypes binding of libtpmlp.so (include/tpmlp.h).

Argument marshalling only: tensors become device pointers, lists of shard
tensors become host arrays of pointers, the current torch stream becomes the
cudaStream_t. Every step of the computation runs in the library's CUDA
kernels; there is no fallback. If the shared library is missing, loading
raises instead of silently doing something else.
"""

import ctypes
import os
import re
from typing import List, Optional, Sequence

import torch

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libtpmlp.so")
HEADER_PATH = os.path.join(os.path.dirname(_PKG), "include", "tpmlp.h")

MAX_SHARDS = 16
OK, ERR_ARG, ERR_SHAPE, ERR_ALIGN, ERR_DTYPE, ERR_CUDA, ERR_TIMEOUT, ERR_WORKSPACE = range(8)
ACT = {"relu": 0, "gelu_tanh": 1, "gelu_erf": 2, "gelu_sigmoid": 3}
DTYPE = {torch.float32: 0, torch.bfloat16: 1}
MODE = {"partials": 0, "splitk": 1}
OP_FORWARD, OP_BACKWARD, OP_SWIGLU_BACKWARD = 0, 1, 2
OP_LINEAR, OP_LINEAR_BACKWARD, OP_LINEAR_BACKWARD_ACT = 3, 4, 5
LINEAR_ACT = {None: -1, **ACT}
MAX_TOP, MAX_TEACHER = 128, 1024


class TpmlpError(RuntimeError):
    def __init__(self, status: int, msg: str):
        super().__init__(msg)
        self.status = status


class KernelTiming(ctypes.Structure):
    _fields_ = [("name", ctypes.c_char * 48), ("launches", ctypes.c_int64),
                ("total_ms", ctypes.c_double)]


_lib = None

_vp = ctypes.c_void_p
_i64 = ctypes.c_int64
_int = ctypes.c_int
_f32 = ctypes.c_float
_PP = ctypes.POINTER(ctypes.c_void_p)

_SIGNATURES = {
    "tpmlp_forward": (_int, [_int, _i64, _i64, _i64, _int, _int, _vp, _PP, _PP, _PP, _vp, _vp,
                             _PP, _PP, _int, _vp, ctypes.c_size_t, _vp]),
    "tpmlp_forward_noalloc": (_int, [_int, _i64, _i64, _i64, _int, _int, _vp, _PP, _PP, _PP, _vp,
                                     _vp, _PP, _PP, _vp]),
    "tpmlp_swiglu_forward": (_int, [_int, _i64, _i64, _i64, _int, _vp, _PP, _PP, _PP, _vp, _PP, _PP,
                                    _PP, _int, _vp, ctypes.c_size_t, _vp]),
    "tpmlp_backward": (_int, [_int, _i64, _i64, _i64, _int, _int, _vp, _PP, _PP, _PP, _PP, _vp,
                              _vp, _PP, _PP, _PP, _vp, _int, _vp, ctypes.c_size_t, _vp]),
    "tpmlp_swiglu_backward": (_int, [_int, _i64, _i64, _i64, _int, _vp, _PP, _PP, _PP, _PP, _PP,
                                     _PP, _vp, _vp, _PP, _PP, _PP, _int, _vp, ctypes.c_size_t, _vp]),
    "tpmlp_vocab_logprobs": (_int, [_int, _i64, _i64, _int, _int, _vp, _i64, _vp, _vp, _vp, _vp,
                                    _vp, _vp, _vp, _vp]),
    "tpmlp_vocab_distill": (_int, [_int, _i64, _i64, _int, _int, _vp, _i64, _vp, _vp, _f32, _vp,
                                   _vp, _vp, _vp]),
    "tpmlp_vocab_distill_backward": (_int, [_int, _i64, _i64, _int, _int, _vp, _i64, _vp, _vp,
                                            _f32, _vp, _vp, _f32, _vp, _i64, _vp]),
    "tpmlp_vocab_distill_with_grad": (_int, [_int, _i64, _i64, _int, _int, _vp, _i64, _vp, _vp,
                                             _f32, _vp, _vp, _vp, _vp, _f32, _vp, _i64, _vp]),
    "tpmlp_vocab_embedding_scaled": (_int, [_int, _i64, _i64, _i64, _int, _vp, _PP, _f32, _vp, _vp]),
    "tpmlp_vocab_embedding_backward": (_int, [_int, _int, _i64, _i64, _i64, _int, _vp, _vp, _f32,
                                              _int, _PP, _vp, ctypes.c_size_t, _vp]),
    "tpmlp_vocab_embedding_backward_workspace_bytes": (ctypes.c_size_t, [_i64, _i64, _i64]),
    "tpmlp_vocab_policy": (_int, [_int, _i64, _i64, _int, _vp, _i64, _vp, _vp, _vp, _vp, _f32, _f32,
                                  _f32, _f32, _vp, _vp, _vp, _vp, _vp]),
    "tpmlp_vocab_policy_backward": (_int, [_int, _i64, _i64, _int, _vp, _i64, _vp, _vp, _vp, _vp,
                                           _f32, _f32, _f32, _f32, _vp, _vp, _f32, _vp, _i64, _vp]),
    "tpmlp_vocab_policy_with_grad": (_int, [_int, _i64, _i64, _int, _vp, _i64, _vp, _vp, _vp, _vp,
                                            _f32, _f32, _f32, _f32, _vp, _vp, _vp, _vp, _vp, _f32,
                                            _vp, _i64, _vp]),
    "tpmlp_layernorm": (_int, [_int, _int, _i64, _i64, _vp, _i64, _vp, _vp, _f32, _vp, _i64, _vp, _vp,
                               _vp]),
    "tpmlp_layernorm_backward": (_int, [_int, _int, _i64, _i64, _vp, _i64, _vp, _i64, _vp, _vp, _vp,
                                        _vp, _i64, _vp, _i64, _vp, _vp, _vp, ctypes.c_size_t, _vp]),
    "tpmlp_layernorm_backward_workspace_bytes": (ctypes.c_size_t, [_i64, _i64]),
    "tpmlp_column_linear": (_int, [_int, _i64, _i64, _i64, _int, _int, _vp, _i64, _PP, _PP, _vp, _i64,
                                   _vp, _i64, _vp, _i64, _vp, ctypes.c_size_t, _vp]),
    "tpmlp_row_linear": (_int, [_int, _i64, _i64, _i64, _int, _vp, _i64, _PP, _vp, _vp, _i64, _vp, _i64,
                                _vp, ctypes.c_size_t, _vp]),
    "tpmlp_column_linear_backward": (_int, [_int, _i64, _i64, _i64, _int, _int, _vp, _i64, _PP, _vp,
                                            _i64, _vp, _i64, _vp, _i64, _PP, _PP, _vp,
                                            ctypes.c_size_t, _vp]),
    "tpmlp_row_linear_backward": (_int, [_int, _i64, _i64, _i64, _int, _vp, _i64, _PP, _vp, _i64, _vp,
                                         _i64, _PP, _vp, _vp, ctypes.c_size_t, _vp]),
    "tpmlp_block_reduce": (_int, [_int, _i64, _i64, _int, _PP, _vp, _vp, _vp]),
    "tpmlp_block_reduce_scatter": (_int, [_int, _i64, _i64, _int, _PP, _vp, _PP, _vp]),
    "tpmlp_forward_reduce_scatter": (_int, [_int, _i64, _i64, _i64, _int, _int, _vp, _PP, _PP, _PP,
                                            _vp, _PP, _PP, _PP, _int, _vp, ctypes.c_size_t, _vp]),
    "tpmlp_vocab_embedding": (_int, [_int, _i64, _i64, _i64, _int, _vp, _PP, _vp, _vp]),
    "tpmlp_vocab_ce": (_int, [_i64, _i64, _int, _vp, _vp, _vp, _vp, _vp, _vp, _vp]),
    "tpmlp_vocab_ce_backward": (_int, [_i64, _i64, _int, _vp, _vp, _vp, ctypes.c_float, _vp, _vp]),
    "tpmlp_workspace_bytes": (ctypes.c_size_t, [_int, _int, _i64, _i64, _i64, _int, _int]),
    "tpmlp_workspace_bytes_balanced": (ctypes.c_size_t, [_int, _int, _i64, _i64, _i64, _int, _int]),
    "tpmlp_status_str": (ctypes.c_char_p, [_int]),
    "tpmlp_check_device_error": (_int, [_vp]),
    "tpmlp_set_wait_timeout_ns": (None, [ctypes.c_uint64]),
    "tpmlp_selftest_wait_timeout": (_int, [ctypes.c_uint64, _vp]),
    "tpmlp_selftest_gemm_stall": (_int, [_int]),
    "tpmlp_selftest_weight_grad_stall": (_int, [_int]),
    "tpmlp_selftest_row_stall": (_int, [_int]),
    "tpmlp_launch_count": (ctypes.c_int64, []),
    "tpmlp_gemm_plan": (_int, [ctypes.c_int64, ctypes.c_int64, ctypes.c_int64, _int, _int, _int,
                               _int, ctypes.POINTER(_int), ctypes.POINTER(_int),
                               ctypes.POINTER(_int)]),
    "tpmlp_timing_enable": (None, [_int]),
    "tpmlp_timing_read": (_int, [ctypes.POINTER(KernelTiming), _int]),
    "tpmlp_timing_reset": (None, []),
}


def lib():
    """The loaded library (loads it on first use; raises if it is missing)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise ImportError(
                f"{LIB_PATH} is missing: build it first "
                "(python -c 'import __graft_entry__ as g; g.build()')")
        l = ctypes.CDLL(LIB_PATH)
        for name, (res, args) in _SIGNATURES.items():
            fn = getattr(l, name)
            fn.restype = res
            fn.argtypes = args
        _lib = l
    return _lib


def header_functions() -> List[str]:
    """Names of the functions include/tpmlp.h declares."""
    src = open(HEADER_PATH).read()
    src = re.sub(r"/\*.*?\*/", "", src, flags=re.S)
    return sorted(set(re.findall(r"\b(tpmlp_[a-z_]+)\s*\(", src)))


def status_str(status: int) -> str:
    return lib().tpmlp_status_str(int(status)).decode()


def _check(status: int):
    if status != OK:
        raise TpmlpError(status, status_str(status))


# Marshalling is on the clock of every small call (a call's kernels may take 4
# us), hence integers instead of ctypes objects, arrays instead of casts, and
# the stream's handle without a stream object where torch offers that.

def _ptr(t: Optional[torch.Tensor]):
    return None if t is None else t.data_ptr()


def _ptrs(ts: Optional[Sequence[torch.Tensor]]):
    """Host array of the tensors' addresses (a POINTER(c_void_p) argument)."""
    if ts is None:
        return None
    return (ctypes.c_void_p * len(ts))(*[t.data_ptr() for t in ts])


_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _stream(t: torch.Tensor):
    if not t.is_cuda:
        return None
    if _raw_stream is not None:
        return _raw_stream(t.get_device())
    return torch.cuda.current_stream(t.device).cuda_stream


def _dtype_code(t: torch.Tensor) -> int:
    if t.dtype not in DTYPE:
        raise TypeError(f"unsupported dtype {t.dtype}")
    return DTYPE[t.dtype]


def _require(ts, device, dtype):
    index = device.index   # None for the host
    for t in ts:
        if t is None:
            continue
        if t.get_device() != index:   # -1 for a host tensor
            raise ValueError("all tensors must live on the same CUDA device")
        if dtype is not None and t.dtype is not dtype:
            raise TypeError(f"expected {dtype}, got {t.dtype}")
        if not t.is_contiguous():
            raise ValueError("tensors must be contiguous (row-major)")


def _shards(ts, T: int, shape, device, dtype):
    """_require and _ptrs of T shards of one shape."""
    if len(ts) != T:
        raise ValueError(f"expected {T} shards, got {len(ts)}")
    index = device.index
    at = (ctypes.c_void_p * T)()
    for k, t in enumerate(ts):
        if t.shape != shape or t.dtype is not dtype or t.get_device() != index or not t.is_contiguous():
            _require([t], device, dtype)
            raise ValueError(f"expected a shard of {tuple(shape)}, got {tuple(t.shape)}")
        at[k] = t.data_ptr()
    return at


def _require_rows(t, what: str) -> int:
    """Row pitch of a [N, V] matrix whose rows are contiguous."""
    if t.dim() != 2:
        raise ValueError(f"{what} must be a matrix")
    N, V = t.shape
    if not t.is_cuda:
        raise ValueError("all tensors must live on the same CUDA device")
    if V > 1 and t.stride(1) != 1:
        raise ValueError(f"the rows of {what} must be contiguous")
    if N <= 1:
        return max(V, 1)
    if t.stride(0) < V:
        raise ValueError(f"the rows of {what} must not overlap")
    return t.stride(0)


def _run(t: torch.Tensor, fn, *args):
    """A call on t's device, which need not be the current one."""
    device = t.get_device()
    if device == torch._C._cuda_getDevice():
        _check(fn(*args))
        return
    with torch.cuda.device(device):
        _check(fn(*args))


def _require_matrix(t, shape, device, dtype, what: str) -> int:
    """Row pitch of a matrix of this shape whose rows are contiguous; 0 for None."""
    if t is None:
        return 0
    if t.get_device() != device.index:
        raise ValueError("all tensors must live on the same CUDA device")
    if t.dtype is not dtype:
        raise TypeError(f"expected {dtype} for {what}, got {t.dtype}")
    if t.shape != shape:
        raise ValueError(f"expected {what} of {tuple(shape)}, got {tuple(t.shape)}")
    return _require_rows(t, what)


def _bytes(workspace, device) -> int:
    _require([workspace], device, None)
    return 0 if workspace is None else workspace.numel() * workspace.element_size()


def _require_len(t, n: int, what: str):
    if t is not None and t.numel() != n:
        raise ValueError(f"{what} must hold {n} elements")


# ---------------------------------------------------------------------------
# The C-ABI calls, same names, tensors in place of pointers
# ---------------------------------------------------------------------------

def tpmlp_workspace_bytes(op: int, dtype: torch.dtype, N: int, D: int, F: int, T: int,
                          mode: str) -> int:
    return int(lib().tpmlp_workspace_bytes(op, DTYPE[dtype], N, D, F, T, MODE[mode]))


def tpmlp_workspace_bytes_balanced(op: int, dtype: torch.dtype, N: int, D: int, F: int, T: int,
                                   mode: str) -> int:
    """Workspace size that also holds the few-token GEMMs' stream-K scratch
    (see include/tpmlp.h)."""
    return int(lib().tpmlp_workspace_bytes_balanced(op, DTYPE[dtype], N, D, F, T, MODE[mode]))


def tpmlp_forward(X, W1, b1, W2, b2, Y, H, Z, act: str, mode: str, workspace=None):
    """Y = sum_r act(X W1[r] + b1[r]) W2[r] + b2 (see include/tpmlp.h).
    W1, W2, H, Z, b1 are lists of T tensors (b1, Z may be None)."""
    T = len(W1)
    N, D = X.shape
    Fs = W1[0].shape[1]
    _require([X, b2, Y, *W1, *W2, *H, *(b1 or []), *(Z or [])], X.device, X.dtype)
    _require([workspace], X.device, None)
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    _check(lib().tpmlp_forward(_dtype_code(X), N, D, Fs * T, T, ACT[act], _ptr(X), _ptrs(W1),
                               _ptrs(b1), _ptrs(W2), _ptr(b2), _ptr(Y), _ptrs(H), _ptrs(Z),
                               MODE[mode], _ptr(workspace), ws_bytes, _stream(X)))


def tpmlp_forward_noalloc(X, W1, b1, W2, b2, Y, H, Z, act: str):
    """tpmlp_forward in PARTIALS mode with the partial sums in the library's
    own fixed scratch array (no workspace, no device allocation); see
    include/tpmlp.h for its size limit and the sharing rules."""
    T = len(W1)
    N, D = X.shape
    Fs = W1[0].shape[1]
    _require([X, b2, Y, *W1, *W2, *H, *(b1 or []), *(Z or [])], X.device, X.dtype)
    _check(lib().tpmlp_forward_noalloc(_dtype_code(X), N, D, Fs * T, T, ACT[act], _ptr(X),
                                       _ptrs(W1), _ptrs(b1), _ptrs(W2), _ptr(b2), _ptr(Y),
                                       _ptrs(H), _ptrs(Z), _stream(X)))


def tpmlp_swiglu_forward(X, Wg, Wu, Wd, Y, H, G, U, mode: str, workspace=None):
    """Gated block: H^(r) = SiLU(X Wg[r]) * (X Wu[r]), Y = sum_r H^(r) Wd[r]."""
    T = len(Wg)
    N, D = X.shape
    Fs = Wg[0].shape[1]
    _require([X, Y, *Wg, *Wu, *Wd, *H, *(G or []), *(U or [])], X.device, X.dtype)
    _require([workspace], X.device, None)
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    _check(lib().tpmlp_swiglu_forward(_dtype_code(X), N, D, Fs * T, T, _ptr(X), _ptrs(Wg),
                                      _ptrs(Wu), _ptrs(Wd), _ptr(Y), _ptrs(H), _ptrs(G), _ptrs(U),
                                      MODE[mode], _ptr(workspace), ws_bytes, _stream(X)))


def tpmlp_backward(X, W1, W2, H, Z, dY, dX, dW1, dW2, db1, db2, act: str, mode: str, workspace):
    """Gradients of the block for upstream dY (see include/tpmlp.h)."""
    T = len(W1)
    N, D = X.shape
    Fs = W1[0].shape[1]
    _require([X, dY, dX, db2, *W1, *W2, *H, *Z, *dW1, *dW2, *(db1 or [])], X.device, X.dtype)
    _require([workspace], X.device, None)
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    _check(lib().tpmlp_backward(_dtype_code(X), N, D, Fs * T, T, ACT[act], _ptr(X), _ptrs(W1),
                                _ptrs(W2), _ptrs(H), _ptrs(Z), _ptr(dY), _ptr(dX), _ptrs(dW1),
                                _ptrs(dW2), _ptrs(db1), _ptr(db2), MODE[mode], _ptr(workspace),
                                ws_bytes, _stream(X)))


def tpmlp_block_reduce(partials: Sequence[torch.Tensor], b2, Y):
    """Y = sum_r partials[r] + b2, fp32 partials, Y fp32 or bf16."""
    T = len(partials)
    N, D = Y.shape
    _require([*partials], Y.device, torch.float32)
    _require([b2, Y], Y.device, Y.dtype)
    for p in partials:
        if p.dtype != torch.float32:
            raise TypeError("partial sums are fp32")
    _check(lib().tpmlp_block_reduce(_dtype_code(Y), N, D, T, _ptrs(partials), _ptr(b2), _ptr(Y),
                                    _stream(Y)))


def tpmlp_block_reduce_scatter(partials: Sequence[torch.Tensor], b2, Y_rows: Sequence[torch.Tensor]):
    """Rows [r N/T, (r+1) N/T) of sum_r partials[r] + b2 into Y_rows[r]."""
    T = len(partials)
    N, D = partials[0].shape
    _require([*partials], partials[0].device, torch.float32)
    _require([b2, *Y_rows], partials[0].device, Y_rows[0].dtype)
    _check(lib().tpmlp_block_reduce_scatter(_dtype_code(Y_rows[0]), N, D, T, _ptrs(partials),
                                            _ptr(b2), _ptrs(Y_rows), _stream(partials[0])))


def tpmlp_forward_reduce_scatter(X, W1, b1, W2, b2, Y_rows, H, Z, act: str, mode: str,
                                 workspace=None):
    """tpmlp_forward with the reduce-scatter block end: rank r's rows in Y_rows[r]."""
    T = len(W1)
    N, D = X.shape
    Fs = W1[0].shape[1]
    _require([X, b2, *Y_rows, *W1, *W2, *H, *(b1 or []), *(Z or [])], X.device, X.dtype)
    _require([workspace], X.device, None)
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    _check(lib().tpmlp_forward_reduce_scatter(
        _dtype_code(X), N, D, Fs * T, T, ACT[act], _ptr(X), _ptrs(W1), _ptrs(b1), _ptrs(W2),
        _ptr(b2), _ptrs(Y_rows), _ptrs(H), _ptrs(Z), MODE[mode], _ptr(workspace), ws_bytes,
        _stream(X)))


def tpmlp_vocab_embedding(ids, table: Sequence[torch.Tensor], out):
    """out[n] = table row ids[n] (table split by rows into len(table) shards)."""
    T = len(table)
    Vs, Hd = table[0].shape
    _require([ids], out.device, torch.int64)
    _require([*table, out], out.device, out.dtype)
    _check(lib().tpmlp_vocab_embedding(_dtype_code(out), ids.shape[0], Vs * T, Hd, T, _ptr(ids),
                                       _ptrs(table), _ptr(out), _stream(out)))


def tpmlp_vocab_ce(logits, targets, T: int, loss_per_token, loss_mean=None, argmax=None,
                   target_owner=None):
    """Vocab-parallel cross-entropy over T contiguous vocab shards."""
    N, V = logits.shape
    _require([logits], logits.device, torch.float32)
    _require([targets], logits.device, torch.int64)
    _require([loss_per_token, loss_mean], logits.device, torch.float32)
    _require([argmax, target_owner], logits.device, torch.int32)
    _check(lib().tpmlp_vocab_ce(N, V, T, _ptr(logits), _ptr(targets), _ptr(loss_per_token),
                                _ptr(loss_mean), _ptr(argmax), _ptr(target_owner),
                                _stream(logits)))


def tpmlp_vocab_ce_backward(logits, targets, T: int, loss_per_token, grad_scale: float, dlogits):
    """dlogits = grad_scale * (softmax(logits) - onehot(targets)); dlogits may
    be logits itself (in place)."""
    N, V = logits.shape
    _require([logits, loss_per_token, dlogits], logits.device, torch.float32)
    _require([targets], logits.device, torch.int64)
    _check(lib().tpmlp_vocab_ce_backward(N, V, T, _ptr(logits), _ptr(targets), _ptr(loss_per_token),
                                         float(grad_scale), _ptr(dlogits), _stream(logits)))


def tpmlp_swiglu_backward(X, Wg, Wu, Wd, H, G, U, dY, dX, dWg, dWu, dWd, mode: str, workspace):
    """Gradients of the gated block for upstream dY (see include/tpmlp.h)."""
    T = len(Wg)
    N, D = X.shape
    Fs = Wg[0].shape[1]
    dev, dt = X.device, X.dtype
    _require([X, dY, dX], dev, dt)
    if dY.shape != X.shape or dX.shape != X.shape:
        raise ValueError("dY and dX must have the shape of X")
    _require([workspace], dev, None)
    up, down, act = (D, Fs), (Fs, D), (N, Fs)
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    _check(lib().tpmlp_swiglu_backward(
        _dtype_code(X), N, D, Fs * T, T, X.data_ptr(), _shards(Wg, T, up, dev, dt),
        _shards(Wu, T, up, dev, dt), _shards(Wd, T, down, dev, dt), _shards(H, T, act, dev, dt),
        _shards(G, T, act, dev, dt), _shards(U, T, act, dev, dt), dY.data_ptr(), dX.data_ptr(),
        _shards(dWg, T, up, dev, dt), _shards(dWu, T, up, dev, dt), _shards(dWd, T, down, dev, dt),
        MODE[mode], _ptr(workspace), ws_bytes, _stream(X)))


def tpmlp_vocab_logprobs(logits, targets, T: int, K: int, logprob=None, rank=None, entropy=None,
                         lse=None, top_ids=None, top_logprobs=None):
    """Log probabilities and ranks of `targets`, entropies and the K most
    likely tokens of each row (see include/tpmlp.h)."""
    ld = _require_rows(logits, "logits")
    N, V = logits.shape
    _require([targets], logits.device, torch.int64)
    _require([logprob, entropy, lse, top_logprobs], logits.device, torch.float32)
    _require([rank, top_ids], logits.device, torch.int32)
    for t in (targets, logprob, rank, entropy, lse):
        _require_len(t, N, "a per-token tensor")
    for t in (top_ids, top_logprobs):
        _require_len(t, N * K, "a top list")
    _check(lib().tpmlp_vocab_logprobs(_dtype_code(logits), N, V, T, K, _ptr(logits), ld,
                                      _ptr(targets), _ptr(logprob), _ptr(rank), _ptr(entropy),
                                      _ptr(lse), _ptr(top_ids), _ptr(top_logprobs),
                                      _stream(logits)))


def _require_teacher(logits, teacher_ids, teacher_logits) -> int:
    _require([teacher_ids], logits.device, torch.int32)
    _require([teacher_logits], logits.device, torch.float32)
    N = logits.shape[0]
    if teacher_ids.dim() != 2 or teacher_ids.shape[0] != N or teacher_ids.shape != teacher_logits.shape:
        raise ValueError("teacher_ids and teacher_logits must be [N, K]")
    return teacher_ids.shape[1]


def tpmlp_vocab_distill(logits, teacher_ids, teacher_logits, T: int, tau: float, loss_per_token,
                        loss_mean=None, lse=None):
    """Distillation loss per token from the teacher's top tokens."""
    ld = _require_rows(logits, "logits")
    N, V = logits.shape
    K = _require_teacher(logits, teacher_ids, teacher_logits)
    _require([loss_per_token, loss_mean, lse], logits.device, torch.float32)
    for t in (loss_per_token, lse):
        _require_len(t, N, "a per-token tensor")
    _check(lib().tpmlp_vocab_distill(_dtype_code(logits), N, V, T, K, _ptr(logits), ld,
                                     _ptr(teacher_ids), _ptr(teacher_logits), float(tau),
                                     _ptr(loss_per_token), _ptr(loss_mean), _ptr(lse),
                                     _stream(logits)))


def _require_dlogits(logits, dlogits) -> int:
    ldd = _require_rows(dlogits, "dlogits")
    if (dlogits.shape != logits.shape or dlogits.dtype is not logits.dtype
            or dlogits.get_device() != logits.get_device()):
        raise ValueError("dlogits must have the shape, type and device of logits")
    return ldd


def tpmlp_vocab_distill_backward(logits, teacher_ids, teacher_logits, T: int, tau: float, lse,
                                 grad_tokens, grad_scale: float, dlogits):
    """Gradient of the distillation loss from the forward's lse; dlogits may be
    logits itself (in place)."""
    ld = _require_rows(logits, "logits")
    N, V = logits.shape
    K = _require_teacher(logits, teacher_ids, teacher_logits)
    ldd = _require_dlogits(logits, dlogits)
    _require([lse, grad_tokens], logits.device, torch.float32)
    for t in (lse, grad_tokens):
        _require_len(t, N, "a per-token tensor")
    _check(lib().tpmlp_vocab_distill_backward(_dtype_code(logits), N, V, T, K, _ptr(logits), ld,
                                              _ptr(teacher_ids), _ptr(teacher_logits), float(tau),
                                              _ptr(lse), _ptr(grad_tokens), float(grad_scale),
                                              _ptr(dlogits), ldd, _stream(logits)))


def tpmlp_vocab_distill_with_grad(logits, teacher_ids, teacher_logits, T: int, tau: float,
                                  loss_per_token, loss_mean, lse, grad_tokens, grad_scale: float,
                                  dlogits):
    """Loss and gradient in one launch; dlogits may be logits itself."""
    ld = _require_rows(logits, "logits")
    N, V = logits.shape
    K = _require_teacher(logits, teacher_ids, teacher_logits)
    ldd = _require_dlogits(logits, dlogits)
    _require([loss_per_token, loss_mean, lse, grad_tokens], logits.device, torch.float32)
    for t in (loss_per_token, lse, grad_tokens):
        _require_len(t, N, "a per-token tensor")
    _check(lib().tpmlp_vocab_distill_with_grad(
        _dtype_code(logits), N, V, T, K, _ptr(logits), ld, _ptr(teacher_ids), _ptr(teacher_logits),
        float(tau), _ptr(loss_per_token), _ptr(loss_mean), _ptr(lse), _ptr(grad_tokens),
        float(grad_scale), _ptr(dlogits), ldd, _stream(logits)))


def tpmlp_vocab_embedding_scaled(ids, table: Sequence[torch.Tensor], scale: float, out):
    """out[n] = scale * table row ids[n] (table split by rows into len(table) shards)."""
    T = len(table)
    Vs, Hd = table[0].shape
    _require([ids], out.device, torch.int64)
    _require([out], out.device, out.dtype)
    shards = _shards(table, T, (Vs, Hd), out.device, out.dtype)
    _require_len(out, ids.numel() * Hd, "out")
    _check(lib().tpmlp_vocab_embedding_scaled(_dtype_code(out), ids.numel(), Vs * T, Hd, T,
                                              _ptr(ids), shards, float(scale), _ptr(out),
                                              _stream(out)))


def tpmlp_vocab_embedding_backward_workspace_bytes(N: int, V: int, Hd: int) -> int:
    return int(lib().tpmlp_vocab_embedding_backward_workspace_bytes(N, V, Hd))


def tpmlp_vocab_embedding_backward(ids, dout, scale: float, accumulate: bool,
                                   dtable: Sequence[torch.Tensor], workspace):
    """dtable[v] = scale * sum of dout rows whose id is v (added to dtable with
    `accumulate`); dtable is split by rows into len(dtable) shards."""
    T = len(dtable)
    Vs, Hd = dtable[0].shape
    _require([ids], dout.device, torch.int64)
    _require([dout], dout.device, None)
    shards = _shards(dtable, T, (Vs, Hd), dout.device, dtable[0].dtype)
    _require([workspace], dout.device, None)
    _require_len(dout, ids.numel() * Hd, "dout")
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    _check(lib().tpmlp_vocab_embedding_backward(_dtype_code(dout), _dtype_code(dtable[0]),
                                                ids.numel(), Vs * T, Hd, T, _ptr(ids), _ptr(dout),
                                                float(scale), 1 if accumulate else 0,
                                                shards, _ptr(workspace), ws_bytes,
                                                _stream(dout)))


def _require_tokens(logits, targets, old_logprobs, advantages, ref_logprobs):
    N = logits.shape[0]
    _require([targets], logits.device, torch.int64)
    _require([old_logprobs, advantages, ref_logprobs], logits.device, torch.float32)
    for t in (targets, old_logprobs, advantages, ref_logprobs):
        _require_len(t, N, "a per-token tensor")


def tpmlp_vocab_policy(logits, targets, old_logprobs, advantages, ref_logprobs, T: int,
                       kl_coef: float, clip_low: float, clip_high: float, tau: float,
                       loss_per_token, loss_mean=None, logprob=None, kl=None):
    """Clipped policy loss of the given tokens with a KL term (see include/tpmlp.h)."""
    ld = _require_rows(logits, "logits")
    N, V = logits.shape
    _require_tokens(logits, targets, old_logprobs, advantages, ref_logprobs)
    _require([loss_per_token, loss_mean, logprob, kl], logits.device, torch.float32)
    for t in (loss_per_token, logprob, kl):
        _require_len(t, N, "a per-token tensor")
    _run(logits, lib().tpmlp_vocab_policy, _dtype_code(logits), N, V, T, _ptr(logits), ld, _ptr(targets),
         _ptr(old_logprobs), _ptr(advantages), _ptr(ref_logprobs), float(kl_coef), float(clip_low),
         float(clip_high), float(tau), _ptr(loss_per_token), _ptr(loss_mean), _ptr(logprob), _ptr(kl),
         _stream(logits))


def tpmlp_vocab_policy_backward(logits, targets, old_logprobs, advantages, ref_logprobs, T: int,
                                kl_coef: float, clip_low: float, clip_high: float, tau: float, logprob,
                                grad_tokens, grad_scale: float, dlogits):
    """Gradient of the policy loss from the forward's logprob; dlogits may be
    logits itself (in place)."""
    ld = _require_rows(logits, "logits")
    N, V = logits.shape
    _require_tokens(logits, targets, old_logprobs, advantages, ref_logprobs)
    ldd = _require_dlogits(logits, dlogits)
    _require([logprob, grad_tokens], logits.device, torch.float32)
    for t in (logprob, grad_tokens):
        _require_len(t, N, "a per-token tensor")
    _run(logits, lib().tpmlp_vocab_policy_backward, _dtype_code(logits), N, V, T, _ptr(logits), ld,
         _ptr(targets), _ptr(old_logprobs), _ptr(advantages), _ptr(ref_logprobs), float(kl_coef),
         float(clip_low), float(clip_high), float(tau), _ptr(logprob), _ptr(grad_tokens),
         float(grad_scale), _ptr(dlogits), ldd, _stream(logits))


def tpmlp_vocab_policy_with_grad(logits, targets, old_logprobs, advantages, ref_logprobs, T: int,
                                 kl_coef: float, clip_low: float, clip_high: float, tau: float,
                                 loss_per_token, loss_mean, logprob, kl, grad_tokens,
                                 grad_scale: float, dlogits):
    """Loss and gradient in one launch; dlogits may be logits itself."""
    ld = _require_rows(logits, "logits")
    N, V = logits.shape
    _require_tokens(logits, targets, old_logprobs, advantages, ref_logprobs)
    ldd = _require_dlogits(logits, dlogits)
    _require([loss_per_token, loss_mean, logprob, kl, grad_tokens], logits.device, torch.float32)
    for t in (loss_per_token, logprob, kl, grad_tokens):
        _require_len(t, N, "a per-token tensor")
    _run(logits, lib().tpmlp_vocab_policy_with_grad, _dtype_code(logits), N, V, T, _ptr(logits), ld,
         _ptr(targets), _ptr(old_logprobs), _ptr(advantages), _ptr(ref_logprobs), float(kl_coef),
         float(clip_low), float(clip_high), float(tau), _ptr(loss_per_token), _ptr(loss_mean),
         _ptr(logprob), _ptr(kl), _ptr(grad_tokens), float(grad_scale), _ptr(dlogits), ldd,
         _stream(logits))


def _require_params(x, *params):
    """Element type of a layer norm's parameters: one for all, x's where there are none."""
    given = [p for p in params if p is not None]
    dtype = given[0].dtype if given else x.dtype
    _require(given, x.device, dtype)
    for p in given:
        _require_len(p, x.shape[1], "a parameter")
    return _dtype_code(given[0] if given else x)


def tpmlp_layernorm(x, weight, bias, eps: float, y, mean=None, rstd=None):
    """y = (x - mean) rstd weight + bias over the rows of x; y may be x itself."""
    ldx = _require_rows(x, "x")
    N, D = x.shape
    ldy = _require_matrix(y, x.shape, x.device, x.dtype, "y")
    param_dt = _require_params(x, weight, bias)
    _require([mean, rstd], x.device, torch.float32)
    for t in (mean, rstd):
        _require_len(t, N, "a per-row tensor")
    _run(x, lib().tpmlp_layernorm, _dtype_code(x), param_dt, N, D, _ptr(x), ldx, _ptr(weight), _ptr(bias),
         float(eps), _ptr(y), ldy, _ptr(mean), _ptr(rstd), _stream(x))


def tpmlp_layernorm_backward_workspace_bytes(N: int, D: int) -> int:
    return int(lib().tpmlp_layernorm_backward_workspace_bytes(N, D))


def tpmlp_layernorm_backward(dy, x, weight, mean, rstd, dresidual, dx, dweight, dbias, workspace):
    """Gradients of the layer norm; dx may be dy, x or dresidual itself."""
    ldx = _require_rows(x, "x")
    N, D = x.shape
    lddy, lddres, lddx = (_require_matrix(t, x.shape, x.device, x.dtype, what) for t, what in
                          ((dy, "dy"), (dresidual, "dresidual"), (dx, "dx")))
    param_dt = _require_params(x, weight, dweight, dbias)
    _require([mean, rstd], x.device, torch.float32)
    for t in (mean, rstd):
        _require_len(t, N, "a per-row tensor")
    ws_bytes = _bytes(workspace, x.device)
    _run(x, lib().tpmlp_layernorm_backward, _dtype_code(x), param_dt, N, D, _ptr(dy), lddy, _ptr(x), ldx,
         _ptr(weight), _ptr(mean), _ptr(rstd), _ptr(dresidual), lddres, _ptr(dx), lddx, _ptr(dweight),
         _ptr(dbias), _ptr(workspace), ws_bytes, _stream(x))


def tpmlp_column_linear(X, W, b, act, R, Y, Z, workspace=None):
    """Y = act(X W + b) + R, W's columns in len(W) shards (b: a list, or None);
    Z, if given, receives X W + b."""
    ldx = _require_rows(X, "X")
    N, D = X.shape
    T, Fs = len(W), W[0].shape[1]
    dev, dt, out = X.device, X.dtype, (N, T * Fs)
    ldr, ldy, ldz = (_require_matrix(t, out, dev, dt, what) for t, what in ((R, "R"), (Y, "Y"), (Z, "Z")))
    ws_bytes = _bytes(workspace, dev)
    _run(X, lib().tpmlp_column_linear, _dtype_code(X), N, D, Fs * T, T, LINEAR_ACT[act], _ptr(X), ldx,
         _shards(W, T, (D, Fs), dev, dt), None if b is None else _shards(b, T, (Fs,), dev, dt), _ptr(R),
         ldr, _ptr(Y), ldy, _ptr(Z), ldz, _ptr(workspace), ws_bytes, _stream(X))


def tpmlp_row_linear(X, W, b, R, Y, workspace=None):
    """Y = sum_r X[:, shard r] W[r] + b + R, W's rows in len(W) shards."""
    ldx = _require_rows(X, "X")
    T = len(W)
    Fs, D = W[0].shape
    dev, dt, out = X.device, X.dtype, (X.shape[0], D)
    if X.shape[1] != T * Fs:
        raise ValueError(f"X has {X.shape[1]} columns, W {T * Fs} rows")
    ldr, ldy = (_require_matrix(t, out, dev, dt, what) for t, what in ((R, "R"), (Y, "Y")))
    _require([b], dev, dt)
    _require_len(b, D, "b")
    ws_bytes = _bytes(workspace, dev)
    _run(X, lib().tpmlp_row_linear, _dtype_code(X), X.shape[0], D, Fs * T, T, _ptr(X), ldx,
         _shards(W, T, (Fs, D), dev, dt), _ptr(b), _ptr(R), ldr, _ptr(Y), ldy, _ptr(workspace), ws_bytes,
         _stream(X))


def tpmlp_column_linear_backward(X, W, Z, dY, act, dX, dW, db, workspace=None):
    """Gradients of column_linear for upstream dY (db: a list, or None)."""
    ldx = _require_rows(X, "X")
    N, D = X.shape
    T, Fs = len(W), W[0].shape[1]
    dev, dt, out = X.device, X.dtype, (N, T * Fs)
    ldz, lddy = (_require_matrix(t, out, dev, dt, what) for t, what in ((Z, "Z"), (dY, "dY")))
    lddx = _require_matrix(dX, X.shape, dev, dt, "dX")
    ws_bytes = _bytes(workspace, dev)
    _run(X, lib().tpmlp_column_linear_backward, _dtype_code(X), N, D, Fs * T, T, LINEAR_ACT[act], _ptr(X),
         ldx, _shards(W, T, (D, Fs), dev, dt), _ptr(Z), ldz, _ptr(dY), lddy, _ptr(dX), lddx,
         _shards(dW, T, (D, Fs), dev, dt), None if db is None else _shards(db, T, (Fs,), dev, dt),
         _ptr(workspace), ws_bytes, _stream(X))


def tpmlp_row_linear_backward(X, W, dY, dX, dW, db, workspace=None):
    """Gradients of row_linear for upstream dY (db: [D], or None)."""
    ldx = _require_rows(X, "X")
    T = len(W)
    Fs, D = W[0].shape
    dev, dt = X.device, X.dtype
    if X.shape[1] != T * Fs:
        raise ValueError(f"X has {X.shape[1]} columns, W {T * Fs} rows")
    lddy = _require_matrix(dY, (X.shape[0], D), dev, dt, "dY")
    lddx = _require_matrix(dX, X.shape, dev, dt, "dX")
    _require([db], dev, dt)
    _require_len(db, D, "db")
    ws_bytes = _bytes(workspace, dev)
    _run(X, lib().tpmlp_row_linear_backward, _dtype_code(X), X.shape[0], D, Fs * T, T, _ptr(X), ldx,
         _shards(W, T, (Fs, D), dev, dt), _ptr(dY), lddy, _ptr(dX), lddx, _shards(dW, T, (Fs, D), dev, dt),
         _ptr(db), _ptr(workspace), ws_bytes, _stream(X))


def tpmlp_check_device_error(device=None) -> int:
    """Synchronizes the current stream and returns (and clears) the device
    error word: OK, ERR_TIMEOUT or ERR_ARG."""
    s = torch.cuda.current_stream(device).cuda_stream
    return int(lib().tpmlp_check_device_error(ctypes.c_void_p(s)))


def tpmlp_set_wait_timeout_ns(ns: int):
    lib().tpmlp_set_wait_timeout_ns(int(ns))


def tpmlp_selftest_wait_timeout(timeout_ns: int, device=None):
    s = torch.cuda.current_stream(device).cuda_stream
    _check(lib().tpmlp_selftest_wait_timeout(int(timeout_ns), ctypes.c_void_p(s)))


def tpmlp_selftest_gemm_stall(role: int):
    """While role is 1 (epilogue), 2 (MMA issuer) or 3 (TMA producer), every
    bf16 GEMM launch makes that role stall on a barrier nothing completes
    until the bounded wait runs out; 0 turns it off."""
    _check(lib().tpmlp_selftest_gemm_stall(int(role)))


def tpmlp_selftest_weight_grad_stall(role: int):
    """The same for the launch of few-token weight gradients alone."""
    _check(lib().tpmlp_selftest_weight_grad_stall(int(role)))


def tpmlp_selftest_row_stall(on: int):
    """While on is 1, every kernel that takes rows in turn waits on a barrier that
    nothing completes until the bounded wait runs out."""
    _check(lib().tpmlp_selftest_row_stall(int(on)))


def tpmlp_launch_count() -> int:
    return int(lib().tpmlp_launch_count())


def tpmlp_gemm_plan(M: int, N: int, K: int, G: int, fold: bool = False, dual: bool = False,
                    balanced: bool = False):
    """Launch configuration of the bf16 tensor-core GEMM for this shape on the
    current device: (accumulator columns, CTAs per MMA, K split: cluster size,
    or 0 for stream-K, which needs balanced=True)."""
    bn, ctas, ks = _int(0), _int(0), _int(0)
    _check(lib().tpmlp_gemm_plan(M, N, K, G, 1 if fold else 0, 1 if dual else 0,
                                 1 if balanced else 0, ctypes.byref(bn), ctypes.byref(ctas),
                                 ctypes.byref(ks)))
    return bn.value, ctas.value, ks.value


def tpmlp_timing_enable(on: bool):
    lib().tpmlp_timing_enable(1 if on else 0)


def tpmlp_timing_read() -> dict:
    buf = (KernelTiming * 64)()
    n = lib().tpmlp_timing_read(buf, 64)
    if n < 0:
        raise TpmlpError(ERR_CUDA, "timing read failed")
    return {buf[i].name.decode(): {"launches": int(buf[i].launches), "total_ms": float(buf[i].total_ms)}
            for i in range(n)}


def tpmlp_timing_reset():
    lib().tpmlp_timing_reset()
