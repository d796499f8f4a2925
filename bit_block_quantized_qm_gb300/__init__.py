"""GGML Q4_0 x f32 quantized matmul, Q4_0 dequant and Q8_0 dequant/quantize on
GB300 (sm_103a).

A thin Python binding over the C ABI of ``libqm.so`` (``include/qm.h``): it
only marshals arguments.  Every step of the computation runs in the library's
CUDA kernels; there is no host fallback, and calls fail loudly when the
library has not been built.  PyTorch supplies device memory and streams.

Entry points (same names as the C ABI):

* ``qm_dequant_q4_0(wq, out=None, stream=None)`` -> f32 tensor ``[n_blocks*32]``
* ``qm_dequant_q8_0(wq, out=None, stream=None)`` -> f32 tensor ``[n_blocks*32]``
* ``qm_quantize_q8_0(x, out=None, stream=None)`` -> uint8 tensor ``[n/32*34]``
* ``qm_matmul_q4_0(A, wq, N, out=None, stream=None)`` -> f32 tensor ``[M, N]``
* ``qm_matmul_q4_0_algo(A, wq, N, algo, out=None, stream=None)``
* ``qm_gemv_q4_0_list(problems, M, counters=None, stream=None)``: a list of
  GEMV problems ``(A, wq, C, N, wait_for)`` in one persistent launch
* ``KVCache(k_pages, v_pages, page_table, lengths, ...)``: a paged 4-bit
  key/value cache, with ``qm_kv_append_q4_0``, ``qm_kv_read_q4_0``,
  ``qm_attn_q4_0`` and ``qm_kv_evict_q4_0`` over it
* ``qm_device_status(stream=None, clear=True)``, ``qm_status_string(code)``,
  ``qm_version()``

The ``*_ptr`` variants take raw device addresses (ints) instead of tensors.
"""
from __future__ import annotations

import contextlib
import ctypes
import os
import struct
import threading

__all__ = [
    "QMError", "load_library", "library_path", "qm_version", "qm_status_string",
    "qm_dequant_q4_0", "qm_matmul_q4_0", "qm_matmul_q4_0_algo", "qm_device_status",
    "qm_launch_count",
    "qm_dequant_q4_0_ptr", "qm_matmul_q4_0_ptr", "qm_matmul_q4_0_algo_ptr",
    "qm_dequant_q8_0", "qm_quantize_q8_0", "qm_dequant_q8_0_ptr", "qm_quantize_q8_0_ptr",
    "QM_OK", "QM_ERR_NULL", "QM_ERR_SHAPE", "QM_ERR_ALIGN", "QM_ERR_ALIAS", "QM_ERR_CUDA",
    "QM_ERR_TIMEOUT", "QM_ERR_UNSUPPORTED", "QM_ERR_POINTER", "QM_ERR_TOO_LARGE",
    "qm_matmul_q4_0_noalloc_ptr", "qm_selftest_wait_timeout",
    "qm_matmul_q4_0_q8act", "qm_matmul_q4_0_q8act_ptr", "qm_gemv_q4_0_q8act_list_ptr",
    "QM_ALGO_AUTO", "QM_ALGO_GEMV", "QM_ALGO_GEMM_SIMT", "QM_ALGO_GEMV_SIMT", "QM_ALGO_GEMM_TC",
    "QM_ALGO_GEMV_PK", "qm_gemv_plan", "GEMV_PLAN_FIELDS", "qm_gemm_plan", "GEMM_PLAN_FIELDS",
    "EXPORTED_SYMBOLS", "QmGemvProblem", "qm_gemv_q4_0_list_ptr", "qm_gemv_q4_0_list",
    "gemv_problem_array",
    "QM_ERR_RANGE", "QM_ERR_WORKSPACE", "QM_F32", "QM_BF16", "QmKVCache", "QmAttnArgs", "KVCache", "kv_page_bytes",
    "ATTN_WORKSPACE_ZEROED",
    "qm_kv_append_q4_0", "qm_kv_read_q4_0", "qm_attn_q4_0", "qm_attn_workspace", "qm_kv_evict_q4_0",
]

QM_OK = 0
QM_ERR_NULL = -1
QM_ERR_SHAPE = -2
QM_ERR_ALIGN = -3
QM_ERR_ALIAS = -4
QM_ERR_CUDA = -5
QM_ERR_TIMEOUT = -6
QM_ERR_UNSUPPORTED = -7
QM_ERR_POINTER = -8
QM_ERR_TOO_LARGE = -9
QM_ERR_RANGE = -10
QM_ERR_WORKSPACE = -11

QM_F32 = 0
QM_BF16 = 1

ATTN_WORKSPACE_ZEROED = 4096

QM_ALGO_AUTO = 0
QM_ALGO_GEMV = 1
QM_ALGO_GEMM_SIMT = 2
QM_ALGO_GEMV_SIMT = 3
QM_ALGO_GEMM_TC = 4
QM_ALGO_GEMV_PK = 5

BLOCK_BYTES = 18
BLOCK_ELEMS = 32
Q8_0_BLOCK_BYTES = 34

# Every symbol include/qm.h declares.
EXPORTED_SYMBOLS = ("qm_version", "qm_status_string", "qm_dequant_q4_0", "qm_matmul_q4_0",
                    "qm_matmul_q4_0_algo", "qm_device_status", "qm_launch_count", "qm_gemv_plan", "qm_gemm_plan",
                    "qm_matmul_q4_0_noalloc", "qm_dequant_q8_0", "qm_quantize_q8_0",
                    "qm_selftest_wait_timeout", "qm_gemv_q4_0_list", "qm_matmul_q4_0_q8act",
                    "qm_gemv_q4_0_q8act_list", "qm_kv_append_q4_0", "qm_kv_read_q4_0", "qm_attn_q4_0",
                    "qm_attn_workspace", "qm_attn_workspace_exact", "qm_kv_evict_q4_0")

_HERE = os.path.dirname(os.path.abspath(__file__))
_LIB_PATH = os.path.join(_HERE, "_build", "libqm.so")
_lock = threading.Lock()
_lib = None


class QmGemvProblem(ctypes.Structure):
    """One problem of qm_gemv_q4_0_list (the C struct qm_gemv_problem)."""
    _fields_ = [("A", ctypes.c_void_p), ("wq", ctypes.c_void_p), ("C", ctypes.c_void_p),
                ("N", ctypes.c_int64), ("K", ctypes.c_int64), ("wait_for", ctypes.c_int32),
                ("reserved", ctypes.c_int32)]


class QmKVCache(ctypes.Structure):
    """The C struct qm_kv_cache (see include/qm.h)."""
    _fields_ = [("k_pages", ctypes.c_void_p), ("v_pages", ctypes.c_void_p), ("page_table", ctypes.c_void_p),
                ("lengths", ctypes.c_void_p), ("n_pages", ctypes.c_int64), ("table_stride", ctypes.c_int64),
                ("max_len", ctypes.c_int64), ("n_seqs", ctypes.c_int32), ("n_kv_heads", ctypes.c_int32),
                ("head_dim", ctypes.c_int32), ("page_tokens", ctypes.c_int32), ("reserved", ctypes.c_int32)]


class QmAttnArgs(ctypes.Structure):
    """The C struct qm_attn_args (see include/qm.h)."""
    _fields_ = [("q", ctypes.c_void_p), ("out", ctypes.c_void_p), ("lse", ctypes.c_void_p),
                ("weights", ctypes.c_void_p), ("q_starts", ctypes.c_void_p), ("workspace", ctypes.c_void_p),
                ("workspace_bytes", ctypes.c_int64), ("n_tokens", ctypes.c_int64), ("max_q", ctypes.c_int64),
                ("q_stride", ctypes.c_int64), ("out_stride", ctypes.c_int64), ("weights_stride", ctypes.c_int64),
                ("window", ctypes.c_int64), ("sinks", ctypes.c_int64), ("n_heads", ctypes.c_int64),
                ("scale", ctypes.c_float), ("dtype", ctypes.c_int32), ("reserved", ctypes.c_int32)]


_ATTN_ARGS = struct.Struct("@6P9qfii4x")  # the same, packed
assert _ATTN_ARGS.size == ctypes.sizeof(QmAttnArgs)


class QMError(RuntimeError):
    """A negative status returned by libqm."""

    def __init__(self, code: int, where: str):
        self.code = code
        super().__init__(f"{where}: {qm_status_string(code)} (status {code})")


def library_path() -> str:
    return _LIB_PATH


def load_library() -> ctypes.CDLL:
    """Load libqm.so (built by ``bit_block_quantized_qm_gb300.build.build()``)."""
    global _lib
    if _lib is not None:
        return _lib
    with _lock:
        if _lib is None:
            if not os.path.exists(_LIB_PATH):
                raise RuntimeError(
                    f"libqm.so is not built ({_LIB_PATH}); run "
                    "`python -c 'import __graft_entry__ as g; g.build()'` first")
            lib = ctypes.CDLL(_LIB_PATH)
            i64, p, i32 = ctypes.c_int64, ctypes.c_void_p, ctypes.c_int
            lib.qm_version.argtypes = []
            lib.qm_version.restype = i32
            lib.qm_status_string.argtypes = [i32]
            lib.qm_status_string.restype = ctypes.c_char_p
            lib.qm_dequant_q4_0.argtypes = [p, i64, p, p]
            lib.qm_dequant_q4_0.restype = i32
            lib.qm_matmul_q4_0.argtypes = [p, p, p, i64, i64, i64, p]
            lib.qm_matmul_q4_0.restype = i32
            lib.qm_matmul_q4_0_algo.argtypes = [p, p, p, i64, i64, i64, i32, p]
            lib.qm_matmul_q4_0_algo.restype = i32
            lib.qm_gemv_plan.argtypes = [i64, i64, i64, i32, i32, i32, i32, i32, i32, i32, p]
            lib.qm_gemv_plan.restype = i32
            lib.qm_gemm_plan.argtypes = [i64, i64, i64, i32, i32, i32, i32, p]
            lib.qm_gemm_plan.restype = i32
            lib.qm_device_status.argtypes = [p, i32]
            lib.qm_selftest_wait_timeout.argtypes = [p]
            lib.qm_selftest_wait_timeout.restype = i32
            lib.qm_device_status.restype = i32
            lib.qm_matmul_q4_0_noalloc.argtypes = [p, p, p, i64, i64, i64, p]
            lib.qm_matmul_q4_0_noalloc.restype = i32
            lib.qm_matmul_q4_0_q8act.argtypes = [p, p, p, i64, i64, i64, p]
            lib.qm_matmul_q4_0_q8act.restype = i32
            lib.qm_dequant_q8_0.argtypes = [p, i64, p, p]
            lib.qm_dequant_q8_0.restype = i32
            lib.qm_quantize_q8_0.argtypes = [p, i64, p, p]
            lib.qm_quantize_q8_0.restype = i32
            lib.qm_gemv_q4_0_list.argtypes = [p, i64, i64, p, p]
            lib.qm_gemv_q4_0_list.restype = i32
            lib.qm_gemv_q4_0_q8act_list.argtypes = [p, i64, i64, p, p]
            lib.qm_gemv_q4_0_q8act_list.restype = i32
            lib.qm_kv_append_q4_0.argtypes = [p, p, p, i32, i64, i64, i64, p, p]
            lib.qm_kv_append_q4_0.restype = i32
            lib.qm_kv_read_q4_0.argtypes = [p, p, p, i64, p, p]
            lib.qm_kv_read_q4_0.restype = i32
            lib.qm_attn_q4_0.argtypes = [p, p, p]
            lib.qm_attn_q4_0.restype = i32
            lib.qm_attn_workspace.argtypes = [p, i64, i64, i64, i32]
            lib.qm_attn_workspace.restype = i64
            lib.qm_attn_workspace_exact.argtypes = [p, i64, i64, i64, i32]
            lib.qm_attn_workspace_exact.restype = i64
            lib.qm_kv_evict_q4_0.argtypes = [p, p, p, i64, i64, i64, i64, p, p, i64, p]
            lib.qm_kv_evict_q4_0.restype = i32
            lib.qm_launch_count.argtypes = []
            lib.qm_launch_count.restype = ctypes.c_uint64
            _lib = lib
    return _lib


def qm_version() -> int:
    return load_library().qm_version()


def qm_status_string(code: int) -> str:
    return load_library().qm_status_string(int(code)).decode()


def _check(code: int, where: str) -> int:
    if code != QM_OK:
        raise QMError(code, where)
    return code


# ------------------------------------------------------------ raw pointers

def qm_dequant_q4_0_ptr(wq: int, n_blocks: int, out: int, stream: int = 0) -> int:
    return load_library().qm_dequant_q4_0(wq, n_blocks, out, stream)


def qm_dequant_q8_0_ptr(wq: int, n_blocks: int, out: int, stream: int = 0) -> int:
    return load_library().qm_dequant_q8_0(wq, n_blocks, out, stream)


def qm_quantize_q8_0_ptr(x: int, n_elements: int, out: int, stream: int = 0) -> int:
    return load_library().qm_quantize_q8_0(x, n_elements, out, stream)


def qm_matmul_q4_0_ptr(A: int, wq: int, C: int, M: int, N: int, K: int, stream: int = 0) -> int:
    return load_library().qm_matmul_q4_0(A, wq, C, M, N, K, stream)


def qm_matmul_q4_0_algo_ptr(A: int, wq: int, C: int, M: int, N: int, K: int, algo: int,
                            stream: int = 0) -> int:
    return load_library().qm_matmul_q4_0_algo(A, wq, C, M, N, K, algo, stream)


def qm_selftest_wait_timeout(stream=None) -> int:
    """Enqueue the failure-path self-test kernel (a bounded wait that runs
    out); the next qm_device_status reports QM_ERR_TIMEOUT.  Returns the C
    status."""
    return load_library().qm_selftest_wait_timeout(_stream_handle(stream))


def qm_matmul_q4_0_noalloc_ptr(A: int, wq: int, C: int, M: int, N: int, K: int,
                               stream: int = 0) -> int:
    """The allocation-free GEMV (M <= 8); see include/qm.h."""
    return load_library().qm_matmul_q4_0_noalloc(A, wq, C, M, N, K, stream)


def qm_matmul_q4_0_q8act_ptr(A: int, wq: int, C: int, M: int, N: int, K: int,
                             stream: int = 0) -> int:
    """The product with the activations quantized to Q8_0 first (M <= 8);
    see include/qm.h."""
    return load_library().qm_matmul_q4_0_q8act(A, wq, C, M, N, K, stream)


def qm_gemv_q4_0_list_ptr(problems, M: int, counters: int = 0, stream: int = 0,
                          q8act: bool = False) -> int:
    """The list GEMV on raw addresses: `problems` is a sequence of (A, wq, C, N,
    K, wait_for) tuples of ints, or an array built once by
    gemv_problem_array; `counters` the device address of len(problems)
    uint32 (0 for none).  With `q8act`, qm_gemv_q4_0_q8act_list (the
    act-quant product).  Returns the C status."""
    arr = problems if isinstance(problems, ctypes.Array) else gemv_problem_array(problems)
    fn = load_library().qm_gemv_q4_0_q8act_list if q8act else load_library().qm_gemv_q4_0_list
    return fn(ctypes.cast(arr, ctypes.c_void_p), len(problems), M, counters or None, stream)


def gemv_problem_array(problems):
    """The C array of qm_gemv_problem for a sequence of (A, wq, C, N, K,
    wait_for) tuples, for callers that pass the same list many times."""
    arr = (QmGemvProblem * len(problems))()
    for i, (A, wq, C, N, K, wait_for) in enumerate(problems):
        arr[i] = QmGemvProblem(A, wq, C, N, K, wait_for, 0)
    return arr


def qm_gemv_q4_0_q8act_list_ptr(problems, M: int, counters: int = 0, stream: int = 0) -> int:
    """qm_gemv_q4_0_q8act_list on raw addresses (see qm_gemv_q4_0_list_ptr)."""
    return qm_gemv_q4_0_list_ptr(problems, M, counters, stream, q8act=True)


# ------------------------------------------------------------ torch tensors

_torch = None


def _torch_module():
    """torch, which the package itself does not import: an import statement in
    every call costs a small call 2 us of its 18."""
    global _torch
    if _torch is None:
        import torch
        _torch = torch
    return _torch


def _stream_handle(stream) -> int:
    torch = _torch or _torch_module()
    if stream is None:
        # The current stream's handle without building a Stream object around it
        # (6 us of a small call's 25).
        raw = getattr(torch._C, "_cuda_getCurrentRawStream", None)
        if raw is not None and torch.cuda.is_initialized():
            return raw(torch._C._cuda_getDevice())
        stream = torch.cuda.current_stream()
    return int(stream.cuda_stream)


def _require(t, dtype, name):
    torch = _torch or _torch_module()
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


def qm_dequant_q4_0(wq, out=None, stream=None):
    """Dequantize a Q4_0 block stream (uint8 CUDA tensor, n_blocks*18 bytes)
    into f32 ``[n_blocks*32]``."""
    import torch
    _require(wq, torch.uint8, "wq")
    if wq.numel() % BLOCK_BYTES:
        raise ValueError("wq length is not a multiple of 18 bytes")
    n_blocks = wq.numel() // BLOCK_BYTES
    if out is None:
        out = torch.empty(n_blocks * BLOCK_ELEMS, dtype=torch.float32, device=wq.device)
    _require(out, torch.float32, "out")
    if out.numel() != n_blocks * BLOCK_ELEMS:
        raise ValueError("out has the wrong number of elements")
    _check(qm_dequant_q4_0_ptr(wq.data_ptr(), n_blocks, out.data_ptr(), _stream_handle(stream)),
           "qm_dequant_q4_0")
    return out


def qm_dequant_q8_0(wq, out=None, stream=None):
    """Dequantize a Q8_0 block stream (uint8 CUDA tensor, n_blocks*34 bytes)
    into f32 ``[n_blocks*32]``."""
    import torch
    _require(wq, torch.uint8, "wq")
    if wq.numel() % Q8_0_BLOCK_BYTES:
        raise ValueError("wq length is not a multiple of 34 bytes")
    n_blocks = wq.numel() // Q8_0_BLOCK_BYTES
    if out is None:
        out = torch.empty(n_blocks * BLOCK_ELEMS, dtype=torch.float32, device=wq.device)
    _require(out, torch.float32, "out")
    if out.numel() != n_blocks * BLOCK_ELEMS:
        raise ValueError("out has the wrong number of elements")
    _check(qm_dequant_q8_0_ptr(wq.data_ptr(), n_blocks, out.data_ptr(), _stream_handle(stream)),
           "qm_dequant_q8_0")
    return out


def qm_quantize_q8_0(x, out=None, stream=None):
    """Quantize f32 (a CUDA tensor of a multiple of 32 elements) into a Q8_0
    block stream (uint8 ``[n/32*34]``)."""
    import torch
    _require(x, torch.float32, "x")
    if x.numel() % BLOCK_ELEMS:
        raise ValueError("x has a number of elements that is not a multiple of 32")
    n_out = x.numel() // BLOCK_ELEMS * Q8_0_BLOCK_BYTES
    if out is None:
        out = torch.empty(n_out, dtype=torch.uint8, device=x.device)
    _require(out, torch.uint8, "out")
    if out.numel() != n_out:
        raise ValueError("out has the wrong number of bytes")
    _check(qm_quantize_q8_0_ptr(x.data_ptr(), x.numel(), out.data_ptr(), _stream_handle(stream)),
           "qm_quantize_q8_0")
    return out


def qm_matmul_q4_0_algo(A, wq, N: int, algo: int, out=None, stream=None):
    """C[M, N] = A[M, K] x dequant(W)^T with the algorithm forced."""
    import torch
    _require(A, torch.float32, "A")
    _require(wq, torch.uint8, "wq")
    if A.dim() != 2:
        raise ValueError("A must be 2-D [M, K]")
    M, K = A.shape
    if K % BLOCK_ELEMS or wq.numel() != N * (K // BLOCK_ELEMS) * BLOCK_BYTES:
        raise ValueError("wq size does not match N x K")
    if out is None:
        out = torch.empty((M, N), dtype=torch.float32, device=A.device)
    _require(out, torch.float32, "out")
    if out.numel() != M * N:
        raise ValueError("out has the wrong number of elements")
    _check(qm_matmul_q4_0_algo_ptr(A.data_ptr(), wq.data_ptr(), out.data_ptr(), M, N, K, algo,
                                   _stream_handle(stream)), "qm_matmul_q4_0")
    return out


def qm_matmul_q4_0(A, wq, N: int, out=None, stream=None):
    """C[M, N] = A[M, K] x dequant(W)^T; GEMV kernels for M <= 8, GEMM above."""
    return qm_matmul_q4_0_algo(A, wq, N, QM_ALGO_AUTO, out=out, stream=stream)


def qm_matmul_q4_0_q8act(A, wq, N: int, out=None, stream=None):
    """C[M, N] = dequant_q8_0(quantize_q8_0(A)) x dequant(W)^T for M <= 8."""
    import torch
    _require(A, torch.float32, "A")
    _require(wq, torch.uint8, "wq")
    if A.dim() != 2:
        raise ValueError("A must be 2-D [M, K]")
    M, K = A.shape
    if K % BLOCK_ELEMS or wq.numel() != N * (K // BLOCK_ELEMS) * BLOCK_BYTES:
        raise ValueError("wq size does not match N x K")
    if out is None:
        out = torch.empty((M, N), dtype=torch.float32, device=A.device)
    _require(out, torch.float32, "out")
    if out.numel() != M * N:
        raise ValueError("out has the wrong number of elements")
    _check(qm_matmul_q4_0_q8act_ptr(A.data_ptr(), wq.data_ptr(), out.data_ptr(), M, N, K,
                                    _stream_handle(stream)), "qm_matmul_q4_0_q8act")
    return out


def qm_gemv_q4_0_list(problems, M: int = 1, counters=None, stream=None):
    """Run a list of GEMV problems ``(A, wq, C, N, wait_for)`` (A f32 [M, K], wq
    the uint8 block stream of N x K, C f32 [M, N] written in place) in one
    persistent launch where the shapes allow; ``counters`` is a uint32 or int32
    CUDA tensor of len(problems) entries, needed for launches in which a
    problem waits on another (see include/qm.h)."""
    import torch
    raw = []
    for A, wq, C, N, wait_for in problems:
        _require(A, torch.float32, "A")
        _require(wq, torch.uint8, "wq")
        _require(C, torch.float32, "C")
        K = A.shape[-1]
        if A.numel() != M * K or C.numel() != M * N or K % BLOCK_ELEMS or \
                wq.numel() != N * (K // BLOCK_ELEMS) * BLOCK_BYTES:
            raise ValueError("problem operands do not match M, N, K")
        raw.append((A.data_ptr(), wq.data_ptr(), C.data_ptr(), N, K, wait_for))
    ctr = 0
    if counters is not None:
        if not counters.is_cuda or counters.element_size() != 4 or counters.numel() < len(problems):
            raise ValueError("counters must be a CUDA tensor of len(problems) 32-bit entries")
        ctr = counters.data_ptr()
    _check(qm_gemv_q4_0_list_ptr(raw, M, ctr, _stream_handle(stream)), "qm_gemv_q4_0_list")


GEMV_PLAN_FIELDS = ("RG", "U", "S", "rps", "c", "hs", "rbpc", "nu_max", "stages", "grid", "smem", "W",
                    "cl")


def qm_gemv_plan(M: int, N: int, K: int, packed: bool = False, sm_count: int = 152,
                 smem_optin: int = 232448, fit=(76, 38, 19), noalloc: bool = False):
    """The decode GEMV's launch plan (host only, see include/qm.h) as a dict,
    or None when no plan fits; raises on invalid arguments.  `fit` = resident
    clusters of 2, 4 and 8 CTAs (the regular path's K split); with `noalloc`
    the plan of qm_matmul_q4_0_noalloc."""
    out = (ctypes.c_int64 * 13)()
    rc = load_library().qm_gemv_plan(M, N, K, 1 if packed else 0, sm_count, smem_optin, fit[0], fit[1],
                                     fit[2], 1 if noalloc else 0, ctypes.cast(out, ctypes.c_void_p))
    if rc == QM_ERR_UNSUPPORTED:
        return None
    _check(rc, "qm_gemv_plan")
    return dict(zip(GEMV_PLAN_FIELDS, (int(v) for v in out)))


GEMM_PLAN_FIELDS = ("BN", "nt", "tiles", "n_full", "s_rem", "hw", "items", "cl")


def qm_gemm_plan(M: int, N: int, K: int, sm_count: int = 152, fit=(76, 38, 19)):
    """The prefill GEMM's work items (host only, see include/qm.h) as a dict;
    `fit` = resident clusters of 2, 4 and 8 CTAs."""
    out = (ctypes.c_int64 * 8)()
    _check(load_library().qm_gemm_plan(M, N, K, sm_count, fit[0], fit[1], fit[2],
                                       ctypes.cast(out, ctypes.c_void_p)), "qm_gemm_plan")
    return dict(zip(GEMM_PLAN_FIELDS, (int(v) for v in out)))


def qm_launch_count() -> int:
    """Kernels enqueued by the library so far in this process."""
    return int(load_library().qm_launch_count())


def qm_device_status(stream=None, clear: bool = True) -> int:
    """Synchronize the stream and return the device error status (QM_OK,
    QM_ERR_TIMEOUT or QM_ERR_RANGE); see include/qm.h."""
    return load_library().qm_device_status(_stream_handle(stream), 1 if clear else 0)


# ------------------------------------------------------- the 4-bit key/value cache

def kv_page_bytes(page_tokens: int, head_dim: int) -> int:
    """Bytes of one page of one kv head (keys or values)."""
    return page_tokens // 16 * 9 * head_dim


class KVCache:
    """A paged 4-bit key/value cache over the caller's tensors (see
    include/qm.h for the layout): ``k_pages`` and ``v_pages`` uint8 ``[n_pages,
    n_kv_heads, kv_page_bytes(page_tokens, head_dim)]``, ``page_table`` int32
    ``[n_seqs, pages]``, ``lengths`` int32 ``[n_seqs]``.  ``max_len`` bounds the
    lengths (default, and at most: what the page table can hold); a tighter
    bound may be set at any time and gives smaller launches.  Keeps the tensors alive, and
    one attention workspace for each stream it is used on (see qm_attn_q4_0)."""

    def __init__(self, k_pages, v_pages, page_table, lengths, head_dim: int, page_tokens: int, max_len=None):
        import torch
        for t, dtype, dims, name in ((k_pages, torch.uint8, 3, "k_pages"), (v_pages, torch.uint8, 3, "v_pages"),
                                     (page_table, torch.int32, 2, "page_table"), (lengths, torch.int32, 1, "lengths")):
            _require(t, dtype, name)
            if t.dim() != dims:
                raise ValueError(f"{name} must be {dims}-D")
            if t.device != k_pages.device:
                raise ValueError(f"{name} is on another device than k_pages")
        if page_tokens < 16 or head_dim < 32 or k_pages.shape[2] != kv_page_bytes(page_tokens, head_dim):
            raise ValueError("a page of k_pages is not page_tokens / 16 cells of 9 * head_dim bytes")
        if v_pages.shape != k_pages.shape:
            raise ValueError("k_pages and v_pages differ in shape")
        if page_table.shape[0] != lengths.shape[0]:
            raise ValueError("page_table and lengths differ in their number of sequences")
        self.k_pages, self.v_pages, self.page_table, self.lengths = k_pages, v_pages, page_table, lengths
        self.n_seqs, self.n_kv_heads, self.head_dim = lengths.shape[0], k_pages.shape[1], head_dim
        self.struct = QmKVCache(k_pages.data_ptr(), v_pages.data_ptr(), page_table.data_ptr(), lengths.data_ptr(),
                                k_pages.shape[0], page_table.shape[1], 0, self.n_seqs, self.n_kv_heads, head_dim,
                                page_tokens, 0)
        self.ref = ctypes.addressof(self.struct)
        self.capacity = page_table.shape[1] * page_tokens
        self.max_len = self.capacity if max_len is None else max_len
        self._workspaces = {}
        self._sizes = {}

    @property
    def max_len(self) -> int:
        return self.struct.max_len

    @max_len.setter
    def max_len(self, n: int):
        if n < 0:
            raise ValueError("max_len is negative")
        self.struct.max_len = min(n, self.capacity)

    def _workspace(self, n_heads: int, n_tokens: int, max_q: int, weights: bool, stream: int, current: bool):
        key = (n_heads, n_tokens, max_q, weights, self.struct.max_len)
        need = self._sizes.get(key)
        if need is None:
            need = qm_attn_workspace(self, n_heads, n_tokens, max_q, weights, exact=True)
            if len(self._sizes) > 256:
                self._sizes.clear()
            self._sizes[key] = need
        if need == 0:
            return None
        torch = _torch or _torch_module()
        if current:
            capturing = torch.cuda.is_current_stream_capturing()
        else:
            with _on_stream(self.k_pages.device, stream):
                capturing = torch.cuda.is_current_stream_capturing()
        # A graph keeps the address and replays the fill, so a call that is captured has a
        # workspace of its own, from the graph's memory, and no other call ever uses it.
        ws = None if capturing else self._workspaces.get(stream)
        if ws is None or ws.numel() < need:
            with _on_stream(self.k_pages.device, stream):
                ws = torch.empty(need, dtype=torch.uint8, device=self.k_pages.device)
                ws[:ATTN_WORKSPACE_ZEROED].zero_()
            if not capturing:
                self._workspaces[stream] = ws
        return ws


@contextlib.contextmanager
def _on_stream(device, handle: int):
    """Makes the stream with this handle torch's current one."""
    torch = _torch or _torch_module()
    with torch.cuda.device(device), \
            torch.cuda.stream(torch.cuda.ExternalStream(handle) if handle else torch.cuda.default_stream()):
        yield


def _rows(t, heads, dim, name):
    """Check a [n_tokens, heads, dim] tensor whose rows may be strided; (dtype code, row stride)."""
    torch = _torch or _torch_module()
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dtype == torch.float32:
        code = QM_F32
    elif t.dtype == torch.bfloat16:
        code = QM_BF16
    else:
        raise TypeError(f"{name} must be torch.float32 or torch.bfloat16, got {t.dtype}")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    shape = t.shape
    if len(shape) != 3 or (heads is not None and shape[1] != heads) or shape[2] != dim:
        raise ValueError(f"{name} must be [n_tokens, heads, {dim}]")
    stride = t.stride()
    if stride[2] != 1 or (stride[1] != dim and shape[1] != 1 and shape[0] != 0):  # (one head has no stride)
        raise ValueError(f"{name}: the heads of a token must be contiguous")
    return code, (stride[0] if shape[0] > 1 else shape[1] * dim)


def _starts(q_starts, n_seqs):
    torch = _torch or _torch_module()
    if q_starts is None:
        return 0
    _require(q_starts, torch.int32, "q_starts")
    if q_starts.numel() != n_seqs + 1:
        raise ValueError("q_starts must have n_seqs + 1 entries")
    return q_starts.data_ptr()


def qm_kv_append_q4_0(cache, k, v, q_starts=None, stream=None):
    """Quantize k and v (f32 or bf16 ``[n_tokens, n_kv_heads, head_dim]``, rows
    may be strided) into the last places of their sequences; ``cache.lengths``
    already counts them.  Row ranges ``q_starts`` int32 ``[n_seqs + 1]``, or
    None for the same number of rows each."""
    code, ks = _rows(k, cache.n_kv_heads, cache.head_dim, "k")
    code_v, vs = _rows(v, cache.n_kv_heads, cache.head_dim, "v")
    if code != code_v or v.shape != k.shape:
        raise ValueError("k and v differ in type or shape")
    _check(load_library().qm_kv_append_q4_0(cache.ref, k.data_ptr(), v.data_ptr(), code, k.shape[0], ks, vs,
                                            _starts(q_starts, cache.n_seqs), _stream_handle(stream)),
           "qm_kv_append_q4_0")


def qm_kv_read_q4_0(cache, n_tokens: int, q_starts=None, k=None, v=None, stream=None):
    """The f32 values of the last rows of each sequence, ``(k, v)`` of shape
    ``[n_tokens, n_kv_heads, head_dim]``."""
    torch = _torch or _torch_module()
    shape = (n_tokens, cache.n_kv_heads, cache.head_dim)
    for t, name in ((k, "k"), (v, "v")):
        if t is not None:
            _require(t, torch.float32, name)
            if tuple(t.shape) != shape:
                raise ValueError(f"{name} must be {shape}")
    if k is None:
        k = torch.empty(shape, dtype=torch.float32, device=cache.k_pages.device)
    if v is None:
        v = torch.empty(shape, dtype=torch.float32, device=cache.k_pages.device)
    _check(load_library().qm_kv_read_q4_0(cache.ref, k.data_ptr(), v.data_ptr(), n_tokens,
                                          _starts(q_starts, cache.n_seqs), _stream_handle(stream)),
           "qm_kv_read_q4_0")
    return k, v


def qm_attn_workspace(cache, n_heads: int, n_tokens: int, max_q: int, weights: bool = False, exact: bool = False) -> int:
    """Bytes of workspace that qm_attn_q4_0 needs for any call of at most these
    sizes, or (``exact``) for a call of these sizes; see include/qm.h."""
    lib = load_library()
    n = (lib.qm_attn_workspace_exact if exact else lib.qm_attn_workspace)(cache.ref, n_heads, n_tokens, max_q,
                                                                         1 if weights else 0)
    if n < 0:
        raise QMError(n, "qm_attn_workspace")
    return n


def qm_attn_q4_0(cache, q, scale=None, window: int = 0, sinks: int = 0, q_starts=None, max_q=None, weights=None,
                 return_lse: bool = False, out=None, lse=None, stream=None, workspace=None):
    """Causal attention of the rows ``q`` (f32 or bf16 ``[n_tokens, n_heads,
    head_dim]``, rows may be strided) over the cache; returns ``out``, or
    ``(out, lse)`` with ``return_lse`` (or an ``lse`` tensor).  ``scale`` defaults
    to head_dim ** -0.5; ``window`` > 0 with ``sinks`` limits what a row sees to
    its last ``window`` tokens and the first ``sinks``; ``weights`` f32 ``[n_seqs,
    n_kv_heads, >= max_len]`` is added each token's attention weight; ``max_q``
    bounds the rows of one sequence (default: all rows, which makes a prompt's call of
    a batch of single tokens with ``q_starts``: give it there).

    ``workspace``: a uint8 tensor of at least ``qm_attn_workspace`` bytes whose first
    ``ATTN_WORKSPACE_ZEROED`` were zeroed once; calls that cannot run at the same time
    can share it, those of other caches too (the layers of a model).  Without it the
    cache has its own, one per stream, kept at its largest size; a call that is
    captured into a CUDA graph gets one from the graph's memory, and a fill of those
    first bytes is captured with it."""
    torch = _torch or _torch_module()
    code, qs = _rows(q, None, cache.head_dim, "q")
    n_tokens, n_heads = q.shape[0], q.shape[1]
    if out is None:
        out, os_ = torch.empty(q.shape, dtype=q.dtype, device=q.device), n_heads * cache.head_dim
    else:
        code_o, os_ = _rows(out, n_heads, cache.head_dim, "out")
        if code_o != code or out.shape[0] != n_tokens:
            raise ValueError("out differs from q in type or shape")
    if lse is None:
        if return_lse:
            lse = torch.empty((n_tokens, n_heads), dtype=torch.float32, device=q.device)
    else:
        _require(lse, torch.float32, "lse")
        if tuple(lse.shape) != (n_tokens, n_heads):
            raise ValueError("lse must be [n_tokens, n_heads]")
    ws_stride = 0
    if weights is not None:
        _require(weights, torch.float32, "weights")
        if weights.dim() != 3 or weights.shape[0] != cache.n_seqs or weights.shape[1] != cache.n_kv_heads:
            raise ValueError("weights must be [n_seqs, n_kv_heads, max_len]")
        ws_stride = weights.shape[2]
    starts = _starts(q_starts, cache.n_seqs)
    if q_starts is None:
        max_q = n_tokens // cache.n_seqs if cache.n_seqs else 0
    elif max_q is None:
        max_q = n_tokens
    handle = _stream_handle(stream)
    if workspace is None:
        ws = cache._workspace(n_heads, n_tokens, max_q, weights is not None, handle, stream is None)
    else:
        ws = workspace
        _require(ws, torch.uint8, "workspace")
    # (The struct's bytes; filling a ctypes object field by field takes 2 us more.)
    args = _ATTN_ARGS.pack(q.data_ptr(), out.data_ptr(), lse.data_ptr() if lse is not None else 0,
                           weights.data_ptr() if weights is not None else 0, starts,
                           ws.data_ptr() if ws is not None else 0, ws.numel() if ws is not None else 0, n_tokens, max_q,
                           qs, os_, ws_stride, window, sinks, n_heads,
                           cache.head_dim ** -0.5 if scale is None else scale, code, 0)
    _check(load_library().qm_attn_q4_0(cache.ref, args, handle), "qm_attn_q4_0")
    return out if lse is None else (out, lse)


def qm_kv_evict_q4_0(cache, to, weights, budget: int, sinks: int = 0, recent: int = 0, kept=None, weights_out=None,
                     stream=None):
    """Cut every sequence and kv head of ``cache`` back to ``budget`` tokens,
    ranked by ``weights`` (f32 ``[n_seqs, n_kv_heads, >= max_len]``), into the
    cache ``to`` (or in place, with ``to`` the same cache); see include/qm.h.
    Returns ``(kept, weights_out)``."""
    torch = _torch or _torch_module()
    lists = (cache.n_seqs, cache.n_kv_heads)
    _require(weights, torch.float32, "weights")
    if weights.dim() != 3 or tuple(weights.shape[:2]) != lists:
        raise ValueError("weights must be [n_seqs, n_kv_heads, max_len]")
    if kept is None:
        kept = torch.empty((*lists, budget), dtype=torch.int32, device=weights.device)
    else:
        _require(kept, torch.int32, "kept")
    if weights_out is None:
        weights_out = torch.empty((*lists, budget), dtype=torch.float32, device=weights.device)
    else:
        _require(weights_out, torch.float32, "weights_out")
    if tuple(kept.shape) != (*lists, budget) or weights_out.dim() != 3 or tuple(weights_out.shape[:2]) != lists:
        raise ValueError("kept must be [n_seqs, n_kv_heads, budget], weights_out [n_seqs, n_kv_heads, >= budget]")
    _check(load_library().qm_kv_evict_q4_0(cache.ref, to.ref, weights.data_ptr(), weights.shape[2], budget, sinks,
                                           recent, kept.data_ptr(), weights_out.data_ptr(), weights_out.shape[2],
                                           _stream_handle(stream)),
           "qm_kv_evict_q4_0")
    return kept, weights_out
