"""Thin ctypes binding over the C ABI in ``include/mma_gb300.h``.

Argument marshalling only: every step of D = A*B + C runs in the CUDA
library ``libmma_gb300.so`` built in-tree from ``csrc/``.  PyTorch supplies
device memory and the current stream.  If the library is missing, or no
CUDA device is present, calls raise; nothing here computes on the CPU.
"""
from __future__ import annotations

import ctypes
import os
import threading

_HERE = os.path.dirname(os.path.abspath(__file__))
_LIBNAME = "libmma_gb300.so"

MMA_F16, MMA_BF16, MMA_I8, MMA_F64, MMA_F32, MMA_I32 = 1, 2, 3, 4, 5, 6
MMA_F8E4M3, MMA_F8E5M2 = 7, 8
MMA_COL_MAJOR, MMA_ROW_MAJOR = 0, 1
MMA_MAX_GROUPS = 1024
STATUS = {0: "MMA_OK", 1: "MMA_ERR_INVALID_ARG", 2: "MMA_ERR_UNSUPPORTED",
          3: "MMA_ERR_MISALIGNED", 4: "MMA_ERR_LAUNCH", 5: "MMA_ERR_TIMEOUT",
          6: "MMA_ERR_NO_DEVICE", 7: "MMA_ERR_NO_MEMORY"}

# The exported entry points and their ctypes signatures (kept in step with
# include/mma_gb300.h; tests check both lists against the header).
_p, _i64, _int = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int
_f32 = ctypes.c_float
SIGNATURES = {
    "mma_gemm": (_int, [_int, _int, _i64, _i64, _i64, _p, _i64, _p, _i64, _p,
                        _i64, _p, _i64, _p]),
    "mma_gemm_ex": (_int, [_int, _int, _i64, _i64, _i64, _p, _i64, _p, _i64,
                           _int, _p, _i64, _p, _i64, _p]),
    "mma_gemm_batched": (_int, [_int, _int, _i64, _i64, _i64, _p, _i64, _p,
                                _i64, _p, _i64, _p, _i64, _i64, _int, _int,
                                _p]),
    "mma_gemm_batched_ex": (_int, [_int, _int, _i64, _i64, _i64, _p, _i64, _p,
                                   _i64, _p, _i64, _p, _i64, _i64, _int, _int,
                                   _int, _p]),
    "mma_gemm_i8_ex": (_int, [_i64, _i64, _i64, _p, _i64, _int, _p, _i64,
                              _int, _int, _p, _i64, _p, _i64, _int, _p]),
    "mma_gemm_i8_noalloc": (_int, [_i64, _i64, _i64, _p, _i64, _p, _i64, _p,
                                   _i64, _p, _i64, _p]),
    "mma_rmsnorm_f8": (_int, [_int, _int, _i64, _i64, _p, _i64, _p, _i64, _p,
                              _f32, _int, _p, _i64, _p, _i64, _p, _i64, _p,
                              _i64, _i64, _p]),
    "mma_rmsnorm_backward": (_int, [_int, _int, _i64, _i64, _p, _i64, _p, _i64,
                                    _p, _f32, _p, _i64, _p, _i64, _p, _p, _i64,
                                    _p]),
    "mma_rmsnorm_backward_workspace": (_i64, [_i64, _i64]),
    "mma_quantize_f8": (_int, [_int, _int, _i64, _i64, _int, _int, _int, _p,
                               _i64, _p, _i64, _p, _i64, _i64, _p]),
    "mma_gemm_f8": (_int, [_int, _int, _int, _i64, _i64, _i64, _p, _i64, _p,
                           _i64, _i64, _p, _i64, _p, _int, _i64, _i64, _p,
                           _i64, _p, _i64, _p]),
    "mma_gemm_grouped": (_int, [_int, _int, _i64, _i64, _i64, _i64, _p, _i64,
                                _p, _i64, _i64, _int, _p, _p, _i64, _p, _i64,
                                _p]),
    "mma_gemm_grouped_wgrad": (_int, [_int, _int, _i64, _i64, _i64, _i64, _p,
                                      _i64, _p, _i64, _p, _p, _i64, _i64, _p,
                                      _i64, _i64, _p]),
    "mma_gemm_grouped_f8": (_int, [_int, _int, _int, _i64, _i64, _i64, _i64,
                                   _p, _i64, _p, _i64, _i64, _p, _i64, _i64,
                                   _p, _int, _i64, _i64, _i64, _p, _p, _i64,
                                   _p, _i64, _p]),
    "mma_device_status": (_int, [_p]),
    "mma_selftest_wait_timeout": (_int, [_i64, _p]),
    "mma_selftest_gemm_abort": (_int, [_int, _i64, _p, _p, _p, _p]),
    "mma_selftest_f8_abort": (_int, [_int, _i64, _p, _p, _p, _p, _p]),
    "mma_peak_probe": (_int, [_int, _i64, ctypes.POINTER(ctypes.c_double), _p]),
    "mma_profile_begin": (_int, []),
    "mma_profile_end": (_int, [ctypes.POINTER(ctypes.c_float), _int,
                               ctypes.POINTER(_int)]),
    "mma_status_string": (ctypes.c_char_p, [_int]),
    "mma_version": (_int, []),
}

_lib = None
_lock = threading.Lock()


class MMAError(RuntimeError):
    def __init__(self, fn: str, status: int):
        self.status = status
        super().__init__(f"{fn} returned {STATUS.get(status, status)}")


def library_path() -> str:
    return os.path.join(_HERE, _LIBNAME)


def load() -> ctypes.CDLL:
    """Load the CUDA library (raises if it has not been built)."""
    global _lib
    if _lib is not None:
        return _lib
    with _lock:
        if _lib is None:
            path = library_path()
            if not os.path.exists(path):
                raise RuntimeError(
                    f"{_LIBNAME} is not built (expected at {path}); run "
                    "`python -m mixed_precision_dense_02_gb300.build`")
            L = ctypes.CDLL(path)
            for name, (res, args) in SIGNATURES.items():
                fn = getattr(L, name)
                fn.restype = res
                fn.argtypes = args
            _lib = L
    return _lib


def _check(fn: str, status: int) -> None:
    if status != 0:
        raise MMAError(fn, status)


# --------------------------------------------------------------------------
# raw-pointer entry points (same names as the C ABI)

def mma_gemm(dtype_in, dtype_acc, M, N, K, A, lda, B, ldb, C, ldc, D, ldd,
             stream) -> int:
    return load().mma_gemm(dtype_in, dtype_acc, M, N, K, A, lda, B, ldb, C,
                           ldc, D, ldd, stream)


def mma_gemm_ex(dtype_in, dtype_acc, M, N, K, A, lda, B, ldb, layout_b, C,
                ldc, D, ldd, stream) -> int:
    return load().mma_gemm_ex(dtype_in, dtype_acc, M, N, K, A, lda, B, ldb,
                              layout_b, C, ldc, D, ldd, stream)


def mma_gemm_batched(dtype_in, dtype_acc, M, N, K, A, lda, B, ldb, C, ldc, D,
                     ldd, batch, group, abid, stream) -> int:
    return load().mma_gemm_batched(dtype_in, dtype_acc, M, N, K, A, lda, B,
                                   ldb, C, ldc, D, ldd, batch, group, abid,
                                   stream)


def mma_gemm_batched_ex(dtype_in, dtype_acc, M, N, K, A, lda, B, ldb, C, ldc,
                        D, ldd, batch, group, abid, blgp, stream) -> int:
    return load().mma_gemm_batched_ex(dtype_in, dtype_acc, M, N, K, A, lda, B,
                                      ldb, C, ldc, D, ldd, batch, group, abid,
                                      blgp, stream)


def mma_gemm_i8_ex(M, N, K, A, lda, a_neg, B, ldb, b_neg, layout_b, C, ldc,
                   D, ldd, clamp, stream) -> int:
    """8-bit integer GEMM, int8 or uint8 per operand, optional saturation."""
    return load().mma_gemm_i8_ex(M, N, K, A, lda, a_neg, B, ldb, b_neg,
                                 layout_b, C, ldc, D, ldd, clamp, stream)


def mma_gemm_i8_noalloc(M, N, K, A, lda, B, ldb, C, ldc, D, ldd,
                        stream) -> int:
    """INT8 -> INT32 GEMM that allocates no device memory (fixed scratch)."""
    return load().mma_gemm_i8_noalloc(M, N, K, A, lda, B, ldb, C, ldc, D, ldd,
                                      stream)


def mma_device_status(stream) -> int:
    return load().mma_device_status(stream)


def mma_selftest_wait_timeout(limit_ns, stream) -> int:
    """Run one bounded wait that is made to run out (failure-detection
    self-test); mma_device_status then reports MMA_ERR_TIMEOUT once."""
    return load().mma_selftest_wait_timeout(limit_ns, stream)


MMA_PEAK_TC_F16, MMA_PEAK_DMMA, MMA_PEAK_IMMA, MMA_PEAK_DFMA = 1, 2, 3, 4


def mma_peak_probe(kind, iterations, stream) -> tuple:
    """Enqueue one issue-rate probe; returns (status, operations per launch)."""
    ops = ctypes.c_double(0.0)
    st = load().mma_peak_probe(kind, iterations, ctypes.byref(ops), stream)
    return st, ops.value


def mma_selftest_gemm_abort(cluster, limit_ns, A, B, D, stream) -> int:
    """Run the tcgen05 GEMM kernel with no operand loads and waits limited to
    limit_ns, so its own abort path runs; mma_device_status then reports
    MMA_ERR_TIMEOUT once."""
    return load().mma_selftest_gemm_abort(cluster, limit_ns, A, B, D, stream)


def mma_selftest_f8_abort(kernel, limit_ns, X, Q, S, workspace, stream) -> int:
    """Run a tile quantiser (kernel 0, 1), the norm's gradient (2) or a product
    (3, 4, 5) with no loads and bounded waits; mma_device_status then reports
    MMA_ERR_TIMEOUT once."""
    return load().mma_selftest_f8_abort(kernel, limit_ns, X, Q, S, workspace, stream)


def mma_status_string(status: int) -> str:
    return load().mma_status_string(status).decode()


# --------------------------------------------------------------------------
# torch-tensor convenience layer (still marshalling only)

def _torch():
    import torch
    return torch


def _dtypes(t):
    torch = _torch()
    m = {torch.float16: (MMA_F16, MMA_F32, torch.float32),
         torch.bfloat16: (MMA_BF16, MMA_F32, torch.float32),
         torch.int8: (MMA_I8, MMA_I32, torch.int32),
         torch.float64: (MMA_F64, MMA_F64, torch.float64)}
    if t.dtype not in m:
        raise TypeError(f"unsupported input dtype {t.dtype}")
    return m[t.dtype]


def _ld(t) -> int:
    if t.dim() != 2 or t.stride(1) != 1:
        raise ValueError("2-D tensors with unit inner stride are required")
    return t.stride(0)


def _stream(stream):
    if stream is None:
        return _torch().cuda.current_stream().cuda_stream
    return getattr(stream, "cuda_stream", stream)


def _under(stream, index, call, *args, **kw):
    """`call` with `stream` (a torch stream or a cudaStream_t) as the current
    one.  Results and scratch memory are then allocated on it: a block of
    another stream's may still be in use by that stream's earlier work, and
    goes to its later work while the call runs."""
    cuda = _torch().cuda
    if not isinstance(stream, cuda.Stream):
        handle = getattr(stream, "cuda_stream", stream)
        stream = (cuda.ExternalStream(handle, device=index) if handle
                  else cuda.default_stream(index))
    with cuda.stream(stream):
        return call(*args, **kw)


def _empty(shape, dtype, like, stream):
    """A result beside `like`, allocated on the call's stream."""
    torch = _torch()
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=like.device)
    return _under(stream, like.get_device(), torch.empty, shape, dtype=dtype,
                  device=like.device)


def gemm_ex(A, B, C=None, D=None, *, b_layout: str = "col", acc=None,
            stream=None):
    """D = A @ B + C on the GPU.

    ``A``: (M, K) row-major; ``B`` as stored: (N, K) for column-major B
    (``b_layout="col"``) or (K, N) for row-major B; ``C``/``D``: (M, N).
    Input dtype float16/bfloat16 -> float32 output, int8 -> int32,
    float64 -> float64.  FP16/BF16 inputs accumulate into a 16-bit addend
    and result of their own type when ``acc="same"`` or when C or D has
    that dtype.  ``D`` is allocated when not given.  Returns D.
    """
    torch = _torch()
    dt_in, dt_acc, out_dtype = _dtypes(A)
    if A.dtype in (torch.float16, torch.bfloat16):
        given = D if D is not None else C
        if acc == "same" or (acc is None and given is not None
                             and given.dtype == A.dtype):
            dt_acc, out_dtype = dt_in, A.dtype
    if B.dtype != A.dtype:
        raise TypeError("A and B must have the same dtype")
    M, K = A.shape
    if b_layout == "col":
        N, Kb = B.shape
        layout = MMA_COL_MAJOR
    elif b_layout == "row":
        Kb, N = B.shape
        layout = MMA_ROW_MAJOR
    else:
        raise ValueError(b_layout)
    if Kb != K:
        raise ValueError(f"K mismatch: {K} vs {Kb}")
    if D is None:
        D = _empty((M, N), out_dtype, A, stream)
    for t in (C, D):
        if t is not None and (t.dtype != out_dtype or tuple(t.shape) != (M, N)):
            raise ValueError("C/D must be (M, N) of the accumulator dtype")
    st = mma_gemm_ex(dt_in, dt_acc, M, N, K, A.data_ptr(), _ld(A),
                     B.data_ptr(), _ld(B), layout,
                     None if C is None else C.data_ptr(),
                     0 if C is None else _ld(C), D.data_ptr(), _ld(D),
                     _stream(stream))
    _check("mma_gemm_ex", st)
    return D


def gemm_i8_ex(A, B, C=None, D=None, *, clamp: bool = False,
               b_layout: str = "col", stream=None):
    """8-bit integer D = A @ B + C (INT32 C and D) on the GPU.

    Each of ``A`` and ``B`` is a torch.int8 (signed) or torch.uint8
    (unsigned) tensor; shapes and layouts as in ``gemm_ex``.  With ``clamp``
    D is the exact result saturated to the INT32 range, else it wraps
    modulo 2^32.  ``D`` is allocated when not given.  Returns D.
    """
    torch = _torch()
    sign = {torch.int8: 1, torch.uint8: 0}
    if A.dtype not in sign or B.dtype not in sign:
        raise TypeError("A and B must be int8 or uint8 tensors")
    M, K = A.shape
    if b_layout == "col":
        N, Kb = B.shape
        layout = MMA_COL_MAJOR
    elif b_layout == "row":
        Kb, N = B.shape
        layout = MMA_ROW_MAJOR
    else:
        raise ValueError(b_layout)
    if Kb != K:
        raise ValueError(f"K mismatch: {K} vs {Kb}")
    if D is None:
        D = _empty((M, N), torch.int32, A, stream)
    for t in (C, D):
        if t is not None and (t.dtype != torch.int32 or tuple(t.shape) != (M, N)):
            raise ValueError("C/D must be (M, N) int32")
    st = mma_gemm_i8_ex(M, N, K, A.data_ptr(), _ld(A), sign[A.dtype],
                        B.data_ptr(), _ld(B), sign[B.dtype], layout,
                        None if C is None else C.data_ptr(),
                        0 if C is None else _ld(C), D.data_ptr(), _ld(D),
                        int(bool(clamp)), _stream(stream))
    _check("mma_gemm_i8_ex", st)
    return D


def gemm(A, B, C=None, D=None, *, acc=None, stream=None):
    """D = A @ B + C with B given column-major as an (N, K) tensor."""
    return gemm_ex(A, B, C, D, b_layout="col", acc=acc, stream=stream)


def gemm_batched(A, B, C=None, D=None, *, group: int = 1, abid: int = 0,
                 blgp: int = 0, acc=None, stream=None):
    """Batched D_b = A_{(b//group)*group + abid} @ B_{bsrc(b)} + C_b with
    bsrc(b) = (b//4)*4 + (quarter read under lane-group pattern ``blgp``).

    ``A``: (batch, M, K); ``B``: (batch, N, K) column-major tiles;
    ``C``/``D``: (batch, M, N); all contiguous.  Dtypes as in ``gemm_ex``
    (FP16/BF16 accumulate into their own type with ``acc="same"`` or a C/D
    of that type).
    """
    torch = _torch()
    dt_in, dt_acc, out_dtype = _dtypes(A)
    if A.dtype in (torch.float16, torch.bfloat16):
        given = D if D is not None else C
        if acc == "same" or (acc is None and given is not None
                             and given.dtype == A.dtype):
            dt_acc, out_dtype = dt_in, A.dtype
    batch, M, K = A.shape
    _, N, Kb = B.shape
    if Kb != K or B.shape[0] != batch:
        raise ValueError("shape mismatch")
    for t in (A, B, C, D):
        if t is not None and not t.is_contiguous():
            raise ValueError("batched operands must be contiguous")
    if D is None:
        D = _empty((batch, M, N), out_dtype, A, stream)
    st = mma_gemm_batched_ex(dt_in, dt_acc, M, N, K, A.data_ptr(), K,
                             B.data_ptr(), K,
                             None if C is None else C.data_ptr(), N,
                             D.data_ptr(), N, batch, group, abid, blgp,
                             _stream(stream))
    _check("mma_gemm_batched_ex", st)
    return D


# --------------------------------------------------------------------------
# 8-bit operands with scales, products grouped by expert

# These calls serve single tokens too, where the kernel takes a few
# microseconds and Python's share counts.  So what a call's argument layouts
# (types, shapes, strides, device) settle is worked out once per layout and
# kept as a plan: the checks, the ABI's codes and leading dimensions, the
# layouts of the results.  A plan holds no tensor and no address.
#
# With `stream` given a call runs as if that stream were the current one: its
# results are that stream's tensors, and what it reads must be ready there.

_KIND = {}
_PLANS = {}
_MOST_PLANS = 4096


def _kinds():
    """Tensor types: their ABI codes, and the sets that arguments may have."""
    global _KIND
    if not _KIND:
        torch = _torch()
        # (put together aside: another thread sees all of it or nothing)
        _KIND = {
            "wide": {torch.float32: MMA_F32, torch.float16: MMA_F16,
                     torch.bfloat16: MMA_BF16},
            "half": {torch.float16: MMA_F16, torch.bfloat16: MMA_BF16},
            "f8": {torch.float8_e4m3fn: MMA_F8E4M3,
                   torch.float8_e5m2: MMA_F8E5M2},
            "scale": {torch.float32: MMA_F32},
            "offset": {torch.int32: MMA_I32},
            "fmt": {"e4m3": torch.float8_e4m3fn, "e5m2": torch.float8_e5m2},
        }
    return _KIND


def _key(t):
    """What a plan may depend on of a tensor."""
    return None if t is None else (t.dtype, t.shape, t.stride(), t.get_device())


def _plan(key, make, *args):
    """The plan of a call whose argument layouts are `key`."""
    plan = _PLANS.get(key)
    if plan is None:
        if len(_PLANS) >= _MOST_PLANS:
            _PLANS.clear()
        plan = make(*args)  # raises what the arguments deserve
        _PLANS[key] = plan
    return plan


def _raw_stream(index):
    """The cudaStream_t of the current stream of the tensors' device, which has
    to be the current one: the library launches there."""
    c = _torch()._C
    if c._cuda_getDevice() != index:
        raise ValueError(f"the tensors are on cuda:{index}, the current device is "
                         f"cuda:{c._cuda_getDevice()}")
    return c._cuda_getCurrentRawStream(index)


def _take(name, t, kinds, *shape):
    """Check a tensor argument: its type, its shape (None: any extent) and
    that it is on the GPU.  Returns the type's ABI code."""
    code = kinds.get(t.dtype)
    if code is None:
        raise TypeError(f"{name}: unsupported dtype {t.dtype}")
    got = t.shape
    if len(got) != len(shape) or any(w is not None and w != g
                                     for w, g in zip(shape, got)):
        want = tuple("*" if s is None else s for s in shape)
        raise ValueError(f"{name} must have shape {want}, not {tuple(got)}")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    return code


def _one_device(*tensors):
    """The index of the device that all the tensors are on."""
    at = {t.get_device() for t in tensors if t is not None}
    if len(at) > 1:
        raise ValueError("the tensors must be on one device")
    return at.pop()


def _rows(name, t) -> int:
    """Leading dimension of the last two axes: contiguous rows.  A single
    row has any leading dimension; its own length rounded up to 16 bytes
    meets every rule."""
    shape, stride = t.shape, t.stride()
    if stride[-1] != 1 and shape[-1] > 1:
        raise ValueError(f"{name}: the last axis must be contiguous")
    if shape[-2] > 1:
        return stride[-2]
    return _row_of(shape[-1], t.dtype)


def _row_of(n, dtype) -> int:
    """Elements of a row of n that ends on a 16-byte boundary."""
    per = 16 // dtype.itemsize
    return -(-n // per) * per


def _scale_strides(t):
    """(row, block) strides of a scale tensor, in elements."""
    shape, stride = t.shape, t.stride()
    return (stride[-2] if shape[-2] > 1 else 1, stride[-1] if shape[-1] > 1 else 0)


def _weight(W, X, n):
    """The ABI code of a norm's weights: of X's type or float32."""
    code = _take("W", W, _kinds()["wide"], n)
    if code != MMA_F32 and W.dtype != X.dtype:
        raise TypeError(f"W must be {X.dtype} or torch.float32, not {W.dtype}")
    if n > 1 and W.stride(0) != 1:
        raise ValueError("W must be contiguous")
    return code


def _same(name, t, X, *shape):
    if t.dtype != X.dtype:
        raise TypeError(f"{name} must be {X.dtype}, not {t.dtype}")
    _take(name, t, _kinds()["wide"], *shape)


def _result(name, C, D, shape, out_dtype):
    """The type of a product's C and D and its code."""
    given = D if D is not None else C
    if given is not None:
        if out_dtype is not None and given.dtype != out_dtype:
            raise TypeError(f"{name}: C and D must be of type {out_dtype}")
        out_dtype = given.dtype
    kinds = _kinds()["wide"]
    for n, t in (("C", C), ("D", D)):
        if t is not None:
            if t.dtype != out_dtype:
                raise TypeError(f"{name}: C and D must have one type")
            _take(f"{name}: {n}", t, kinds, *shape)
    code = kinds.get(out_dtype)
    if code is None:
        raise TypeError(f"{name}: unsupported result type {out_dtype}")
    return out_dtype, code


def _plan_rmsnorm(X, W, residual):
    kinds = _kinds()
    code = _take("X", X, kinds["wide"], None, None)
    M, N = X.shape
    w_code = _weight(W, X, N)
    ldr = 0
    if residual is not None:
        _same("residual", residual, X, M, N)
        ldr = _rows("residual", residual)
    q = kinds["fmt"]["e4m3"]
    return (code, w_code, M, N, _rows("X", X), ldr, _row_of(N, X.dtype),
            q, _row_of(N, q), -(-N // 128), _one_device(X, W, residual))


def rmsnorm_f8(X, W, residual=None, *, eps: float = 1e-6, pow2: bool = False,
               y: bool = False, stream=None):
    """Root-mean-square norm of ``X + residual`` with an 8-bit output.

    ``h = X + residual``, ``y = h * W / sqrt(mean(h**2) + eps)`` per row, and
    ``y`` in E4M3 with one FP32 scale for each 128 columns (with ``pow2`` a
    power of two).  ``X``, ``residual``: (M, N) float16, bfloat16 or float32;
    ``W``: (N,) of that type or float32.  Returns ``(Q, S, H)``: Q (M, N)
    float8_e4m3fn, S (M, ceil(N / 128)), H the sum in X's type (X itself
    without a residual); with ``y=True`` also y in X's type.
    """
    torch = _torch()
    (code, w_code, M, N, ldx, ldr, ldh, f8, ldq, blocks, index) = _plan(
        ("norm", _key(X), _key(W), _key(residual)), _plan_rmsnorm, X, W, residual)
    if stream is not None:
        return _under(stream, index, rmsnorm_f8, X, W, residual, eps=eps, pow2=pow2, y=y)
    dtype, device = X.dtype, X.device
    H, r_ptr, h_ptr = X, None, None
    if residual is not None:
        H = torch.empty_strided((M, N), (ldh, 1), dtype=dtype, device=device)
        r_ptr, h_ptr = residual.data_ptr(), H.data_ptr()
    Q = torch.empty_strided((M, N), (ldq, 1), dtype=f8, device=device)
    # the scales of one block side by side
    S = torch.empty_strided((M, blocks), (1, M), dtype=torch.float32, device=device)
    Y = (torch.empty_strided((M, N), (ldh, 1), dtype=dtype, device=device)
         if y else None)
    st = load().mma_rmsnorm_f8(
        code, w_code, M, N, X.data_ptr(), ldx, r_ptr, ldr, W.data_ptr(), eps,
        1 if pow2 else 0, h_ptr, ldh, None if Y is None else Y.data_ptr(), ldh,
        Q.data_ptr(), ldq, S.data_ptr(), 1, M, _raw_stream(index))
    if st:
        _check("mma_rmsnorm_f8", st)
    return (Q, S, H, Y) if y else (Q, S, H)


def _plan_rmsnorm_backward(dY, H, W, dH):
    code = _take("H", H, _kinds()["wide"], None, None)
    M, N = H.shape
    _same("dY", dY, H, M, N)
    w_code = _weight(W, H, N)
    if dH is not None:
        _same("dH", dH, H, M, N)
    return (code, w_code, M, N, _rows("dY", dY), _rows("H", H),
            0 if dH is None else _rows("dH", dH), _row_of(N, H.dtype),
            load().mma_rmsnorm_backward_workspace(M, N),
            _one_device(dY, H, W, dH))


def rmsnorm_backward(dY, H, W, dH=None, *, eps: float = 1e-6, stream=None):
    """Gradient of the norm of ``rmsnorm_f8`` (taken at the unrounded y).

    ``dY``: gradient of y; ``H``: the sum that the forward returned; ``dH``:
    gradient that reaches H from elsewhere.  Returns ``(dX, dW)``: dX, the
    gradient of X and of the residual alike, in H's type, and dW (N,)
    float32.
    """
    torch = _torch()
    code, w_code, M, N, ldy, ldh, ldr, ldx, need, index = _plan(
        ("back", _key(dY), _key(H), _key(W), _key(dH)), _plan_rmsnorm_backward,
        dY, H, W, dH)
    if stream is not None:
        return _under(stream, index, rmsnorm_backward, dY, H, W, dH, eps=eps)
    device = H.device
    dX = torch.empty_strided((M, N), (ldx, 1), dtype=H.dtype, device=device)
    dW = torch.empty((N,), dtype=torch.float32, device=device)
    # (its memory goes to other work of the current stream only after the call's)
    ws = torch.empty((need,), dtype=torch.uint8, device=device)
    st = load().mma_rmsnorm_backward(
        code, w_code, M, N, dY.data_ptr(), ldy, H.data_ptr(), ldh, W.data_ptr(),
        eps, None if dH is None else dH.data_ptr(), ldr, dX.data_ptr(), ldx,
        dW.data_ptr(), ws.data_ptr(), need, _raw_stream(index))
    if st:
        _check("mma_rmsnorm_backward", st)
    return dX, dW


def _plan_quantize(X, fmt, block_rows, transpose):
    kinds = _kinds()
    code = _take("X", X, kinds["wide"], None, None)
    f8 = kinds["fmt"].get(fmt)
    if f8 is None:
        raise ValueError(f"fmt must be e4m3 or e5m2, not {fmt!r}")
    if block_rows != 1 and block_rows != 128:
        raise ValueError("block_rows must be 1 or 128")
    M, N = X.shape
    m, n = (N, M) if transpose else (M, N)
    return (code, f8, kinds["f8"][f8], M, N, _rows("X", X), m, n, _row_of(n, f8),
            -(-m // block_rows), -(-n // 128), X.get_device())


def quantize_f8(X, *, fmt: str = "e4m3", block_rows: int = 1,
                transpose: bool = False, pow2: bool = False, stream=None):
    """``X`` (M, N) in 8-bit floating point with a scale for each block.

    ``fmt``: "e4m3" or "e5m2"; blocks of ``block_rows`` (1 or 128) x 128 of
    the result, which is X or, with ``transpose``, its transpose (N, M).
    Returns ``(Q, S)`` with S (ceil(rows / block_rows), ceil(columns / 128)).
    """
    torch = _torch()
    transpose = bool(transpose)
    code, f8, f8_code, M, N, ldx, m, n, ldq, s_rows, blocks, index = _plan(
        ("quantize", _key(X), fmt, block_rows, transpose), _plan_quantize, X, fmt,
        block_rows, transpose)
    if stream is not None:
        return _under(stream, index, quantize_f8, X, fmt=fmt, block_rows=block_rows,
                      transpose=transpose, pow2=pow2)
    device = X.device
    Q = torch.empty_strided((m, n), (ldq, 1), dtype=f8, device=device)
    # the scales of one block side by side
    S = torch.empty_strided((s_rows, blocks), (1, s_rows), dtype=torch.float32,
                            device=device)
    st = load().mma_quantize_f8(
        code, f8_code, M, N, block_rows, 1 if transpose else 0, 1 if pow2 else 0,
        X.data_ptr(), ldx, Q.data_ptr(), ldq, S.data_ptr(), 1, s_rows,
        _raw_stream(index))
    if st:
        _check("mma_quantize_f8", st)
    return Q, S


def _scale_rows(SB, N):
    """Rows of B that share a scale, from the scales' shape."""
    rows = SB.shape[-2]
    if rows == N:
        return 1
    if rows == -(-N // 128):
        return 128
    raise ValueError(f"SB must have {N} or {-(-N // 128)} rows, not {rows}")


def _plan_gemm_f8(A, SA, B, SB, C, D, out_dtype):
    kinds = _kinds()
    f8, scale = kinds["f8"], kinds["scale"]
    a_code = _take("A", A, f8, None, None)
    M, K = A.shape
    b_code = _take("B", B, f8, None, K)
    N = B.shape[0]
    kb = -(-K // 128)
    _take("SA", SA, scale, M, kb)
    _take("SB", SB, scale, None, kb)
    if out_dtype is None and C is None and D is None:
        out_dtype = _torch().bfloat16
    dtype, d_code = _result("gemm_f8", C, D, (M, N), out_dtype)
    return (a_code, b_code, d_code, M, N, K, _rows("A", A), *_scale_strides(SA),
            _rows("B", B), _scale_rows(SB, N), *_scale_strides(SB),
            0 if C is None else _rows("C", C), N if D is None else _rows("D", D),
            dtype, _one_device(A, SA, B, SB, C, D))


def gemm_f8(A, SA, B, SB, C=None, D=None, *, out_dtype=None, stream=None):
    """D = A @ B^T + C for 8-bit operands with scales.

    ``A``: (M, K), ``B``: (N, K), each float8_e4m3fn or float8_e5m2;
    ``SA``: (M, ceil(K / 128)) float32; ``SB``: (N, ceil(K / 128)) or, a scale
    for each 128 x 128 block, (ceil(N / 128), ceil(K / 128)).  ``C``, ``D``:
    (M, N) bfloat16, float16 or float32 (``out_dtype``, bfloat16 unless C or D
    is given).  Any strides of the scales; those of ``quantize_f8`` are read
    fastest.  Returns D.
    """
    (a_code, b_code, d_code, M, N, K, lda, sa_row, sa_blk, ldb, sb_rows, sb_row,
     sb_blk, ldc, ldd, dtype, index) = _plan(
        ("f8", _key(A), _key(SA), _key(B), _key(SB), _key(C), _key(D), out_dtype),
        _plan_gemm_f8, A, SA, B, SB, C, D, out_dtype)
    if stream is not None:
        return _under(stream, index, gemm_f8, A, SA, B, SB, C, D, out_dtype=out_dtype)
    if D is None:
        D = _torch().empty((M, N), dtype=dtype, device=A.device)
    st = load().mma_gemm_f8(
        a_code, b_code, d_code, M, N, K, A.data_ptr(), lda, SA.data_ptr(), sa_row,
        sa_blk, B.data_ptr(), ldb, SB.data_ptr(), sb_rows, sb_row, sb_blk,
        None if C is None else C.data_ptr(), ldc, D.data_ptr(), ldd,
        _raw_stream(index))
    if st:
        _check("mma_gemm_f8", st)
    return D


def _check_offsets(offsets, groups):
    _take("offsets", offsets, _kinds()["offset"], groups + 1)
    if groups and offsets.stride(0) != 1:
        raise ValueError("offsets must be contiguous")


def _slices(name, t) -> int:
    """Elements between the matrices of a (groups, rows, columns) tensor."""
    return t.stride(0) if t.shape[0] > 1 else t.shape[1] * _rows(name, t)


def _plan_grouped(A, B, offsets, C, D, b_layout, out_dtype):
    code = _take("A", A, _kinds()["half"], None, None)
    T, K = A.shape
    if b_layout not in ("col", "row"):
        raise ValueError(b_layout)
    row = b_layout == "row"
    if row:
        _same("B", B, A, None, K, None)
    else:
        _same("B", B, A, None, None, K)
    groups, N = B.shape[0], B.shape[2 if row else 1]
    _check_offsets(offsets, groups)
    if out_dtype is None and C is None and D is None:
        out_dtype = A.dtype
    dtype, d_code = _result("gemm_grouped", C, D, (T, N), out_dtype)
    return (code, d_code, groups, T, N, K, _rows("A", A), _rows("B", B),
            _slices("B", B), MMA_ROW_MAJOR if row else MMA_COL_MAJOR,
            0 if C is None else _rows("C", C), N if D is None else _rows("D", D),
            dtype, _one_device(A, B, offsets, C, D))


def gemm_grouped(A, B, offsets, C=None, D=None, *, b_layout: str = "col",
                 out_dtype=None, stream=None):
    """Products grouped by expert: ``D[i] = A[i] @ B[e]^T + C[i]`` for the rows
    i in ``[offsets[e], offsets[e + 1])`` of each expert e.

    ``A``: (T, K) float16 or bfloat16, rows sorted by expert; ``B``: (E, N, K),
    or (E, K, N) with ``b_layout="row"`` (then ``A[i] @ B[e]``: the gradient of
    the input); ``offsets``: (E + 1,) int32 on the GPU; ``C``, ``D``: (T, N) of
    A's type or float32 (``out_dtype``, A's unless C or D is given).  Rows of
    no expert are not written.  Returns D.
    """
    (code, d_code, groups, T, N, K, lda, ldb, stride_b, layout, ldc, ldd, dtype,
     index) = _plan(
        ("grouped", _key(A), _key(B), _key(offsets), _key(C), _key(D), b_layout,
         out_dtype),
        _plan_grouped, A, B, offsets, C, D, b_layout, out_dtype)
    if stream is not None:
        return _under(stream, index, gemm_grouped, A, B, offsets, C, D, b_layout=b_layout,
                      out_dtype=out_dtype)
    if D is None:
        D = _torch().empty((T, N), dtype=dtype, device=A.device)
    st = load().mma_gemm_grouped(
        code, d_code, groups, T, N, K, A.data_ptr(), lda, B.data_ptr(), ldb,
        stride_b, layout, offsets.data_ptr(), None if C is None else C.data_ptr(),
        ldc, D.data_ptr(), ldd, _raw_stream(index))
    if st:
        _check("mma_gemm_grouped", st)
    return D


def _plan_wgrad(dY, X, offsets, C, D, out_dtype):
    code = _take("dY", dY, _kinds()["half"], None, None)
    T, N = dY.shape
    _same("X", X, dY, T, None)
    K = X.shape[1]
    if offsets.dim() != 1 or offsets.shape[0] < 1:
        raise ValueError("offsets must hold one value more than there are experts")
    groups = offsets.shape[0] - 1
    _check_offsets(offsets, groups)
    if out_dtype is None and C is None and D is None:
        out_dtype = _torch().float32
    dtype, d_code = _result("gemm_grouped_wgrad", C, D, (groups, N, K), out_dtype)
    return (code, d_code, groups, T, N, K, _rows("dY", dY), _rows("X", X),
            0 if C is None else _rows("C", C), 0 if C is None else _slices("C", C),
            K if D is None else _rows("D", D),
            N * K if D is None else _slices("D", D), dtype,
            _one_device(dY, X, offsets, C, D))


def gemm_grouped_wgrad(dY, X, offsets, C=None, D=None, *, out_dtype=None,
                       stream=None):
    """Weight gradient of ``gemm_grouped``: ``D[e] = dY_e^T @ X_e + C[e]`` over
    the rows of expert e.

    ``dY``: (T, N), ``X``: (T, K), float16 or bfloat16; ``C``, ``D``: (E, N, K)
    of that type or float32 (``out_dtype``, float32 unless C or D is given;
    C may be D, to accumulate).  An expert without rows gives C[e], or zeros.
    Returns D.
    """
    (code, d_code, groups, T, N, K, ldy, ldx, ldc, stride_c, ldd, stride_d, dtype,
     index) = _plan(
        ("wgrad", _key(dY), _key(X), _key(offsets), _key(C), _key(D), out_dtype),
        _plan_wgrad, dY, X, offsets, C, D, out_dtype)
    if stream is not None:
        return _under(stream, index, gemm_grouped_wgrad, dY, X, offsets, C, D,
                      out_dtype=out_dtype)
    if D is None:
        D = _torch().empty((groups, N, K), dtype=dtype, device=dY.device)
    st = load().mma_gemm_grouped_wgrad(
        code, d_code, groups, T, N, K, dY.data_ptr(), ldy, X.data_ptr(), ldx,
        offsets.data_ptr(), None if C is None else C.data_ptr(), ldc, stride_c,
        D.data_ptr(), ldd, stride_d, _raw_stream(index))
    if st:
        _check("mma_gemm_grouped_wgrad", st)
    return D


def _plan_grouped_f8(A, SA, B, SB, offsets, C, D, out_dtype):
    kinds = _kinds()
    f8, scale = kinds["f8"], kinds["scale"]
    a_code = _take("A", A, f8, None, None)
    T, K = A.shape
    b_code = _take("B", B, f8, None, None, K)
    groups, N = B.shape[0], B.shape[1]
    kb = -(-K // 128)
    _take("SA", SA, scale, T, kb)
    _take("SB", SB, scale, groups, None, kb)
    _check_offsets(offsets, groups)
    if out_dtype is None and C is None and D is None:
        out_dtype = _torch().bfloat16
    dtype, d_code = _result("gemm_grouped_f8", C, D, (T, N), out_dtype)
    return (a_code, b_code, d_code, groups, T, N, K, _rows("A", A),
            *_scale_strides(SA), _rows("B", B), _slices("B", B),
            _scale_rows(SB, N), SB.stride(0), *_scale_strides(SB),
            0 if C is None else _rows("C", C), N if D is None else _rows("D", D),
            dtype, _one_device(A, SA, B, SB, offsets, C, D))


def gemm_grouped_f8(A, SA, B, SB, offsets, C=None, D=None, *, out_dtype=None,
                    stream=None):
    """``gemm_grouped`` for 8-bit operands with scales.

    ``A``: (T, K) and ``SA``: (T, ceil(K / 128)) as in ``gemm_f8``; ``B``:
    (E, N, K); ``SB``: (E, N, ceil(K / 128)) or (E, ceil(N / 128),
    ceil(K / 128)).  Returns D (T, N), bfloat16 unless given otherwise.
    """
    (a_code, b_code, d_code, groups, T, N, K, lda, sa_row, sa_blk, ldb, stride_b,
     sb_rows, sb_group, sb_row, sb_blk, ldc, ldd, dtype, index) = _plan(
        ("grouped_f8", _key(A), _key(SA), _key(B), _key(SB), _key(offsets), _key(C),
         _key(D), out_dtype),
        _plan_grouped_f8, A, SA, B, SB, offsets, C, D, out_dtype)
    if stream is not None:
        return _under(stream, index, gemm_grouped_f8, A, SA, B, SB, offsets, C, D,
                      out_dtype=out_dtype)
    if D is None:
        D = _torch().empty((T, N), dtype=dtype, device=A.device)
    st = load().mma_gemm_grouped_f8(
        a_code, b_code, d_code, groups, T, N, K, A.data_ptr(), lda, SA.data_ptr(),
        sa_row, sa_blk, B.data_ptr(), ldb, stride_b, SB.data_ptr(), sb_rows,
        sb_group, sb_row, sb_blk, offsets.data_ptr(),
        None if C is None else C.data_ptr(), ldc, D.data_ptr(), ldd,
        _raw_stream(index))
    if st:
        _check("mma_gemm_grouped_f8", st)
    return D


def profile_begin() -> None:
    """Start recording the duration of each call's dominant kernel."""
    _check("mma_profile_begin", load().mma_profile_begin())


def profile_end(max_count: int = 4096) -> list:
    """Stop recording; durations (ms) of the recorded dominant kernels."""
    buf = (ctypes.c_float * max_count)()
    n = _int(0)
    _check("mma_profile_end", load().mma_profile_end(buf, max_count, ctypes.byref(n)))
    return [float(buf[i]) for i in range(min(n.value, max_count))]


def device_status(stream=None) -> None:
    """Raise MMAError if an in-kernel wait has run out since the last check."""
    _check("mma_device_status", mma_device_status(_stream(stream)))
