"""ctypes binding of libdmp_gemm.so (argument marshalling only)."""
from __future__ import annotations

import ctypes
import os
import threading

_HERE = os.path.dirname(os.path.abspath(__file__))
_LIB_NAME = "libdmp_gemm.so"

GEMM_F16, GEMM_BF16, GEMM_I8, GEMM_F64 = 0, 1, 2, 3
GEMM_A_COLMAJOR, GEMM_B_COLMAJOR, GEMM_A_SHARED, GEMM_B_SHARED = 1, 2, 4, 8
GEMM_OUT_F32, GEMM_OUT_F16, GEMM_OUT_BF16, GEMM_OUT_I32, GEMM_OUT_F64 = 0, 1, 2, 3, 4
GEMM_OK = 0

EXPORTED_SYMBOLS = ("gemm_create", "gemm_run", "gemm_run_ex", "gemm_run_noalloc", "gemm_prune24",
                    "gemm_run_sparse24", "gemm_run_grouped", "gemm_run_grouped_wgrad", "gemm_quant8",
                    "gemm_run_scaled8", "gemm_destroy", "gemm_status_string", "gemm_plan")
GEMM_OFFSETS_I32 = 16
GEMM_E4M3, GEMM_E5M2 = 0, 1
GEMM_ERR_SCRATCH = 5
NOALLOC_SCRATCH_BYTES = 64 << 20

_lib = None
_lock = threading.Lock()


class Q8Operand(ctypes.Structure):
    """gemm_q8_t: an 8-bit operand of gemm_run_scaled8."""
    _fields_ = [("q", ctypes.c_void_p), ("scale", ctypes.c_void_p), ("ld", ctypes.c_int64),
                ("scale_row", ctypes.c_int64), ("scale_k", ctypes.c_int64), ("group", ctypes.c_int64),
                ("scale_group", ctypes.c_int64), ("type", ctypes.c_int)]


class GemmError(RuntimeError):
    def __init__(self, status: int, what: str):
        self.status = status
        super().__init__(f"{what}: {status_string(status)} ({status})")


def lib_path() -> str:
    return os.path.join(_HERE, _LIB_NAME)


def load_library():
    """Load the built library.  Raises if it is missing: there is no fallback path."""
    global _lib
    with _lock:
        if _lib is not None:
            return _lib
        path = lib_path()
        if not os.path.exists(path):
            raise RuntimeError(f"{path} is not built; run __graft_entry__.build() "
                               "(or python -m dense_mixed_precision_02_amd.build)")
        lib = ctypes.CDLL(path)
        i64, vp = ctypes.c_int64, ctypes.c_void_p
        lib.gemm_create.restype = ctypes.c_int
        lib.gemm_create.argtypes = [ctypes.POINTER(vp)]
        lib.gemm_destroy.restype = ctypes.c_int
        lib.gemm_destroy.argtypes = [vp]
        lib.gemm_status_string.restype = ctypes.c_char_p
        lib.gemm_status_string.argtypes = [ctypes.c_int]
        lib.gemm_run.restype = ctypes.c_int
        lib.gemm_run.argtypes = [vp, vp, vp, vp, vp, i64, i64, i64, i64, i64, i64,
                                 ctypes.c_int, ctypes.c_uint, i64, vp]
        lib.gemm_run_ex.restype = ctypes.c_int
        lib.gemm_run_ex.argtypes = [vp, vp, vp, vp, vp, i64, i64, i64, i64, i64, i64,
                                    ctypes.c_int, ctypes.c_uint, i64, ctypes.c_float,
                                    ctypes.c_float, ctypes.c_int, ctypes.c_int, vp]
        lib.gemm_run_noalloc.restype = ctypes.c_int
        lib.gemm_run_noalloc.argtypes = lib.gemm_run_ex.argtypes
        lib.gemm_prune24.restype = ctypes.c_int
        lib.gemm_prune24.argtypes = [vp, vp, i64, i64, i64, ctypes.c_int, i64, vp, vp, vp]
        lib.gemm_run_sparse24.restype = ctypes.c_int
        lib.gemm_run_sparse24.argtypes = [vp, vp, vp, vp, vp, vp, i64, i64, i64, i64, i64,
                                          ctypes.c_int, ctypes.c_uint, i64, vp]
        cf, ci, cu = ctypes.c_float, ctypes.c_int, ctypes.c_uint
        lib.gemm_run_grouped.restype = ci
        lib.gemm_run_grouped.argtypes = [vp, vp, vp, vp, vp, vp, i64, i64, i64, i64, i64, i64, i64, ci,
                                         cu, cf, cf, ci, ci, vp]
        lib.gemm_run_grouped_wgrad.restype = ci
        lib.gemm_run_grouped_wgrad.argtypes = lib.gemm_run_grouped.argtypes
        lib.gemm_quant8.restype = ci
        lib.gemm_quant8.argtypes = [vp, vp, i64, i64, i64, ci, cu, i64, ci, ci, vp, vp, vp]
        lib.gemm_run_scaled8.restype = ci
        lib.gemm_run_scaled8.argtypes = [vp, ctypes.POINTER(Q8Operand), ctypes.POINTER(Q8Operand), vp, vp,
                                         vp, i64, i64, i64, i64, i64, cu, cf, cf, ci, ci, vp]
        lib.gemm_plan.restype = ctypes.c_int
        lib.gemm_plan.argtypes = [vp, i64, i64, i64, i64, i64, i64, ctypes.c_int, ctypes.c_uint,
                                  i64, ctypes.c_char_p, ctypes.c_size_t]
        _lib = lib
        return lib


def status_string(status: int) -> str:
    return load_library().gemm_status_string(int(status)).decode()


def plan_label(M, N, K, lda, ldb, ldc, dtype, flags=0, batch=1, handle=None) -> str:
    """Which kernel path gemm_run takes for these sizes (no launch; handle optional)."""
    lib = load_library()
    buf = ctypes.create_string_buffer(256)
    h = handle.ptr if handle is not None else None
    rc = lib.gemm_plan(h, M, N, K, lda, ldb, ldc, dtype, flags, batch, buf, 256)
    if rc != GEMM_OK:
        raise GemmError(rc, "gemm_plan")
    return buf.value.decode()


class Handle:
    """Owns one gemm_handle_t (bound to the HIP device current at creation)."""

    def __init__(self):
        lib = load_library()
        p = ctypes.c_void_p()
        rc = lib.gemm_create(ctypes.byref(p))
        if rc != GEMM_OK:
            raise GemmError(rc, "gemm_create")
        self.ptr = p

    def close(self):
        if self.ptr:
            rc = load_library().gemm_destroy(self.ptr)
            self.ptr = None
            if rc != GEMM_OK:
                raise GemmError(rc, "gemm_destroy")

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    def run(self, A: int, B: int, C: int, D: int, M: int, N: int, K: int, lda: int, ldb: int,
            ldc: int, dtype: int, flags: int = 0, batch: int = 1, stream: int = 0) -> None:
        """Raw-pointer call of gemm_run (device addresses as ints, stream as hipStream_t int)."""
        rc = load_library().gemm_run(self.ptr, A, B, C, D, M, N, K, lda, ldb, ldc, dtype, flags,
                                     batch, stream)
        if rc != GEMM_OK:
            raise GemmError(rc, "gemm_run")

    def status(self, A, B, C, D, M, N, K, lda, ldb, ldc, dtype, flags=0, batch=1, stream=0) -> int:
        """Like run() but returns the status code instead of raising."""
        return load_library().gemm_run(self.ptr, A, B, C, D, M, N, K, lda, ldb, ldc, dtype, flags,
                                       batch, stream)

    def status_ex(self, A, B, C, D, M, N, K, lda, ldb, ldc, dtype, flags=0, batch=1,
                  alpha=1.0, beta=1.0, c_type=GEMM_OUT_F32, d_type=GEMM_OUT_F32,
                  stream=0) -> int:
        """Raw-pointer call of gemm_run_ex; returns the status code."""
        return load_library().gemm_run_ex(self.ptr, A, B, C, D, M, N, K, lda, ldb, ldc, dtype,
                                          flags, batch, alpha, beta, c_type, d_type, stream)

    def status_noalloc(self, A, B, C, D, M, N, K, lda, ldb, ldc, dtype, flags=0, batch=1,
                       alpha=1.0, beta=1.0, c_type=GEMM_OUT_F32, d_type=GEMM_OUT_F32,
                       stream=0) -> int:
        """Raw-pointer call of gemm_run_noalloc (fixed scratch, no device allocation);
        returns the status code."""
        return load_library().gemm_run_noalloc(self.ptr, A, B, C, D, M, N, K, lda, ldb, ldc, dtype,
                                               flags, batch, alpha, beta, c_type, d_type, stream)

    def prune24(self, A, M, K, lda, dtype, batch, Ac, meta, stream=0) -> int:
        """Raw-pointer call of gemm_prune24; returns the status code."""
        return load_library().gemm_prune24(self.ptr, A, M, K, lda, dtype, batch, Ac, meta, stream)

    def run_sparse24(self, Ac, meta, B, C, D, M, N, K, ldb, ldc, dtype, flags=0, batch=1,
                     stream=0) -> int:
        """Raw-pointer call of gemm_run_sparse24; returns the status code."""
        return load_library().gemm_run_sparse24(self.ptr, Ac, meta, B, C, D, M, N, K, ldb, ldc,
                                                dtype, flags, batch, stream)

    def run_grouped(self, A, B, C, D, offsets, groups, M, N, K, lda, ldb, ldc, dtype, flags=0, alpha=1.0,
                    beta=0.0, c_type=GEMM_OUT_F32, d_type=GEMM_OUT_F32, stream=0) -> int:
        """Raw-pointer call of gemm_run_grouped; returns the status code."""
        return load_library().gemm_run_grouped(self.ptr, A, B, C, D, offsets, groups, M, N, K, lda, ldb,
                                               ldc, dtype, flags, alpha, beta, c_type, d_type, stream)

    def run_grouped_wgrad(self, X, Y, C, D, offsets, groups, M, N, K, ldx, ldy, ldc, dtype, flags=0,
                          alpha=1.0, beta=0.0, c_type=GEMM_OUT_F32, d_type=GEMM_OUT_F32, stream=0) -> int:
        """Raw-pointer call of gemm_run_grouped_wgrad; returns the status code."""
        return load_library().gemm_run_grouped_wgrad(self.ptr, X, Y, C, D, offsets, groups, M, N, K, ldx,
                                                     ldy, ldc, dtype, flags, alpha, beta, c_type, d_type,
                                                     stream)

    def quant8(self, X, M, K, ldx, x_type, flags, batch, block, q_type, Q, scale, stream=0) -> int:
        """Raw-pointer call of gemm_quant8; returns the status code."""
        return load_library().gemm_quant8(self.ptr, X, M, K, ldx, x_type, flags, batch, block, q_type, Q,
                                          scale, stream)

    def run_scaled8(self, A: Q8Operand, B: Q8Operand, C, D, offsets, groups, M, N, K, ldc, flags=0,
                    alpha=1.0, beta=0.0, c_type=GEMM_OUT_F32, d_type=GEMM_OUT_F32, stream=0) -> int:
        """Raw-pointer call of gemm_run_scaled8; returns the status code."""
        return load_library().gemm_run_scaled8(self.ptr, ctypes.byref(A), ctypes.byref(B), C, D, offsets,
                                               groups, M, N, K, ldc, flags, alpha, beta, c_type, d_type,
                                               stream)

    def run_ex(self, *args, **kw) -> None:
        """Like status_ex() but raises on a non-zero status."""
        rc = self.status_ex(*args, **kw)
        if rc != GEMM_OK:
            raise GemmError(rc, "gemm_run_ex")




def sparse24_kp(K: int, dtype: int = GEMM_F16) -> int:
    """Dense k per compressed row (Kp/2 values, Kp/16 16-bit index words):
    64 * ceil(K / 64) for fp16/bf16, 128 * ceil(K / 128) for int8."""
    g = 128 if dtype == GEMM_I8 else 64
    return -(-K // g) * g


def sparse24_mp(M: int) -> int:
    """Rows of the compressed form: 16 * ceil(M / 16) (16-row blocks)."""
    return -(-M // 16) * 16


_tls = threading.local()


def default_handle() -> Handle:
    """The handle the torch front ends use: one per host thread, device and
    stream, since a handle's workspace must not serve two calls that can run at
    the same time (one thread at a time, one stream at a time).  Each cached
    handle keeps its workspace until release_default_handles() is called on
    the thread that created it (or the thread ends)."""
    import torch
    dev = torch.cuda.current_device()
    key = (dev, torch.cuda.current_stream(dev).cuda_stream)
    handles = getattr(_tls, "handles", None)
    if handles is None:
        handles = _tls.handles = {}
    h = handles.get(key)
    if h is None:
        h = Handle()
        handles[key] = h
    return h


def release_default_handles() -> int:
    """Close this thread's cached front-end handles and free their workspaces
    (each close waits for its device's queued work).  A program that creates
    many streams or threads calls this when it is done with one; the next
    front-end call makes a new handle.  Returns the number of handles closed."""
    handles = getattr(_tls, "handles", None) or {}
    n = len(handles)
    for h in handles.values():
        h.close()
    _tls.handles = {}
    return n


def _operand_layout(X, rows: int, cols: int, name: str):
    """(col_major, ld) of a logical rows x cols matrix view (last two dims)."""
    s_r, s_c = X.stride(-2), X.stride(-1)
    if s_c == 1 and (s_r >= max(1, cols) or rows == 1):
        return False, max(s_r, cols, 1)
    if s_r == 1 and (s_c >= max(1, rows) or cols == 1):
        return True, max(s_c, rows, 1)
    raise ValueError(f"{name} must be row-major or column-major in its last two dims")


_OUT_CODES: dict = {}


def _out_code(dtype):
    if not _OUT_CODES:
        import torch
        _OUT_CODES.update({torch.float32: GEMM_OUT_F32, torch.float16: GEMM_OUT_F16,
                           torch.bfloat16: GEMM_OUT_BF16, torch.int32: GEMM_OUT_I32,
                           torch.float64: GEMM_OUT_F64})
    return _OUT_CODES.get(dtype)


def gemm(A, B, C=None, out=None, alpha: float = 1.0, beta: float = 1.0, out_dtype=None,
         handle: Handle | None = None):
    """D = alpha * (A @ B) + beta * C on the current stream.

    A: (..., M, K) float16 / bfloat16 / int8 / float64;  B: (..., K, N) same dtype (row-major,
    or a transposed view = column-major);  C: (..., M, N) row-major, float32 / float16 /
    bfloat16 for 16-bit inputs, int32 for int8, float64 for float64 (None means beta = 0).
    D has ``out_dtype`` (default: float32; int32 for int8; float64 for float64), a new tensor
    with C's strides unless ``out`` is given (``out`` may be C itself when the dtypes agree).
    Leading batch dims (one at most) must be contiguous in the library's sense.  int8 and
    float64 take alpha == 1 and beta in {0, 1} only."""
    import torch
    dt = {torch.float16: GEMM_F16, torch.bfloat16: GEMM_BF16, torch.int8: GEMM_I8,
          torch.float64: GEMM_F64}.get(A.dtype)
    if dt is None or B.dtype != A.dtype:
        raise TypeError("A and B must both be float16, bfloat16, int8 or float64")
    acc = {GEMM_I8: torch.int32, GEMM_F64: torch.float64}.get(dt, torch.float32)
    if A.dim() not in (2, 3) or B.dim() not in (2, 3):
        raise ValueError("A and B must be 2-D or 3-D")
    if not (A.is_cuda and B.is_cuda) or B.device != A.device:
        raise ValueError("A and B must be on the same GPU")
    M, K = A.shape[-2], A.shape[-1]
    N = B.shape[-1]
    nd = max(A.dim(), B.dim())
    batch = A.shape[0] if A.dim() == 3 else (B.shape[0] if B.dim() == 3 else 1)
    a_shared = A.dim() == 2 and nd == 3
    b_shared = B.dim() == 2 and nd == 3
    if B.shape[-2] != K or (A.dim() == 3 and B.dim() == 3 and B.shape[0] != batch):
        raise ValueError("shape mismatch between A and B")
    if C is None:
        beta = 0.0
    else:
        if C.device != A.device or C.dim() != nd or C.shape[-2:] != (M, N) or \
                (nd == 3 and C.shape[0] != batch):
            raise ValueError("C must be a tensor of shape ((batch,) M, N) on A's GPU")
        if C.stride(-1) != 1 or (M > 1 and C.stride(-2) < N):
            raise ValueError("C must be row-major with a row stride of at least N")
    c_code = _out_code(C.dtype if C is not None else acc)
    if c_code is None:
        raise TypeError("C must be float32, float16, bfloat16 or int32")
    d_dtype = out.dtype if out is not None else (out_dtype if out_dtype is not None else acc)
    d_code = _out_code(d_dtype)
    if d_code is None:
        raise TypeError("out dtype must be float32, float16, bfloat16 or int32")
    a_col, lda = _operand_layout(A, M, K, "A")
    b_col, ldb = _operand_layout(B, K, N, "B")
    shape = (batch, M, N) if nd == 3 else (M, N)
    if C is not None:
        ldc = max(C.stride(-2), N, 1)
        strides = C.stride()
    else:
        ldc = max(N, 1)
        strides = (M * ldc, ldc, 1) if nd == 3 else (ldc, 1)
    if out is None:
        out = torch.empty_strided(shape, strides, dtype=d_dtype, device=A.device)
    if out.device != A.device or tuple(out.shape) != shape or out.stride() != strides:
        raise ValueError("out must have shape (..., M, N) and C's strides, on A's GPU")
    if batch > 1:
        want_a = (K if a_col else M) * lda
        want_b = (N if b_col else K) * ldb
        if (not a_shared and A.stride(0) != want_a) or (not b_shared and B.stride(0) != want_b) \
                or out.stride(0) != M * ldc:
            raise ValueError("batched operands must have contiguous batch strides")
    flags = (GEMM_A_COLMAJOR if a_col else 0) | (GEMM_B_COLMAJOR if b_col else 0) | \
        (GEMM_A_SHARED if a_shared else 0) | (GEMM_B_SHARED if b_shared else 0)
    with torch.cuda.device(A.device):  # the handle and the stream of A's GPU
        h = handle if handle is not None else default_handle()
        stream = torch.cuda.current_stream(A.device).cuda_stream
        h.run_ex(A.data_ptr(), B.data_ptr(), C.data_ptr() if C is not None else 0, out.data_ptr(),
                 M, N, K, lda, ldb, ldc, dt, flags, batch, alpha=float(alpha), beta=float(beta),
                 c_type=c_code, d_type=d_code, stream=stream)
    return out


class Sparse24:
    """A 2:4-compressed A (the library's blocked form): values ``Ac``, index words
    ``meta``, and the dense sizes M, K, the input code and the batch."""

    def __init__(self, Ac, meta, M: int, K: int, dtype: int, batch: int):
        self.Ac, self.meta, self.M, self.K, self.dtype, self.batch = Ac, meta, M, K, dtype, batch


def prune24(A, handle: Handle | None = None) -> Sparse24:
    """Compress A ((batch,) M, K; float16, bfloat16 or int8; rows K-contiguous with
    contiguous batches) to 2:4 form on the current stream: in every group of four
    consecutive k of a row the two entries of largest magnitude are kept."""
    import torch
    dt = {torch.float16: GEMM_F16, torch.bfloat16: GEMM_BF16, torch.int8: GEMM_I8}.get(A.dtype)
    if dt is None:
        raise TypeError("A must be float16, bfloat16 or int8")
    if A.dim() not in (2, 3) or not A.is_cuda:
        raise ValueError("A must be a 2-D or 3-D GPU tensor")
    M, K = A.shape[-2], A.shape[-1]
    batch = A.shape[0] if A.dim() == 3 else 1
    if A.stride(-1) != 1 or (M > 1 and A.stride(-2) < K):
        raise ValueError("A must be row-major (K-contiguous rows)")
    lda = max(A.stride(-2), K, 1)
    if batch > 1 and A.stride(0) != M * lda:
        raise ValueError("batched A must have a contiguous batch stride")
    kp, mp = sparse24_kp(K, dt), sparse24_mp(M)
    Ac = torch.empty((batch, mp, kp // 2), dtype=torch.int8 if dt == GEMM_I8 else torch.int16,
                     device=A.device)
    meta = torch.empty((batch, mp, kp // 16), dtype=torch.int16, device=A.device)
    with torch.cuda.device(A.device):
        h = handle if handle is not None else default_handle()
        rc = h.prune24(A.data_ptr(), M, K, lda, dt, batch, Ac.data_ptr(), meta.data_ptr(),
                       torch.cuda.current_stream(A.device).cuda_stream)
    if rc != GEMM_OK:
        raise GemmError(rc, "gemm_prune24")
    return Sparse24(Ac, meta, M, K, dt, batch)


def gemm_sparse24(sp: Sparse24, B, C=None, out=None, handle: Handle | None = None):
    """D = prune(A) @ B + C from a Sparse24 on the current stream.  B: ((batch,) K, N)
    of A's type, row-major or a transposed (column-major) view; C: ((batch,) M, N)
    row-major float32 (16-bit inputs) or int32 (int8), or None for a zero C.  D is a
    new tensor with C's strides unless ``out`` is given (``out`` may be C)."""
    import torch
    want = {GEMM_F16: torch.float16, GEMM_BF16: torch.bfloat16, GEMM_I8: torch.int8}[sp.dtype]
    if B.dtype != want:
        raise TypeError("B must have the compressed A's type")
    if not B.is_cuda or B.device != sp.Ac.device or B.dim() not in (2, 3):
        raise ValueError("B must be a 2-D or 3-D tensor on A's GPU")
    M, K, N, batch = sp.M, sp.K, B.shape[-1], sp.batch
    if B.shape[-2] != K or (B.dim() == 3 and B.shape[0] != batch) or (B.dim() == 2 and batch > 1):
        raise ValueError("B must be (batch, K, N) with the compressed A's K and batch")
    acc = torch.int32 if sp.dtype == GEMM_I8 else torch.float32
    b_col, ldb = _operand_layout(B, K, N, "B")
    shape = (batch, M, N) if B.dim() == 3 else (M, N)
    if C is None:
        C = torch.zeros(shape, dtype=acc, device=B.device)
    if C.dtype != acc or tuple(C.shape) != shape or C.device != B.device:
        raise ValueError(f"C must be {acc} of shape {shape} on B's GPU")
    if C.stride(-1) != 1 or (M > 1 and C.stride(-2) < N):
        raise ValueError("C must be row-major with a row stride of at least N")
    ldc = max(C.stride(-2), N, 1)
    if out is None:
        out = torch.empty_strided(shape, C.stride(), dtype=acc, device=B.device)
    if out.dtype != acc or tuple(out.shape) != shape or out.stride() != C.stride():
        raise ValueError("out must match C's dtype, shape and strides")
    if batch > 1 and (B.stride(0) != (N if b_col else K) * ldb or C.stride(0) != M * ldc):
        raise ValueError("batched operands must have contiguous batch strides")
    with torch.cuda.device(B.device):
        h = handle if handle is not None else default_handle()
        rc = h.run_sparse24(sp.Ac.data_ptr(), sp.meta.data_ptr(), B.data_ptr(), C.data_ptr(),
                            out.data_ptr(), M, N, K, ldb, ldc, sp.dtype,
                            GEMM_B_COLMAJOR if b_col else 0, batch,
                            torch.cuda.current_stream(B.device).cuda_stream)
    if rc != GEMM_OK:
        raise GemmError(rc, "gemm_run_sparse24")
    return out


def _on(device, handle, call):
    """call(handle, stream) with `device` current: `handle`, or the default one of the
    device's current stream, and that stream."""
    import torch
    index = device.index
    if torch.cuda.current_device() != index:
        with torch.cuda.device(index):
            return _on(device, handle, call)
    stream = torch._C._cuda_getCurrentRawStream(index)
    if handle is None:
        handles = getattr(_tls, "handles", None)
        handle = handles.get((index, stream)) if handles else None
        if handle is None:
            handle = default_handle()
    return call(handle, stream)


_FLOAT_OUT = (GEMM_OUT_F32, GEMM_OUT_F16, GEMM_OUT_BF16)


def _check_offsets(offsets, device):
    """(groups, flag) of the row offsets of a grouped product."""
    import torch
    if offsets.dtype not in (torch.int32, torch.int64):
        raise TypeError("offsets must be int32 or int64")
    n = offsets.shape[0] if offsets.dim() == 1 else 0
    if n < 1 or offsets.device != device:
        raise ValueError("offsets must be a vector of groups + 1 row numbers on the operands' GPU")
    if n > 1 and offsets.stride(0) != 1:
        raise ValueError("offsets must be contiguous")
    return n - 1, GEMM_OFFSETS_I32 if offsets.dtype == torch.int32 else 0


def _output(C, out, shape, out_dtype, beta, device, name):
    """(C's address, C's code, D, D's code, ldc, beta) of a grouped product with outputs `shape`."""
    import torch
    rows, n = shape[-2], shape[-1]
    ldc = None  # the row stride that C and out share, where rows have one
    for X, what in ((C, "C"), (out, "out")):
        if X is None:
            continue
        if X.device != device or X.shape != shape:
            raise ValueError(f"{what} must be a tensor of shape {name} on the operands' GPU")
        if _out_code(X.dtype) not in _FLOAT_OUT:
            raise TypeError(f"{what} must be float32, float16 or bfloat16")
        strides = X.stride()
        if (n > 1 and strides[-1] != 1) or (rows > 1 and strides[-2] < n):
            raise ValueError(f"{what} must be row-major with a row stride of at least N")
        ld = max(strides[-2] if rows > 1 else n, 1)
        if (ldc is not None and ld != ldc) or (len(shape) == 3 and shape[0] > 1 and strides[0] != rows * ld):
            raise ValueError("C and out must have the same row stride, and contiguous groups")
        ldc = ld
    if ldc is None:
        ldc = max(n, 1)
    if out is None:
        dtype = out_dtype if out_dtype is not None else torch.float32
        if _out_code(dtype) not in _FLOAT_OUT:
            raise TypeError("out dtype must be float32, float16 or bfloat16")
        out = torch.empty_strided(shape, (rows * ldc, ldc, 1) if len(shape) == 3 else (ldc, 1), dtype=dtype,
                                  device=device)
    if C is None:
        return 0, GEMM_OUT_F32, out, _out_code(out.dtype), ldc, 0.0
    return C.data_ptr(), _out_code(C.dtype), out, _out_code(out.dtype), ldc, float(beta)


def _sixteen_bit(A, B, what):
    dt = {GEMM_OUT_F16: GEMM_F16, GEMM_OUT_BF16: GEMM_BF16}.get(_out_code(A.dtype))
    if dt is None or B.dtype != A.dtype:
        raise TypeError(f"{what} must both be float16 or bfloat16")
    if not A.is_cuda or B.device != A.device:
        raise ValueError(f"{what} must be on the same GPU")
    return dt


def _rows_of(X, name):
    """Leading dimension of a row-major matrix."""
    rows, cols = X.shape if X.dim() == 2 else (-1, -1)
    s = X.stride()
    if rows < 0 or (cols > 1 and s[1] != 1) or (rows > 1 and s[0] < cols):
        raise ValueError(f"{name} must be a row-major matrix")
    return max(s[0] if rows > 1 else cols, 1)


def gemm_grouped(A, B, offsets, C=None, out=None, alpha: float = 1.0, beta: float = 1.0, out_dtype=None,
                 handle: Handle | None = None):
    """D[i] = alpha * A[i] @ B[g] + beta * C[i] for the rows i of every group g, on the
    current stream: the experts' products of rows sorted by expert.

    A: (T, K) float16 / bfloat16, row-major;  B: (groups, K, N) of the same dtype,
    contiguous (row-major), or a contiguous (groups, N, K) tensor's transpose(1, 2)
    (column-major);  offsets: groups + 1 ascending row numbers, int32 or int64, on the
    GPU: group g owns the rows offsets[g] .. offsets[g+1] - 1;  C: (T, N) float32 /
    float16 / bfloat16 row-major, or None (beta = 0).  D (T, N) has ``out_dtype``
    (default float32), a new tensor unless ``out`` is given (``out`` may be C when the
    dtypes agree).  Rows that no group owns are left as they are in ``out`` (in a new
    tensor they are undefined).

    The input gradient of Y = gemm_grouped(A, W, offsets) is
    gemm_grouped(dY, W.transpose(1, 2), offsets); the weight gradient is
    gemm_grouped_wgrad(A, dY, offsets)."""
    dt = _sixteen_bit(A, B, "A and B")
    if B.dim() != 3 or A.dim() != 2 or B.shape[1] != A.shape[1]:
        raise ValueError("A must be (T, K) and B (groups, K, N)")
    groups, flags = _check_offsets(offsets, A.device)
    (T, K), N = A.shape, B.shape[2]
    if B.shape[0] != groups:
        raise ValueError("offsets must hold one number more than B has groups")
    lda = _rows_of(A, "A")
    b_col, ldb = _operand_layout(B, K, N, "B")
    if groups > 1 and K > 0 and N > 0 and B.stride(0) != (N if b_col else K) * ldb:
        raise ValueError("B's groups must be contiguous")
    c, c_code, out, d_code, ldc, beta = _output(C, out, (T, N), out_dtype, beta, A.device, "(T, N)")
    rc = _on(A.device, handle, lambda h, stream: h.run_grouped(
        A.data_ptr(), B.data_ptr(), c, out.data_ptr(), offsets.data_ptr(), groups, T, N, K, lda, ldb, ldc, dt,
        flags | (GEMM_B_COLMAJOR if b_col else 0), alpha, beta, c_code, d_code, stream))
    if rc != GEMM_OK:
        raise GemmError(rc, "gemm_run_grouped")
    return out


def gemm_grouped_wgrad(X, Y, offsets, C=None, out=None, alpha: float = 1.0, beta: float = 1.0,
                       out_dtype=None, handle: Handle | None = None):
    """D[g] = alpha * X_g^T @ Y_g + beta * C[g] for every group g, X_g and Y_g the group's
    rows (see gemm_grouped), on the current stream: the experts' weight gradients.

    X: (T, M), Y: (T, N), float16 / bfloat16, row-major;  C: (groups, M, N) float32 /
    float16 / bfloat16 with contiguous groups, or None (beta = 0).  D has ``out_dtype``
    (default float32), a new tensor unless ``out`` is given (``out`` may be C when the
    dtypes agree).  An empty group's D is beta * C (zero without C).  Rows that no group
    owns are not read."""
    dt = _sixteen_bit(X, Y, "X and Y")
    ldx, ldy = _rows_of(X, "X"), _rows_of(Y, "Y")
    if Y.shape[0] != X.shape[0]:
        raise ValueError("X and Y must have the same rows")
    groups, flags = _check_offsets(offsets, X.device)
    (T, M), N = X.shape, Y.shape[1]
    c, c_code, out, d_code, ldc, beta = _output(C, out, (groups, M, N), out_dtype, beta, X.device,
                                                "(groups, M, N)")
    rc = _on(X.device, handle, lambda h, stream: h.run_grouped_wgrad(
        X.data_ptr(), Y.data_ptr(), c, out.data_ptr(), offsets.data_ptr(), groups, M, N, T, ldx, ldy, ldc, dt,
        flags, alpha, beta, c_code, d_code, stream))
    if rc != GEMM_OK:
        raise GemmError(rc, "gemm_run_grouped_wgrad")
    return out


_F8_CODES: dict = {}


def _f8_code(dtype):
    if not _F8_CODES:
        import torch
        _F8_CODES.update({torch.float8_e4m3fn: GEMM_E4M3, torch.float8_e5m2: GEMM_E5M2})
    return _F8_CODES.get(dtype)


class Scaled8:
    """An 8-bit operand of gemm_scaled8: ``q`` ((groups,) rows, Kp), float8_e4m3fn or
    float8_e5m2, K-contiguous rows of Kp = 16 * ceil(K / 16) values, zeros past K; and
    ``scale`` ((groups,) ceil(rows / block), ceil(K / 128)) float32 of any strides: the
    value stands for q times the scale of its block of ``block`` rows by 128 k.  Made
    by quant8, or from tensors that are there.  Both may be changed in place or replaced;
    a product reads what the operand holds when it is called."""

    def __init__(self, q, scale, block: int = 1, K: int | None = None):
        self.type = _f8_code(q.dtype)
        if self.type is None or _out_code(scale.dtype) != GEMM_OUT_F32:
            raise TypeError("q must be float8_e4m3fn or float8_e5m2, and scale float32")
        if block != 1 and block != 128:
            raise ValueError("block must be 1 or 128")
        shape = q.shape
        dims = len(shape)
        K = shape[-1] if K is None else K
        kp = -(-K // 16) * 16
        if dims not in (2, 3) or shape[-1] != kp:
            raise ValueError("q must be ((groups,) rows, 16 * ceil(K / 16))")
        rows = shape[-2]
        groups = shape[0] if dims == 3 else None
        blocks = (-(-rows // block), -(-K // 128))
        if scale.shape != (blocks if groups is None else (groups, *blocks)):
            raise ValueError("scale must be ((groups,) ceil(rows / block), ceil(K / 128))")
        if scale.device != q.device or not q.is_cuda:
            raise ValueError("q and scale must be on the same GPU")
        s, at = q.stride(), q.data_ptr()
        if 0 not in shape and (s[-1] != 1 or (rows > 1 and (s[-2] < kp or s[-2] % 16)) or
                          (dims == 3 and groups > 1 and s[0] % 16) or at % 16):
            raise ValueError("q's rows must be contiguous and begin at multiples of 16 bytes")
        self._set(q, scale, block, K, rows, groups, at, s[-2] if rows > 1 and kp else kp,
                  s[0] if dims == 3 else 0)

    def _set(self, q, scale, block, K, rows, groups, at, ld, group):
        t, scale_at = scale.stride(), scale.data_ptr()
        self.q, self.scale, self.block, self.K, self.rows, self.groups = q, scale, block, K, rows, groups
        self._operand = Q8Operand(at, scale_at, ld, t[-2], t[-1], group, t[0] if groups is not None else 0, self.type)
        self._of = q, scale, at, scale_at, block, K

    @property
    def operand(self) -> Q8Operand:
        """The operand as it is now: ``q`` and ``scale`` may have been replaced, or their
        memory moved, since the structure was filled in; it is then checked and filled in anew."""
        q, scale, at, scale_at, block, K = self._of
        if self.q is not q or self.scale is not scale or q.data_ptr() != at or scale.data_ptr() != scale_at or \
                self.block != block or self.K != K:
            self.__init__(self.q, self.scale, self.block, self.K)
        return self._operand

    def __reduce__(self):  # copies and saved operands: of the tensors, not of addresses
        return Scaled8, (self.q, self.scale, self.block, self.K)


def quant8(X, block: int = 1, dtype=None, handle: Handle | None = None) -> Scaled8:
    """Quantize X ((batch,) M, K; float32, float16 or bfloat16; row-major or a transposed
    view) to 8-bit floats (``dtype``: torch.float8_e4m3fn, the default, or float8_e5m2)
    with a scale for every block of 128 consecutive k of one row (block = 1: activations)
    or of 128 rows (block = 128: weights), on the current stream.  The result is
    K-contiguous whatever X's layout: the operand B of gemm_scaled8 for weights stored
    (K, N) is quant8(W.t(), block=128)."""
    import torch
    dtype = torch.float8_e4m3fn if dtype is None else dtype
    code = _f8_code(dtype)
    x_code = _out_code(X.dtype)
    if code is None or x_code not in _FLOAT_OUT:
        raise TypeError("X must be float32, float16 or bfloat16, and dtype float8_e4m3fn or float8_e5m2")
    if X.dim() not in (2, 3) or not X.is_cuda:
        raise ValueError("X must be a 2-D or 3-D GPU tensor")
    if block not in (1, 128):
        raise ValueError("block must be 1 or 128")
    M, K = X.shape[-2], X.shape[-1]
    lead = X.shape[:-2]
    batch = X.shape[0] if lead else 1
    col, ldx = _operand_layout(X, M, K, "X")
    if batch > 1 and X.numel() and X.stride(0) != (K if col else M) * ldx:
        raise ValueError("batched X must have a contiguous batch stride")
    kb, mb = -(-K // 128), -(-M // block)
    kp = -(-K // 16) * 16
    q = torch.empty((*lead, M, kp), dtype=dtype, device=X.device)
    scale = torch.empty((*lead, kb, mb), dtype=torch.float32, device=X.device)
    at = q.data_ptr()
    rc = _on(X.device, handle, lambda h, stream: h.quant8(
        X.data_ptr(), M, K, ldx, x_code, GEMM_A_COLMAJOR if col else 0, batch, block, code, at, scale.data_ptr(),
        stream))
    if rc != GEMM_OK:
        raise GemmError(rc, "gemm_quant8")
    r = Scaled8.__new__(Scaled8)  # what the constructor would check holds
    r.type = code
    r._set(q, scale.transpose(-1, -2), block, K, M, batch if lead else None, at, kp, M * kp)
    return r


def gemm_scaled8(A: Scaled8, B: Scaled8, offsets=None, C=None, out=None, alpha: float = 1.0,
                 beta: float = 1.0, out_dtype=None, handle: Handle | None = None):
    """D = alpha * (A @ B^T) + beta * C of 8-bit operands with block scales, on the current
    stream.  A: (T, K) with blocks of one row;  B: (N, K) with blocks of 128 rows (the N
    columns of a K x N matrix as rows);  formats may differ.  With ``offsets`` (see
    gemm_grouped) B is (groups, N, K) and the rows of group g meet B[g].  C, ``out`` and
    ``out_dtype`` (default float32) as in gemm_grouped.

    A float32 result sums exact products in 32 bits.  For a float16 or bfloat16 one the
    8-bit matrix instruction keeps, of 8 products with consecutive k, what lies within 13
    bits of the largest (an error of at most 2^-9 of the sum of magnitudes, about 1.5e-5 of
    a random result's norm), except where rows are few (up to 16 to a group, or 64 where the
    groups' columns are few too), where every result is exact in this sense."""
    a, b = A.operand, B.operand
    if A.block != 1 or B.block != 128:
        raise ValueError("A must have blocks of one row and B blocks of 128 rows")
    device = A.q.device
    if A.groups is not None or A.K != B.K or B.q.device != device:
        raise ValueError("A must be (T, K) and B ((groups,) N, K) on the same GPU")
    groups, flags = (1, 0) if offsets is None else _check_offsets(offsets, device)
    if (offsets is None) != (B.groups is None) or (offsets is not None and B.groups != groups):
        raise ValueError("a grouped B needs offsets that hold one number more than it has groups")
    T, N = A.rows, B.rows
    c, c_code, out, d_code, ldc, beta = _output(C, out, (T, N), out_dtype, beta, device, "(T, N)")
    rc = _on(device, handle, lambda h, stream: h.run_scaled8(
        a, b, c, out.data_ptr(), offsets.data_ptr() if offsets is not None else 0, groups, T, N,
        A.K, ldc, flags, alpha, beta, c_code, d_code, stream))
    if rc != GEMM_OK:
        raise GemmError(rc, "gemm_run_scaled8")
    return out
