"""ctypes binding of libsgemm.so (argument marshalling only).

Every computing function here hands pointers, sizes and a stream to the C ABI
in include/sgemm.h; no arithmetic of the GEMM happens in Python.  Importing
this module raises ImportError when the library has not been built (there is
no fallback path).
"""
from __future__ import annotations

import ctypes
import os

from .build import LIB_DEBUG_BOUNDS_PATH, LIB_PATH

# SGEMM_LIBRARY=debug_bounds loads the range-checked test build instead of the
# library (a test switch; the library is always one of this package's builds)
library_path = LIB_DEBUG_BOUNDS_PATH if os.environ.get("SGEMM_LIBRARY") == "debug_bounds" \
    else LIB_PATH

if not os.path.exists(library_path):
    raise ImportError(
        f"{os.path.basename(library_path)} is not built at {library_path}; run "
        "`python -c 'import __graft_entry__ as g; g.build()'` or "
        "`python -m dense_fp32_gemm_02_gb300.build`")

lib = ctypes.CDLL(library_path)

_i, _f, _p = ctypes.c_int, ctypes.c_float, ctypes.c_void_p
_ull, _ll, _d = ctypes.c_ulonglong, ctypes.c_longlong, ctypes.c_double

lib.sgemm.argtypes = [_i, _i, _i, _f, _p, _i, _p, _i, _f, _p, _i, _p]
lib.sgemm.restype = _i
lib.sgemm_host.argtypes = [_i, _i, _i, _f, _p, _i, _p, _i, _f, _p, _i, _p]
lib.sgemm_host.restype = _i
lib.sgemm_ex.argtypes = [_i, _i, _i, _f, _p, _i, _ll, _p, _i, _ll, _f, _p, _i, _ll, _i, _p, _ll,
                         _i, _p]
lib.sgemm_ex.restype = _i
lib.sgemm_noalloc.argtypes = [_i, _i, _i, _f, _p, _i, _p, _i, _f, _p, _i, _p]
lib.sgemm_noalloc.restype = _i
lib.sgemm_3xtf32.argtypes = [_i, _i, _i, _f, _p, _i, _p, _i, _f, _p, _i, _p]
lib.sgemm_3xtf32.restype = _i
lib.sgemm_host_3xtf32.argtypes = [_i, _i, _i, _f, _p, _i, _p, _i, _f, _p, _i, _p]
lib.sgemm_host_3xtf32.restype = _i
lib.sgemm_lora.argtypes = [_i] * 6 + [_p, _i, _p, _i, _p, _i, _ll, _p, _i, _ll, _p, _p, _p, _p,
                                      _p, _i, _p, _i, _p]
lib.sgemm_lora.restype = _i
lib.sgemm_lora_backward.argtypes = [_i] * 6 + [_p, _i, _p, _i, _p, _i, _p, _i, _p, _i, _p, _i, _ll,
                                               _p, _i, _ll, _p, _p, _p, _p, _i, _p, _i, _p, _i,
                                               _ll, _p, _i, _ll, _p]
lib.sgemm_lora_backward.restype = _i
lib.sgemm_act8_store.argtypes = [_i, _i, _i, _p, _i, _i, _p, _i, _p, _i, _p, _i, _p]
lib.sgemm_act8_store.restype = _i
lib.sgemm_act8_load.argtypes = [_i, _i, _i, _p, _i, _p, _i, _p, _i, _p]
lib.sgemm_act8_load.restype = _i
lib.sgemm_act8_grad.argtypes = [_i, _i, _i, _p, _i, _p, _i, _i, _p, _i, _p, _i, _p]
lib.sgemm_act8_grad.restype = _i
lib.sgemm_act8_weight_grad.argtypes = [_i, _i, _i, _i, _p, _i, _p, _i, _p, _i, _f, _p, _i, _p]
lib.sgemm_act8_weight_grad.restype = _i
lib.sgemm_status_string.argtypes = [_i]
lib.sgemm_status_string.restype = ctypes.c_char_p
lib.sgemm_version.argtypes = []
lib.sgemm_version.restype = _i
lib.sgemm_last_cuda_error.argtypes = []
lib.sgemm_last_cuda_error.restype = _i
lib.sgemm_device_status.argtypes = [_p]
lib.sgemm_device_status.restype = _i
lib.sgemm_set_wait_timeout_ns.argtypes = [_ull]
lib.sgemm_set_wait_timeout_ns.restype = _i
lib.sgemm_selftest_wait_timeout.argtypes = [_ull, _p]
lib.sgemm_selftest_wait_timeout.restype = _i
lib.sgemm_profile_enable.argtypes = [_i]
lib.sgemm_profile_enable.restype = _i
lib.sgemm_profile_collect.argtypes = [ctypes.POINTER(_d), ctypes.POINTER(_ll),
                                      ctypes.POINTER(_d), ctypes.POINTER(_ll)]
lib.sgemm_profile_collect.restype = _i
lib.sgemm_kernel_launch_count.argtypes = []
lib.sgemm_kernel_launch_count.restype = _ll
lib.sgemm_config_string.argtypes = [_i, _i, _i]
lib.sgemm_config_string.restype = ctypes.c_char_p
lib.sgemm_last_kernel.argtypes = []
lib.sgemm_last_kernel.restype = ctypes.c_char_p
lib.sgemm_variant_count.argtypes = []
lib.sgemm_variant_count.restype = _i
lib.sgemm_variant_name.argtypes = [_i]
lib.sgemm_variant_name.restype = ctypes.c_char_p
lib.sgemm_set_variant.argtypes = [_i]
lib.sgemm_set_variant.restype = _i
lib.sgemm_set_3xtf32_kernel.argtypes = [_i]
lib.sgemm_set_3xtf32_kernel.restype = _i
lib.sgemm_debug_drop_release.argtypes = [_i]
lib.sgemm_debug_drop_release.restype = _i
lib.sgemm_debug_bounds_checks.argtypes = []
lib.sgemm_debug_bounds_checks.restype = _i

SGEMM_OK = 0
SGEMM_ERR_INVALID_ARG = 1
SGEMM_ERR_UNSUPPORTED_DEVICE = 2
SGEMM_ERR_CUDA = 3
SGEMM_ERR_TIMEOUT = 4
SGEMM_ERR_ALLOC = 5
SGEMM_ERR_TOO_LARGE = 6
SGEMM_ERR_BOUNDS = 7


class SgemmError(RuntimeError):
    def __init__(self, status: int):
        self.status = status
        msg = lib.sgemm_status_string(status).decode()
        if status in (SGEMM_ERR_CUDA, SGEMM_ERR_ALLOC):
            msg += f" (cuda error {lib.sgemm_last_cuda_error()})"
        super().__init__(msg)


def check(status: int) -> int:
    if status != SGEMM_OK:
        raise SgemmError(status)
    return status


def status_string(status: int) -> str:
    return lib.sgemm_status_string(status).decode()


def version() -> int:
    return lib.sgemm_version()


# ------------------------------------------------------------------ tensors
_INT_MAX = 2 ** 31 - 1   # sizes and pitches are C ints, which ctypes cuts to 32 bits


def _ld(t, width: int) -> int:
    """Row pitch (elements) of a 2-D row-major tensor/array view."""
    if t.dim() != 2:
        raise ValueError("expected a 2-D tensor")
    if t.numel() > 0 and t.size(1) > 1 and t.stride(1) != 1:
        raise ValueError("rows must be contiguous (stride(1) == 1)")
    if t.size(0) <= 1 or t.numel() == 0:
        return max(width, 1)
    ld = t.stride(0)
    if ld < t.size(1):
        raise ValueError(f"rows must not overlap (stride(0) is {ld}, below the {t.size(1)} columns, "
                         "as in an expanded tensor)")
    if ld > _INT_MAX:
        raise ValueError(f"rows are too far apart (stride(0) is {ld}, past 2^31 - 1)")
    return max(ld, width)


def _stream_handle(stream, device):
    import torch
    if stream is None:
        stream = torch.cuda.current_stream(device)
    return ctypes.c_void_p(stream.cuda_stream)


def _shapes(A, B, C):
    M, K = A.shape
    K2, N = B.shape
    if K2 != K:
        raise ValueError(f"inner dimensions differ: A {tuple(A.shape)}, B {tuple(B.shape)}")
    if tuple(C.shape) != (M, N):
        raise ValueError(f"C must be {(M, N)}, got {tuple(C.shape)}")
    if max(M, N, K) > _INT_MAX:
        raise SgemmError(SGEMM_ERR_TOO_LARGE)
    return M, N, K


def _cuda_f32(*named):
    """TypeError unless every (name, tensor) pair holds a CUDA float32 tensor;
    ValueError unless they all sit on one device."""
    import torch
    for name, t in named:
        if not isinstance(t, torch.Tensor) or t.dtype != torch.float32 or not t.is_cuda:
            raise TypeError(f"{name} must be a CUDA float32 tensor")
    if len({t.device for _, t in named}) > 1:
        raise ValueError(", ".join(n for n, _ in named) + " must be on one device")


def sgemm_into(A, B, C, alpha: float = 1.0, beta: float = 0.0, stream=None):
    """C <- alpha*A@B + beta*C on CUDA float32 tensors (row-major, any row pitch).
    Asynchronous on `stream` (default: torch's current stream of C's device)."""
    import torch
    _cuda_f32(("A", A), ("B", B), ("C", C))
    M, N, K = _shapes(A, B, C)
    with torch.cuda.device(C.device):
        st = lib.sgemm(M, N, K, float(alpha), A.data_ptr(), _ld(A, K), B.data_ptr(), _ld(B, N),
                       float(beta), C.data_ptr(), _ld(C, N), _stream_handle(stream, C.device))
    check(st)
    return C


ACTIVATIONS = {"none": 0, "relu": 1, "gelu": 2}


def _batched(t, name):
    """(2-D view of batch 0, batch count, batch stride in elements) of a 2-D or
    3-D tensor; a 2-D tensor is one matrix used by every batch (stride 0)."""
    if t.dim() == 2:
        return t, 1, 0
    if t.dim() != 3:
        raise ValueError(f"{name} must be 2-D or 3-D")
    return t[0], t.size(0), (t.stride(0) if t.size(0) > 1 else 0)


def sgemm_ex_into(A, B, C, alpha: float = 1.0, beta: float = 0.0, bias=None, act: str = "none",
                  stream=None):
    """C[b] <- act(alpha*A[b]@B[b] + beta*C[b] + bias[b]) on CUDA float32 tensors.
    C is 3-D (batch, M, N) or 2-D (one batch); A and B are 3-D with the same
    batch or 2-D (shared by all batches); bias is None, a length-N vector
    (shared) or (batch, N).  Asynchronous on `stream`."""
    import torch
    _cuda_f32(("A", A), ("B", B), ("C", C), *((("bias", bias),) if bias is not None else ()))
    if act not in ACTIVATIONS:
        raise ValueError(f"act must be one of {sorted(ACTIVATIONS)}, got {act!r}")
    C0, batch, sc = _batched(C, "C")
    A0, ba, sa = _batched(A, "A")
    B0, bb, sb = _batched(B, "B")
    for name, t, n in (("A", A, ba), ("B", B, bb)):
        if t.dim() == 3 and n != batch:
            raise ValueError(f"{name} has {n} batches, C has {batch}")
    M, N, K = _shapes(A0, B0, C0)
    bias_ptr, sbias = None, 0
    if bias is not None:
        if bias.dim() == 1 and bias.size(0) == N:
            sbias = 0
        elif bias.dim() == 2 and tuple(bias.shape) == (batch, N):
            sbias = bias.stride(0) if batch > 1 else 0
        else:
            raise ValueError(f"bias must be ({N},) or ({batch}, {N})")
        if bias.size(-1) > 1 and bias.stride(-1) != 1:
            raise ValueError("bias rows must be contiguous")
        bias_ptr = bias.data_ptr()
    with torch.cuda.device(C.device):
        st = lib.sgemm_ex(M, N, K, float(alpha), A0.data_ptr(), _ld(A0, K), sa, B0.data_ptr(),
                          _ld(B0, N), sb, float(beta), C0.data_ptr(), _ld(C0, N), sc, batch,
                          bias_ptr, sbias, ACTIVATIONS[act], _stream_handle(stream, C.device))
    check(st)
    return C


def sgemm_3xtf32_into(A, B, C, alpha: float = 1.0, beta: float = 0.0, stream=None):
    """Like sgemm_into(), on the tensor cores by the 3xTF32 split (same FP32
    tolerance, not bitwise equal to sgemm_into)."""
    import torch
    _cuda_f32(("A", A), ("B", B), ("C", C))
    M, N, K = _shapes(A, B, C)
    with torch.cuda.device(C.device):
        st = lib.sgemm_3xtf32(M, N, K, float(alpha), A.data_ptr(), _ld(A, K), B.data_ptr(),
                              _ld(B, N), float(beta), C.data_ptr(), _ld(C, N),
                              _stream_handle(stream, C.device))
    check(st)
    return C


def sgemm_noalloc_into(A, B, C, alpha: float = 1.0, beta: float = 0.0, stream=None):
    """Like sgemm_into(), through the entry point that allocates no device
    memory (its workspace is a fixed array; see include/sgemm.h)."""
    import torch
    _cuda_f32(("A", A), ("B", B), ("C", C))
    M, N, K = _shapes(A, B, C)
    with torch.cuda.device(C.device):
        st = lib.sgemm_noalloc(M, N, K, float(alpha), A.data_ptr(), _ld(A, K), B.data_ptr(),
                               _ld(B, N), float(beta), C.data_ptr(), _ld(C, N),
                               _stream_handle(stream, C.device))
    check(st)
    return C


# floats in the fixed scratch array of sgemm_noalloc (see include/sgemm.h)
NOALLOC_SCRATCH_FLOATS = 8 * 1024 * 1024


def sgemm(A, B, C=None, alpha: float = 1.0, beta: float = 0.0, stream=None):
    """alpha*A@B + beta*C.  With C=None a new tensor is returned (beta must be 0);
    otherwise C is updated in place and returned."""
    import torch
    if C is None:
        if beta != 0.0:
            raise ValueError("beta != 0 needs an input C")
        C = torch.empty((A.shape[0], B.shape[1]), dtype=torch.float32, device=A.device)
    return sgemm_into(A, B, C, alpha, beta, stream)


def sgemm_host(A, B, C, alpha: float = 1.0, beta: float = 0.0, stream=None, device=None,
               tensor_cores: bool = False):
    """The host-buffer entry point: A, B, C are CPU float32 tensors (pinned for
    speed).  C is overwritten with alpha*A@B + beta*C; synchronous.  Copies and
    compute are pipelined over row blocks.  tensor_cores=True uses the 3xTF32
    path (sgemm_host_3xtf32)."""
    import torch
    for name, t in (("A", A), ("B", B), ("C", C)):
        if not isinstance(t, torch.Tensor) or t.dtype != torch.float32 or t.is_cuda:
            raise TypeError(f"{name} must be a CPU float32 tensor")
    M, N, K = _shapes(A, B, C)
    device = torch.device(device) if device is not None else \
        torch.device("cuda", torch.cuda.current_device())
    fn = lib.sgemm_host_3xtf32 if tensor_cores else lib.sgemm_host
    with torch.cuda.device(device):
        st = fn(M, N, K, float(alpha), A.data_ptr(), _ld(A, K), B.data_ptr(), _ld(B, N),
                float(beta), C.data_ptr(), _ld(C, N), _stream_handle(stream, device))
    check(st)
    return C


# ------------------------------------------------------------------ linear layers
# (include/sgemm_layers.h: float32 or bfloat16 tensors, all of one type.  A matrix's rows are
# contiguous, any distance apart, and do not overlap: what was expanded, the gradient of a sum
# over rows for one, needs contiguous() first.)
ACT8_BLOCK = 32   # columns of a row that share an exponent of an 8-bit checkpoint


# A decode step makes one such call per projection, so the checks below are written for
# the calls that pass them: what is wrong is worked out only once something is.
torch = None   # imported by the first call (this module loads without it)


def _import_torch():
    global torch
    import torch as module
    torch = module


def _layer_type(names, *tensors):
    """(sgemm_type, device number) of CUDA tensors (or None, past the first) of one type,
    float32 or bfloat16, on one device."""
    if torch is None:
        _import_torch()
    first = tensors[0]
    try:
        dtype, device = first.dtype, first.get_device()
        for t in tensors:
            if t is not None and (t.dtype is not dtype or t.get_device() != device):
                break
        else:
            if device >= 0:
                if dtype is torch.float32:
                    return 0, device
                if dtype is torch.bfloat16:
                    return 1, device
    except AttributeError:
        pass
    for name, t in zip(names, tensors):
        if t is None and t is not first:
            continue
        if not isinstance(t, torch.Tensor) or not t.is_cuda or \
                t.dtype not in (torch.float32, torch.bfloat16):
            raise TypeError(f"{name} must be a CUDA float32 or bfloat16 tensor")
        if t.dtype != first.dtype:
            raise TypeError(f"{name} must have the type of {names[0]}, {first.dtype}")
    raise ValueError(", ".join(names) + " must be on one device")


def _missing(names, *tensors):
    """TypeError for the first of these that is None."""
    for name, t in zip(names, tensors):
        if t is None:
            raise TypeError(f"{name} must be a CUDA tensor, not None")


def _typed(name, t, dtype, device):
    """TypeError / ValueError unless t is a tensor of this type on CUDA device number `device`."""
    try:
        if t.dtype is dtype and t.get_device() == device:
            return
    except AttributeError:
        pass
    if torch is None:
        _import_torch()
    if not isinstance(t, torch.Tensor) or t.dtype != dtype or not t.is_cuda:
        raise TypeError(f"{name} must be a CUDA {str(dtype).replace('torch.', '')} tensor")
    raise ValueError(f"{name} must be on cuda:{device}")


def _vector(name, t, dtype, n, device):
    """Address of a contiguous vector of n elements, or None."""
    if t is None:
        return None
    try:
        typed = t.dtype is dtype and t.get_device() == device
    except AttributeError:
        typed = False
    if not typed:
        _typed(name, t, dtype, device)
    if t.shape != (n,):
        raise ValueError(f"{name} must be {(n,)}, got {tuple(t.shape)}")
    if n > 1 and t.stride(0) != 1:
        raise ValueError(f"{name} must be contiguous")
    return t.data_ptr()


def _pitch(name, rows, cols, row_stride, col_stride):
    if rows > _INT_MAX or cols > _INT_MAX:
        raise SgemmError(SGEMM_ERR_TOO_LARGE)
    if cols > 1 and col_stride != 1 and rows > 0:
        raise ValueError(f"{name}: rows must be contiguous (stride(-1) == 1)")
    if rows <= 1 or cols == 0:
        return max(cols, 1)
    if row_stride < cols:
        raise ValueError(f"{name}: rows must not overlap (stride(-2) is {row_stride}, below the {cols} "
                         "columns, as in an expanded tensor)")
    if row_stride > _INT_MAX:
        raise ValueError(f"{name}: rows are too far apart (stride(-2) is {row_stride}, past 2^31 - 1)")
    return row_stride


def _matrix(name, t, rows, cols):
    """(address, row pitch) of a rows x cols row-major view; (None, 0) for None."""
    if t is None:
        return None, 0
    if t.shape != (rows, cols):
        raise ValueError(f"{name} must be {(rows, cols)}, got {tuple(t.shape)}")
    row_stride, col_stride = t.stride()
    if col_stride == 1 and 0 < cols <= row_stride <= _INT_MAX and 1 < rows <= _INT_MAX:   # (what _pitch would say)
        return t.data_ptr(), row_stride
    return t.data_ptr(), _pitch(name, rows, cols, row_stride, col_stride)


def _stack(name, t, count, rows, cols):
    """(address, row pitch, matrix stride) of count x rows x cols; (None, 0, 0) for None."""
    if t is None:
        return None, 0, 0
    if t.shape != (count, rows, cols):
        raise ValueError(f"{name} must be {(count, rows, cols)}, got {tuple(t.shape)}")
    if count == 0:
        return None, max(cols, 1), 0
    stride, row_stride, col_stride = t.stride()
    if col_stride == 1 and 0 < cols <= row_stride <= _INT_MAX and 1 < rows <= _INT_MAX:
        return t.data_ptr(), row_stride, stride if count > 1 else 0
    return t.data_ptr(), _pitch(name, rows, cols, row_stride, col_stride), stride if count > 1 else 0


def _checkpoint(q, e, rows, cols, device):
    """(address, pitch, address, pitch) of an 8-bit checkpoint of a rows x cols matrix."""
    _typed("q", q, torch.int8, device)
    _typed("e", e, torch.int8, device)
    return (*_matrix("q", q, rows, cols), *_matrix("e", e, rows, -(-cols // ACT8_BLOCK)))


def _adapters(A, B, ids, M, scale, ranks, device):
    """(L, R, ids, ranks, scale) of a stack A (L, K, R), B (L, R, N): sizes and addresses."""
    if torch is None:
        _import_torch()
    if A.dim() != 3:
        raise ValueError("A must be 3-D (adapters, K, R)")
    L, _, R = A.shape
    if L > 0 and not 1 <= R <= 128:
        raise ValueError(f"the adapters' rank must be 1 to 128, got {R}")
    if L > 1024:
        raise ValueError(f"at most 1024 adapters, got {L}")
    if ids is None and L > 0:
        _missing(("ids",), ids)
    return (L, R, _vector("ids", ids, torch.int32, M, device),
            _vector("ranks", ranks, torch.int32, L, device),
            _vector("scale", scale, torch.float32, L, device))


def _call(device, stream, fn, *args):
    """fn(*args, stream) with CUDA device number `device` current, on `stream` or torch's
    current stream of that device."""
    handle = torch._C._cuda_getCurrentRawStream(device) if stream is None else stream.cuda_stream
    if torch._C._cuda_getDevice() == device:
        status = fn(*args, handle)
        return check(status) if status else status
    with torch.cuda.device(device):
        return check(fn(*args, handle))


def lora_into(X, W, A, B, ids, Y, scale=None, ranks=None, bias=None, H=None, stream=None):
    """Y[i] <- X[i]@W + bias + scale[a]*(X[i]@A[a])@B[a] with a = ids[i]: the adapters
    of many requests beside one projection, for one token up to a long prefill.

    X (M, K), W (K, N), A (L, K, R), B (L, R, N), Y (M, N) and bias (N,) or None: CUDA
    float32 or bfloat16, one type.  ids (M,) int32; a row whose id is not in [0, L)
    uses no adapter.  scale (L,) float32 or None (1).  ranks (L,) int32 or None: only
    the first ranks[a] columns of A[a] and rows of B[a] are used.  H (M, R) float32,
    where given, receives X[i]@A[a] for lora_backward_into().  Asynchronous on `stream`
    (default: torch's current stream)."""
    kind, device = _layer_type(("X", "W", "A", "B", "Y", "bias"), X, W, A, B, Y, bias)
    if W is None or A is None or B is None or Y is None:
        _missing(("W", "A", "B", "Y"), W, A, B, Y)
    if X.dim() != 2 or W.dim() != 2:
        raise ValueError("X and W must be 2-D")
    (M, K), N = X.shape, W.shape[1]
    L, R, ids_p, ranks_p, scale_p = _adapters(A, B, ids, M, scale, ranks, device)
    if H is not None:
        _typed("H", H, torch.float32, device)
    _call(device, stream, lib.sgemm_lora, kind, M, N, K, L, R, *_matrix("X", X, M, K),
          *_matrix("W", W, K, N), *_stack("A", A, L, K, R), *_stack("B", B, L, R, N), ids_p, ranks_p,
          scale_p, _vector("bias", bias, Y.dtype, N, device), *_matrix("H", H, M, R),
          *_matrix("Y", Y, M, N))
    return Y


def lora_backward_into(dY, X, W, A, B, ids, H, dX=None, dA=None, dB=None, scale=None, ranks=None,
                       stream=None):
    """Gradients of lora_into() for dY (M, N), W being frozen: with
    G[i] = scale[a]*dY[i]@B[a].T, dX <- dY@W.T + G[i]@A[a].T, dA[a] <- sum_i X[i].T@G[i]
    and dB[a] <- sum_i scale[a]*H[i].T@dY[i] (zero for adapters without rows).

    X is the forward call's input or the pair (q, e) that act8_store_into() kept of it;
    H what the forward call wrote.  dX (M, K) may be None, and dA (L, K, R) and
    dB (L, R, N) may be None together; X and H may then be None too.  Returns (dX, dA, dB)."""
    kept = isinstance(X, tuple)
    kind, device = _layer_type(("dY", "X", "W", "A", "B", "dX", "dA", "dB"), dY, None if kept else X,
                               W, A, B, dX, dA, dB)
    if W is None or A is None or B is None:
        _missing(("W", "A", "B"), W, A, B)
    if (dA is None) != (dB is None):
        raise ValueError("dA and dB must be given together")
    if dA is not None and (X is None or H is None):   # (dX needs neither)
        _missing(("X", "H"), X, H)
    if dY.dim() != 2 or W.dim() != 2:
        raise ValueError("dY and W must be 2-D")
    M, (K, N) = dY.shape[0], W.shape
    L, R, ids_p, ranks_p, scale_p = _adapters(A, B, ids, M, scale, ranks, device)
    if H is not None:
        _typed("H", H, torch.float32, device)
    x = (None, 0, *_checkpoint(*X, M, K, device)) if kept else (*_matrix("X", X, M, K), None, 0, None, 0)
    _call(device, stream, lib.sgemm_lora_backward, kind, M, N, K, L, R, *_matrix("dY", dY, M, N), *x,
          *_matrix("W", W, K, N), *_stack("A", A, L, K, R), *_stack("B", B, L, R, N), ids_p, ranks_p,
          scale_p, *_matrix("H", H, M, R), *_matrix("dX", dX, M, K), *_stack("dA", dA, L, K, R),
          *_stack("dB", dB, L, R, N))
    return dX, dA, dB


def act8_empty(M: int, K: int, device=None):
    """A checkpoint's two tensors for an M x K matrix: q (M, K) and e (M, ceil(K/32)), int8."""
    if torch is None:
        _import_torch()
    if device is None:
        device = torch.device("cuda", torch.cuda.current_device())
    return (torch.empty((M, K), dtype=torch.int8, device=device),
            torch.empty((M, -(-K // ACT8_BLOCK)), dtype=torch.int8, device=device))


def _act_number(act):
    if act not in ACTIVATIONS:
        raise ValueError(f"act must be one of {sorted(ACTIVATIONS)}, got {act!r}")
    return ACTIVATIONS[act]


def _sizes(name, t):
    if t.dim() != 2:
        raise ValueError(f"{name} must be 2-D")
    return t.shape


def act8_store_into(Z, q, e, act: str = "none", Y=None, stream=None):
    """(q, e) <- the 8-bit checkpoint of Z (M, K): for each block of 32 columns of a row
    an exponent e and q = rint(z / 2^e) in int8.  With Y, also Y <- act(Z) in the same
    pass (Y may be Z).  Returns (q, e)."""
    kind, device = _layer_type(("Z", "Y"), Z, Y)
    number = _act_number(act)
    if number and Y is None:
        raise ValueError("an activation needs an output Y")
    M, K = _sizes("Z", Z)
    _call(device, stream, lib.sgemm_act8_store, kind, M, K, *_matrix("Z", Z, M, K), number,
          *_checkpoint(q, e, M, K, device), *_matrix("Y", Y, M, K))
    return q, e


def act8_load_into(q, e, X, stream=None):
    """X <- the values q * 2^e that a checkpoint stands for."""
    kind, device = _layer_type(("X",), X)
    M, K = _sizes("X", X)
    _call(device, stream, lib.sgemm_act8_load, kind, M, K, *_checkpoint(q, e, M, K, device),
          *_matrix("X", X, M, K))
    return X


def act8_grad_into(q, e, dY, dZ, act: str = "none", stream=None):
    """dZ <- dY * act'(z), z the values of the checkpoint (q, e) of the activation's
    input (dZ may be dY)."""
    kind, device = _layer_type(("dY", "dZ"), dY, dZ)
    if dZ is None:
        _missing(("dZ",), dZ)
    number = _act_number(act)
    M, K = _sizes("dY", dY)
    _call(device, stream, lib.sgemm_act8_grad, kind, M, K, *_checkpoint(q, e, M, K, device), number,
          *_matrix("dY", dY, M, K), *_matrix("dZ", dZ, M, K))
    return dZ


def act8_weight_grad_into(q, e, dY, dW, beta: float = 0.0, stream=None):
    """dW <- x.T@dY + beta*dW, x (M, K) the values of the checkpoint (q, e) of a layer's
    input, dY (M, N), dW (K, N)."""
    kind, device = _layer_type(("dY", "dW"), dY, dW)
    if dW is None:
        _missing(("dW",), dW)
    (M, N), K = _sizes("dY", dY), _sizes("dW", dW)[0]
    _call(device, stream, lib.sgemm_act8_weight_grad, kind, M, N, K,
          *_checkpoint(q, e, M, K, device), *_matrix("dY", dY, M, N), float(beta),
          *_matrix("dW", dW, K, N))
    return dW


# ------------------------------------------------------------------ control
def device_status(stream=None, device=None) -> int:
    """Synchronise and read/clear the device error word: 0 or SGEMM_ERR_TIMEOUT."""
    import torch
    if device is None:
        device = torch.device("cuda", torch.cuda.current_device())
    with torch.cuda.device(device):
        return lib.sgemm_device_status(_stream_handle(stream, device))


def set_wait_timeout_ns(ns: int) -> None:
    check(lib.sgemm_set_wait_timeout_ns(int(ns)))


def selftest_wait_timeout(ns: int, stream=None, device=None) -> int:
    import torch
    if device is None:
        device = torch.device("cuda", torch.cuda.current_device())
    with torch.cuda.device(device):
        return lib.sgemm_selftest_wait_timeout(int(ns), _stream_handle(stream, device))


def profile_enable(on: bool = True) -> None:
    check(lib.sgemm_profile_enable(1 if on else 0))


def profile_collect() -> dict:
    mm, pm = ctypes.c_double(0), ctypes.c_double(0)
    mn, pn = ctypes.c_longlong(0), ctypes.c_longlong(0)
    check(lib.sgemm_profile_collect(ctypes.byref(mm), ctypes.byref(mn), ctypes.byref(pm),
                                    ctypes.byref(pn)))
    return {"main_ms": mm.value, "main_launches": mn.value,
            "pack_ms": pm.value, "pack_launches": pn.value}


def kernel_launch_count() -> int:
    return lib.sgemm_kernel_launch_count()


def config_string(M: int, N: int, K: int) -> str:
    return lib.sgemm_config_string(M, N, K).decode()


def last_kernel() -> str:
    """Configuration of the last main kernel this thread's calls launched."""
    return lib.sgemm_last_kernel().decode()


def variants() -> list:
    """Descriptions of the compiled kernel variants, by index."""
    return [lib.sgemm_variant_name(i).decode() for i in range(lib.sgemm_variant_count())]


def set_variant(variant_id: int) -> None:
    """Force a kernel variant for later calls (-1: automatic choice)."""
    check(lib.sgemm_set_variant(int(variant_id)))


def set_3xtf32_kernel(pair) -> None:
    """3xTF32 main kernel for later calls: the CTA pair (True), the single-CTA
    kernel (False) or the automatic choice per shape (None, the default)."""
    check(lib.sgemm_set_3xtf32_kernel(-1 if pair is None else (1 if pair else 0)))


def debug_drop_release(on: bool) -> None:
    """Failure-detection test switch: while on, plain sgemm() calls run the
    test build of the default kernel in which one release is left out, so a
    bounded wait expires and the kernel's abort path runs (include/sgemm.h)."""
    check(lib.sgemm_debug_drop_release(1 if on else 0))
