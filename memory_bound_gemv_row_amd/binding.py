"""ctypes binding over the C ABI in ``include/gemv.h``,
``include/gemv_quant.h``, ``include/gemv_softmax.h``,
``include/gemv_tokens.h`` and ``include/gemv_attention.h``.

Argument marshalling only: every step of the product runs in the HIP
library.  PyTorch supplies device memory and the current stream; no torch
operator is on the path.  If the library is missing the first call raises:
there is no fallback.
"""
from __future__ import annotations

import ctypes
import os
import threading

PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(PKG, "libgemv_amd.so")

KIND = {"f32": 0, "f16": 1, "q8": 2, "q4": 3, "f16x32": 4, "f16_acc16": 5}
DTYPE = {"float32": 0, "float16": 1, "bfloat16": 2}   # gemv_dtype
STATUS = {0: "GEMV_OK", 1: "GEMV_E_INVAL", 2: "GEMV_E_UNSUPPORTED", 3: "GEMV_E_LAUNCH", 4: "GEMV_E_DEVICE"}

_lock = threading.Lock()
_lib = None


class GemvError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        super().__init__(f"{where}: {STATUS.get(status, status)} ({status_string(status)})")


class LaunchInfo(ctypes.Structure):
    _fields_ = [("variant", ctypes.c_int), ("grid", ctypes.c_int), ("block", ctypes.c_int),
                ("rows_per_wave", ctypes.c_int), ("units_in_flight", ctypes.c_int), ("lds_bytes", ctypes.c_int),
                ("stage_order", ctypes.c_int)]


class Plan(ctypes.Structure):
    """gemv_plan: an explicit launch plan (variant, waves, units_in_flight,
    rows_per_wave, stage_order, cap)."""
    _fields_ = [("variant", ctypes.c_int), ("waves", ctypes.c_int), ("units_in_flight", ctypes.c_int),
                ("rows_per_wave", ctypes.c_int), ("stage_order", ctypes.c_int), ("cap", ctypes.c_int)]


class KvCache(ctypes.Structure):
    """gemv_kv_cache: the pages of a key-value cache and how they lie."""
    _fields_ = [("k", ctypes.c_void_p), ("v", ctypes.c_void_p), ("dtype", ctypes.c_int), ("pages", ctypes.c_int),
                ("page_size", ctypes.c_int), ("heads", ctypes.c_int), ("head_dim", ctypes.c_int),
                ("stride_page", ctypes.c_int64), ("stride_slot", ctypes.c_int64), ("stride_head", ctypes.c_int64)]


class KvBatch(ctypes.Structure):
    """gemv_kv_batch: the sequences of a call."""
    _fields_ = [("table", ctypes.c_void_p), ("table_stride", ctypes.c_int64), ("width", ctypes.c_int),
                ("lens", ctypes.c_void_p), ("batch", ctypes.c_int), ("max_len", ctypes.c_int)]


def load():
    """Load the in-tree library (raises if it has not been built)."""
    global _lib
    if _lib is not None:
        return _lib
    with _lock:
        if _lib is not None:
            return _lib
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"HIP library not built: {LIB_PATH} is missing "
                               "(run python -m memory_bound_gemv_row_amd.build)")
        lib = ctypes.CDLL(LIB_PATH)
        p, i = ctypes.c_void_p, ctypes.c_int
        for name in ("gemv_f32", "gemv_f16", "gemv_f16x32", "gemv_f16_acc16"):
            getattr(lib, name).argtypes = [p, p, p, i, i, p]
            getattr(lib, name).restype = i
        for name in ("gemv_q8", "gemv_q4"):
            getattr(lib, name).argtypes = [p, p, p, p, i, i, p]
            getattr(lib, name).restype = i
        for name in ("gemv_quantize_q8", "gemv_quantize_q4"):
            getattr(lib, name).argtypes = [p, p, p, p, i, i, p]
            getattr(lib, name).restype = i
        lib.gemv_softmax_f16.argtypes = [p, p, i, i, p]
        lib.gemv_softmax_f16.restype = i
        lib.gemv_status_string.argtypes = [i]
        lib.gemv_status_string.restype = ctypes.c_char_p
        lib.gemv_probe_read.argtypes = [p, ctypes.c_size_t, p, ctypes.c_uint32, p]
        lib.gemv_probe_read.restype = i
        lib.gemv_probe_copy.argtypes = [p, p, ctypes.c_size_t, p]
        lib.gemv_probe_copy.restype = i
        lib.gemv_describe_launch.argtypes = [i, i, i, i, ctypes.POINTER(LaunchInfo)]
        lib.gemv_describe_launch.restype = i
        lib.gemv_describe_launch_for.argtypes = [i, i, i, i, i, i, ctypes.POINTER(LaunchInfo)]
        lib.gemv_describe_launch_for.restype = i
        lib.gemv_check_plan_for.argtypes = [i, i, i, i, i, ctypes.POINTER(Plan), ctypes.POINTER(LaunchInfo)]
        lib.gemv_check_plan_for.restype = i
        lib.gemv_launch_plan.argtypes = [i, p, p, p, p, i, i, ctypes.POINTER(Plan), p]
        lib.gemv_launch_plan.restype = i
        i64, z = ctypes.c_int64, ctypes.c_size_t
        lib.gemv_quantize_tokens_q8.argtypes = [p, i, i64, p, p, i, i, p]
        lib.gemv_quantize_tokens_q8.restype = i
        lib.gemv_gemm_q8.argtypes = [p, p, p, p, p, i, i, i, i, p]
        lib.gemv_gemm_q8.restype = i
        cache, batch = ctypes.POINTER(KvCache), ctypes.POINTER(KvBatch)
        lib.gemv_attention_workspace.argtypes = [cache, batch, i, i]
        lib.gemv_attention_workspace.restype = z
        lib.gemv_attention.argtypes = [cache, batch, p, i64, i, ctypes.c_float, p, p, i64, p, z, p]
        lib.gemv_attention.restype = i
        lib.gemv_kv_append.argtypes = [cache, batch, p, p, i64, p, i64, i, p, p, p, i64, p]
        lib.gemv_kv_append.restype = i
        lib.gemv_kv_evict_workspace.argtypes = [cache, batch, i]
        lib.gemv_kv_evict_workspace.restype = z
        lib.gemv_kv_evict.argtypes = [cache, batch, p, p, p, i64, i, i, p, p, p, p, z, p]
        lib.gemv_kv_evict.restype = i
        _lib = lib
        return lib


def status_string(status: int) -> str:
    return load().gemv_status_string(int(status)).decode()


def _check(rc: int, where: str):
    if rc != 0:
        raise GemvError(rc, where)


# ---------------------------------------------------------------- raw pointers
# Device pointers as integers, stream as an integer handle (0 = null stream).
def gemv_f32_ptr(A: int, x: int, y: int, M: int, N: int, stream: int = 0) -> int:
    return load().gemv_f32(A, x, y, M, N, stream)


def gemv_f16_ptr(A: int, x: int, y: int, M: int, N: int, stream: int = 0) -> int:
    return load().gemv_f16(A, x, y, M, N, stream)


def gemv_f16x32_ptr(A: int, x: int, y: int, M: int, N: int, stream: int = 0) -> int:
    return load().gemv_f16x32(A, x, y, M, N, stream)


def gemv_f16_acc16_ptr(A: int, x: int, y: int, M: int, N: int, stream: int = 0) -> int:
    return load().gemv_f16_acc16(A, x, y, M, N, stream)


def gemv_q8_ptr(A: int, scale: int, x: int, y: int, M: int, N: int, stream: int = 0) -> int:
    return load().gemv_q8(A, scale, x, y, M, N, stream)


def gemv_q4_ptr(A: int, scale: int, x: int, y: int, M: int, N: int, stream: int = 0) -> int:
    return load().gemv_q4(A, scale, x, y, M, N, stream)


def quantize_q8_ptr(W: int, q: int, scale: int, row_sse: int, M: int, N: int, stream: int = 0) -> int:
    return load().gemv_quantize_q8(W, q, scale, row_sse, M, N, stream)


def quantize_q4_ptr(W: int, q: int, scale: int, row_sse: int, M: int, N: int, stream: int = 0) -> int:
    return load().gemv_quantize_q4(W, q, scale, row_sse, M, N, stream)


def softmax_f16_ptr(x: int, y: int, M: int, N: int, stream: int = 0) -> int:
    return load().gemv_softmax_f16(x, y, M, N, stream)


def probe_read_ptr(buf: int, nbytes: int, sink: int, guard: int = 0xA5A5A5A5, stream: int = 0) -> int:
    return load().gemv_probe_read(buf, nbytes, sink, guard, stream)


def probe_copy_ptr(src: int, dst: int, nbytes: int, stream: int = 0) -> int:
    return load().gemv_probe_copy(src, dst, nbytes, stream)


def describe_launch(kind: str, M: int, N: int, aligned: bool = True) -> dict:
    info = LaunchInfo()
    _check(load().gemv_describe_launch(KIND[kind], M, N, int(aligned), ctypes.byref(info)), "gemv_describe_launch")
    return {f: getattr(info, f) for f, _ in LaunchInfo._fields_}


def describe_launch_for(kind: str, M: int, N: int, cus: int, lds_max: int, aligned: bool = True) -> dict:
    """describe_launch for a device of `cus` CUs and `lds_max` bytes of LDS
    per workgroup; touches no device."""
    info = LaunchInfo()
    _check(load().gemv_describe_launch_for(KIND[kind], M, N, int(aligned), cus, lds_max, ctypes.byref(info)),
           "gemv_describe_launch_for")
    return {f: getattr(info, f) for f, _ in LaunchInfo._fields_}


# ---------------------------------------------------------------- torch tensors
def _stream(stream):
    import torch

    s = torch.cuda.current_stream() if stream is None else stream
    return s.cuda_stream


def _need(t, name, dtypes, shape):
    import torch

    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a device tensor")
    if t.device.index != torch.cuda.current_device():
        # the C ABI launches on the current device's stream
        raise ValueError(f"{name} is on {t.device}, the current device is cuda:{torch.cuda.current_device()}")
    if t.dtype not in dtypes:
        raise TypeError(f"{name}: dtype {t.dtype} not in {dtypes}")
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name}: shape {tuple(t.shape)} != {tuple(shape)}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return t.data_ptr()


_INT_MAX = (1 << 31) - 1


def _dims(*dims):
    # the C ABI takes M and N as int: larger values would wrap in ctypes
    for d in dims:
        if not 0 <= d <= _INT_MAX:
            raise ValueError(f"dimension {d} outside the C ABI's int range [0, 2^31 - 1]")


def _out(out, M, device):
    import torch

    if out is None:
        return torch.empty(M, dtype=torch.float32, device=device)
    _need(out, "out", (torch.float32,), (M,))
    return out


def gemv_f32(A, x, out=None, stream=None):
    import torch

    M, N = A.shape
    _dims(M, N)
    a = _need(A, "A", (torch.float32,), (M, N))
    xp = _need(x, "x", (torch.float32,), (N,))
    y = _out(out, M, A.device)
    _check(gemv_f32_ptr(a, xp, y.data_ptr(), M, N, _stream(stream)), "gemv_f32")
    return y


def gemv_f16(A, x, out=None, stream=None):
    import torch

    h = (torch.float16, torch.int16, torch.uint16)
    M, N = A.shape
    _dims(M, N)
    a = _need(A, "A", h, (M, N))
    xp = _need(x, "x", h, (N,))
    y = _out(out, M, A.device)
    _check(gemv_f16_ptr(a, xp, y.data_ptr(), M, N, _stream(stream)), "gemv_f16")
    return y


def gemv_f16x32(A, x, out=None, stream=None):
    """A: binary16 [M, N], x: float32 [N]."""
    import torch

    h = (torch.float16, torch.int16, torch.uint16)
    M, N = A.shape
    _dims(M, N)
    a = _need(A, "A", h, (M, N))
    xp = _need(x, "x", (torch.float32,), (N,))
    y = _out(out, M, A.device)
    _check(gemv_f16x32_ptr(a, xp, y.data_ptr(), M, N, _stream(stream)), "gemv_f16x32")
    return y


def gemv_f16_acc16(A, x, out=None, stream=None):
    """LOSSY: binary16 running sums (see gemv_f16_acc16 in include/gemv.h).
    A: binary16 [M, N], x: binary16 [N]."""
    import torch

    h = (torch.float16, torch.int16, torch.uint16)
    M, N = A.shape
    _dims(M, N)
    a = _need(A, "A", h, (M, N))
    xp = _need(x, "x", h, (N,))
    y = _out(out, M, A.device)
    _check(gemv_f16_acc16_ptr(a, xp, y.data_ptr(), M, N, _stream(stream)), "gemv_f16_acc16")
    return y


def gemv_q8(A, scale, x, out=None, stream=None):
    import torch

    h = (torch.float16, torch.int16, torch.uint16)
    M, N = A.shape
    _dims(M, N)
    a = _need(A, "A", (torch.int8,), (M, N))
    s = _need(scale, "scale", h, (M,))
    xp = _need(x, "x", h, (N,))
    y = _out(out, M, A.device)
    _check(gemv_q8_ptr(a, s, xp, y.data_ptr(), M, N, _stream(stream)), "gemv_q8")
    return y


def gemv_q4(A, scale, x, out=None, stream=None):
    """A: uint8 [M, N/2] (two INT4 per byte, low nibble = even column),
    scale: binary16 [M, N/128], x: binary16 [N]."""
    import torch

    h = (torch.float16, torch.int16, torch.uint16)
    M, half = A.shape
    N = 2 * half
    _dims(M, N)
    a = _need(A, "A", (torch.uint8,), (M, half))
    if N % 128:
        raise ValueError("INT4 needs N % 128 == 0")
    s = _need(scale, "scale", h, (M, N // 128))
    xp = _need(x, "x", h, (N,))
    y = _out(out, M, A.device)
    _check(gemv_q4_ptr(a, s, xp, y.data_ptr(), M, N, _stream(stream)), "gemv_q4")
    return y


def quantize_q8(W, with_error=True, stream=None):
    """FP32 W [M, N] -> (q int8 [M, N], scale float16 [M], row_sse float32 [M]
    or None).  RMSE = sqrt(row_sse.sum() / (M * N))."""
    import torch

    M, N = W.shape
    _dims(M, N)
    w = _need(W, "W", (torch.float32,), (M, N))
    q = torch.empty((M, N), dtype=torch.int8, device=W.device)
    s = torch.empty(M, dtype=torch.float16, device=W.device)
    e = torch.empty(M, dtype=torch.float32, device=W.device) if with_error else None
    _check(quantize_q8_ptr(w, q.data_ptr(), s.data_ptr(), e.data_ptr() if e is not None else 0, M, N,
                           _stream(stream)), "gemv_quantize_q8")
    return q, s, e


def quantize_q4(W, with_error=True, stream=None):
    """FP32 W [M, N], N % 128 == 0 -> (q uint8 [M, N/2] two INT4 per byte,
    low nibble = even column; scale float16 [M, N/128]; row_sse float32 [M]
    or None)."""
    import torch

    M, N = W.shape
    _dims(M, N)
    if N % 128:
        raise ValueError("INT4 quantisation needs N % 128 == 0")
    w = _need(W, "W", (torch.float32,), (M, N))
    q = torch.empty((M, N // 2), dtype=torch.uint8, device=W.device)
    s = torch.empty((M, N // 128), dtype=torch.float16, device=W.device)
    e = torch.empty(M, dtype=torch.float32, device=W.device) if with_error else None
    _check(quantize_q4_ptr(w, q.data_ptr(), s.data_ptr(), e.data_ptr() if e is not None else 0, M, N,
                           _stream(stream)), "gemv_quantize_q4")
    return q, s, e


def softmax_f16(x, out=None, stream=None):
    """Row-wise softmax of binary16 x [M, N] -> binary16 [M, N]."""
    import torch

    h = (torch.float16, torch.int16, torch.uint16)
    M, N = x.shape
    _dims(M, N)
    xp = _need(x, "x", h, (M, N))
    if out is None:
        out = torch.empty((M, N), dtype=torch.float16, device=x.device)
    else:
        _need(out, "out", h, (M, N))
    _check(softmax_f16_ptr(xp, out.data_ptr(), M, N, _stream(stream)), "gemv_softmax_f16")
    return out


def probe_read(buf, sink, guard: int = 0xA5A5A5A5, stream=None):
    _check(probe_read_ptr(buf.data_ptr(), buf.numel() * buf.element_size(), sink.data_ptr(), guard,
                          _stream(stream)), "gemv_probe_read")


def probe_copy(src, dst, stream=None):
    n = src.numel() * src.element_size()
    if dst.numel() * dst.element_size() < n:
        raise ValueError("dst smaller than src")
    _check(probe_copy_ptr(src.data_ptr(), dst.data_ptr(), n, _stream(stream)), "gemv_probe_copy")


def check_plan_for(kind: str, M: int, N: int, cus: int, lds_max: int, plan: tuple) -> dict | None:
    """The launch an explicit plan (variant, waves, units_in_flight,
    rows_per_wave, stage_order, cap) makes on a device of `cus` CUs and
    `lds_max` bytes of LDS per workgroup, or None where the library holds no
    kernel for it or it does not fit the shape; touches no device."""
    _dims(M, N)
    info = LaunchInfo()
    rc = load().gemv_check_plan_for(KIND[kind], M, N, cus, lds_max, ctypes.byref(Plan(*plan)), ctypes.byref(info))
    if rc == 2:
        return None
    _check(rc, "gemv_check_plan_for")
    return {f: getattr(info, f) for f, _ in LaunchInfo._fields_}


def launch_plan_ptr(kind: str, A: int, scale: int, x: int, y: int, M: int, N: int, plan: tuple,
                    stream: int = 0) -> int:
    """gemv_launch_plan on raw device pointers (scale 0 for FP formats)."""
    _dims(M, N)
    return load().gemv_launch_plan(KIND[kind], A, scale or None, x, y, M, N, ctypes.byref(Plan(*plan)), stream)


# ---------------------------------------------------------------- several tokens, and the key-value cache
# These take strided rows where the C ABI does, and make their outputs and
# workspaces on the stream that the work runs on.  A decode step makes many
# such calls, each shorter on the GPU than on the host, so the checks of a
# right call are few steps: what fails them goes to _need for its reason.
def _here():
    import torch

    get = getattr(torch._C, "_cuda_getDevice", None)   # current_device() without its check for a first use
    return get() if get is not None else torch.cuda.current_device()


def _work_stream(stream, device):
    """(handle, maker of empty tensors) of `stream`, or of the current stream."""
    import torch

    if stream is None:
        raw = getattr(torch._C, "_cuda_getCurrentRawStream", None)   # current_stream() without its wrapper object
        return raw(device) if raw is not None else torch.cuda.current_stream().cuda_stream, torch.empty
    if stream.device.index != device:
        raise ValueError(f"stream is on {stream.device}, the current device is cuda:{device}")

    def empty(*args, **kw):
        # the allocator hands memory out by stream: what is freed when this
        # call returns must not go to another stream while the work runs
        with torch.cuda.stream(stream):
            return torch.empty(*args, **kw)

    return stream.cuda_stream, empty


def _ptr(t, name, dtype, shape, device):
    """Data pointer of a dense tensor of `dtype` and `shape` on `device`, the current one."""
    try:
        if t.dtype is dtype and t.shape == shape and t.get_device() == device and t.is_contiguous():
            return t.data_ptr()
    except AttributeError:
        pass
    return _need(t, name, (dtype,), shape)


def _rows(t, name, dtype, shape, device, dense):
    """Data pointer and row stride of a tensor whose rows, of `dense` elements
    each, may lie apart."""
    import torch

    try:
        if t.dtype is dtype and t.shape == shape and t.get_device() == device and t.is_contiguous():
            return t.data_ptr(), dense
    except AttributeError:
        pass
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.is_contiguous():
        return _need(t, name, (dtype,), shape), dense
    if t.dim() < 2 or t.stride(0) < dense or not t[0].is_contiguous():
        raise ValueError(f"{name}: the rows must be contiguous and not overlap")
    _need(t[0], name, (dtype,), tuple(shape)[1:])
    if t.shape != tuple(shape):
        raise ValueError(f"{name}: shape {tuple(t.shape)} != {tuple(shape)}")
    return t.data_ptr(), t.stride(0)


def _apart(outs, ins):
    """Refuses outputs that share memory with each other or with inputs, each
    given as (address, bytes)."""
    for i, (p, n) in enumerate(outs):
        for q, m in outs[i + 1:] + ins:
            if n and m and p < q + m and q < p + n:
                raise ValueError("the outputs must not overlap the inputs or each other")


_codes = {}


def _code(dtype):
    code = _codes.get(dtype)
    if code is None:
        code = DTYPE.get(str(dtype)[6:])   # "torch.float16"
        if code is None:
            raise TypeError(f"dtype {dtype} is none of {sorted(DTYPE)}")
        _codes[dtype] = code
    return code


def quantize_tokens_q8_ptr(x: int, dtype: int, stride: int, q: int, scale: int, T: int, N: int, stream: int = 0) -> int:
    return load().gemv_quantize_tokens_q8(x, dtype, stride, q, scale, T, N, stream)


def gemm_q8_ptr(A: int, scale: int, x: int, x_scale: int, y: int, dtype: int, T: int, M: int, N: int,
                stream: int = 0) -> int:
    return load().gemv_gemm_q8(A, scale, x, x_scale, y, dtype, T, M, N, stream)


def quantize_tokens_q8(x, stream=None):
    """Activations x [T, N] (float32, float16 or bfloat16; rows may lie apart)
    -> (q int8 [T, N], scale float32 [T]), one scale per token."""
    import torch

    T, N = x.shape
    _dims(T, N)
    here = _here()
    code = _code(x.dtype)
    xp, stride = _rows(x, "x", x.dtype, (T, N), here, N)
    handle, empty = _work_stream(stream, here)
    q = empty((T, N), dtype=torch.int8, device=x.device)
    s = empty(T, dtype=torch.float32, device=x.device)
    _check(quantize_tokens_q8_ptr(xp, code, stride, q.data_ptr(), s.data_ptr(), T, N, handle), "gemv_quantize_tokens_q8")
    return q, s


def gemm_q8(A, scale, x, x_scale, out=None, out_dtype=None, stream=None):
    """The INT8 product of several tokens: A int8 [M, N] with scale float16 [M]
    (the weights of gemv_q8), x int8 [T, N] with x_scale float32 [T] ->
    y [T, M] of `out_dtype` (float16 unless given, or `out`'s)."""
    import torch

    M, N = A.shape
    T = x.shape[0]
    _dims(T, M, N)
    here = _here()
    a = _ptr(A, "A", torch.int8, (M, N), here)
    s = _ptr(scale, "scale", torch.float16, (M,), here) if getattr(scale, "dtype", None) is torch.float16 else \
        _need(scale, "scale", (torch.float16, torch.int16, torch.uint16), (M,))
    xp = _ptr(x, "x", torch.int8, (T, N), here)
    xs = _ptr(x_scale, "x_scale", torch.float32, (T,), here)
    handle, empty = _work_stream(stream, here)
    if out is None:
        out_dtype = out_dtype or torch.float16
        code = _code(out_dtype)
        out = empty((T, M), dtype=out_dtype, device=A.device)
        y = out.data_ptr()
    else:
        if out_dtype is not None and out.dtype != out_dtype:
            raise TypeError(f"out is {out.dtype}, out_dtype {out_dtype}")
        code = _code(out.dtype)
        y = _ptr(out, "out", out.dtype, (T, M), here)
    _check(gemm_q8_ptr(a, s, xp, xs, y, code, T, M, N, handle), "gemv_gemm_q8")
    return out


class PagedCache:
    """A paged key-value cache: k and v [pages, page_size, heads, head_dim],
    float16 or bfloat16, the last dimension dense and the others in any order
    in memory, the same for both (so a cache kept as [pages, heads, page_size,
    head_dim] is given as ``t.transpose(1, 2)``).  Keeps the tensors; their
    contents belong to the caller."""

    def __init__(self, k, v):
        import torch

        for t, name in ((k, "k"), (v, "v")):
            if not isinstance(t, torch.Tensor):
                raise TypeError(f"{name} must be a torch.Tensor")
            if not t.is_cuda:
                raise ValueError(f"{name} must be a device tensor")
            if t.dtype not in (torch.float16, torch.bfloat16):
                raise TypeError(f"{name}: dtype {t.dtype} is neither float16 nor bfloat16")
            if t.dim() != 4:
                raise ValueError(f"{name} must be [pages, page_size, heads, head_dim]")
        if k.shape != v.shape or k.dtype != v.dtype or k.device != v.device:
            raise ValueError("k and v must have the same shape, type and device")
        pages, page_size, heads, dim = k.shape
        _dims(pages, page_size, heads, dim)
        if page_size < 1 or heads < 1:
            raise ValueError("a page holds at least one slot of at least one head")
        if dim < 8 or dim > 256 or dim % 8:
            raise ValueError(f"head_dim {dim} is no multiple of 8 from 8 to 256")
        # a dimension of size 1 is never stepped over: its stride is free
        strides = [tuple(dim if t.shape[d] == 1 else t.stride(d) for d in range(3)) for t in (k, v)]
        if strides[0] != strides[1]:
            raise ValueError("k and v must have the same strides")
        if k.stride(3) != 1 or v.stride(3) != 1 or min(strides[0]) < dim:
            raise ValueError("the last dimension must be dense and rows must not overlap")
        if any(s % 8 for s in strides[0]) or k.data_ptr() % 16 or v.data_ptr() % 16:
            raise ValueError("k, v and their rows must be 16-byte aligned")
        self.k, self.v = k, v
        self.pages, self.page_size, self.heads, self.head_dim = pages, page_size, heads, dim
        self.dtype, self.device, self.index = k.dtype, k.device, k.get_device()
        self.c = KvCache(k.data_ptr(), v.data_ptr(), _code(k.dtype), pages, page_size, heads, dim, *strides[0])
        self._by_ref = ctypes.byref(self.c)
        self._needs = {}   # bytes of workspace by the shape of a call

    def _batch(self, table, lens, max_len, here):
        """gemv_kv_batch of a call, and the slots that its sequences may use."""
        import torch

        if self.index != here:
            raise ValueError(f"the cache is on {self.device}, the current device is cuda:{here}")
        B, width = table.shape
        tp, stride = _rows(table, "table", torch.int32, (B, width), here, width)
        lp = _ptr(lens, "lens", torch.int32, (B,), here)
        room = min(width * self.page_size, _INT_MAX)
        if max_len is None:
            max_len = room
        if not 0 <= max_len <= _INT_MAX:
            raise ValueError(f"max_len {max_len} outside [0, 2^31 - 1]")
        return KvBatch(tp, stride, width, lp, B, max_len), min(room, max_len)

    def _need(self, key, ask):
        need = self._needs.get(key)
        if need is None:
            if len(self._needs) > 4096:
                self._needs.clear()
            need = self._needs[key] = ask()
        return need


def _tracked(t, name, dtype, batch, heads, room, here):
    if t.dim() != 3 or t.shape[2] < room:
        raise ValueError(f"{name} must be [batch, heads, slots] with at least {room} slots")
    return _ptr(t, name, dtype, (batch, heads, t.shape[2]), here)


def paged_attention(cache, table, lens, q, scale=None, max_len=None, weights=None, out=None, stream=None):
    """Attention of one new token per sequence over a paged cache: q
    [batch, q_heads, head_dim] of the cache's type (sequences may lie apart)
    -> [batch, q_heads, head_dim].  table int32 [batch, pages per sequence],
    lens int32 [batch]; scale 1 / sqrt(head_dim) unless given; max_len the
    longest length, where the host knows one below the table's room.
    weights float32 [batch, heads, slots]: each token's attention weights,
    summed over the query heads of its head, are added to it.  out may be a
    dense q itself."""
    import torch

    here = _here()
    batch, room = cache._batch(table, lens, max_len, here)
    B, heads, dim = q.shape
    if B != batch.batch or dim != cache.head_dim or heads < 1 or heads % cache.heads:
        raise ValueError(f"q: shape {tuple(q.shape)} does not fit {batch.batch} sequences, {cache.heads} heads of "
                         f"{cache.head_dim}")
    qp, q_stride = _rows(q, "q", cache.dtype, (B, heads, dim), here, heads * dim)
    handle, empty = _work_stream(stream, here)
    if out is None:
        out = empty((B, heads, dim), dtype=cache.dtype, device=cache.device)
        op = out.data_ptr()
    else:
        op = _ptr(out, "out", cache.dtype, (B, heads, dim), here)
    wp, slots = None, 0
    if weights is not None:
        wp, slots = _tracked(weights, "weights", torch.float32, B, cache.heads, room, here), weights.shape[2]
    scale = dim ** -0.5 if scale is None else scale
    lib, c, s = load(), cache._by_ref, ctypes.byref(batch)
    need = cache._need((B, heads, room, wp is None), lambda: lib.gemv_attention_workspace(c, s, heads, wp is not None))
    work = empty(need, dtype=torch.uint8, device=cache.device) if need else None
    _check(lib.gemv_attention(c, s, qp, q_stride, heads, scale, op, wp, slots, work.data_ptr() if need else None, need,
                              handle), "gemv_attention")
    return out


def kv_append(cache, table, lens, starts, k, v, weights=None, positions=None, seen=None, stream=None):
    """Writes new tokens to a paged cache: rows starts[b] .. starts[b+1] - 1 of
    k and v [rows, heads, head_dim] (rows may lie apart) become the last tokens
    of sequence b, which with them holds lens[b].  starts int32 [batch + 1].
    With weights float32 and positions int32 [batch, heads, slots] and seen
    int32 [batch], the slots' weights become 0 and their positions those of
    the sequence's last tokens, of seen[b] in all."""
    import torch

    here = _here()
    batch, _ = cache._batch(table, lens, None, here)
    B, rows = batch.batch, k.shape[0]
    _dims(rows)
    shape, dense = (rows, cache.heads, cache.head_dim), cache.heads * cache.head_dim
    kp, k_stride = _rows(k, "k", cache.dtype, shape, here, dense)
    vp, v_stride = _rows(v, "v", cache.dtype, shape, here, dense)
    sp = _ptr(starts, "starts", torch.int32, (B + 1,), here)
    if (weights is None) != (positions is None) or (weights is None) != (seen is None):
        raise ValueError("weights, positions and seen go together")
    wp = pp = np = None
    slots = 0
    if weights is not None:
        wp = _tracked(weights, "weights", torch.float32, B, cache.heads, 0, here)
        slots = weights.shape[2]
        pp = _ptr(positions, "positions", torch.int32, (B, cache.heads, slots), here)
        np = _ptr(seen, "seen", torch.int32, (B,), here)
    handle, _ = _work_stream(stream, here)
    _check(load().gemv_kv_append(cache._by_ref, ctypes.byref(batch), sp, kp, k_stride, vp, v_stride, rows, wp, pp, np,
                                 slots, handle), "gemv_kv_append")


def kv_evict(cache, table, lens, seen, weights, positions, budget, recent, max_len=None, out=None, stream=None):
    """Evicts from a paged cache by accumulated attention weight: each head of
    a sequence over `budget` keeps its tokens of the last `recent` positions
    and of the others those of the largest weight, `budget` in all (keep
    recent <= budget: of more newest tokens than that, those in the lower slots
    stay, not the latest); keys and values move in place.  weights float32 and
    positions int32 [batch, heads, slots], seen int32 [batch] (see kv_append).
    Returns, or writes to ``out``, (weights, positions, lens) afterwards."""
    import torch

    here = _here()
    batch, room = cache._batch(table, lens, max_len, here)
    B = batch.batch
    wp = _tracked(weights, "weights", torch.float32, B, cache.heads, room, here)
    shape = weights.shape
    pp = _ptr(positions, "positions", torch.int32, shape, here)
    np = _ptr(seen, "seen", torch.int32, (B,), here)
    _dims(budget, recent)
    handle, empty = _work_stream(stream, here)
    if out is None:
        new_w = empty(shape, dtype=torch.float32, device=cache.device)
        new_p = empty(shape, dtype=torch.int32, device=cache.device)
        left = empty(B, dtype=torch.int32, device=cache.device)
        outs = new_w.data_ptr(), new_p.data_ptr(), left.data_ptr()
    else:
        new_w, new_p, left = out
        outs = (_ptr(new_w, "out[0]", torch.float32, shape, here), _ptr(new_p, "out[1]", torch.int32, shape, here),
                _ptr(left, "out[2]", torch.int32, (B,), here))
        tracked = 4 * weights.numel()
        _apart([(outs[0], tracked), (outs[1], tracked), (outs[2], 4 * B)],
               [(wp, tracked), (pp, tracked), (batch.lens, 4 * B), (np, 4 * B)])
    lib, c, s = load(), cache._by_ref, ctypes.byref(batch)
    need = cache._need((B, budget, room), lambda: lib.gemv_kv_evict_workspace(c, s, budget))
    work = empty(need, dtype=torch.uint8, device=cache.device) if need else None
    _check(lib.gemv_kv_evict(c, s, np, wp, pp, shape[2], budget, recent, *outs, work.data_ptr() if need else None, need,
                             handle), "gemv_kv_evict")
    return new_w, new_p, left
