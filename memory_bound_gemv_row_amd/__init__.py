"""Row-major GEMV, y[M] = A[M,N] . x[N], on MI355X (gfx950), with the INT8
product of several tokens and attention over a paged key-value cache.

The compute lives in a hand-written HIP library behind a C ABI
(``include/*.h``); ``binding`` is a thin ctypes layer over it.  The
library is loaded on first use and its absence is an error: there is no CPU
fallback.
"""

from .binding import (  # noqa: F401,E402  (no library load at import time)
    GemvError,
    gemv_f32,
    gemv_f16,
    gemv_f16x32,
    gemv_f16_acc16,
    gemv_q8,
    gemv_q4,
    describe_launch,
    quantize_q8,
    quantize_q4,
    softmax_f16,
    quantize_tokens_q8,
    gemm_q8,
    PagedCache,
    paged_attention,
    kv_append,
    kv_evict,
)
