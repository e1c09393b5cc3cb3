"""Every kernel that the serving operators' launch rules can choose, against
plain 64-bit forms: the product at each of its tilings."""
import numpy as np
import pytest
import torch

from memory_bound_gemv_row_amd import binding

import serving_ref as ref
import serving_rules as rules
from gpu_util import say

pytestmark = pytest.mark.gpu

TYPES = [torch.float32, torch.float16, torch.bfloat16]


def _cus():
    return torch.cuda.get_device_properties(0).multi_processor_count


# ---------------------------------------------------------------- product
def _check_products(T, M, N, seed, shift=0):
    rng = np.random.default_rng(seed)
    A, x = rng.integers(-127, 128, (M, N), dtype=np.int8), rng.integers(-127, 128, (T, N), dtype=np.int8)
    scale, xs = rng.uniform(1e-4, 2e-3, M).astype(np.float16), rng.uniform(1e-3, 0.05, T).astype(np.float32)
    # sums of whole numbers below 2^53, exact in binary64 in any order
    want = (x.astype(np.float64) @ A.astype(np.float64).T) * (xs.astype(np.float64)[:, None] * scale.astype(np.float64)[None])
    room = torch.zeros(M * N + shift, dtype=torch.int8, device="cuda")
    dA = room[shift:].view(M, N)
    dA.copy_(torch.from_numpy(A))
    rest = [torch.from_numpy(t).cuda() for t in (scale, x, xs)]
    for dtype in TYPES:
        say(f"[gemm q8] {T}x{M}x{N} {dtype}, A {shift} bytes off")
        y = binding.gemm_q8(dA, *rest, out_dtype=dtype)
        torch.cuda.synchronize()
        off = np.abs(y.cpu().double().numpy() - want)
        assert np.all(off <= ref.product_bound(want, dtype)), (T, M, N, dtype)


@pytest.mark.parametrize("T,M,N", rules.STREAMED)
def test_products_of_every_streaming_tile(gpu, T, M, N):
    assert rules.product_kernel(T, M, N, _cus())[0] == "stream"
    _check_products(T, M, N, T + M)


@pytest.mark.parametrize("T,M,N", rules.LOOSE)
def test_products_of_every_loose_tile(gpu, T, M, N):
    assert rules.product_kernel(T, M, N, _cus())[0] == "any"
    _check_products(T, M, N, T + M)


@pytest.mark.parametrize("T,M,N", [(19, 43, 3088), (133, 638, 784)])
def test_products_of_whole_columns_in_unaligned_rows(gpu, T, M, N):
    _check_products(T, M, N, T + M, shift=1)


@pytest.mark.parametrize("T,M,N", rules.LARGE)
def test_products_of_large_tiles(gpu, T, M, N):
    assert rules.product_kernel(T, M, N, _cus())[0] == "tiles"
    _check_products(T, M, N, T + M)
