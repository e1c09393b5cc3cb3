"""Every kernel that the serving operators' launch rules can choose, against
plain 64-bit forms: the product at each of its tilings, and attention over
whole and loose pages at each head size, in one part, by one workgroup of
eight waves, and split."""
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


# ---------------------------------------------------------------- attention
def _check_attention(pool, q, label, scale=None):
    say(f"[attention] {label}")
    scale = pool.dim ** -0.5 if scale is None else scale
    want, bound, want_w, wbound = ref.attention_by_slot(pool, q, scale)
    cache = binding.PagedCache(pool.dk, pool.dv)
    out = binding.paged_attention(cache, pool.dtable, pool.dlens, q.cuda(), scale=scale)
    off = np.abs(out.cpu().double().numpy() - want)
    assert np.all(off <= bound), (label, float(np.nanmax(off / bound)), int(np.isnan(off).sum()))
    before = np.random.default_rng(1).uniform(0, 2, want_w.shape).astype(np.float32)
    w = torch.from_numpy(before.copy()).cuda()
    again = binding.paged_attention(cache, pool.dtable, pool.dlens, q.cuda(), scale=scale, weights=w)
    assert torch.equal(again, out), label
    got = w.cpu().double().numpy()
    assert np.all(np.abs(got - (before + want_w)) <= wbound + ref.U32 * (before + want_w)), label
    for b, n in enumerate(pool.lens):
        assert np.array_equal(got[b, :, n:], before[b, :, n:]), label


def _query(B, heads, dim, dtype, seed):
    return torch.randn((B, heads, dim), generator=torch.Generator().manual_seed(seed)).to(dtype)


@pytest.mark.parametrize("dtype", TYPES[1:], ids=str)
@pytest.mark.parametrize("dim", rules.DIMS)
@pytest.mark.parametrize("page", rules.PAGES)
@pytest.mark.parametrize("name", list(rules.LENGTHS))
def test_attention_in_every_form(gpu, name, page, dim, dtype):
    lens, kv, heads = rules.LENGTHS[name]
    pool = ref.Pool(lens, kv, dim, page, dtype, seed=dim + page)
    _check_attention(pool, _query(len(lens), heads, dim, dtype, page), f"{name}: dim {dim} page {page} {dtype}")


@pytest.mark.parametrize("dtype", TYPES[1:], ids=str)
@pytest.mark.parametrize("page,n", [(16, 64), (5, 64), (16, 1500)])
def test_masked_keys_weigh_nothing(gpu, page, n, dtype):
    # tokens masked by the lowest finite key, and one by a key of -inf
    pool = ref.Pool([n], 1, 64, page, dtype, seed=12)
    for j in (0, 5, 40, n - 1):
        pool.k[pool.table[0, j // page], j % page, 0] = -65504.0
    pool.k[pool.table[0, 19 // page], 19 % page] = -float("inf")
    pool.dk = pool.k.cuda()
    _check_attention(pool, torch.ones((1, 2, 64), dtype=dtype), f"masked keys, {n} in pages of {page} {dtype}", scale=0.125)


@pytest.mark.parametrize("dim", [8, 64, 72, 128, 256])
def test_parts_are_those_of_the_rule(gpu, dim):
    # the workspace holds a maximum, a sum and `dim` values of every query head and part
    import ctypes

    lib, cus = binding.load(), _cus()
    for batch, limit, kv, heads in ((16, 2048, 16, 16), (64, 1504, 8, 8), (8, 4000, 32, 32), (1, 30000, 4, 16), (2, 8192, 8, 32),
                                    (32, 1024, 8, 32), (8, 4000, 4, 28), (1, 250, 2, 4), (40, 500, 4, 4), (3, 77, 1, 50)):
        for page in (16, 24):
            k = torch.empty((1, page, kv, dim), dtype=torch.float16, device="cuda")
            cache = binding.PagedCache(k, k)
            width = -(-limit // page)
            call = binding.KvBatch(cache.c.k, width, width, cache.c.k, batch, limit)
            got = lib.gemv_attention_workspace(ctypes.byref(cache.c), ctypes.byref(call), heads, 0)
            _, _, _, parts = rules.attention_form(batch, limit, kv, heads, dim, page, cus)
            want = 0 if parts == 1 else -(-batch * heads * parts * 8 // 16) * 16 + batch * heads * parts * dim * 4
            assert got == want, (batch, limit, kv, heads, page)
