"""That the shapes of the GPU tests reach every kernel of the serving
operators, and that the bounds they are held to catch mistakes."""
import numpy as np
import pytest
import torch

import serving_ref as ref
import serving_rules as rules

CUS = 256


def _limit(lens, page):
    return max(-(-n // page) for n in lens) * page


def test_every_tiling_of_the_product_is_reached():
    every = rules.tilings()
    for kind, shapes in (("stream", rules.STREAMED), ("any", rules.LOOSE)):
        reached = set()
        for T, M, N in shapes:
            got, t = rules.product_kernel(T, M, N, CUS)
            assert got == kind
            if N > 2 * t.stages * t.columns and N % t.columns and T % t.tokens and M % t.outputs:
                reached.add(t)
        assert reached == set(every[kind]), set(every[kind]) - reached


def test_large_tiles_are_reached_whole_and_halved():
    forms = set()
    for T, M, N in rules.LARGE:
        assert rules.product_kernel(T, M, N, CUS) == ("tiles", None)
        tiles = -(-T // 256) * -(-M // 256)
        left = tiles % CUS
        forms.add((tiles < CUS, tiles > CUS and 0 < left <= CUS // 2))
        assert N > 512      # more than two rounds of the buffers
    assert forms == {(True, False), (False, True), (False, False)}
    # of the halved ones, one ends in the first half of its last tile
    assert any(0 < M % 256 <= 128 and -(-T // 256) * -(-M // 256) > CUS for T, M, _ in rules.LARGE)


def test_every_form_of_the_attention_is_reached():
    forms = set()
    for dim in rules.DIMS:
        for page in rules.PAGES:
            for lens, kv, heads in rules.LENGTHS.values():
                dp, whole, lone, parts = rules.attention_form(len(lens), _limit(lens, page), kv, heads, dim, page, CUS)
                forms.add((dp, whole, whole and dim == dp, lone, parts > 1))
    for dp in (64, 128, 256):
        for split in (False, True):
            assert (dp, False, False, False, split) in forms, (dp, split)
        for exact in (False, True):
            assert (dp, True, exact, True, False) in forms
            for split in (False, True):
                assert (dp, True, exact, False, split) in forms, (dp, exact, split)


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16], ids=str)
def test_the_bound_catches_attention_to_masked_tokens(dtype):
    # keys of the lowest value: their logits' large error must not widen the bound
    pool = ref.Pool([64], 1, 64, 16, dtype, seed=12, device="cpu")
    for j in (0, 5, 40):
        pool.k[pool.table[0, j // 16], j % 16, 0] = -65504.0
    pool.k[pool.table[0, 1], 3] = -float("inf")
    q = torch.ones((1, 2, 64), dtype=dtype)
    out, bound, w, wbound = ref.attention_by_slot(pool, q, 0.125)
    assert np.all(w[0, 0, [0, 5, 19, 40]] == 0) and np.all(np.isfinite(bound)) and np.all(wbound < 1e-3)
    v = ref.gathered(pool, pool.v, 0, 64)[0][0]
    for wrong in (v.mean(0), np.zeros(64), v[[0, 5, 40]].mean(0), v[1], 1.02 * out[0, 0]):
        assert np.any(np.abs(wrong - out[0, 0]) > bound[0, 0])


def test_the_bounds_agree_where_both_apply():
    pool = ref.Pool([130, 0, 33], 2, 80, 5, torch.float16, seed=3, device="cpu")
    pool.table[0, 2] = -1
    q = torch.randn((3, 6, 80), generator=torch.Generator().manual_seed(1)).half()
    for a, b in zip(ref.attention(pool, q, 0.1)[::2], ref.attention_by_slot(pool, q, 0.1)[::2]):
        assert np.allclose(a, b, rtol=1e-12, atol=1e-15)
    wide, narrow = ref.attention(pool, q, 0.1)[1], ref.attention_by_slot(pool, q, 0.1)[1]
    assert np.all(narrow <= 2 * wide) and np.all(narrow > 0)


# parts of the length for heads of 64, with what the other rule took: one that
# aims at eight workgroups per CU, or the estimate of what the busiest CU reads
@pytest.mark.parametrize("batch,limit,kv,heads,parts", [
    (16, 2048, 16, 16, 8),      # 23.8 us, by the estimate (2 parts) 26.2
    (64, 1504, 8, 8, 4),        # 29.8 us, by the estimate 37.3
    (8, 4000, 32, 32, 8),       # 38.3 us, by the estimate 49.1
    (1, 30000, 4, 16, 59),      # 15.5 us, by workgroups per CU (469 parts) 39.9
    (2, 8192, 8, 32, 16),       # 13.1 us, by workgroups per CU (128 parts) 23.5
    (32, 1024, 8, 32, 1),       # 15.0 us, by workgroups per CU (8 parts) 21.3
    (8, 4000, 4, 28, 8)])       # 13.6 us, by workgroups per CU (63 parts) 22.1
def test_parts_of_small_heads(batch, limit, kv, heads, parts):
    assert rules.attention_form(batch, limit, kv, heads, 64, 16, CUS)[2:] == (False, parts)
