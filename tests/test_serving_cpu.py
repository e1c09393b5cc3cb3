"""Host-side checks of the serving entry points that need no GPU: every call
that the headers refuse returns its status before a device is touched, and
the plain forms that the GPU tests compare with hold against closed forms."""
import ctypes
import os
import subprocess

import numpy as np
import pytest
import torch

from memory_bound_gemv_row_amd import binding, build

import serving_ref as ref

OK, INVAL, UNSUPPORTED = 0, 1, 2
P = 1 << 20     # stands for a device pointer: refused calls do not read it


@pytest.fixture(scope="module")
def lib():
    if build.stale():
        build.build()
    return binding.load()


def test_headers_are_plain_c(tmp_path):
    src = tmp_path / "h.c"
    src.write_text('#include "gemv_tokens.h"\n#include "gemv_attention.h"\nint main(void) { return GEMV_F32; }\n')
    subprocess.run(["gcc", "-std=c11", "-Wall", "-Wextra", "-Werror", "-pedantic", "-fsyntax-only", "-I", build.INCLUDE,
                    str(src)], check=True)


@pytest.mark.parametrize("args,status", [
    ((P, 1, 64, P, P, -1, 64), INVAL), ((P, 1, 64, P, P, 4, -1), INVAL), ((P, 1, 63, P, P, 4, 64), INVAL),
    ((P, 3, 64, P, P, 4, 64), INVAL), ((P, -1, 64, P, P, 4, 64), INVAL), ((0, 1, 64, P, P, 4, 64), INVAL),
    ((P, 1, 64, 0, P, 4, 64), INVAL), ((P, 1, 64, P, 0, 4, 64), INVAL), ((0, 1, 64, 0, 0, 0, 64), OK)])
def test_quantize_tokens_status(lib, args, status):
    assert lib.gemv_quantize_tokens_q8(*args, None) == status


@pytest.mark.parametrize("args,status", [
    ((P, P, P, P, P, 1, -1, 4, 64), INVAL), ((P, P, P, P, P, 1, 4, -1, 64), INVAL), ((P, P, P, P, P, 1, 4, 4, -1), INVAL),
    ((P, P, P, P, P, 3, 4, 4, 64), INVAL), ((0, P, P, P, P, 1, 4, 4, 64), INVAL), ((P, 0, P, P, P, 1, 4, 4, 64), INVAL),
    ((P, P, 0, P, P, 1, 4, 4, 64), INVAL), ((P, P, P, 0, P, 1, 4, 4, 64), INVAL), ((P, P, P, P, 0, 1, 4, 4, 64), INVAL),
    ((P, P, P, P, P, 1, 4, 4, 131072), UNSUPPORTED), ((0, 0, 0, 0, 0, 1, 0, 4, 64), OK), ((0, 0, 0, 0, 0, 1, 4, 0, 64), OK),
    ((P, P, P, P, P, 1, (1 << 31) - 1, (1 << 31) - 1, 64), (UNSUPPORTED, 4))])
def test_gemm_status(lib, args, status):
    assert lib.gemv_gemm_q8(*args, None) in (status if isinstance(status, tuple) else (status,))


def _cache(**kw):
    f = dict(k=P, v=P, dtype=1, pages=10, page_size=16, heads=2, head_dim=64, stride_page=2048, stride_slot=128,
             stride_head=64)
    f.update(kw)
    return binding.KvCache(*(f[n] for n, _ in binding.KvCache._fields_))


def _batch(**kw):
    f = dict(table=P, table_stride=4, width=4, lens=P, batch=2, max_len=64)
    f.update(kw)
    return binding.KvBatch(*(f[n] for n, _ in binding.KvBatch._fields_))


BAD_CACHE = [(dict(dtype=0), INVAL), (dict(dtype=3), INVAL), (dict(pages=-1), INVAL), (dict(page_size=0), INVAL),
             (dict(heads=0), INVAL), (dict(head_dim=0), INVAL), (dict(stride_page=56), INVAL), (dict(stride_slot=0), INVAL),
             (dict(stride_head=-64), INVAL), (dict(k=None), INVAL), (dict(v=None), INVAL), (dict(head_dim=60), UNSUPPORTED),
             (dict(head_dim=264, stride_page=8192, stride_slot=528, stride_head=264), UNSUPPORTED),
             (dict(stride_page=2049), UNSUPPORTED), (dict(stride_slot=132), UNSUPPORTED), (dict(stride_head=68), UNSUPPORTED),
             (dict(k=P + 8), UNSUPPORTED), (dict(v=P + 2), UNSUPPORTED)]
BAD_BATCH = [(dict(batch=-1), INVAL), (dict(width=-1), INVAL), (dict(max_len=-1), INVAL), (dict(table_stride=3), INVAL),
             (dict(table=None), INVAL), (dict(lens=None), INVAL)]


def _attend(lib, c, b, q=P, q_stride=256, heads=4, out=P, weights=None, slots=0, ws=P, nws=1 << 30):
    return lib.gemv_attention(ctypes.byref(c), ctypes.byref(b), q, q_stride, heads, 0.125, out, weights, slots, ws, nws, None)


def _append(lib, c, b, starts=P, k=P, k_stride=128, v=P, v_stride=128, rows=2, weights=None, positions=None, seen=None,
            slots=0):
    return lib.gemv_kv_append(ctypes.byref(c), ctypes.byref(b), starts, k, k_stride, v, v_stride, rows, weights, positions,
                              seen, slots, None)


def _evict(lib, c, b, seen=P, w=P, p=P, slots=64, budget=8, recent=2, wo=P, po=P, lo=P, ws=P, nws=1 << 30):
    return lib.gemv_kv_evict(ctypes.byref(c), ctypes.byref(b), seen, w, p, slots, budget, recent, wo, po, lo, ws, nws, None)


@pytest.mark.parametrize("call", [_attend, _append, _evict])
def test_cache_and_batch_status(lib, call):
    for kw, status in BAD_CACHE:
        assert call(lib, _cache(**kw), _batch()) == status, kw
    for kw, status in BAD_BATCH:
        if call is _append and "max_len" in kw:
            continue                  # not used there
        assert call(lib, _cache(), _batch(**kw)) == status, kw
    assert call(lib, _cache(), _batch(batch=0, lens=None)) == OK


def test_call_status(lib):
    c, b = _cache(), _batch()
    for kw in (dict(heads=0), dict(heads=3), dict(q_stride=248), dict(weights=P, slots=63), dict(q=None), dict(out=None)):
        assert _attend(lib, c, b, **kw) == INVAL, kw
    for kw in (dict(q=P + 8), dict(q_stride=260)):
        assert _attend(lib, c, b, **kw) == UNSUPPORTED, kw
    for kw in (dict(rows=-1), dict(k_stride=120), dict(v_stride=127), dict(weights=P), dict(weights=P, positions=P),
               dict(seen=P), dict(starts=None), dict(k=None), dict(v=None),
               dict(weights=P, positions=P, seen=P, slots=-1)):
        assert _append(lib, c, b, **kw) == INVAL, kw
    for kw in (dict(k=P + 8), dict(v=P + 4), dict(k_stride=132), dict(v_stride=130)):
        assert _append(lib, c, b, **kw) == UNSUPPORTED, kw
    assert _append(lib, c, b, rows=0, k=None, v=None) == OK
    for kw in (dict(budget=-1), dict(recent=-1), dict(slots=63), dict(seen=None), dict(w=None), dict(p=None), dict(wo=None),
               dict(po=None), dict(lo=None)):
        assert _evict(lib, c, b, **kw) == INVAL, kw
    assert lib.gemv_attention_workspace(None, None, 4, 0) == 0
    assert lib.gemv_kv_evict_workspace(None, None, 4) == 0
    assert lib.gemv_kv_evict_workspace(ctypes.byref(c), ctypes.byref(b), -1) == 0


def test_torch_wrappers_refuse_host_tensors():
    k = torch.zeros((4, 16, 2, 64), dtype=torch.float16)
    with pytest.raises(ValueError):
        binding.PagedCache(k, k)
    with pytest.raises(TypeError):
        binding.PagedCache(k.numpy(), k.numpy())


# ---------------------------------------------------------------- the plain forms themselves
def test_reference_codes():
    x = np.array([[127.0, 0.5, 1.5, -2.5, 126.5, -0.49]])
    q, s = ref.quantize_tokens(x)
    assert s[0] == 1.0 and q[0].tolist() == [127, 0, 2, -2, 126, 0]
    assert np.all(np.isnan(ref.quantize_tokens(np.array([[1.0, np.inf]]))[1]))


def test_reference_attention():
    # equal logits average the values; one dominant logit takes its value; holes and empty sequences
    pool = ref.Pool([5, 0], 1, 8, 2, device="cpu", seed=1)
    q = torch.zeros((2, 2, 8), dtype=torch.float16)
    out, bound, w, _ = ref.attention(pool, q, 1.0)
    v, _ = pool.rows(pool.v, 0, 0, 5)
    assert np.allclose(out[0, 0], v.mean(0)) and np.all(out[1] == 0) and np.allclose(w[0, 0, :5], 2 / 5)
    assert np.all(bound[0] < 1e-2)
    for j in range(5):
        pool.k[pool.table[0, j // 2], j % 2, 0] = 0.0
    pool.k[pool.table[0, 1], 1, 0, 0] = 100.0
    q[0, 0, 0] = 10.0
    out, _, w, _ = ref.attention(pool, q, 1.0)
    assert np.allclose(out[0, 0], v[3]) and np.isclose(w[0, 0, 3], 1 + 1 / 5)
    pool.table[0, 0] = -1
    out, _, w, _ = ref.attention(pool, torch.zeros((2, 2, 8), dtype=torch.float16), 1.0)
    assert np.allclose(out[0, 1], v[2:].mean(0)) and np.all(w[0, 0, :2] == 0)


def test_reference_attention_bound_catches_a_lost_token():
    # a mistake planted in the reference: the last token left out
    pool = ref.Pool([40], 1, 16, 8, device="cpu", seed=2)
    q = torch.randn((1, 1, 16), generator=torch.Generator().manual_seed(1)).half()
    out, bound, _, _ = ref.attention(pool, q, 0.25)
    pool.lens = [39]
    wrong, _, _, _ = ref.attention(pool, q, 0.25)
    assert np.any(np.abs(wrong - out) > 2 * bound)


def test_reference_eviction():
    w = np.array([[[5, 1, 3, 1, 4, 9, 2, 0]]], np.float32)
    pos = np.arange(8, dtype=np.int32).reshape(1, 1, 8)
    source, w2, p2, left = ref.evict([8], [8], w, pos, 4, 2, 8)
    # positions 6 and 7 are recent; 9 and 5 weigh most: slots 0, 5, 6, 7 stay; 5, 6, 7 go to 1, 2, 3
    assert source[0, 0, :4].tolist() == [0, 5, 6, 7] and left.tolist() == [4]
    assert w2[0, 0].tolist() == [5, 9, 2, 0, 0, 0, 0, 0] and p2[0, 0].tolist() == [0, 5, 6, 7, -1, -1, -1, -1]
    source, _, _, _ = ref.evict([8], [8], np.ones_like(w), pos, 4, 0, 8)
    assert source[0, 0].tolist() == list(range(8))     # ties: the lower slots stay


def test_package_exports_the_operators():
    import memory_bound_gemv_row_amd as amd

    for name in ("quantize_tokens_q8", "gemm_q8", "PagedCache", "paged_attention", "kv_append", "kv_evict"):
        assert getattr(amd, name) is getattr(binding, name)
    assert os.path.exists(os.path.join(build.INCLUDE, "gemv_attention.h"))


def test_outputs_that_share_memory_are_refused():
    apart = binding._apart
    apart([(100, 40), (140, 40), (180, 4)], [(0, 100), (200, 40), (184, 4)])
    apart([(100, 0), (100, 40)], [(100, 0)])              # nothing shares nothing
    for outs, ins in (([(100, 40)], [(100, 40)]), ([(100, 40)], [(139, 1)]), ([(100, 40)], [(0, 101)]),
                      ([(100, 40)], [(110, 2)]), ([(100, 40), (120, 40)], []), ([(0, 4), (8, 4), (11, 4)], [])):
        with pytest.raises(ValueError):
            apart(outs, ins)
