"""Host-side checks of the entry points of include/gemv_prompt.h that need no
GPU: refused calls return their status before a device is touched, and the
plain forms that the GPU tests compare with hold against closed forms."""
import ctypes
import subprocess

import numpy as np
import pytest
import torch

from memory_bound_gemv_row_amd import binding, build

import prompt_ref as pref
import serving_ref as ref
from test_serving_cpu import BAD_BATCH, BAD_CACHE, INVAL, OK, P, UNSUPPORTED, _batch, _cache


@pytest.fixture(scope="module")
def lib():
    if build.stale():
        build.build()
    return binding.load()


def test_header_is_plain_c(tmp_path):
    src = tmp_path / "h.c"
    src.write_text('#include "gemv_prompt.h"\nint main(void) { return GEMV_F32; }\n')
    subprocess.run(["gcc", "-std=c11", "-Wall", "-Wextra", "-Werror", "-pedantic", "-fsyntax-only", "-I", build.INCLUDE, str(src)],
                   check=True)


def _prompt(lib, c, b, starts=P, rows=8, max_new=4, q=P, q_stride=256, heads=4, window=0, sinks=0, out=P, ws=P, nws=1 << 30):
    return lib.gemv_prompt_attention(ctypes.byref(c), ctypes.byref(b), starts, rows, max_new, q, q_stride, heads, 0.125, window,
                                     sinks, out, ws, nws, None)


def _prefix(lib, c, b, far=None, starts=P, q=P, q_stride=256, heads=4, out=P, ws=P, nws=1 << 30):
    far = _batch() if far is None else far
    return lib.gemv_prefix_attention(ctypes.byref(c), ctypes.byref(far), starts, ctypes.byref(b), q, q_stride, heads, 0.125, out, ws,
                                     nws, None)


@pytest.mark.parametrize("call", [_prompt, _prefix])
def test_cache_and_batch_status(lib, call):
    for kw, status in BAD_CACHE:
        assert call(lib, _cache(**kw), _batch()) == status, kw
    for kw, status in BAD_BATCH:
        assert call(lib, _cache(), _batch(**kw)) == status, kw
        if call is _prefix:
            assert call(lib, _cache(), _batch(), far=_batch(**kw)) == status, kw
    assert call(lib, _cache(), _batch(batch=0, lens=None)) == OK


def test_call_status(lib):
    c, b = _cache(), _batch()
    for kw in (dict(heads=0), dict(heads=3), dict(q_stride=248), dict(q=None), dict(out=None)):
        assert _prompt(lib, c, b, **kw) == INVAL, kw
        assert _prefix(lib, c, b, **kw) == INVAL, kw
    for kw in (dict(q=P + 8), dict(q_stride=260), dict(out=P + 8)):
        assert _prompt(lib, c, b, **kw) == UNSUPPORTED, kw
        assert _prefix(lib, c, b, **kw) == UNSUPPORTED, kw
    for kw in (dict(rows=-1), dict(max_new=-1), dict(window=-1), dict(sinks=-1), dict(starts=None),
               dict(starts=None, max_new=1, rows=1)):
        assert _prompt(lib, c, b, **kw) == INVAL, kw
    for kw in (dict(rows=0, q=None, out=None), dict(max_new=0)):
        assert _prompt(lib, c, b, **kw) == OK, kw
    assert _prefix(lib, c, b, starts=None) == INVAL
    most = (1 << 31) - 1
    one = _cache(heads=1, stride_slot=64)
    assert _prompt(lib, one, b, rows=most, q_stride=most * 64 // 8 * 8 + 64, heads=most) == UNSUPPORTED
    assert _prompt(lib, c, _batch(batch=most), rows=8) == UNSUPPORTED
    assert _prefix(lib, one, b, q_stride=most * 64 // 8 * 8 + 64, heads=most) == UNSUPPORTED
    assert _prefix(lib, c, _batch(batch=most)) == UNSUPPORTED
    assert _prefix(lib, c, b, far=_batch(batch=most)) == UNSUPPORTED
    assert lib.gemv_prompt_attention_workspace(ctypes.byref(one), ctypes.byref(b), most, 4, most, 0, 0) == 0
    assert lib.gemv_prompt_attention_workspace(None, None, 8, 4, 4, 0, 0) == 0
    assert lib.gemv_prefix_attention_workspace(None, None, None, 4) == 0
    for bad in ((-1, 4, 4, 0, 0), (8, -1, 4, 0, 0), (8, 4, 3, 0, 0), (8, 4, 4, -1, 0), (8, 4, 4, 0, -1)):
        assert lib.gemv_prompt_attention_workspace(ctypes.byref(c), ctypes.byref(b), *bad) == 0


def test_window_arguments():
    assert binding._window(None, 4) == (0, 4) and binding._window(3, 0) == (3, 0)
    for bad in ((0, 0), (-2, 0), (4, -1), (1 << 31, 0), (4, 1 << 31)):
        with pytest.raises(ValueError):
            binding._window(*bad)


# ---------------------------------------------------------------- the plain forms
def test_seen():
    assert pref.seen(2, 4).tolist() == [[True, True, True, False], [True] * 4]
    assert pref.seen(1, 6, window=2).tolist() == [[False] * 4 + [True] * 2]
    assert pref.seen(1, 6, window=2, sinks=1).tolist() == [[True] + [False] * 3 + [True] * 2]
    assert pref.seen(3, 2).tolist() == [[False, False], [True, False], [True, True]]


def test_a_window_past_the_length_is_the_whole():
    pool = ref.Pool([20], 2, 16, 4, seed=1, device="cpu")
    q = torch.randn((5, 4, 16)).half()
    a, b = (pref.prompt(pool, q, [0, 5], 0.25, w)[0] for w in (None, 20))
    assert np.array_equal(a, b)


def test_single_visible_token_returns_its_value():
    # a window of one: every row gets its own token's value
    pool = ref.Pool([9], 1, 16, 4, seed=2, device="cpu")
    out, bound, _ = pref.prompt(pool, torch.randn((9, 2, 16)).half(), [0, 9], 0.25, window=1)
    v, _ = pool.rows(pool.v, 0, 0, 9)
    assert np.allclose(out, np.repeat(v[:, None], 2, 1), rtol=0, atol=1e-12) and np.all(bound > 0)


def test_equal_logits_average_what_is_seen():
    pool = ref.Pool([12], 1, 8, 4, seed=3, device="cpu")
    out, _, _ = pref.prompt(pool, torch.zeros((3, 1, 8)).half(), [0, 3], 1.0, window=4, sinks=2)
    v, _ = pool.rows(pool.v, 0, 0, 12)
    for t, p in enumerate((9, 10, 11)):
        assert np.allclose(out[t, 0], v[[0, 1] + list(range(p - 3, p + 1))].mean(0), atol=1e-12)


def test_a_prefix_continues_the_sequence():
    whole = ref.Pool([14], 1, 16, 4, seed=4, device="cpu")
    far, near = (ref.Pool([n], 1, 16, 4, seed=5, device="cpu") for n in (8, 6))
    k, _ = whole.rows(whole.k, 0, 0, 14)
    v, _ = whole.rows(whole.v, 0, 0, 14)
    for p, first, n in ((far, 0, 8), (near, 8, 6)):
        for j in range(n):
            p.k[p.table[0, j // 4], j % 4, 0] = torch.from_numpy(k[first + j]).half()
            p.v[p.table[0, j // 4], j % 4, 0] = torch.from_numpy(v[first + j]).half()
    q = torch.randn((1, 2, 16)).half()
    a, _ = pref.prefix(far, near, [0, 1], q, 0.25)
    b, _, _ = pref.prompt(whole, q, [0, 1], 0.25)
    assert np.allclose(a, b, atol=1e-12)
