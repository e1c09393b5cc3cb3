"""Host-side checks of the entry points of include/gemv_rotate.h and
include/gemv_pages.h that need no GPU: refused calls return their status before
a device is touched, the wrappers refuse what does not fit, and the plain forms
that the GPU tests compare with hold against closed forms."""
import ctypes
import subprocess

import numpy as np
import pytest
import torch

from memory_bound_gemv_row_amd import binding, build

import between_ref as bref
from test_serving_cpu import INVAL, OK, P, UNSUPPORTED, _cache


@pytest.fixture(scope="module")
def lib():
    if build.stale():
        build.build()
    return binding.load()


def test_headers_are_plain_c(tmp_path):
    src = tmp_path / "h.c"
    src.write_text('#include "gemv_rotate.h"\n#include "gemv_pages.h"\nint main(void) { return GEMV_F32; }\n')
    subprocess.run(["gcc", "-std=c11", "-Wall", "-Wextra", "-Werror", "-pedantic", "-fsyntax-only", "-I", build.INCLUDE, str(src)],
                   check=True)


def _of(cls, base, kw):
    base = dict(base, **kw)
    return cls(*(base[n] for n, _ in cls._fields_))


def _how(**kw):
    return _of(binding.Rotation, dict(head_dim=64, rotated=64, interleaved=0, freqs=P, norm=1, eps=1e-6, weight_dtype=1), kw)


def _heads(heads=2, **kw):
    return _of(binding.Heads, dict(x=P, stride=64 * max(heads, 0), heads=heads, weight=P, out=2 * P, out_stride=64 * max(heads, 0)), kw)


def _turn(lib, how=None, q=None, k=None, dtype=1, out_dtype=1, positions=P, rows=2):
    how, q, k = how or _how(), q or _heads(4), k or _heads(2)
    return lib.gemv_norm_rotate(ctypes.byref(how), ctypes.byref(q), ctypes.byref(k), dtype, out_dtype, positions, rows, None)


def _put(lib, how=None, q=None, k=None, v=None, dtype=1, positions=P, rows=2, cache=None, slots=P):
    how, q, k, v, cache = how or _how(), q or _heads(4), k or _heads(2), v or _heads(2), cache or _cache()
    return lib.gemv_norm_rotate_append(ctypes.byref(how), ctypes.byref(q), ctypes.byref(k), ctypes.byref(v), dtype, positions, rows,
                                       ctypes.byref(cache), slots, None)


@pytest.mark.parametrize("call", [_turn, _put])
def test_rotation_status(lib, call):
    for kw in (dict(head_dim=0), dict(rotated=-2), dict(rotated=63), dict(rotated=66), dict(freqs=None), dict(weight_dtype=3),
               dict(weight_dtype=-1)):
        assert call(lib, how=_how(**kw)) == INVAL, kw
    for kw in (dict(q=_heads(-1)), dict(q=_heads(4, stride=255)), dict(q=_heads(4, x=None)), dict(q=_heads(4, out=None)),
               dict(q=_heads(4, out_stride=255)), dict(k=_heads(2, stride=100)), dict(k=_heads(2, x=None)), dict(dtype=3), dict(dtype=-1),
               dict(positions=None), dict(rows=-1)):
        assert call(lib, **kw) == INVAL, kw
    for kw in (dict(q=_heads(4, out=P + 64, x=P + 64, out_stride=264)), dict(q=_heads(4, out=P + 64, x=P + 64), dtype=0)):
        assert call(lib, **kw) == INVAL, kw
    assert call(lib, rows=0, positions=None, q=_heads(4, x=None, out=None)) == OK


def test_rotation_status_of_each(lib):
    assert _turn(lib, how=_how(head_dim=257), q=_heads(1, stride=257, out_stride=257), k=_heads(0)) == UNSUPPORTED
    for kw in (dict(out_dtype=3), dict(k=_heads(2, out=None)), dict(k=_heads(2, out_stride=127))):
        assert _turn(lib, **kw) == INVAL, kw
    assert lib.gemv_norm_rotate(None, ctypes.byref(_heads()), None, 1, 1, P, 2, None) == INVAL
    assert lib.gemv_norm_rotate(ctypes.byref(_how()), None, None, 1, 1, P, 2, None) == INVAL
    for kw in (dict(k=_heads(3)), dict(v=_heads(1)), dict(v=_heads(2, x=None)), dict(v=_heads(2, stride=127)), dict(slots=None),
               dict(cache=_cache(head_dim=32)), dict(cache=_cache(dtype=0)), dict(cache=_cache(k=None)), dict(cache=_cache(v=None)),
               dict(cache=_cache(pages=-1)), dict(cache=_cache(page_size=0)), dict(cache=_cache(heads=0)),
               dict(cache=_cache(stride_slot=56))):
        assert _put(lib, **kw) == INVAL, kw
    for kw in (dict(cache=_cache(k=P + 8)), dict(cache=_cache(v=P + 2)), dict(cache=_cache(stride_page=2049)),
               dict(cache=_cache(stride_slot=132)), dict(cache=_cache(stride_head=68))):
        assert _put(lib, **kw) == UNSUPPORTED, kw


def _pool(**kw):
    return _of(binding.Pool, dict(free_pages=P, count=P, pages=8, page_size=16, table=P, table_stride=4, width=4, batch=2), kw)


BAD_POOL = [dict(pages=-1), dict(page_size=0), dict(width=-1), dict(batch=-1), dict(table_stride=3), dict(count=None),
            dict(free_pages=None), dict(table=None)]


def test_pages_status(lib):
    def take(lens=P, added=P, rows=2, outs=(P + 64,) * 5, **kw):
        return lib.gemv_reserve_pages(ctypes.byref(_pool(**kw)), lens, added, rows, *outs, None)

    def give(keep=P, out=P + 64, ws=P, n=1 << 20, **kw):
        return lib.gemv_release_pages(ctypes.byref(_pool(**kw)), keep, out, ws, n, None)

    for kw in BAD_POOL:
        assert take(**kw) == INVAL and give(**kw) == INVAL, kw
    for kw in [dict(lens=None), dict(added=None), dict(rows=-1)] + \
            [dict(outs=tuple(None if i == j else P + 64 for j in range(5))) for i in range(5)]:
        assert take(**kw) == INVAL, kw
    assert take(rows=(1 << 30) + 1) == UNSUPPORTED
    for kw in (dict(keep=None), dict(out=None), dict(out=P), dict(ws=None), dict(n=7), dict(ws=P + 4)):
        assert give(**kw) == INVAL, kw
    assert give(batch=65537) == UNSUPPORTED
    assert lib.gemv_release_pages_workspace(ctypes.byref(_pool(batch=5))) == 20
    assert lib.gemv_release_pages_workspace(ctypes.byref(_pool(batch=65537))) == 0
    assert lib.gemv_reserve_pages(None, P, P, 2, P, P, P, P, P, None) == INVAL
    assert lib.gemv_release_pages(None, P, P, P, 4, None) == INVAL


def test_rotation_arguments():
    q, k = torch.zeros((3, 4, 64)), torch.zeros((3, 2, 64))
    at, freqs, w = torch.zeros(3, dtype=torch.int32), torch.zeros(32, dtype=torch.float64), torch.ones(64)
    for args in ((q[0], k, at, freqs, None, None, 1e-6), (q, k[:2], at, freqs, None, None, 1e-6), (q, k, at, freqs[None], None, None, 1e-6),
                 (q, k, at, torch.zeros(33, dtype=torch.float64), None, None, 1e-6), (q, k, at, freqs, w, None, None)):
        with pytest.raises(ValueError):
            binding._rotation(*args, False, 0)
    with pytest.raises(TypeError):
        binding._rotation(q, k, at, freqs, w, w.half(), 1e-6, False, 0)
    with pytest.raises((ValueError, TypeError)):
        binding._rotation(q, k, at, freqs, w, w, 1e-6, False, 0)   # host tensors


# ---------------------------------------------------------------- the plain forms
def test_turned():
    x = torch.tensor([[[3.0, 4.0, 0.0, 0.0]]])
    y, bound = bref.turned(x, None, np.array([1]), np.array([np.pi / 2, 0.0]), None, False, torch.float32)
    assert np.allclose(y, [[[0, 4, 3, 0]]], atol=1e-12) and np.all(bound > 0)
    y, _ = bref.turned(x, None, np.array([1]), np.array([np.pi / 2, 0.0]), None, True, torch.float32)
    assert np.allclose(y, [[[-4, 3, 0, 0]]], atol=1e-12)
    y, _ = bref.turned(x, np.array([2.0, 1, 1, 1]), np.array([0]), np.array([]), 0.0, False, torch.float32)
    assert np.allclose(y, [[[2.4, 1.6, 0, 0]]], atol=1e-12)


def test_the_series_of_the_angles():
    # the kernel's polynomials in binary32, without fused operations: two units of one at most
    f = np.float32
    exact = np.linspace(-np.pi / 4, np.pi / 4, 200001)
    r = exact.astype(f)
    z = r * r
    s = r + r * z * (f(-1 / 6) + z * (f(1 / 120) + z * (f(-1 / 5040) + z * f(1 / 362880))))
    c = f(1) - f(0.5) * z + z * z * (f(1 / 24) + z * (f(-1 / 720) + z * f(1 / 40320)))
    assert np.abs(s - np.sin(exact)).max() <= 2 * bref.U32 and np.abs(c - np.cos(exact)).max() <= 2 * bref.U32


def test_reserve_and_release():
    table = [[4, -1, -1], [2, 3, -1]]
    count, lens, starts, positions, slots, after = bref.reserve([7, 6, 5, 0, 0, 0, 0, 0], 3, table, [3, 8], [2, 9], 4, 12, 8)
    assert count == [1, 0] and lens == [5, 17] and starts == [0, 2, 11]
    assert positions == [3, 4, 8, 9, 10, 11, 12, 13, 14, 15, 16, 0]
    assert slots == [19, 20, 24, 25, 26, 27, -1, -1, -1, -1, -1, -1]
    assert after.tolist() == [[4, 5, -1], [2, 3, 6]]
    free, n, table = bref.release([7, 6, 5, 0, 0, 0, 0, 0], 1, after, [4, 0], 4, 8)
    assert free[:n] == [7, 5, 2, 3, 6] and table.tolist() == [[4, -1, -1], [-1, -1, -1]]
    count, *_ = bref.reserve([1], 1, [[-1, -1]], [0], [8], 4, 8, 1)
    assert count == [0, 1]
