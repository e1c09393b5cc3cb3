"""Results of norms with rotation that are laid over inputs otherwise than in their
own places, or over each other, are refused, before a device is touched."""
import ctypes

import pytest
import torch

from memory_bound_gemv_row_amd import binding

from test_between_cpu import _heads, _how, lib  # noqa: F401
from test_serving_cpu import INVAL, P, _cache

# four heads of queries, two of keys and of values, of 64 elements: parts of rows of 512 in binary16
ROW, Q, K, V = 1024, P, P + 512, P + 768
FAR, FARTHER = P + (1 << 20), P + (1 << 21)


def _parts(q_out, q_stride, k_out, k_stride):
    return (_heads(4, x=Q, stride=512, out=q_out, out_stride=q_stride), _heads(2, x=K, stride=512, out=k_out, out_stride=k_stride),
            _heads(2, x=V, stride=512))


def _turn(lib, q, k, rows, out_dtype=1):   # noqa: F811
    return lib.gemv_norm_rotate(ctypes.byref(_how()), ctypes.byref(q), ctypes.byref(k), 1, out_dtype, P, rows, None)


def _put(lib, q, k, v, rows):   # noqa: F811
    return lib.gemv_norm_rotate_append(ctypes.byref(_how()), ctypes.byref(q), ctypes.byref(k), ctypes.byref(v), 1, P, rows,
                                       ctypes.byref(_cache(k=FARTHER, v=2 * FARTHER)), P, None)


BAD = [(K, 512, FAR, 128), (FAR, 256, Q, 512),                      # the other's place
       (FAR, 256, FAR, 128), (FAR, 256, FAR + 256, 128),            # one place for both
       (FAR, 256, FAR + 256 * 2 * 9 - 2, 128),
       (Q, 256, FAR, 128), (Q, 520, FAR, 128), (FAR, 256, K, 128),  # their own place in other rows
       (Q + 16, 512, FAR, 128), (Q - 16, 512, FAR, 128), (FAR, 256, K + 2, 512),
       (Q + ROW, 512, FAR, 128), (FAR, 256, K - ROW, 512), (Q + 9 * ROW + 510, 512, FAR, 128)]


@pytest.mark.parametrize("place", BAD, ids=str)
def test_refused(lib, place):   # noqa: F811
    q, k, v = _parts(*place)
    assert _turn(lib, q, k, 10) == INVAL


@pytest.mark.parametrize("q_out,q_stride", [(K, 512), (V, 512), (Q, 256), (Q + 16, 512), (V - ROW, 512), (K - 16, 520)])
def test_refused_before_the_cache(lib, q_out, q_stride):   # noqa: F811
    q, k, v = _parts(q_out, q_stride, None, 0)
    assert _put(lib, q, k, v, 10) == INVAL


@pytest.mark.skipif(torch.cuda.is_available(), reason="the calls would run, and the addresses are made up")
def test_not_refused(lib):   # noqa: F811
    for place in [(FAR, 256, FARTHER, 128), (Q, 512, K, 512), (FAR, 384, FAR + 512, 384), (FAR, 256, FAR + 256 * 2 * 10, 128),
                  (P + 10 * ROW, 256, P - 256 * 10, 128)]:
        q, k, v = _parts(*place)
        assert _turn(lib, q, k, 10) != INVAL, place
    q, k, v = _parts(Q, 256, FAR, 128)
    assert _turn(lib, q, k, 1) != INVAL                              # one row has no stride
    assert _turn(lib, q, _heads(0, x=K, out=Q), 1) != INVAL          # nor have no heads a place
    for place in [(Q, 512), (FAR, 256), (P + 10 * ROW, 256)]:
        q, k, v = _parts(*place, None, 0)
        assert _put(lib, q, k, v, 10) != INVAL, place


def _rows(at, width, step, rows):
    return {b for i in range(rows) for b in range(at + i * step, at + i * step + width)}


def test_against_sets_of_bytes(lib):   # noqa: F811
    # results of two bytes an element about inputs of four: every way that their rows can lie
    dim, rows = 8, 4
    for heads in (1, 2):
        for stride in (heads * dim, heads * dim + 8, 40):
            for out_stride in (heads * dim, heads * dim + 4, 40, 80):
                for shift in range(-200, 900, 22):
                    q = binding.Heads(P, stride, heads, None, P + shift, out_stride)
                    meets = _rows(P, heads * dim * 4, stride * 4, rows) & _rows(P + shift, heads * dim * 2, out_stride * 2, rows)
                    if not meets and torch.cuda.is_available():
                        continue
                    got = lib.gemv_norm_rotate(ctypes.byref(_how(head_dim=8, rotated=8, norm=0)), ctypes.byref(q), None, 0, 1, P - (1 << 19),
                                               rows, None)
                    assert (got == INVAL) == bool(meets), (heads, stride, out_stride, shift)


def test_more_heads_than_are_counted(lib):   # noqa: F811
    most, wide = (1 << 31) - 1, 64 << 31
    q, k, v = (_heads(n, x=P, stride=wide, out=P + (at << 50), out_stride=wide) for n, at in ((most, 1), (most, 2), (2, 0)))
    assert _turn(lib, q, k, 1) == 2 and _turn(lib, q, _heads(0), 1) == 2 and _turn(lib, _heads(0), k, 1) == 2
    assert _put(lib, q, v, v, 1) == 2
