"""Outputs of the calls on a cache's pages that share memory with each other or with
the inputs are refused, before a device is touched."""
import ctypes

import pytest
import torch

from test_between_cpu import _pool, lib  # noqa: F401
from test_serving_cpu import INVAL, P

# two sequences of four entries, eight pages; each array in a room of its own
ROOM = 1 << 16
FREE, COUNT, TABLE, LENS, ADDED, KEEP = (P + i * ROOM for i in range(6))
OUTS = dict(count_out=P + 8 * ROOM, lens_out=P + 9 * ROOM, starts=P + 10 * ROOM, positions=P + 11 * ROOM, slots=P + 12 * ROOM)
WORK = P + 13 * ROOM


def _take(lib, **kw):   # noqa: F811
    outs = dict(OUTS, **kw)
    pool = _pool(free_pages=FREE, count=COUNT, table=TABLE)
    return lib.gemv_reserve_pages(ctypes.byref(pool), LENS, ADDED, 5000, *outs.values(), None)


@pytest.mark.skipif(torch.cuda.is_available(), reason="the call would run, and the addresses are made up")
def test_what_lies_apart_is_not_refused(lib):   # noqa: F811
    assert _take(lib) != INVAL
    pool = _pool(free_pages=FREE, count=COUNT, table=TABLE)
    assert lib.gemv_release_pages(ctypes.byref(pool), KEEP, OUTS["count_out"], WORK, 1 << 10, None) != INVAL


@pytest.mark.parametrize("kw", [
    dict(count_out=COUNT), dict(count_out=COUNT - 4), dict(lens_out=LENS), dict(lens_out=ADDED), dict(lens_out=LENS + 4),
    dict(starts=LENS), dict(starts=ADDED - 8), dict(starts=COUNT), dict(positions=LENS - 4 * 4999), dict(slots=ADDED),
    dict(count_out=FREE + 28), dict(lens_out=TABLE + 28), dict(starts=TABLE - 8), dict(positions=TABLE), dict(slots=FREE),
    dict(starts=OUTS["lens_out"]), dict(count_out=OUTS["starts"] + 8), dict(slots=OUTS["positions"] - 39996), dict(count_out=OUTS["slots"]),
], ids=str)
def test_reserve(lib, kw):   # noqa: F811
    assert _take(lib, **kw) == INVAL


@pytest.mark.parametrize("kw", [dict(out=COUNT), dict(out=COUNT - 4), dict(out=FREE + 28), dict(out=TABLE + 16), dict(out=KEEP), dict(out=KEEP + 4),
                                dict(out=WORK), dict(work=COUNT), dict(work=KEEP), dict(work=TABLE)], ids=str)
def test_release(lib, kw):   # noqa: F811
    pool = _pool(free_pages=FREE, count=COUNT, table=TABLE)
    out, work = kw.get("out", OUTS["count_out"]), kw.get("work", WORK)
    assert lib.gemv_release_pages(ctypes.byref(pool), KEEP, out, work, 1 << 10, None) == INVAL
