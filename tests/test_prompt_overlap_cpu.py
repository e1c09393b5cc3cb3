"""Outputs of prompt and prefix attention that share memory with the queries
otherwise than as the same dense rows are refused, before a device is touched."""
import pytest

from test_prompt_cpu import _prefix, _prompt, lib  # noqa: F401
from test_serving_cpu import INVAL, P, _batch, _cache

ROW = 4 * 64 * 2   # bytes of a row of four heads of 64


@pytest.mark.parametrize("out,stride", [
    (P, 264),                           # the first part of wider rows, and dense rows from there on
    (P, 512),
    (P + ROW, 256), (P - ROW, 256),     # a row on, a row back
    (P + 16, 256), (P - 16, 256),
    (P + 7 * ROW, 256), (P - 7 * ROW, 256),
    (P + ROW, 512),                     # begins between two rows, ends past the next
    (P + ROW + 64, 512), (P + 6 * 2 * ROW + ROW, 512),
    (P + 7 * 2 * ROW, 512),             # the last row
    (P + 7 * 2 * ROW + ROW - 16, 512),
])
def test_refused(lib, out, stride):   # noqa: F811
    c, rows = _cache(), 8
    assert _prompt(lib, c, _batch(), rows=rows, q_stride=stride, out=out) == INVAL
    assert _prompt(lib, c, _batch(batch=rows), starts=None, rows=rows, max_new=1, q_stride=stride, out=out) == INVAL
    assert _prefix(lib, c, _batch(batch=rows), q_stride=stride, out=out) == INVAL
