"""Outputs of prompt and prefix attention beside and in place of the queries."""
import pytest
import torch

from memory_bound_gemv_row_amd import binding

import serving_ref as ref
from gpu_util import say
from test_gpu_prompt import _query

pytestmark = pytest.mark.gpu


def _ints(*v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def _calls():
    """(name, call(q, out), rows) of heads of 64, eight of queries."""
    pool = ref.Pool([300, 90], 2, 64, 16, seed=81)
    cache = binding.PagedCache(pool.dk, pool.dv)
    starts, groups = _ints(0, 20, 30), _ints(0, 2)
    return [
        ("prompt", lambda q, out: binding.prompt_attention(cache, pool.dtable, pool.dlens, starts, q, out=out), 30),
        ("window", lambda q, out: binding.paged_attention(cache, pool.dtable, pool.dlens, q, window=40, out=out), 2),
        ("prefix", lambda q, out: binding.prefix_attention(cache, pool.dtable[:1], pool.dlens[:1], groups, pool.dtable, pool.dlens, q,
                                                           out=out), 2),
    ]


def test_dense_rows_over_strided_ones_are_refused(gpu):
    for name, call, rows in _calls():
        say(f"[overlap] {name}")
        made = _query(rows, 12, 64, torch.float16, 82).cuda()
        q = made[:, :8]                                                      # the first part of a product's rows
        before = made.clone()
        for first in (0, 64, 8 * 64):
            out = made.view(-1)[first: first + rows * 512].view(rows, 8, 64)
            with pytest.raises(binding.GemvError):
                call(q, out)
        assert torch.equal(made, before)


def test_outputs_beside_the_queries(gpu):
    # behind their last row, before their first, between two of them, and a single row in its own place
    for name, call, rows in _calls():
        say(f"[overlap] {name}, beside")
        width = rows * 512
        room = torch.zeros(3 * width + rows * (width + 512), dtype=torch.float16, device="cuda")
        want = None
        for q_at, step, out_at in ((0, 512, width), (width, 512, 0), (0, 512 + width, 512), (0, 512 + width, 512 + (rows - 2) * (512 + width))):
            q = room[q_at: q_at + rows * step].view(rows, step)[:, :512].view(rows, 8, 64)
            q.copy_(_query(rows, 8, 64, torch.float16, 83))
            out = room[out_at: out_at + width].view(rows, 8, 64)
            call(q, out)
            want = out.clone() if want is None else want
            assert torch.equal(out, want), (name, q_at, step, out_at)
    pool = ref.Pool([300], 2, 64, 16, seed=84)
    cache = binding.PagedCache(pool.dk, pool.dv)
    made = _query(1, 12, 64, torch.float16, 85).cuda()
    q = made[:, :8]
    want = binding.prompt_attention(cache, pool.dtable, pool.dlens, _ints(0, 1), q)
    assert torch.equal(binding.prompt_attention(cache, pool.dtable, pool.dlens, _ints(0, 1), q, out=q), want)
