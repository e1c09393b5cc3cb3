"""Calls with nothing to do, without room, with pages that are shared, and graphs that
are captured together and replayed in turn."""
import numpy as np
import pytest
import torch

from memory_bound_gemv_row_amd import binding

import prompt_ref as pref
import serving_ref as ref
from gpu_util import say
from test_gpu_prompt import _query, _starts

pytestmark = pytest.mark.gpu


def _ints(*v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def test_nothing_to_do(gpu):
    say("[edges] no rows, no sequences, no room")
    pool = ref.Pool([40, 9], 2, 64, 16, seed=91)
    cache = binding.PagedCache(pool.dk, pool.dv)
    none = _query(0, 4, 64, torch.float16, 1).cuda()
    for starts in (_ints(0, 0, 0), _ints(7, 7, 7)):
        assert binding.prompt_attention(cache, pool.dtable, pool.dlens, starts, none).shape == (0, 4, 64)
    empty = _ints()
    assert binding.prompt_attention(cache, pool.dtable[:0], empty, _ints(0), none).shape == (0, 4, 64)
    assert binding.paged_attention(cache, pool.dtable[:0], empty, none, window=5).shape == (0, 4, 64)
    assert binding.prefix_attention(cache, pool.dtable, pool.dlens, _ints(0, 0, 0), pool.dtable[:0], empty, none).shape == (0, 4, 64)
    # rows without a sequence stay; rows whose sequence has no room see nothing
    q = _query(3, 4, 64, torch.float16, 2).cuda()
    for kw in (dict(), dict(max_new=1), dict(window=3), dict(window=3, max_new=1)):
        out = torch.full_like(q, 7.0)
        binding.prompt_attention(cache, pool.dtable[:0], empty, _ints(0), q, out=out, **kw)
        assert torch.all(out == 7.0)
        binding.prompt_attention(cache, pool.dtable, pool.dlens, _ints(0, 1, 2), q, max_len=0, out=out, **kw)
        assert torch.all(out[:2] == 0) and torch.all(out[2] == 7.0)
        out.fill_(7.0)
        binding.prompt_attention(cache, pool.dtable[:, :0], pool.dlens, _ints(0, 1, 2), q, out=out, **kw)
        assert torch.all(out[:2] == 0) and torch.all(out[2] == 7.0)
    out = binding.prefix_attention(cache, pool.dtable, pool.dlens, _ints(0, 1, 2), pool.dtable, pool.dlens, q[:2], max_prefix=0, max_len=0)
    assert torch.all(out == 0)


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16], ids=str)
def test_shared_pages(gpu, dtype):
    # sequences whose first pages are one another's, and a prefix that is a sequence too
    say(f"[edges] shared pages {dtype}")
    pool = ref.Pool([200, 200, 200], 2, 64, 16, dtype, seed=92)
    for b in (1, 2):
        pool.table[b, :6] = pool.table[0, :6]
    pool.dtable = pool.table.cuda()
    cache = binding.PagedCache(pool.dk, pool.dv)
    news = [80, 3, 1]
    q = _query(84, 4, 64, dtype, 93)
    out = binding.prompt_attention(cache, pool.dtable, pool.dlens, _ints(*_starts(news)), q.cuda()).cpu().double().numpy()
    want, bound, _ = pref.prompt(pool, q, _starts(news), 0.125)
    assert np.all(np.abs(out - want) <= bound)
    far = ref.Pool.__new__(ref.Pool)
    far.__dict__.update(pool.__dict__)
    far.lens, far.table = [96], pool.table[:1]
    out = binding.prefix_attention(cache, pool.dtable[:1], _ints(96), _ints(0, 3), pool.dtable, pool.dlens, q[:3].cuda()).cpu().double().numpy()
    want, bound = pref.prefix(far, pool, [0, 3], q[:3], 0.125)
    assert np.all(np.abs(out - want) <= bound)


def test_graphs_of_one_pool_in_turn(gpu):
    # split calls keep their parts in memory that both graphs hold
    say("[edges] two graphs")
    pools = [ref.Pool([n, 70], 1, 64, 16, seed=94 + n) for n in (3000, 2100)]
    caches = [binding.PagedCache(p.dk, p.dv) for p in pools]
    starts, q = _ints(0, 5, 9), _query(9, 8, 64, torch.float16, 96).cuda()
    calls = [lambda i=i: binding.prompt_attention(caches[i], pools[i].dtable, pools[i].dlens, starts, q) for i in range(2)]
    calls.append(lambda: binding.prefix_attention(caches[0], pools[0].dtable[:1], pools[0].dlens[:1], _ints_kept, pools[0].dtable[1:].expand(9, -1).contiguous(),
                                                  lens_kept, q))
    _ints_kept, lens_kept = _ints(0, 9), _ints(*range(60, 69))
    memory, graphs, outs = torch.cuda.graph_pool_handle(), [], []
    for call in calls:
        call()
    torch.cuda.synchronize()
    for call in calls:
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, pool=memory):
            outs.append(call())
        graphs.append(graph)
    base = q.clone()
    for factor, order in ((1.0, (0, 1, 2)), (-0.5, (2, 1, 0)), (0.25, (1, 0, 2))):
        q.copy_(base * factor)
        want = [call() for call in calls]
        for i in order:
            graphs[i].replay()
            torch.cuda.synchronize()
            assert torch.equal(outs[i], want[i]), (factor, i)


def test_no_heads(gpu):
    say("[edges] no heads, no rows")
    freqs = torch.ones(4, dtype=torch.float64, device="cuda")
    q = _query(3, 2, 8, torch.float16, 97).cuda()
    none = q[:, :0]
    a, b = binding.norm_rotate(none, none, _ints(0, 1, 2), freqs)
    assert a.shape == b.shape == (3, 0, 8)
    a, b = binding.norm_rotate(q[:0], q[:0], _ints(), freqs)
    assert a.shape == (0, 2, 8)
    cache = binding.PagedCache(*(torch.zeros((2, 4, 2, 8), dtype=torch.float16, device="cuda") for _ in range(2)))
    out = binding.norm_rotate_append(cache, torch.empty(0, dtype=torch.int64, device="cuda"), q[:0], q[:0], q[:0], _ints(), freqs)
    assert out.shape == (0, 2, 8) and torch.all(cache.k == 0)
    # keys and values alone
    slots = torch.arange(3, device="cuda")
    out = binding.norm_rotate_append(cache, slots, none, q, q, _ints(0, 0, 0), freqs, eps=None)
    assert out.shape == (3, 0, 8) and torch.equal(cache.k.view(8, 2, 8)[:3], q) and torch.equal(cache.v.view(8, 2, 8)[:3], q)
    assert torch.all(cache.k.view(8, 2, 8)[3:] == 0)
