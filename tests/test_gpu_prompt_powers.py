"""Attention of several new tokens, and behind prefixes, where many keys have small
weights beside a large one: against plain 64-bit forms, with bounds that count a
power's error by the largest power of its row."""
import numpy as np
import pytest
import torch

from memory_bound_gemv_row_amd import binding

import prompt_ref as pref
import serving_ref as ref
from gpu_util import say
from test_gpu_prompt import _pools, _query

pytestmark = pytest.mark.gpu

HALVES = [torch.float16, torch.bfloat16]
# What a power may be off by besides half a step, of its row's largest power: binary16
# holds them raised by 2^7, so half its least step is 2^-25 / 2^7 of the largest.
LOWEST = {torch.float16: 2.0 ** -32, torch.bfloat16: 2.0 ** -133}


def _normaliser(k, q, sees, scale):
    """Sum of the powers of each row, of its largest [R, 1]."""
    x = np.where(sees, (q @ k.T) * scale, -np.inf)
    return np.exp(x - x.max(-1, keepdims=True)).sum(-1, keepdims=True)


def _attend(k, v, q, sees, scale, dtype, rounding=None):
    """(out, bound) of rows q in the type: prompt_ref.attend, whose last argument is of a
    probability, with the powers' least error brought to one."""
    half = pref.HALF_STEP[dtype]
    rounding = np.full(len(k), half) if rounding is None else rounding
    out, bound = pref.attend(k, v, q, sees, scale, rounding, LOWEST[dtype] / _normaliser(k, q, sees, scale))
    return out, pref.stored(out, bound, dtype)


def _sink(pool, b, gap, values=0.0):
    """The first token of sequence b `gap` above the others' mean logit for queries that
    begin with 8 in heads of 64, and its value."""
    page = int(pool.table[b, 0])
    pool.k[page, 0, :, 0], pool.k[page, 0, :, 1:] = gap, 0
    pool.v[page, 0] = values


def _others(pool, b, seed):
    """Keys whose logits are about 0.3 apart, and values about 1."""
    g = torch.Generator().manual_seed(seed)
    pages, n = pool.table[b].long(), pool.lens[b]
    for t, mean, spread in ((pool.k, 0.0, 0.3), (pool.v, 1.0, 0.5)):
        rows = (torch.randn((len(pages) * pool.page, pool.heads, pool.dim), generator=g) * spread + mean).to(t.dtype)
        if t is pool.k:
            rows[..., 0] = 0
        rows[n:] = float("nan")
        t[pages] = rows.view(len(pages), pool.page, pool.heads, pool.dim)


def _rows_for_sink(rows, heads, dtype, seed):
    q = _query(rows, heads, 64, dtype, seed)
    q[..., 0] = 8
    return q


def _empty_pool(lens, heads, page, dtype):
    """A pool whose held slots are to be filled: quick to make at any length."""
    pool = ref.Pool([0] * len(lens), heads, 64, page, dtype, width=max(-(-n // page) for n in lens))
    pool.lens = [int(n) for n in lens]
    pool.dlens = torch.tensor(pool.lens, dtype=torch.int32, device="cuda")
    return pool


@pytest.mark.parametrize("dtype", HALVES, ids=str)
@pytest.mark.parametrize("gap", [8.0, 12.0, 15.0, 16.0, 17.0, 17.5, 19.0, 21.0])
@pytest.mark.parametrize("n,old,heads,window,sinks", [(1200, 18800, 64, None, 0), (2, 39998, 2, None, 0), (1200, 12000, 64, 9000, 4)],
                         ids=["prompt", "draft", "window"])
def test_a_first_token_far_above_the_others(gpu, n, old, heads, window, sinks, gap, dtype):
    say(f"[prompt] {n} after {old}, first token {gap} above, {dtype}")
    pool = _empty_pool([n + old], 1, 16, dtype)
    _others(pool, 0, 61)
    _sink(pool, 0, gap)
    pool.dk, pool.dv = pool.k.cuda(), pool.v.cuda()
    q = _rows_for_sink(n, heads, dtype, 62)
    cache = binding.PagedCache(pool.dk, pool.dv)
    out = binding.prompt_attention(cache, pool.dtable, pool.dlens, torch.tensor([0, n], dtype=torch.int32, device="cuda"), q.cuda(),
                                   window=window, sinks=sinks).cpu().double().numpy()
    # one maximum for all keys, of which a row's are at least 9000: they are not split
    assert n == 2 or list(cache._needs.values()) == [0]
    k, v = (ref.gathered(pool, p, 0, n + old)[0][0] for p in (pool.k, pool.v))
    sample = np.unique(np.array([0, 1, n // 3, n - 1]))
    sees = pref.seen(n, n + old, window, sinks)[sample]
    for h in (0, heads - 1):
        want, bound = _attend(k, v, q[sample, h].double().numpy(), sees, 0.125, dtype)
        off = np.abs(out[sample, h] - want)
        assert np.all(off <= bound), (gap, dtype, float((off / bound).max()), want[0, :2], out[sample[0], h, :2])


@pytest.mark.parametrize("dtype", HALVES, ids=str)
@pytest.mark.parametrize("gap", [12.0, 16.0, 17.5, 20.0])
def test_a_prefix_whose_first_token_is_far_above(gpu, gap, dtype):
    # many rows, so that few parts share the prefix; every sequence has the same token of its own
    say(f"[prefix] 20000, first token {gap} above, {dtype}")
    pool = _empty_pool([20000, 1], 1, 16, dtype)
    for b in range(2):
        _others(pool, b, 63 + b)
    _sink(pool, 0, gap)
    pool.dk, pool.dv = pool.k.cuda(), pool.v.cuda()
    q = _rows_for_sink(128, 128, dtype, 67)
    t = lambda *x: torch.tensor(x, dtype=torch.int32, device="cuda")
    out = binding.prefix_attention(binding.PagedCache(pool.dk, pool.dv), pool.dtable[:1], pool.dlens[:1], t(0, 128),
                                   pool.dtable[1:].expand(128, -1).contiguous(), pool.dlens[1:].expand(128).contiguous(), q.cuda(),
                                   max_len=16).cpu().double().numpy()
    k, v = (np.concatenate([ref.gathered(pool, p, b, pool.lens[b])[0][0] for b in range(2)]) for p in (pool.k, pool.v))
    for b in (0, 77, 127):
        rows = q[b, ::41].double().numpy()
        want, bound = _attend(k, v, rows, np.ones((len(rows), len(k)), bool), 0.125, dtype)
        off = np.abs(out[b, ::41] - want)
        assert np.all(off <= bound), (gap, dtype, b, float((off / bound).max()))


@pytest.mark.parametrize("dtype", HALVES, ids=str)
def test_long_prompts(gpu, dtype):
    """20000 slots, 2500 new tokens; a sample of rows against the plain form."""
    pool = _empty_pool([20000], 1, 16, dtype)
    g = torch.Generator().manual_seed(68)
    pool.k[pool.table[0].long()], pool.v[pool.table[0].long()] = (
        torch.randn((1250, 16, 1, 64), generator=g).to(dtype) for _ in range(2))
    pool.dk, pool.dv = pool.k.cuda(), pool.v.cuda()
    q = _query(2500, 4, 64, dtype, 69)
    starts = torch.tensor([0, 2500], dtype=torch.int32, device="cuda")
    k, v = (ref.gathered(pool, p, 0, 20000)[0][0] for p in (pool.k, pool.v))
    sample = np.array([0, 1, 31, 32, 63, 64, 100, 1023, 1024, 1700, 2047, 2400, 2498, 2499])
    for window, sinks in ((None, 0), (4096, 4), (1000, 0)):
        say(f"[prompt] 2500 of 20000, window {window} {dtype}")
        got = binding.prompt_attention(binding.PagedCache(pool.dk, pool.dv), pool.dtable, pool.dlens, starts, q.cuda(), window=window,
                                       sinks=sinks).cpu().double().numpy()
        sees = pref.seen(2500, 20000, window, sinks)[sample]
        for h in range(4):
            want, bound = _attend(k, v, q[sample, h].double().numpy(), sees, 0.125, dtype)
            assert np.all(np.abs(got[sample, h] - want) <= bound), (window, h)


@pytest.mark.parametrize("dtype", HALVES, ids=str)
@pytest.mark.parametrize("dim,page", [(64, 16), (80, 24), (128, 16), (256, 16)])
@pytest.mark.parametrize("spread", [0.0, 2.0, 8.0, 40.0])
def test_flat_and_peaked_softmax(gpu, spread, dim, page, dtype):
    lens, news, starts = [700, 333], [100, 333], [0, 100, 433]
    say(f"[prompt] spread {spread}, heads of {dim}, {dtype}")
    pool = ref.Pool(lens, 1, dim, page, dtype, seed=7, spread=max(spread, 1e-3))
    q = _query(433, 2, dim, dtype, 7, spread / 4)
    out = binding.prompt_attention(binding.PagedCache(pool.dk, pool.dv), pool.dtable, pool.dlens,
                                   torch.tensor(starts, dtype=torch.int32, device="cuda"), q.cuda()).cpu().double().numpy()
    for b in range(2):
        k, v = (ref.gathered(pool, p, b, lens[b])[0][0] for p in (pool.k, pool.v))
        mine = slice(starts[b], starts[b + 1])
        for h in range(2):
            want, bound = _attend(k, v, q[mine, h].double().numpy(), pref.seen(news[b], lens[b]), dim ** -0.5, dtype)
            assert np.all(np.abs(out[mine, h] - want) <= bound), (spread, dim, b, h)
