"""Attention of several new tokens per sequence, through a window, and behind
shared prefixes, against plain 64-bit forms.  Every slot that no sequence holds
is NaN or infinite, so a read past a length shows."""
import numpy as np
import pytest
import torch

from memory_bound_gemv_row_amd import binding

import prompt_ref as pref
import serving_ref as ref
from gpu_util import say

pytestmark = pytest.mark.gpu

HALVES = [torch.float16, torch.bfloat16]
LEFT = 7.0   # what rows of no sequence hold before


def _starts(counts, before=0):
    return [before] + [before + int(n) for n in np.cumsum(counts)]


def _query(rows, heads, dim, dtype, seed, spread=1.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn((rows, heads, dim), generator=g) * spread).to(dtype)


def _check(pool, news, heads, label, window=None, sinks=0, before=0, after=0, max_new=None, max_len=None, stride=0, seed=1,
           scale=None, q=None):
    say(f"[prompt] {label}")
    starts = _starts(news, before)
    rows, dtype = starts[-1] + after, pool.k.dtype
    q = _query(rows, heads, pool.dim, dtype, seed) if q is None else q
    scale = pool.dim ** -0.5 if scale is None else scale
    cache = binding.PagedCache(pool.dk, pool.dv)
    dq = q.cuda()
    if stride:
        wide = torch.full((rows, heads * pool.dim + stride), float("nan"), dtype=dtype, device="cuda")
        wide[:, : heads * pool.dim] = dq.view(rows, -1)
        dq = wide[:, : heads * pool.dim].view(rows, heads, pool.dim)
    out = torch.full((rows, heads, pool.dim), LEFT, dtype=dtype, device="cuda")
    binding.prompt_attention(cache, pool.dtable, pool.dlens, torch.tensor(starts, dtype=torch.int32, device="cuda"), dq,
                             scale=scale, max_len=max_len, max_new=max_new, window=window, sinks=sinks, out=out)
    got = out.cpu().double().numpy()
    want, bound, mine = pref.prompt(pool, q, starts, scale, window, sinks, rounded=(rows if max_new is None else max_new) > 1)
    assert np.all(got[~mine] == LEFT), label
    off = np.abs(got - want)[mine]
    assert np.all(off <= bound[mine]), (label, float(np.nanmax(off / bound[mine])), int(np.isnan(off).sum()))
    return out


# tiles of 64 keys and of 128 rows: lengths and counts about each border
@pytest.mark.parametrize("dtype", HALVES, ids=str)
@pytest.mark.parametrize("n,old", [(1, 0), (2, 0), (2, 61), (3, 62), (17, 0), (31, 33), (32, 32), (33, 31), (63, 1), (64, 0), (65, 0),
                                   (64, 64), (127, 1), (128, 3), (129, 0), (5, 1000), (130, 500), (300, 0)])
def test_counts(gpu, n, old, dtype):
    _check(ref.Pool([n + old], 2, 64, 16, dtype, seed=n), [n], 4, f"{n} after {old} {dtype}")


@pytest.mark.parametrize("dtype", HALVES, ids=str)
@pytest.mark.parametrize("page", [16, 24, 5])
@pytest.mark.parametrize("dim", [8, 16, 40, 64, 72, 80, 96, 104, 120, 128, 136, 192, 248, 256])
def test_head_sizes(gpu, dim, page, dtype):
    _check(ref.Pool([70, 3, 129], 2, dim, page, dtype, seed=dim), [66, 2, 40], 6, f"dim {dim} page {page} {dtype}")


@pytest.mark.parametrize("heads,kv", [(1, 1), (3, 3), (16, 16), (5, 1), (7, 1), (28, 4), (15, 3), (17, 1), (64, 1), (130, 1), (260, 2)])
def test_head_groups(gpu, heads, kv):
    _check(ref.Pool([100, 37], kv, 64, 16, seed=heads), [41, 37], heads, f"{heads} over {kv}")


@pytest.mark.parametrize("page", [1, 3, 8, 12, 16, 17, 24, 32, 48, 64, 100, 256])
@pytest.mark.parametrize("layout", ["slots", "heads", "padded"])
def test_pages_and_layouts(gpu, page, layout):
    _check(ref.Pool([90, 2, 200], 2, 64, page, torch.bfloat16, seed=page, layout=layout), [90, 2, 33], 4, f"page {page} {layout}")


@pytest.mark.parametrize("kv", [1, 3, 4, 8, 16, 24])
def test_every_order_of_workgroups(gpu, kv):
    # sets of workgroups that are a multiple of eight, and others; one part of the keys and several
    for lens, news in (([333, 150], [333, 150]), ([2000, 1300], [5, 3])):
        _check(ref.Pool(lens, kv, 64, 16, seed=kv), news, 2 * kv, f"{kv} heads, {news}")


@pytest.mark.parametrize("kv", [1, 5, 8])
@pytest.mark.parametrize("news", [[300, 290, 137, 299], [310, 0, 300], [300, 3, 1, 0]], ids=str)
def test_row_tiles_in_runs(gpu, kv, news):
    # seventeen row tiles and fewer, of alike and of unlike sequences, one part of the keys and several
    for old in (0, 900):
        _check(ref.Pool([n + old for n in news], kv, 64, 16, seed=kv), news, 7 * kv, f"{kv} heads, {news} after {old}")


@pytest.mark.parametrize("lens,news", [
    ([0, 5000, 3, 700, 64, 1], [2, 3, 3, 0, 1, 1]),
    ([9000, 65, 64, 63], [4, 2, 0, 4]),
    ([1, 1, 0, 2], [1, 2, 3, 0]),
    ([(i * 131) % 1700 for i in range(64)], [i % 4 for i in range(64)]),
    ([(i * 131) % 700 for i in range(65)], [i % 4 for i in range(65)]),
], ids=["empty", "one long", "short", "64", "65"])
@pytest.mark.parametrize("kv,dim", [(1, 64), (3, 256), (8, 128)])
def test_few_new_tokens_of_unlike_sequences(gpu, lens, news, kv, dim):
    # tables with room for 9000 slots whatever the lengths are: several parts of the keys, shared out by the lengths
    pool = ref.Pool(lens, kv, dim, 16, torch.bfloat16, seed=kv)
    pool.dtable = torch.cat([pool.dtable, pool.dtable[:, :1].expand(-1, 563 - pool.width)], 1).contiguous()
    _check(pool, news, 4 * kv, f"{kv} heads of {dim}, {news}", before=1, after=2, max_new=max(news))


def test_long_prompts(gpu):
    """20000 slots, 2500 new tokens; a sample of rows against the plain form."""
    pool = ref.Pool([20000], 1, 128, 16, torch.bfloat16, seed=31)
    q = _query(2500, 4, 128, torch.bfloat16, 31)
    cache = binding.PagedCache(pool.dk, pool.dv)
    starts = torch.tensor([0, 2500], dtype=torch.int32, device="cuda")
    k, _ = ref.gathered(pool, pool.k, 0, 20000)
    v, _ = ref.gathered(pool, pool.v, 0, 20000)
    sample = np.array([0, 1, 31, 32, 63, 64, 100, 1023, 1024, 1700, 2047, 2400, 2498, 2499])
    half, low = pref._power_errors(torch.bfloat16)
    for window, sinks in ((None, 0), (4096, 4), (1000, 0)):
        say(f"[prompt] 2500 of 20000, window {window}")
        got = binding.prompt_attention(cache, pool.dtable, pool.dlens, starts, q.cuda(), window=window, sinks=sinks).cpu()
        sees = pref.seen(2500, 20000, window, sinks)[sample]
        for h in range(4):
            want, bound = pref.attend(k[0], v[0], q[sample, h].double().numpy(), sees, 128 ** -0.5, np.full(20000, half), low)
            off = np.abs(got[sample, h].double().numpy() - want)
            assert np.all(off <= pref.stored(want, bound, torch.bfloat16)), (window, h)


def test_ragged_batch_with_empty_sequences(gpu):
    lens, news = [0, 500, 5, 0, 33, 257, 9, 64], [0, 70, 5, 0, 33, 0, 1, 64]
    _check(ref.Pool(lens, 2, 128, 16, seed=3, width=40), news, 8, "ragged", before=3, after=5, stride=64)


def test_many_sequences(gpu):
    # more than a wave finds at once, several without new tokens
    rng = np.random.default_rng(4)
    news = rng.integers(0, 4, 300)
    news[::7] = 0
    _check(ref.Pool(news + rng.integers(0, 30, 300), 2, 64, 8, seed=4), news, 4, "300 sequences", after=2)


def test_more_new_tokens_than_the_sequence_holds(gpu):
    _check(ref.Pool([10, 0, 40], 1, 64, 16, seed=5, width=4), [30, 5, 40], 4, "tokens before the first slot")


def test_only_the_last_max_new_rows(gpu):
    pool = ref.Pool([90, 60], 2, 64, 16, seed=6)
    say("[prompt] the last max_new rows")
    q = _query(90, 4, 64, torch.float16, 6)
    cache = binding.PagedCache(pool.dk, pool.dv)
    starts = torch.tensor([0, 50, 90], dtype=torch.int32, device="cuda")
    full = binding.prompt_attention(cache, pool.dtable, pool.dlens, starts, q.cuda())
    for most in (1, 2, 33):
        out = torch.full_like(full, LEFT)
        binding.prompt_attention(cache, pool.dtable, pool.dlens, starts, q.cuda(), max_new=most, out=out)
        mine = torch.zeros(90, dtype=torch.bool)
        mine[50 - most: 50] = mine[90 - most:] = True
        assert torch.all(out.cpu()[~mine] == LEFT)
        want, bound, _ = pref.prompt(pool, q, [0, 50, 90], 0.125, rounded=most > 1)
        off = np.abs(out.cpu().double().numpy() - want)[mine.numpy()]
        assert np.all(off <= bound[mine.numpy()]), most


@pytest.mark.parametrize("dtype", HALVES, ids=str)
@pytest.mark.parametrize("window,sinks", [(1, 0), (1, 1), (2, 5), (16, 0), (63, 64), (64, 65), (65, 3), (100, 16), (128, 0), (400, 4),
                                          (1000, 7), (40, 1000)])
@pytest.mark.parametrize("news", [[1, 1, 1], [300, 2, 90]], ids=["newest", "several"])
def test_windows(gpu, news, window, sinks, dtype):
    for page in (16, 24):
        _check(ref.Pool([500, 66, 90], 2, 64, page, dtype, seed=window), news, 8, f"window {window} sinks {sinks} page {page} {dtype}",
               window=window, sinks=sinks, max_new=max(news))


@pytest.mark.parametrize("dim", [64, 80, 128, 256])
def test_windows_over_head_sizes(gpu, dim):
    for news in ([1, 1], [1, 0], [130, 3]):
        _check(ref.Pool([700, 301], 2, dim, 16, seed=dim), news, 8, f"window, dim {dim}, new {news}", window=200, sinks=4,
               max_new=max(news))


@pytest.mark.parametrize("window,sinks", [(70, 3), (1000, 0), (5000, 4)])
def test_windows_of_paged_attention(gpu, window, sinks):
    # one query per sequence without starts, out in place, rows apart
    pool = ref.Pool([0, 3000, 1, 900], 2, 128, 16, torch.bfloat16, seed=window, width=200)
    q = _query(4, 8, 128, torch.bfloat16, 2)
    say(f"[window] {window} {sinks}")
    cache = binding.PagedCache(pool.dk, pool.dv)
    want, bound, _ = pref.prompt(pool, q, [0, 1, 2, 3, 4], 128 ** -0.5, window, sinks, rounded=False)
    out = binding.paged_attention(cache, pool.dtable, pool.dlens, q.cuda(), window=window, sinks=sinks)
    assert np.all(np.abs(out.cpu().double().numpy() - want) <= bound)
    place = q.cuda()
    assert torch.equal(binding.paged_attention(cache, pool.dtable, pool.dlens, place, window=window, sinks=sinks, out=place), out)


    assert out[0].abs().max() == 0


def test_a_window_past_every_length_is_none(gpu):
    pool = ref.Pool([300, 77], 2, 64, 16, seed=8)
    q = _query(2, 4, 64, torch.float16, 8).cuda()
    say("[window] past every length")
    cache = binding.PagedCache(pool.dk, pool.dv)
    plain = binding.paged_attention(cache, pool.dtable, pool.dlens, q)
    for window in (400, (1 << 31) - 1):
        assert torch.equal(binding.paged_attention(cache, pool.dtable, pool.dlens, q, window=window, sinks=3), plain)


def test_long_keys_few_rows(gpu):
    # the keys are split over workgroups, and the parts joined
    for dtype in HALVES:
        _check(ref.Pool([5000, 4097], 1, 64, 32, dtype, seed=9), [7, 2], 4, f"few rows {dtype}")
        _check(ref.Pool([5000, 4097, 100], 2, 128, 16, dtype, seed=9), [7, 0, 3], 8, f"few rows {dtype}", after=4, before=2)


def test_in_place(gpu):
    for lens, news in (([5000, 4097], [7, 2]), ([300, 200], [300, 100])):
        pool = ref.Pool(lens, 2, 64, 16, seed=10)
        starts = torch.tensor(_starts(news), dtype=torch.int32, device="cuda")
        q = _query(sum(news), 4, 64, torch.float16, 10).cuda()
        say("[prompt] in place")
        cache = binding.PagedCache(pool.dk, pool.dv)
        out = binding.prompt_attention(cache, pool.dtable, pool.dlens, starts, q)
        assert torch.equal(binding.prompt_attention(cache, pool.dtable, pool.dlens, starts, q, out=q), out)


def test_holes(gpu):
    for page in (16, 12):
        pool = ref.Pool([200, 70, 48], 2, 64, page, seed=5)
        for b, i, p in ((0, 3, -1), (0, 11, 1 << 30), (1, 0, pool.k.shape[0])):
            pool.table[b, i] = p
        pool.table[2] = -5
        pool.dtable = pool.table.cuda()
        out = _check(pool, [90, 70, 48], 4, f"holes, pages of {page}")
        assert torch.all(out[160:] == 0)
        _check(pool, [90, 70, 48], 4, f"holes, pages of {page}", window=50, sinks=2)
        _check(pool, [1, 1, 1], 4, f"holes, pages of {page}", window=50, sinks=2, max_new=1)


def test_lengths_are_cut_to_the_room(gpu):
    pool = ref.Pool([96, 96, 96], 2, 64, 16, seed=6)
    q = _query(30, 4, 64, torch.float16, 6).cuda()
    cache = binding.PagedCache(pool.dk, pool.dv)
    starts = torch.tensor([0, 10, 20, 30], dtype=torch.int32, device="cuda")
    full = binding.prompt_attention(cache, pool.dtable, pool.dlens, starts, q)
    wild = torch.tensor([1 << 30, -7, 96], dtype=torch.int32, device="cuda")
    say("[prompt] lengths outside the room")
    out = binding.prompt_attention(cache, pool.dtable, wild, starts, q)
    assert torch.equal(out[:10], full[:10]) and torch.all(out[10:20] == 0) and torch.equal(out[20:], full[20:])
    # starts outside the rows are taken as at most those
    out = torch.full_like(full, LEFT)
    binding.prompt_attention(cache, pool.dtable, pool.dlens, torch.tensor([-4, 10, 20, 1 << 30], dtype=torch.int32, device="cuda"), q,
                             out=out)
    assert torch.equal(out, full)


@pytest.mark.parametrize("spread", [0.0, 8.0, 40.0])
def test_flat_and_peaked_softmax(gpu, spread):
    pool = ref.Pool([700, 333], 2, 64, 16, torch.bfloat16, seed=7, spread=max(spread, 1e-3))
    _check(pool, [100, 333], 4, f"spread {spread}", q=_query(433, 4, 64, torch.bfloat16, 7, spread / 4))


def test_negative_and_zero_scale(gpu):
    pool = ref.Pool([300, 90], 2, 64, 16, seed=11)
    for scale in (-0.3, 0.0, 1e-30):
        _check(pool, [200, 3], 4, f"scale {scale}", scale=scale)


def test_rising_logits(gpu):
    pool = ref.Pool([400], 1, 64, 16, seed=8)
    for j in range(400):
        pool.k[pool.table[0, j // 16], j % 16, 0] = j / 16.0
    pool.dk = pool.k.cuda()
    q = torch.full((300, 2, 64), 1.0, dtype=torch.float16)
    q[:, 1] = -1.0
    _check(pool, [300], 2, "rising and falling", q=q)


@pytest.mark.parametrize("dtype", HALVES, ids=str)
@pytest.mark.parametrize("dim,page", [(64, 16), (64, 24), (64, 5), (96, 16), (128, 16), (200, 16), (256, 16)])
def test_what_a_row_does_not_see_does_not_touch_it(gpu, dim, page, dtype):
    # NaN and infinities in keys and values of later tokens, and of those before the window
    lens, news = [200, 150], [150, 150]
    for window, sinks in ((None, 0), (40, 2)):
        pool = ref.Pool(lens, 1, dim, page, dtype, seed=12)
        q = _query(300, 2, dim, dtype, 12)
        bad = {0: (60, 100, 199), 1: (0, 33, 149)}
        for b, slots in bad.items():
            for i, j in enumerate(slots):
                pool.dv[pool.table[b, j // page], j % page, 0, i::7] = (float("nan"), float("inf"), -float("inf"))[i]
                if i == 1:
                    pool.dk[pool.table[b, j // page], j % page] = float("nan")
        say(f"[prompt] unseen NaN, window {window}")
        cache = binding.PagedCache(pool.dk, pool.dv)
        out = binding.prompt_attention(cache, pool.dtable, pool.dlens, torch.tensor([0, 150, 300], dtype=torch.int32, device="cuda"),
                                       q.cuda(), window=window, sinks=sinks).cpu().double().numpy()
        want, bound, _ = pref.prompt(pool, q, [0, 150, 300], dim ** -0.5, window, sinks)   # of the finite pool
        for b in range(2):
            sees = pref.seen(150, lens[b], window, sinks)
            for t in range(150):
                row, w = out[150 * b + t], want[150 * b + t]
                nan_key = sees[t, bad[b][1]]
                if nan_key:
                    assert np.all(np.isnan(row)), (b, t)
                    continue
                cols = np.zeros(dim, bool)
                for i, j in enumerate(bad[b]):
                    if sees[t, j]:
                        cols[i::7] = True
                assert np.all(~np.isfinite(row[:, cols])), (b, t)
                assert np.all(np.abs(row - w)[:, ~cols] <= bound[150 * b + t][:, ~cols]), (b, t)


def test_seen_infinities_are_infinite(gpu):
    pool = ref.Pool([90], 1, 64, 16, seed=13)
    pool.dv[pool.table[0, 20 // 16], 20 % 16, 0, 7] = float("inf")
    pool.dv[pool.table[0, 80 // 16], 80 % 16, 0, 9] = -float("inf")
    say("[prompt] infinite values")
    out = binding.prompt_attention(binding.PagedCache(pool.dk, pool.dv), pool.dtable, pool.dlens,
                                   torch.tensor([0, 40], dtype=torch.int32, device="cuda"), _query(40, 2, 64, torch.float16, 13).cuda())
    assert torch.all(out[:, :, 7] == float("inf"))
    assert torch.all(out[30:, :, 9] == -float("inf")) and torch.all(torch.isfinite(out[:30, :, 9]))


def test_keys_of_the_lowest_logit_weigh_nothing(gpu):
    for dtype in HALVES:
        pool = ref.Pool([140], 1, 64, 16, dtype, seed=12)
        for j in (0, 5, 40, 139):
            pool.k[pool.table[0, j // 16], j % 16, 0] = -65504.0
        pool.k[pool.table[0, 1], 3] = -float("inf")
        pool.dk = pool.k.cuda()
        _check(pool, [100], 2, f"lowest logits {dtype}", q=torch.ones((100, 2, 64), dtype=dtype), scale=0.125)


def test_a_row_without_a_logit_above_minus_infinity(gpu):
    pool = ref.Pool([80], 1, 64, 16, seed=14)
    pool.k[:] = -float("inf")
    pool.dk = pool.k.cuda()
    say("[prompt] every logit -inf")
    out = binding.prompt_attention(binding.PagedCache(pool.dk, pool.dv), pool.dtable, pool.dlens,
                                   torch.tensor([0, 80], dtype=torch.int32, device="cuda"), torch.ones((80, 2, 64), dtype=torch.float16).cuda())
    assert torch.all(out == 0)


def test_offsets_past_32_bits(gpu):
    pages, page, heads, dim = 8600, 64, 32, 128
    k = torch.zeros((pages, page, heads, dim), dtype=torch.float16, device="cuda")
    v = torch.zeros_like(k)
    table = torch.tensor([[0, pages - 1], [pages - 2, 5]], dtype=torch.int32)
    g = torch.Generator().manual_seed(2)
    for p in table.ravel().tolist():
        k[p] = torch.randn((page, heads, dim), generator=g).to(torch.float16).cuda()
        v[p] = torch.randn((page, heads, dim), generator=g).to(torch.float16).cuda()
    assert k.numel() > 1 << 31
    say("[prompt] offsets past 2^31 elements")
    q = _query(70, 32, 128, torch.float16, 2).cuda()
    rows = table.ravel().long().cuda()
    lens = torch.tensor([100, 128], dtype=torch.int32, device="cuda")
    starts = torch.tensor([0, 50, 70], dtype=torch.int32, device="cuda")
    near = binding.PagedCache(k[rows].contiguous(), v[rows].contiguous())
    small = torch.tensor([[0, 1], [2, 3]], dtype=torch.int32, device="cuda")
    far = binding.PagedCache(k, v)
    out = binding.prompt_attention(far, table.cuda(), lens, starts, q)
    same = binding.prompt_attention(near, small, lens, starts, q)
    assert torch.equal(out, same) and torch.all(torch.isfinite(out)) and out.abs().max() > 0
    out = binding.paged_attention(far, table.cuda(), lens, q[:2].contiguous(), window=70, sinks=3)
    assert torch.equal(out, binding.paged_attention(near, small, lens, q[:2].contiguous(), window=70, sinks=3))


# ---------------------------------------------------------------- shared prefixes
def _pools(far_lens, lens, kv, dim, page, dtype, seed):
    """One pool that holds the prefixes and the sequences, as two tables over it."""
    both = ref.Pool(list(far_lens) + list(lens), kv, dim, page, dtype, seed=seed)
    views = []
    for first, n in ((0, len(far_lens)), (len(far_lens), len(lens))):
        view = ref.Pool.__new__(ref.Pool)
        view.__dict__.update(both.__dict__)
        view.lens = both.lens[first: first + n]
        view.table = both.table[first: first + n]
        view.dtable = view.table.cuda()
        view.dlens = torch.tensor(view.lens, dtype=torch.int32, device="cuda")
        views.append(view)
    return both, *views


def _check_prefix(far_lens, groups, lens, kv, heads, dim, page, dtype, label, seed=1, **kw):
    say(f"[prefix] {label}")
    both, far, near = _pools(far_lens, lens, kv, dim, page, dtype, seed)
    q = _query(len(lens), heads, dim, dtype, seed)
    cache = binding.PagedCache(both.dk, both.dv)
    out = binding.prefix_attention(cache, far.dtable, far.dlens, torch.tensor(groups, dtype=torch.int32, device="cuda"), near.dtable,
                                   near.dlens, q.cuda(), **kw)
    want, bound = pref.prefix(far, near, groups, q, dim ** -0.5)
    off = np.abs(out.cpu().double().numpy() - want)
    assert np.all(off <= bound), (label, float(np.nanmax(off / bound)), int(np.isnan(off).sum()))
    return out


@pytest.mark.parametrize("dtype", HALVES, ids=str)
@pytest.mark.parametrize("far,own", [(1, 1), (63, 1), (64, 17), (65, 300), (500, 0), (0, 40), (2000, 3), (777, 777)])
def test_prefix_lengths(gpu, far, own, dtype):
    _check_prefix([far], [0, 5], [own, 1, max(own - 1, 0), 7, own], 2, 8, 64, 16, dtype, f"{far} and {own} {dtype}")


@pytest.mark.parametrize("dim", [8, 64, 80, 96, 128, 200, 256])
@pytest.mark.parametrize("page", [16, 24])
def test_prefix_head_sizes(gpu, dim, page):
    _check_prefix([150, 20], [0, 2, 4], [70, 3, 9, 0], 2, 6, dim, page, torch.bfloat16, f"dim {dim} page {page}")


@pytest.mark.parametrize("heads,kv", [(1, 1), (7, 1), (28, 4), (64, 2), (130, 1)])
def test_prefix_head_groups(gpu, heads, kv):
    _check_prefix([130], [0, 3], [20, 0, 33], kv, heads, 64, 16, torch.float16, f"{heads} over {kv}")


def test_groups(gpu):
    # empty groups, groups without a prefix, sequences of no group, and neither prefix nor tokens
    lens = [30, 0, 5, 64, 1, 0, 12, 200, 0]
    out = _check_prefix([100, 7, 0, 300], [1, 3, 3, 5, 8], lens, 2, 8, 64, 16, torch.float16, "groups")
    assert torch.all(out[8] == 0)
    _check_prefix([100], [0, 0], lens, 2, 8, 64, 16, torch.float16, "one group of none")


def test_many_prefixed_sequences(gpu):
    rng = np.random.default_rng(3)
    _check_prefix([900, 333], [0, 60, 100], rng.integers(0, 50, 100), 1, 4, 64, 16, torch.bfloat16, "100 sequences, tiles of rows")


def test_prefix_limits(gpu):
    # the longest lengths named by the host, and no groups at all
    _check_prefix([300, 200], [0, 3, 4], [20, 90, 3, 4], 2, 4, 128, 16, torch.float16, "limits", max_prefix=300, max_len=90)
    both, far, near = _pools([10], [20, 30], 2, 64, 16, torch.float16, 5)
    q = _query(2, 4, 64, torch.float16, 5).cuda()
    say("[prefix] no groups")
    cache = binding.PagedCache(both.dk, both.dv)
    out = binding.prefix_attention(cache, far.dtable[:0], far.dlens[:0], torch.zeros(1, dtype=torch.int32, device="cuda"), near.dtable,
                                   near.dlens, q)
    want, bound, _ = pref.prompt(near, q.cpu(), [0, 1, 2], 0.125, rounded=False)
    assert np.all(np.abs(out.cpu().double().numpy() - want) <= bound)
    place = q.clone()
    binding.prefix_attention(cache, far.dtable, far.dlens, torch.tensor([0, 1], dtype=torch.int32, device="cuda"), near.dtable, near.dlens,
                             place, out=place)
    assert torch.equal(place, binding.prefix_attention(cache, far.dtable, far.dlens,
                                                       torch.tensor([0, 1], dtype=torch.int32, device="cuda"), near.dtable, near.dlens, q))


def test_a_prefix_is_as_if_it_were_each_sequences_own(gpu):
    # the same tokens by one table per sequence, within both bounds
    both, far, near = _pools([160], [32, 48, 16], 2, 128, 16, torch.float16, 9)
    q = _query(3, 8, 128, torch.float16, 9)
    say("[prefix] against whole tables")
    cache = binding.PagedCache(both.dk, both.dv)
    out = binding.prefix_attention(cache, far.dtable, far.dlens, torch.tensor([0, 3], dtype=torch.int32, device="cuda"), near.dtable,
                                   near.dlens, q.cuda())
    table = torch.cat([far.dtable[:, :10].expand(3, 10), near.dtable], 1).contiguous()
    whole = binding.paged_attention(cache, table, near.dlens + 160, q.cuda())
    _, bound = pref.prefix(far, near, [0, 3], q, 128 ** -0.5)
    assert np.all((out.double() - whole.double()).abs().cpu().numpy() <= 2 * bound)


# ---------------------------------------------------------------- streams and graphs
def _calls():
    pool = ref.Pool([900, 40, 333], 2, 64, 16, seed=21)
    both, far, near = _pools([500], [30, 41], 2, 64, 16, torch.float16, 22)
    cache, shared = binding.PagedCache(pool.dk, pool.dv), binding.PagedCache(both.dk, both.dv)
    q = _query(500, 8, 64, torch.float16, 21).cuda()
    t = lambda *v: torch.tensor(v, dtype=torch.int32, device="cuda")
    few, all_rows, groups = t(0, 5, 6, 9), t(0, 400, 420, 500), t(0, 2)
    return [
        ("window", lambda **kw: binding.paged_attention(cache, pool.dtable, pool.dlens, q[:3], window=300, sinks=4, **kw)),
        ("few rows", lambda **kw: binding.prompt_attention(cache, pool.dtable, pool.dlens, few, q[:9], **kw)),
        ("prompt", lambda **kw: binding.prompt_attention(cache, pool.dtable, pool.dlens, all_rows, q, **kw)),
        ("prefix", lambda **kw: binding.prefix_attention(shared, far.dtable, far.dlens, groups, near.dtable, near.dlens, q[:2], **kw)),
    ], q


def test_calls_on_another_stream_and_in_graphs(gpu):
    calls, q = _calls()
    side = torch.cuda.Stream()
    for name, call in calls:
        say(f"[streams] {name}")
        want = call()
        torch.cuda.synchronize()
        other = call(stream=side)
        side.synchronize()
        assert torch.equal(other, want), name
    graph, outs = torch.cuda.CUDAGraph(), []
    with torch.cuda.graph(graph):
        for _, call in calls:
            outs.append(call())
    base = q.clone()
    for factor in (1.0, 0.5, -1.0):
        q.copy_(base * factor)
        graph.replay()
        torch.cuda.synchronize()
        for (name, call), out in zip(calls, outs):
            assert torch.equal(out, call()), (name, factor)


def test_two_calls_at_once(gpu):
    calls, _ = _calls()
    streams = [torch.cuda.Stream() for _ in range(2)]
    want = [call() for _, call in calls]
    torch.cuda.synchronize()
    say("[streams] two at once")
    got = [[call(stream=s) for s in streams] for _, call in calls]
    torch.cuda.synchronize()
    for w, pair in zip(want, got):
        assert torch.equal(pair[0], w) and torch.equal(pair[1], w)
