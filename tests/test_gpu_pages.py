"""Pages for new tokens, and pages given back, against whole numbers row by row."""
import numpy as np
import pytest
import torch

from memory_bound_gemv_row_amd import binding

import between_ref as bref
import prompt_ref as pref
import serving_ref as ref
from gpu_util import say

pytestmark = pytest.mark.gpu


def _ints(v, dtype=torch.int32):
    return torch.tensor(np.asarray(v, np.int64), dtype=dtype, device="cuda")


def _state(lens, page, width, spare, seed):
    """(free, count, table, pages): tables that hold the lengths, the rest of the pool on the stack."""
    rng = np.random.default_rng(seed)
    held = [min(-(-max(0, n) // page), width) for n in lens]
    pages = sum(held) + spare
    order = rng.permutation(pages)
    table, at = np.full((len(lens), width), -1, np.int64), 0
    for b, n in enumerate(held):
        table[b, :n] = order[at: at + n]
        at += n
    free = np.concatenate([order[at:], np.zeros(at, np.int64)])
    return free, spare, table, pages


def _reserve(lens, added, page, width, spare, label, rows=None, seed=1, stride=0, free=None, count=None):
    say(f"[reserve] {label}")
    f, c, table, pages = _state(lens, page, width, spare, seed)
    free, count = f if free is None else free, c if count is None else count
    rows = int(sum(max(0, n) for n in added)) if rows is None else rows
    B = len(lens)
    wide = torch.full((B, width + stride), -9, dtype=torch.int32, device="cuda")
    wide[:, :width] = _ints(table).view(B, width)
    df, dc = _ints(free), _ints([count, 77])
    got = binding.reserve_pages(df, dc, wide[:, :width], _ints(lens), _ints(added), page, rows)
    want = bref.reserve(free, count, table, lens, added, page, rows, pages)
    for g, w, name in zip(got, want, ("count", "lens", "starts", "positions", "slots")):
        assert g.cpu().tolist() == list(w), (label, name)
    assert np.array_equal(wide[:, :width].cpu().numpy(), want[5]), label
    assert torch.all(wide[:, width:] == -9)
    assert df.cpu().tolist() == [int(p) for p in free] and dc.cpu().tolist() == [count, 77]
    return got


@pytest.mark.parametrize("page", [1, 2, 16, 24, 128])
def test_decode_steps(gpu, page):
    rng = np.random.default_rng(page)
    for B in (1, 2, 63, 64, 65, 511, 512, 513, 1500):
        lens = rng.integers(0, 200, B)
        _reserve(lens, np.ones(B, int), page, 300 // page + 2, B, f"{B} sequences, pages of {page}", stride=3)


@pytest.mark.parametrize("page", [1, 5, 16, 64])
@pytest.mark.parametrize("counts", [[0], [1], [2047], [2048], [2049], [5000], [100, 0, 0, 7000, 1, 2048, 0], [0, 0, 0]], ids=str)
def test_prompts(gpu, counts, page):
    rng = np.random.default_rng(len(counts))
    lens = rng.integers(0, 40, len(counts))
    width = (max(counts) + 40) // page + 2
    _reserve(lens, counts, page, width, sum(counts) // page + 2 * len(counts), f"{counts}, pages of {page}")
    _reserve(lens, counts, page, width, sum(counts) // page // 2, f"{counts}, pages of {page}, too few")
    _reserve(lens, counts, page, width, 0, f"{counts}, pages of {page}, none")


def test_more_rows_and_fewer(gpu):
    counts, lens = [10, 0, 300, 7], [3, 16, 0, 90]
    for rows in (317, 318, 400, 3000, 316, 310, 10, 9, 1, 0):
        _reserve(lens, counts, 16, 30, 60, f"{rows} rows", rows=rows)
    many = np.full(1300, 3)
    for rows in (3900, 3899, 1536, 1537, 1535, 5000):
        _reserve(np.arange(1300) % 50, many, 16, 6, 3000, f"{rows} rows of 1300 sequences", rows=rows)


def test_odd_state(gpu):
    # lengths past the table, negative numbers, a stack that is said to be larger, pages that are none
    _reserve([70, -5, 40, 64], [5, 3, -2, 10], 16, 4, 20, "past the table's width")
    _reserve([10, 20], [20, 20], 16, 8, 2, "a stack past its room", count=1 << 30)
    _reserve([10, 20], [20, 20], 16, 8, 5, "a stack below zero", count=-4)
    f, c, _, pages = _state([10, 20], 16, 8, 6, 1)
    f[c - 1], f[c - 2] = pages + 4, -7
    _reserve([10, 20], [20, 20], 16, 8, 6, "pages that are none", free=f)
    _reserve([(1 << 31) - 3], [8], 1 << 20, 2048, 1, "the last lengths there are")
    _reserve([], [], 16, 4, 3, "no sequences", rows=5)


def _release(lens, keep, page, width, spare, label, seed=1, stride=0, edit=None):
    say(f"[release] {label}")
    free, count, table, pages = _state(lens, page, width, spare, seed)
    if edit:
        edit(free, table, pages)
    B = len(lens)
    wide = torch.full((B, width + stride), -9, dtype=torch.int32, device="cuda")
    wide[:, :width] = _ints(table).view(B, width)
    df, dc = _ints(free), _ints([count, 3])
    got = binding.release_pages(df, dc, wide[:, :width], _ints(keep), page)
    want_free, want_count, want_table = bref.release(free, count, table, keep, page, pages)
    assert got.cpu().tolist() == [want_count, 0], label
    assert df.cpu().tolist() == want_free and np.array_equal(wide[:, :width].cpu().numpy(), want_table), label
    assert torch.all(wide[:, width:] == -9) and dc.cpu().tolist() == [count, 3]


@pytest.mark.parametrize("page", [1, 5, 16])
def test_release(gpu, page):
    rng = np.random.default_rng(page)
    for B in (1, 3, 64, 300):
        lens = rng.integers(0, 600, B)
        width = 600 // page + 3
        _release(lens, np.where(rng.random(B) < 0.5, 0, lens), page, width, 5, f"half of {B}, pages of {page}", stride=2)
        _release(lens, rng.integers(-3, 700, B), page, width, 0, f"parts of {B}, pages of {page}")
        _release(lens, lens, page, width, 3, f"none of {B}, pages of {page}")


def test_release_of_odd_tables(gpu):
    def holes(free, table, pages):
        table[0, 1], table[1, 0], table[1, 2] = -1, pages, 1 << 30
    _release([90, 70], [0, 0], 16, 8, 4, "holes", edit=holes)
    def twice(free, table, pages):
        table[1] = table[0]
    _release([100, 100], [0, 0], 16, 8, 2, "more pages than the stack has room for", edit=twice)
    _release([], [], 16, 4, 3, "no sequences")


def test_refusals(gpu):
    free, count, table = _ints(range(8)), _ints([8, 0]), _ints(-np.ones((2, 4)))
    lens = _ints([3, 4])
    for bad in (dict(out=(count, lens, _ints([0, 0, 0]), _ints([0]), _ints([0], torch.int64))),
                dict(out=(_ints([0, 0]), _ints([0, 0]), _ints([0, 0, 0]), _ints([0]), _ints([0]))), dict(page_size=-1), dict(rows=-1)):
        kw = dict(page_size=16, rows=1)
        kw.update(bad)
        with pytest.raises((ValueError, TypeError)):
            binding.reserve_pages(free, count, table, lens, _ints([1, 0]), **kw)
    with pytest.raises(binding.GemvError):
        binding.reserve_pages(free, count, table, lens, _ints([1, 0]), 0, 1)
    with pytest.raises(ValueError):
        binding.release_pages(free, count, table, lens, 16, out=count)


def test_streams_and_graphs(gpu):
    free, count, table, _ = _state([5, 60, 16], 16, 12, 30, 3)
    df, dc, dt, dl = _ints(free), _ints([count, 0]), _ints(table), _ints([5, 60, 16])
    added = _ints([1, 9, 40])
    say("[pages] streams and graphs")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = binding.reserve_pages(df, dc, dt, dl, added, 16, 64, stream=side)
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = binding.reserve_pages(df, dc, dt, dl, added, 16, 64)
        back = binding.release_pages(df, out[0], dt, dl, 16)
    for shift in (0, 1, 3):
        added.copy_(_ints([1 + shift, 9, 40 - shift]))
        graph.replay()
        torch.cuda.synchronize()
        want = bref.reserve(free, count, table, [5, 60, 16], added.tolist(), 16, 64, len(free))
        for g, w in zip(out, want):
            assert g.cpu().tolist() == list(w)
        # what was taken has come back, in the order in which it is given back
        assert back.cpu().tolist() == [count, 0] and np.array_equal(dt.cpu().numpy(), table)
        free = np.array(bref.release(free, want[0][0], want[5], [5, 60, 16], 16, len(free))[0])
        assert df.cpu().tolist() == free.tolist()
    assert got[2].cpu().tolist() == [0, 1, 10, 50]


# ---------------------------------------------------------------- a run of them together
@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16], ids=str)
def test_a_prompt_and_decode_steps(gpu, dtype):
    """Two prompts are taken in, then five steps of a token each: pages reserved,
    heads normed, rotated and put into the cache, attention with and without a
    window; at the end one sequence is released.  Against 64-bit forms of every
    stage, on what the stage before has stored."""
    heads, kv, dim, page, pages, width = 8, 2, 64, 16, 40, 16
    half = dim // 2
    freqs = 10000.0 ** -(np.arange(half) / half)
    dfreqs = torch.from_numpy(freqs).cuda()
    weight = (1 + 0.1 * torch.randn(dim, generator=torch.Generator().manual_seed(1))).to(dtype)
    cache = binding.PagedCache(*(torch.full((pages, page, kv, dim), float("nan"), dtype=dtype, device="cuda") for _ in range(2)))
    free, count = torch.arange(pages, dtype=torch.int32, device="cuda").flip(0).contiguous(), _ints([pages, 0])
    table, lens = _ints(-np.ones((2, width))), _ints([0, 0])
    mirror = ref.Pool.__new__(ref.Pool)
    mirror.page, mirror.heads, mirror.dim, mirror.width = page, kv, dim, width
    for step, counts in enumerate([[70, 37]] + [[1, 1]] * 5):
        rows = sum(counts) + 3
        say(f"[run] step {step} {dtype}")
        count, lens, starts, positions, slots = binding.reserve_pages(free, count, table, lens, _ints(counts), page, rows)
        made = (torch.randn((rows, (heads + 2 * kv) * dim), generator=torch.Generator().manual_seed(step)) * 2).to(dtype)
        on = made.cuda()
        q, k, v = (on[:, a * dim: b * dim].view(rows, b - a, dim) for a, b in ((0, heads), (heads, heads + kv), (heads + kv, heads + 2 * kv)))
        queries = binding.norm_rotate_append(cache, slots, q, k, v, positions, dfreqs, weight.cuda(), weight.cuda())
        place = positions.cpu().numpy()
        for x, got in ((q, queries), (k, cache.k.view(-1, kv, dim)[slots.clamp(min=0)])):
            want, bound = bref.turned(x.cpu(), weight.double().numpy(), place, freqs, 1e-6, False, dtype)
            n = rows if got is queries else rows - 3
            assert np.all(np.abs(got.cpu().double().numpy() - want)[:n] <= bound[:n])
        assert torch.equal(cache.v.view(-1, kv, dim)[slots[: rows - 3]], v[: rows - 3])
        mirror.k, mirror.v, mirror.table, mirror.lens = cache.k.cpu(), cache.v.cpu(), table.cpu(), lens.tolist()
        first = starts.tolist()
        for window, sinks in ((None, 0), (20, 2)):
            out = binding.prompt_attention(cache, table, lens, starts, queries, window=window, sinks=sinks, max_new=max(counts),
                                           out=torch.zeros_like(queries))
            want, bound, mine = pref.prompt(mirror, queries.cpu(), first, dim ** -0.5, window, sinks, rounded=max(counts) > 1)
            assert np.all(np.abs(out.cpu().double().numpy() - want)[mine] <= bound[mine]) and torch.all(out[rows - 3:] == 0)
    assert count.tolist() == [pages - 5 - 3, 0] and lens.tolist() == [75, 42]
    count = binding.release_pages(free, count, table, _ints([75, 0]), page)
    assert count.tolist() == [pages - 5, 0] and torch.all(table[1] == -1)
    held = set(table[0].tolist()) - {-1}
    assert len(held) == 5 and held | set(free[: pages - 5].tolist()) == set(range(pages))
