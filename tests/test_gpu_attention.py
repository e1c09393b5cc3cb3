"""Decode attention over a paged key-value cache, its append and its eviction,
against plain 64-bit forms.  Every slot that no sequence holds is NaN or
infinite, so a read past a length shows."""
import numpy as np
import pytest
import torch

from memory_bound_gemv_row_amd import binding

import serving_ref as ref
from gpu_util import say

pytestmark = pytest.mark.gpu

HALVES = [torch.float16, torch.bfloat16]


def _query(B, heads, dim, dtype, seed, spread=1.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn((B, heads, dim), generator=g) * spread).to(dtype)


def _check(pool, q, label, scale=None, weighted=True, max_len=None, stride=0):
    say(f"[attention] {label}")
    B, heads, dim = q.shape
    scale = dim ** -0.5 if scale is None else scale
    cache = binding.PagedCache(pool.dk, pool.dv)
    dq = q.cuda()
    if stride:
        wide = torch.full((B, heads * dim + stride), float("nan"), dtype=q.dtype, device="cuda")
        wide[:, : heads * dim] = dq.view(B, -1)
        dq = wide[:, : heads * dim].view(B, heads, dim)
    slots = pool.width * pool.page
    want, bound, want_w, wbound = ref.attention(pool, q, scale)
    out = binding.paged_attention(cache, pool.dtable, pool.dlens, dq, scale=scale, max_len=max_len)
    off = np.abs(out.cpu().double().numpy() - want)
    assert np.all(off <= bound), (label, float(np.nanmax(off / bound)), np.isnan(off).sum())
    if weighted:
        before = np.random.default_rng(1).uniform(0, 2, want_w.shape).astype(np.float32)
        w = torch.from_numpy(before.copy()).cuda()
        again = binding.paged_attention(cache, pool.dtable, pool.dlens, dq, scale=scale, max_len=max_len, weights=w)
        assert torch.equal(again, out), label
        got = w.cpu().double().numpy()
        assert np.all(np.abs(got - (before + want_w)) <= wbound + ref.U32 * (before + want_w)), label
        for b, n in enumerate(pool.lens):
            assert np.array_equal(got[b, :, max(n, 0):], before[b, :, max(n, 0):]), label
    return out


# tiles of 16 slots, 4 waves of them, parts of the length: lengths about each border
@pytest.mark.parametrize("dtype", HALVES, ids=str)
@pytest.mark.parametrize("n", [1, 2, 15, 16, 17, 31, 33, 63, 64, 65, 127, 129, 255, 256, 257, 300, 511, 513, 1000])
def test_lengths(gpu, n, dtype):
    _check(ref.Pool([n], 2, 64, 16, dtype, seed=n), _query(1, 8, 64, dtype, n), f"one of {n} {dtype}")


@pytest.mark.parametrize("dtype", HALVES, ids=str)
@pytest.mark.parametrize("dim", [8, 16, 24, 40, 64, 72, 80, 96, 120, 128, 136, 192, 248, 256])
def test_head_sizes(gpu, dim, dtype):
    _check(ref.Pool([70, 3, 129], 2, dim, 16, dtype, seed=dim), _query(3, 6, dim, dtype, dim), f"dim {dim} {dtype}")


@pytest.mark.parametrize("heads,kv", [(1, 1), (3, 3), (16, 16), (2, 1), (5, 1), (15, 3), (16, 1), (17, 1), (32, 1), (33, 1),
                                      (40, 2), (64, 4), (28, 4)])
def test_head_groups(gpu, heads, kv):
    _check(ref.Pool([100, 37], kv, 64, 16, seed=heads), _query(2, heads, 64, torch.float16, kv), f"{heads} over {kv}")


@pytest.mark.parametrize("page", [1, 2, 3, 5, 8, 12, 16, 17, 24, 32, 48, 64, 100, 128, 256])
@pytest.mark.parametrize("layout", ["slots", "heads", "padded"])
def test_pages_and_layouts(gpu, page, layout):
    _check(ref.Pool([90, 1, 200], 2, 64, page, torch.bfloat16, seed=page, layout=layout),
           _query(3, 4, 64, torch.bfloat16, page), f"page {page} {layout}")


def test_ragged_batch_with_empty_sequences(gpu):
    lens = [0, 500, 1, 0, 33, 257, 0, 64]
    out = _check(ref.Pool(lens, 2, 128, 16, seed=3, width=40), _query(8, 8, 128, torch.float16, 3), "ragged", stride=64)
    assert torch.all(out[[0, 3, 6]] == 0)


def test_long_sequences_are_split(gpu):
    for dtype in HALVES:
        _check(ref.Pool([5000, 4097], 1, 64, 32, dtype, seed=9), _query(2, 4, 64, dtype, 9), f"long {dtype}")


def test_batches_past_the_card(gpu):
    lens = np.random.default_rng(4).integers(0, 40, 700)
    _check(ref.Pool(lens, 2, 64, 8, seed=4), _query(700, 4, 64, torch.float16, 4), "700 sequences")


def test_holes(gpu):
    # pages outside the pool are left out of the softmax; a sequence of holes gets zeros
    pool = ref.Pool([200, 70, 48], 2, 64, 16, seed=5)
    for b, i, p in ((0, 3, -1), (0, 11, 1 << 30), (1, 0, pool.k.shape[0]), (2, 0, -5), (2, 1, -1), (2, 2, 1 << 29)):
        pool.table[b, i] = p
    pool.dtable = pool.table.cuda()
    out = _check(pool, _query(3, 4, 64, torch.float16, 5), "holes")
    assert torch.all(out[2] == 0)


def test_lengths_are_cut_to_the_room(gpu):
    pool = ref.Pool([96, 96, 96], 2, 64, 16, seed=6)
    q = _query(3, 4, 64, torch.float16, 6)
    cache = binding.PagedCache(pool.dk, pool.dv)
    full = binding.paged_attention(cache, pool.dtable, pool.dlens, q.cuda())
    wild = torch.tensor([1 << 30, -7, 96], dtype=torch.int32, device="cuda")
    say("[attention] lengths outside the room")
    out = binding.paged_attention(cache, pool.dtable, wild, q.cuda())
    assert torch.equal(out[0], full[0]) and torch.all(out[1] == 0) and torch.equal(out[2], full[2])
    pool.lens = [50, 50, 50]
    pool.dlens = torch.tensor([96, 50, 70], dtype=torch.int32, device="cuda")
    short = binding.paged_attention(cache, pool.dtable, pool.dlens, q.cuda(), max_len=50)
    want, bound, _, _ = ref.attention(pool, q, 64 ** -0.5)
    assert np.all(np.abs(short.cpu().double().numpy() - want) <= bound)


@pytest.mark.parametrize("spread", [0.0, 8.0, 40.0])
def test_flat_and_peaked_softmax(gpu, spread):
    # all logits equal, and logits that run past the reference maximum again and again
    pool = ref.Pool([700, 333], 2, 64, 16, torch.bfloat16, seed=7, spread=max(spread, 1e-3))
    _check(pool, _query(2, 4, 64, torch.bfloat16, 7, spread=max(spread, 0.0) / 4), f"spread {spread}")


def test_rising_logits(gpu):
    # each key larger than the last: the maximum moves with every tile
    pool = ref.Pool([400], 1, 64, 16, seed=8)
    for j in range(400):
        pool.k[pool.table[0, j // 16], j % 16, 0] = j / 16.0
    pool.dk = pool.k.cuda()
    q = torch.full((1, 2, 64), 1.0, dtype=torch.float16)
    q[0, 1] = -1.0
    _check(pool, q, "rising and falling")


def test_infinite_and_nan_values(gpu):
    pool = ref.Pool([64, 64, 64], 1, 64, 16, seed=10)
    pool.dk[pool.table[0, 0], 3] = float("nan")
    pool.dv[pool.table[1, 1], 5, 0, 7] = float("inf")
    q = _query(3, 2, 64, torch.float16, 10)
    say("[attention] NaN key, infinite value")
    out = binding.paged_attention(binding.PagedCache(pool.dk, pool.dv), pool.dtable, pool.dlens, q.cuda()).cpu()
    assert torch.all(torch.isnan(out[0]))
    assert torch.all(out[1, :, 7] == float("inf")) and torch.all(torch.isfinite(out[1, :, :7]))
    assert torch.all(torch.isfinite(out[2]))


def test_keys_of_the_lowest_logit_weigh_nothing(gpu):
    # a token masked by a key that drives its logit to the lowest finite value, or below it
    pool = ref.Pool([64], 1, 64, 16, seed=12)
    q = torch.ones((1, 2, 64), dtype=torch.float16)
    for j in (0, 5, 40):
        pool.k[pool.table[0, j // 16], j % 16, 0] = -65504.0
    pool.dk = pool.k.cuda()
    _check(pool, q, "lowest logits")
    pool.dk[pool.table[0, 1], 3] = -float("inf")
    out = binding.paged_attention(binding.PagedCache(pool.dk, pool.dv), pool.dtable, pool.dlens, q.cuda())
    assert torch.all(torch.isfinite(out))


def test_offsets_past_32_bits(gpu):
    # a pool of 2.2 G elements per buffer: pages at both ends
    pages, page, heads, dim = 8600, 64, 32, 128
    say("[attention] offsets past 2^31 elements")
    k = torch.zeros((pages, page, heads, dim), dtype=torch.float16, device="cuda")
    v = torch.zeros_like(k)
    table = torch.tensor([[0, pages - 1], [pages - 2, 5]], dtype=torch.int32)
    g = torch.Generator().manual_seed(2)
    for p in table.ravel().tolist():
        k[p] = torch.randn((page, heads, dim), generator=g).to(torch.float16).cuda()
        v[p] = torch.randn((page, heads, dim), generator=g).to(torch.float16).cuda()
    assert k.numel() > 1 << 31
    q = _query(2, 32, 128, torch.float16, 2)
    small = {p: i for i, p in enumerate(table.ravel().tolist())}
    rows = torch.tensor(list(small))
    cache = binding.PagedCache(k, v)
    out = binding.paged_attention(cache, table.cuda(), torch.tensor([100, 128], dtype=torch.int32, device="cuda"), q.cuda())
    near = binding.PagedCache(k[rows.cuda()].contiguous(), v[rows.cuda()].contiguous())
    same = binding.paged_attention(near, torch.tensor([[0, 1], [2, 3]], dtype=torch.int32, device="cuda"),
                                   torch.tensor([100, 128], dtype=torch.int32, device="cuda"), q.cuda())
    assert torch.equal(out, same) and torch.all(torch.isfinite(out)) and out.abs().max() > 0


# ---------------------------------------------------------------- append
def _append_reference(pool, lens, news, new_k, new_v):
    k, v = pool.k.clone(), pool.v.clone()
    row = 0
    for b, n in enumerate(news):
        for i in range(n):
            j = lens[b] - n + i
            if 0 <= j < pool.width * pool.page:
                p = int(pool.table[b, j // pool.page])
                if 0 <= p < k.shape[0]:
                    k[p, j % pool.page], v[p, j % pool.page] = new_k[row], new_v[row]
            row += 1
    return k, v


def _same(a, b):
    return torch.equal(a.view(torch.int16), b.view(torch.int16))


@pytest.mark.parametrize("layout", ["slots", "heads", "padded"])
@pytest.mark.parametrize("heads,dim,page", [(1, 8, 1), (2, 64, 16), (3, 80, 5), (8, 128, 16), (5, 256, 24)])
def test_append(gpu, heads, dim, page, layout):
    # ragged: nothing, one token, some, a first prompt; rows before and behind stay unread
    news, before = [0, 1, 7, 33, 1, 0, 20], [5, 12, 0, 30, 63, 0, 41]
    lens = [a + n for a, n in zip(before, news)]
    pool = ref.Pool(lens, heads, dim, page, torch.bfloat16, seed=dim, layout=layout, width=-(-70 // page))
    rows = sum(news)
    g = torch.Generator().manual_seed(dim)
    new_k, new_v = (torch.randn((rows, heads, dim), generator=g).to(torch.bfloat16) for _ in range(2))
    want_k, want_v = _append_reference(pool, lens, news, new_k, new_v)
    fused = torch.full((rows + 5, 3 * heads * dim), float("nan"), dtype=torch.bfloat16, device="cuda")
    fused[2: 2 + rows, : heads * dim] = new_k.view(rows, -1).cuda()
    fused[2: 2 + rows, heads * dim: 2 * heads * dim] = new_v.view(rows, -1).cuda()
    starts = torch.tensor(np.concatenate([[0], np.cumsum(news)]) + 2, dtype=torch.int32, device="cuda")
    slots = pool.width * page + 3
    w = torch.full((7, heads, slots), 9.0, device="cuda")
    pos = torch.full((7, heads, slots), -3, dtype=torch.int32, device="cuda")
    seen = torch.tensor([n + 100 * b for b, n in enumerate(lens)], dtype=torch.int32, device="cuda")
    say(f"[append] {heads}x{dim} page {page} {layout}")
    binding.kv_append(binding.PagedCache(pool.dk, pool.dv), pool.dtable, pool.dlens, starts,
                      fused[:, : heads * dim].view(rows + 5, heads, dim),
                      fused[:, heads * dim: 2 * heads * dim].view(rows + 5, heads, dim), weights=w, positions=pos, seen=seen)
    assert _same(pool.dk.cpu().contiguous(), want_k) and _same(pool.dv.cpu().contiguous(), want_v)
    want_w, want_p = np.full(w.shape, 9.0, np.float32), np.full(pos.shape, -3, np.int32)
    for b, n in enumerate(news):
        want_w[b, :, lens[b] - n: lens[b]] = 0
        want_p[b, :, lens[b] - n: lens[b]] = np.arange(n) + 100 * b + lens[b] - n
    assert np.array_equal(w.cpu().numpy(), want_w) and np.array_equal(pos.cpu().numpy(), want_p)


def test_append_leaves_out_what_has_no_slot(gpu):
    # past the table, before slot 0, in a hole, and rows no sequence owns
    pool = ref.Pool([40, 16, 30, 2], 2, 64, 16, seed=1, width=2, extra=2)
    pool.table[2, 1] = -1
    pool.dtable = pool.table.cuda()
    lens, news = [40, 16, 30, 2], [10, 1, 20, 5]
    rows = sum(news) + 4
    g = torch.Generator().manual_seed(1)
    new = torch.randn((rows, 2, 64), generator=g).to(torch.float16)
    want_k, want_v = _append_reference(pool, lens, news, new, new)
    starts = torch.tensor([0, 10, 11, 31, 36], dtype=torch.int32, device="cuda")
    say("[append] rows without a slot")
    binding.kv_append(binding.PagedCache(pool.dk, pool.dv), pool.dtable, pool.dlens, starts, new.cuda(), new.cuda())
    assert _same(pool.dk.cpu(), want_k) and _same(pool.dv.cpu(), want_v)


# ---------------------------------------------------------------- eviction
def _check_evict(lens, heads, dim, page, budget, recent, seed, ties=False, max_len=None, wild=False, slots_more=0, holes=False):
    rng = np.random.default_rng(seed)
    B = len(lens)
    pool = ref.Pool(lens, heads, dim, page, torch.bfloat16, seed=seed)
    if holes:
        pool.table[0, 1] = -1
        pool.table[0, pool.width - 1] = pool.k.shape[0] + 9
        pool.dtable = pool.table.cuda()
    slots = pool.width * page + slots_more
    w = rng.exponential(1.0, (B, heads, slots)).astype(np.float32)
    if ties:
        w = rng.integers(0, 3, w.shape).astype(np.float32) * np.float32(0.5)
        w[rng.random(w.shape) < 0.2] *= -1.0      # -0 among the zeros
    if wild:
        w[rng.random(w.shape) < 0.05] = np.nan
        w[rng.random(w.shape) < 0.05] = np.inf
        w[rng.random(w.shape) < 0.05] = -np.inf
    seen = np.array(lens, np.int32) + rng.integers(0, 50, B).astype(np.int32)
    pos = np.full((B, heads, slots), 1 << 30, np.int32)
    for b, n in enumerate(lens):
        for h in range(heads):
            p = rng.permutation(int(seen[b]))[:n]
            pos[b, h, :n] = p if rng.random() < 0.5 else np.sort(p)
    use = [min(n, max_len) for n in lens] if max_len is not None else lens
    source, want_w, want_p, left = ref.evict(use, seen, w, pos, budget, recent, slots)
    want_k, want_v = pool.k.clone(), pool.v.clone()
    for b in range(B):
        for h in range(heads):
            for j in range(left[b]):
                s = int(source[b, h, j])
                at, frm = int(pool.table[b, j // page]), int(pool.table[b, s // page])
                if s != j and 0 <= at < len(want_k) and 0 <= frm < len(want_k):
                    want_k[at, j % page, h] = pool.k[frm, s % page, h]
                    want_v[at, j % page, h] = pool.v[frm, s % page, h]
    dw, dp = torch.from_numpy(w).cuda(), torch.from_numpy(pos).cuda()
    say(f"[evict] lens {lens[:6]} heads {heads} dim {dim} page {page} budget {budget} recent {recent}")
    new_w, new_p, new_l = binding.kv_evict(binding.PagedCache(pool.dk, pool.dv), pool.dtable, pool.dlens,
                                           torch.from_numpy(seen).cuda(), dw, dp, budget, recent, max_len=max_len)
    assert np.array_equal(new_l.cpu().numpy(), left)
    assert np.array_equal(new_p.cpu().numpy(), want_p)
    assert np.array_equal(new_w.cpu().numpy(), want_w, equal_nan=True)
    assert _same(pool.dk.cpu(), want_k) and _same(pool.dv.cpu(), want_v)
    assert np.array_equal(dw.cpu().numpy(), w, equal_nan=True) and np.array_equal(dp.cpu().numpy(), pos)


@pytest.mark.parametrize("n,budget,recent", [(65, 64, 8), (100, 64, 16), (300, 64, 64), (64, 64, 8), (10, 64, 8), (0, 16, 4),
                                             (50, 1, 0), (50, 1, 1), (50, 0, 0), (1, 0, 0), (1100, 1024, 100), (3000, 700, 0),
                                             (2500, 2499, 2499)])
def test_evict(gpu, n, budget, recent):
    _check_evict([n, max(0, n - 3), n // 2], 2, 64, 16, budget, recent, seed=n + budget)


@pytest.mark.parametrize("dim,page,heads", [(8, 1, 1), (80, 5, 3), (128, 24, 8), (256, 64, 2)])
def test_evict_shapes(gpu, dim, page, heads):
    _check_evict([90, 40, 77], heads, dim, page, 33, 9, seed=dim, slots_more=5)


def test_evict_ties_and_odd_weights(gpu):
    _check_evict([500, 499, 1500], 2, 64, 16, 200, 30, seed=1, ties=True)
    _check_evict([500, 499, 1500], 2, 64, 16, 200, 0, seed=2, wild=True)
    _check_evict([300, 200], 2, 64, 16, 100, 20, seed=3, ties=True, wild=True, max_len=250)


def test_evict_more_recent_than_the_budget(gpu):
    _check_evict([300, 280], 2, 64, 16, 50, 200, seed=4)


def test_evict_leaves_holes_alone(gpu):
    _check_evict([100, 90], 2, 64, 16, 40, 10, seed=5, holes=True)


# ---------------------------------------------------------------- together
def test_decode_steps_with_eviction(gpu):
    """Steps of a small INT8 layer over a paged cache held to a budget, as a
    program runs them: quantise, project, append, attend, evict; the operators'
    results against plain forms carried along, every step."""
    B, H, G, D, page, budget, recent, steps = 3, 2, 3, 64, 8, 40, 8, 30
    rng = np.random.default_rng(0)
    hidden, width = 128, (G * H + 2 * H) * D
    A = rng.integers(-127, 128, (width, hidden), dtype=np.int8)
    scale = np.full(width, 1e-3, np.float16)
    dA, ds = torch.from_numpy(A).cuda(), torch.from_numpy(scale).cuda()
    pool = ref.Pool([0, 0, 0], H, D, page, torch.float16, width=8, seed=1)
    slots = 8 * page
    cache = binding.PagedCache(pool.dk, pool.dv)
    held = [35, 0, 20]
    pool.lens = list(held)
    for b in range(B):
        for j in range(held[b]):
            for t in (pool.k, pool.v):
                t[pool.table[b, j // page], j % page] = torch.from_numpy(rng.standard_normal((H, D))).to(torch.float16)
    pool.dk.copy_(pool.k)
    pool.dv.copy_(pool.v)
    w = rng.uniform(0, 1, (B, H, slots)).astype(np.float32)
    pos = np.broadcast_to(np.arange(slots, dtype=np.int32), (B, H, slots)).copy()
    dw, dp = torch.from_numpy(w).cuda(), torch.from_numpy(pos).cuda()
    lens = torch.tensor(held, dtype=torch.int32, device="cuda")
    seen = lens.clone()
    starts = torch.arange(B + 1, dtype=torch.int32, device="cuda")
    for step in range(steps):
        x = torch.from_numpy(rng.standard_normal((B, hidden))).to(torch.float16).cuda()
        q8, t = binding.quantize_tokens_q8(x)
        fused = binding.gemm_q8(dA, ds, q8, t)
        lens += 1
        seen += 1
        q, k, v = fused.split([G * H * D, H * D, H * D], dim=1)
        binding.kv_append(cache, pool.dtable, lens, starts, k.view(B, H, D), v.view(B, H, D), weights=dw, positions=dp,
                          seen=seen)
        out = binding.paged_attention(cache, pool.dtable, lens, q.view(B, H * G, D), weights=dw)
        attended = dw.cpu().numpy()
        dw, dp, left = binding.kv_evict(cache, pool.dtable, lens, seen, dw, dp, budget, recent)
        # the plain forms, on the operators' own inputs of this step
        want = ref.product(A, scale, q8.cpu().numpy(), t.cpu().numpy())
        assert np.all(np.abs(fused.cpu().double().numpy() - want) <= ref.product_bound(want, torch.float16))
        for b in range(B):
            j = pool.lens[b]
            for mine, new in ((pool.k, k), (pool.v, v)):
                mine[pool.table[b, j // page], j % page] = new[b].cpu().view(H, D)
            pool.lens[b] += 1
            w[b, :, j], pos[b, :, j] = 0, int(seen[b]) - 1
        want, bound, want_w, wbound = ref.attention(pool, q.cpu().view(B, H * G, D), D ** -0.5)
        assert np.all(np.abs(out.cpu().double().numpy() - want) <= bound), step
        for b, n in enumerate(pool.lens):
            assert np.all(np.abs(attended[b, :, :n] - (w + want_w)[b, :, :n]) <= (wbound + ref.U32 * (w + want_w))[b, :, :n])
        source, w, pos, lefts = ref.evict(pool.lens, seen.cpu().numpy(), attended, pos, budget, recent, slots)
        for pool_t in (pool.k, pool.v):
            old = pool_t.clone()
            for b in range(B):
                for h in range(H):
                    for j in range(lefts[b]):
                        s = int(source[b, h, j])
                        pool_t[pool.table[b, j // page], j % page, h] = old[pool.table[b, s // page], s % page, h]
        pool.lens = [int(n) for n in lefts]
        assert np.array_equal(left.cpu().numpy(), lefts) and np.array_equal(dw.cpu().numpy(), w)
        assert np.array_equal(dp.cpu().numpy(), pos)
        assert _same(pool.dk.cpu(), pool.k) and _same(pool.dv.cpu(), pool.v), step
        lens = left
    assert max(pool.lens) == budget and int(seen[0]) == 35 + steps


# ---------------------------------------------------------------- streams, graphs, refusals
def _serving_state(seed):
    pool = ref.Pool([200, 150, 37], 2, 64, 16, seed=seed, width=16)
    q = _query(3, 8, 64, torch.float16, seed).cuda()
    g = torch.Generator(device="cuda").manual_seed(seed)
    return {"pool": pool, "cache": binding.PagedCache(pool.dk, pool.dv), "q": q,
            "k": torch.randn((3, 2, 64), generator=g, device="cuda").half(),
            "starts": torch.arange(4, dtype=torch.int32, device="cuda"),
            "w": torch.rand((3, 2, 256), generator=g, device="cuda"),
            "pos": torch.arange(256, dtype=torch.int32, device="cuda").expand(3, 2, 256).contiguous(),
            "x": torch.randn((5, 512), generator=g, device="cuda"),
            "A": torch.randint(-127, 128, (96, 512), generator=g, device="cuda", dtype=torch.int8),
            "s": torch.rand(96, generator=g, device="cuda").half()}


def _serve(s, stream=None):
    pool = s["pool"]
    q8, t = binding.quantize_tokens_q8(s["x"], stream=stream)
    y = binding.gemm_q8(s["A"], s["s"], q8, t, stream=stream)
    binding.kv_append(s["cache"], pool.dtable, pool.dlens, s["starts"], s["k"], s["k"], stream=stream)
    out = binding.paged_attention(s["cache"], pool.dtable, pool.dlens, s["q"], stream=stream)
    new = binding.kv_evict(s["cache"], pool.dtable, pool.dlens, pool.dlens, s["w"], s["pos"], 100, 20, stream=stream)
    return [q8, t, y, out, *new, pool.dk, pool.dv]


def _bits(ts):
    return [t.contiguous().view(torch.uint8).clone() if t.dtype not in (torch.float16, torch.bfloat16)
            else t.contiguous().view(torch.int16).clone() for t in ts]


def test_graph_replays_match_eager(gpu):
    # the first pass moves rows of the cache; from then on a pass finds the
    # cache as it leaves it, so replays give what an eager pass gives
    a, b = _serving_state(1), _serving_state(2)
    say("[serving graph] eager")
    for s in (a, b):
        _serve(s)
    want = [_bits(_serve(s)) for s in (a, b)]
    graphs = []
    for s in (a, b):      # two graphs, captured in turn and replayed in turn
        g, stream = torch.cuda.CUDAGraph(), torch.cuda.Stream()
        stream.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(stream), torch.cuda.graph(g, stream=stream):
            outs = _serve(s)
        torch.cuda.synchronize()
        graphs.append((g, outs))
    for r in range(4):
        for (g, outs), s in zip(graphs, (a, b)):
            for o in outs[:7]:
                o.zero_()
            say(f"[serving graph] replay {r}")
            g.replay()
            _serve(_serving_state(3))             # eager work of another state between the replays
        torch.cuda.synchronize()
        for (g, outs), ws in zip(graphs, want):
            assert all(torch.equal(x, y) for x, y in zip(_bits(outs), ws)), r


def test_two_streams_and_a_given_stream(gpu):
    a, b = _serving_state(4), _serving_state(5)
    for s in (a, b):
        _serve(s)
    want = [_bits(_serve(s)) for s in (a, b)]
    torch.cuda.synchronize()
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    say("[serving streams]")
    for _ in range(10):
        got = [_serve(a, stream=s1), _serve(b, stream=s2)]
        junk = torch.full((1 << 20,), float("nan"), device="cuda")   # takes what the current stream's pool has free
        del junk
    torch.cuda.synchronize()
    for x, y in zip(got, want):
        assert all(torch.equal(p, q) for p, q in zip(_bits(x), y))


def test_repeated_calls_are_bitwise_equal(gpu):
    pool = ref.Pool([3000, 2900, 10], 2, 128, 16, seed=11)
    cache = binding.PagedCache(pool.dk, pool.dv)
    q = _query(3, 16, 128, torch.float16, 11).cuda()
    w = torch.zeros((3, 2, pool.width * 16), device="cuda")
    first = binding.paged_attention(cache, pool.dtable, pool.dlens, q, weights=w).clone()
    w1 = w.clone()
    for _ in range(3):
        w.zero_()
        assert torch.equal(binding.paged_attention(cache, pool.dtable, pool.dlens, q, weights=w), first)
        assert torch.equal(w, w1)


def test_refusals(gpu):
    pool = ref.Pool([20, 20], 2, 64, 16, seed=1)
    cache = binding.PagedCache(pool.dk, pool.dv)
    q = _query(2, 4, 64, torch.float16, 1).cuda()
    table, lens = pool.dtable, pool.dlens
    w = torch.zeros((2, 2, 32), device="cuda")
    pos = torch.zeros((2, 2, 32), dtype=torch.int32, device="cuda")
    for bad in (lambda: binding.PagedCache(pool.dk, pool.dv.to(torch.bfloat16)),
                lambda: binding.PagedCache(pool.dk, pool.dv[:-1]),
                lambda: binding.PagedCache(pool.dk.float(), pool.dv.float()),
                lambda: binding.PagedCache(pool.k, pool.v),
                lambda: binding.PagedCache(pool.dk[..., :60], pool.dv[..., :60]),
                lambda: binding.PagedCache(pool.dk[:1].expand(4, -1, -1, -1), pool.dv[:1].expand(4, -1, -1, -1)),
                lambda: binding.PagedCache(pool.dk.transpose(2, 3), pool.dv.transpose(2, 3)),
                lambda: binding.PagedCache(pool.dk, pool.dv.transpose(1, 2).contiguous().transpose(1, 2)),
                lambda: binding.paged_attention(cache, table.long(), lens, q),
                lambda: binding.paged_attention(cache, table, lens[:1], q),
                lambda: binding.paged_attention(cache, table, lens, q[:, :3]),
                lambda: binding.paged_attention(cache, table, lens, q[:1]),
                lambda: binding.paged_attention(cache, table, lens, q.to(torch.bfloat16)),
                lambda: binding.paged_attention(cache, table, lens, q, max_len=-1),
                lambda: binding.paged_attention(cache, table, lens, q, weights=w[..., :31]),
                lambda: binding.paged_attention(cache, table, lens, q, weights=w.double()),
                lambda: binding.paged_attention(cache, table, lens, q.transpose(1, 2).contiguous().transpose(1, 2)),
                lambda: binding.kv_append(cache, table, lens, lens, q[:, :2], q[:, :2]),
                lambda: binding.kv_append(cache, table, lens, torch.arange(3, dtype=torch.int32, device="cuda"), q[:, :1],
                                          q[:, :2]),
                lambda: binding.kv_append(cache, table, lens, torch.arange(3, dtype=torch.int32, device="cuda"), q[:, :2],
                                          q[:, :2], weights=w),
                lambda: binding.kv_evict(cache, table, lens, lens, w, pos, -1, 0),
                lambda: binding.kv_evict(cache, table, lens, lens, w, pos, 8, -1),
                lambda: binding.kv_evict(cache, table, lens, lens, w, pos[..., :30], 8, 0),
                lambda: binding.kv_evict(cache, table, lens, lens, w, pos, 8, 0, out=(w, pos, lens))):
        with pytest.raises((ValueError, TypeError, binding.GemvError)):
            bad()


# ---------------------------------------------------------------- edges of the calls
def test_no_sequences_no_slots_no_rows(gpu):
    pool = ref.Pool([20, 20], 2, 64, 16, seed=1)
    cache = binding.PagedCache(pool.dk, pool.dv)
    q = _query(2, 4, 64, torch.float16, 1).cuda()
    w = torch.ones((2, 2, 32), device="cuda")
    pos = torch.zeros((2, 2, 32), dtype=torch.int32, device="cuda")
    say("[attention] nothing to attend to")
    assert torch.all(binding.paged_attention(cache, pool.dtable, pool.dlens, q, max_len=0, weights=w) == 0)
    assert torch.all(binding.paged_attention(cache, pool.dtable[:, :0], pool.dlens, q) == 0)
    assert torch.all(w == 1)
    none = torch.empty(0, dtype=torch.int32, device="cuda")
    assert binding.paged_attention(cache, pool.dtable[:0], none, q[:0]).shape == (0, 4, 64)
    starts = torch.zeros(3, dtype=torch.int32, device="cuda")
    binding.kv_append(cache, pool.dtable, pool.dlens, starts, q[:0, :2], q[:0, :2])
    new_w, new_p, left = binding.kv_evict(cache, pool.dtable, pool.dlens, pool.dlens, w, pos, 4, 0, max_len=0)
    assert torch.all(new_w == 0) and torch.all(new_p == -1) and torch.all(left == 0)
    new_w, _, left = binding.kv_evict(cache, pool.dtable[:0], none, none, w[:0], pos[:0], 4, 0)
    assert new_w.shape == (0, 2, 32) and left.shape == (0,)
    empty = binding.PagedCache(pool.dk[:0], pool.dv[:0])      # a pool without pages: every page is a hole
    assert torch.all(binding.paged_attention(empty, pool.dtable, pool.dlens, q) == 0)
    assert _same(pool.dk.cpu(), pool.k)


@pytest.mark.parametrize("budget,recent", [(5000, 300), (39990, 64), (39998, 0), (20000, 25000)])
def test_evict_past_the_held_keys(gpu, budget, recent):
    # more slots than LDS holds keys of
    _check_evict([40000, 33000], 1, 8, 64, budget, recent, seed=budget, ties=budget == 5000)


@pytest.mark.parametrize("few", [1, 2, 3, 4, 5])
def test_evict_few_among_equals(gpu, few):
    # the last of equals go first, newest or not
    rng = np.random.default_rng(few)
    for recent in (0, 3, 64):
        n, budget = 64 + few, 64
        pool = ref.Pool([n], 1, 8, 16, torch.float16, seed=few)
        w = np.zeros((1, 1, pool.width * 16), np.float32)
        w[0, 0, : n // 2] = rng.integers(0, 2, n // 2)
        pos = np.arange(pool.width * 16, dtype=np.int32).reshape(1, 1, -1)
        source, want_w, want_p, _ = ref.evict([n], [n], w, pos, budget, recent, w.shape[2])
        seen = torch.tensor([n], dtype=torch.int32, device="cuda")
        new_w, new_p, _ = binding.kv_evict(binding.PagedCache(pool.dk, pool.dv), pool.dtable, pool.dlens, seen,
                                           torch.from_numpy(w).cuda(), torch.from_numpy(pos).cuda(), budget, recent)
        assert np.array_equal(new_w.cpu().numpy(), want_w) and np.array_equal(new_p.cpu().numpy(), want_p)


# whole and cut lengths on both sides of the rules that choose how a length is shared out
@pytest.mark.parametrize("n", [256, 257, 320, 511, 512, 767, 768, 769, 1023, 1025, 2049])
def test_sharing_of_lengths(gpu, n):
    for B, kv in ((1, 1), (3, 4), (33, 4)):
        lens = [n] + [1 + (n * i) // B for i in range(1, B)]
        pool = ref.Pool(lens if B < 33 else [n, 1, 17] * 11, kv, 8, 16, seed=n)
        _check(pool, _query(B, kv * 2, 8, torch.float16, n), f"{B} of up to {n}, {kv} heads", weighted=B < 33)


def test_many_query_heads_over_long_lengths(gpu):
    # several sets of 16 query heads read the same keys, in padded groups of workgroups
    pool = ref.Pool([1500, 700, 1499], 1, 16, 16, seed=21)
    _check(pool, _query(3, 40, 16, torch.float16, 21), "40 heads over 1")
    pool = ref.Pool([1500, 700, 1499], 2, 16, 24, seed=22)
    _check(pool, _query(3, 34, 16, torch.float16, 22), "34 heads over 2, loose pages")


def test_first_call_inside_graph_capture(gpu):
    # a fresh process whose first calls of these operators are captured
    import os
    import subprocess
    import sys

    code = """
import torch
from memory_bound_gemv_row_amd import binding as B
g = torch.Generator(device="cuda").manual_seed(1)
k = torch.randn((40, 16, 2, 64), generator=g, device="cuda").half()
c = B.PagedCache(k, k.clone())
t = torch.arange(40, dtype=torch.int32, device="cuda").view(2, 20)
n = torch.tensor([300, 20], dtype=torch.int32, device="cuda")
q = torch.randn((2, 8, 64), generator=g, device="cuda").half()
w = torch.rand((2, 2, 320), generator=g, device="cuda")
p = torch.arange(320, dtype=torch.int32, device="cuda").expand(2, 2, 320).contiguous()
A = torch.randint(-127, 128, (96, 512), generator=g, device="cuda", dtype=torch.int8)
s = torch.rand(96, generator=g, device="cuda").half()
torch.cuda.synchronize()
def work():
    x, xs = B.quantize_tokens_q8(q.view(2, 512))
    return [B.gemm_q8(A, s, x, xs), B.paged_attention(c, t, n, q), *B.kv_evict(c, t, n, n, w, p, 100, 10)]
graph, stream = torch.cuda.CUDAGraph(), torch.cuda.Stream()
with torch.cuda.stream(stream), torch.cuda.graph(graph, stream=stream):
    outs = work()
torch.cuda.synchronize()
graph.replay()      # its eviction moves rows; later passes find the cache so
torch.cuda.synchronize()
graph.replay()
torch.cuda.synchronize()
got = [o.clone() for o in outs]
assert all(torch.equal(a, b) for a, b in zip(got, work()))
print("first-call capture ok", flush=True)
"""
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    say("[serving graph] first call captured, fresh process")
    r = subprocess.run([sys.executable, "-c", code], cwd=root, capture_output=True, text=True, timeout=240)
    assert r.returncode == 0 and "first-call capture ok" in r.stdout, r.stdout[-2000:] + r.stderr[-2000:]


def test_append_tracks_only_what_it_writes(gpu):
    # a token in a hole leaves weights and positions as they were; one past the
    # tracked slots is written without them
    pool = ref.Pool([20, 30], 2, 64, 16, seed=1, width=2)
    pool.table[0, 1] = -1
    pool.dtable = pool.table.cuda()
    g = torch.Generator().manual_seed(1)
    new = torch.randn((2, 2, 64), generator=g).to(torch.float16)
    want_k, _ = _append_reference(pool, [20, 30], [1, 1], new, new)
    w = torch.full((2, 2, 24), 5.0, device="cuda")
    pos = torch.full((2, 2, 24), 7, dtype=torch.int32, device="cuda")
    say("[append] a hole and a slot past the tracked ones")
    binding.kv_append(binding.PagedCache(pool.dk, pool.dv), pool.dtable, pool.dlens,
                      torch.arange(3, dtype=torch.int32, device="cuda"), new.cuda(), new.cuda(), weights=w, positions=pos,
                      seen=pool.dlens)
    assert torch.all(w == 5) and torch.all(pos == 7) and _same(pool.dk.cpu(), want_k)


def test_evict_of_many_sequences(gpu):
    # more heads than the moving launch has blocks for at their usual number
    B, H, n, budget, page = 3000, 2, 160, 70, 16
    g = torch.Generator(device="cuda").manual_seed(1)
    width = n // page
    k = torch.randn((B * width, page, H, 8), generator=g, device="cuda").half()
    table = torch.randperm(B * width, generator=g, device="cuda").to(torch.int32).view(B, width)
    lens = torch.full((B,), n, dtype=torch.int32, device="cuda")
    w = torch.rand((B, H, n), generator=g, device="cuda")
    pos = torch.arange(n, dtype=torch.int32, device="cuda").expand(B, H, n).contiguous()
    before = k.clone()
    say("[evict] 6000 heads")
    cache = binding.PagedCache(k, k.clone())
    new_w, new_p, left = binding.kv_evict(cache, table, lens, lens, w, pos, budget, 5)
    assert torch.all(left == budget) and torch.all(new_p[..., budget:] == -1)
    kept = torch.where(pos >= n - 5, torch.inf, w).topk(budget, dim=2).indices.sort(2).values
    assert torch.equal(new_p[..., :budget].sort(2).values.long(), kept)      # positions are slots here
    assert torch.equal(new_w[..., :budget], w.gather(2, new_p[..., :budget].long()))
    at = new_p[..., :budget].long()
    b = torch.arange(B, device="cuda").view(B, 1, 1)
    h = torch.arange(H, device="cuda").view(1, H, 1)
    old = before[table.long()[b, at // page], at % page, h]
    now = k[table.long()[b, torch.arange(budget, device="cuda").view(1, 1, -1) // page],
            torch.arange(budget, device="cuda").view(1, 1, -1) % page, h]
    assert torch.equal(old, now)


def test_more_query_heads_than_a_join_holds(gpu):
    # the weights of 70 and 130 query heads over one key-value head, short and split
    for heads in (70, 130):
        _check(ref.Pool([300, 40], 1, 64, 16, seed=heads), _query(2, heads, 64, torch.float16, heads), f"{heads} over 1")
        _check(ref.Pool([1300, 7], 1, 128, 16, torch.bfloat16, seed=heads), _query(2, heads, 128, torch.bfloat16, heads),
               f"{heads} over 1, split")


def test_evict_refuses_outputs_that_overlap(gpu):
    # in part, with one another, and `seen`, which workgroups read while another writes the lengths
    pool = ref.Pool([20, 20], 2, 64, 16, seed=1)
    cache = binding.PagedCache(pool.dk, pool.dv)
    w = torch.rand((3, 2, 2, 32), device="cuda")
    pos = torch.zeros((3, 2, 2, 32), dtype=torch.int32, device="cuda")
    seen, left = pool.dlens.clone(), torch.zeros(2, dtype=torch.int32, device="cuda")
    part = w.flatten()[64: 192].view(2, 2, 32)              # the second half of w[0] and the first of w[1]
    say("[evict] outputs that overlap")
    for out in ((part, pos[1], left), (w[1], pos[0], left), (w[1], pos[1], pool.dlens), (w[1], pos[1], seen),
                (w[1], w[1].view(torch.int32), left), (w[1], pos[1], pos[1, 0, 0, :2])):
        with pytest.raises(ValueError):
            binding.kv_evict(cache, pool.dtable, pool.dlens, seen, w[0], pos[0], 8, 2, out=out)
    binding.kv_evict(cache, pool.dtable, pool.dlens, seen, w[0], pos[0], 8, 2, out=(w[1], pos[1], left))
    assert torch.all(left == 8)


@pytest.mark.parametrize("lens,kv,heads", [([60, 3], 2, 6), ([250, 17], 2, 40), ([1500, 700], 1, 34)])
def test_attention_in_place(gpu, lens, kv, heads):
    # the outputs in the queries' memory: one part, one workgroup of eight waves, split and joined
    pool = ref.Pool(lens, kv, 64, 16, torch.bfloat16, seed=heads)
    cache = binding.PagedCache(pool.dk, pool.dv)
    q = _query(len(lens), heads, 64, torch.bfloat16, heads).cuda()
    want = binding.paged_attention(cache, pool.dtable, pool.dlens, q)
    w, again = (torch.zeros((len(lens), kv, pool.width * 16), device="cuda") for _ in range(2))
    say(f"[attention] in place, {heads} heads over {kv}")
    binding.paged_attention(cache, pool.dtable, pool.dlens, q.clone(), weights=w)
    both = q.clone()
    assert binding.paged_attention(cache, pool.dtable, pool.dlens, both, weights=again, out=both) is both
    assert torch.equal(both, want) and torch.equal(w, again)


def test_keys_and_values_of_one_buffer(gpu):
    # the two as parts of one array, page by page, as many programs keep them
    pool = ref.Pool([90, 1, 200], 2, 80, 16, torch.float16, seed=6)
    both = torch.stack([pool.k, pool.v], 1).cuda()
    pool.dk, pool.dv = both[:, 0], both[:, 1]
    _check(pool, _query(3, 4, 80, torch.float16, 6), "keys and values in one buffer")


def test_pages_shared_by_sequences(gpu):
    # a common first part: one page in two tables, and twice in one; only unshared pages are written
    pool = ref.Pool([70, 61, 40], 2, 64, 16, torch.bfloat16, seed=13)
    pool.table[1, 0] = pool.table[0, 0]
    pool.table[2, 1] = pool.table[2, 0]
    pool.dtable = pool.table.cuda()
    q = _query(3, 4, 64, torch.bfloat16, 13)
    _check(pool, q, "shared pages")
    new = torch.randn((3, 2, 64), generator=torch.Generator().manual_seed(13)).to(torch.bfloat16)
    want_k, want_v = _append_reference(pool, pool.lens, [1, 1, 1], new, new)
    binding.kv_append(binding.PagedCache(pool.dk, pool.dv), pool.dtable, pool.dlens,
                      torch.arange(4, dtype=torch.int32, device="cuda"), new.cuda(), new.cuda())
    assert _same(pool.dk.cpu(), want_k) and _same(pool.dv.cpu(), want_v)
