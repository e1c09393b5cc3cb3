"""Norms and rotation of queries and keys, into tensors and into a paged cache,
against the plain 64-bit form."""
import numpy as np
import pytest
import torch

from memory_bound_gemv_row_amd import binding

import between_ref as bref
from gpu_util import say

pytestmark = pytest.mark.gpu

TYPES = [torch.float32, torch.float16, torch.bfloat16]


def _freqs(half, base=10000.0):
    return base ** -(np.arange(half) / max(half, 1))


def _random(shape, dtype, seed, spread=2.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(shape, generator=g) * spread).to(dtype)


def _close(got, want, bound, label):
    off = np.abs(got.cpu().double().numpy() - want)
    assert np.all(off <= bound), (label, float(np.nanmax(off / bound)), int(np.isnan(off).sum()))


def _check(rows, heads, kv, dim, rotated, dtype, out_dtype, label, interleaved=False, weighted=True, eps=1e-6, apart=0, far=1000,
           weight_dtype=None, seed=1, made=None):
    say(f"[rotate] {label}")
    made = _random((rows, (heads + kv) * dim + apart), dtype, seed) if made is None else made
    q, k = made[:, : heads * dim].view(rows, heads, dim), made[:, heads * dim: (heads + kv) * dim].view(rows, kv, dim)
    device = made.cuda()
    dq, dk = device[:, : heads * dim].view(rows, heads, dim), device[:, heads * dim: (heads + kv) * dim].view(rows, kv, dim)
    rng = np.random.default_rng(seed)
    positions = (rng.integers(0, far + 1) + np.arange(rows)).astype(np.int32)
    freqs = _freqs(rotated // 2)
    weights = [_random((dim,), weight_dtype or dtype, seed + 1 + i, 0.5) if weighted else None for i in range(2)]
    dw = [w.cuda() if w is not None else None for w in weights]
    got = binding.norm_rotate(dq, dk, torch.from_numpy(positions).cuda(), torch.from_numpy(freqs).cuda(), *dw, eps=eps,
                              interleaved=interleaved, out_dtype=out_dtype)
    for x, w, y in zip((q, k), weights, got):
        assert y.dtype == out_dtype and y.shape == x.shape
        want, bound = bref.turned(x, None if w is None else w.double().numpy(), positions, freqs, eps, interleaved, out_dtype)
        _close(y, want, bound, label)
    return got


@pytest.mark.parametrize("out_dtype", TYPES, ids=str)
@pytest.mark.parametrize("dtype", TYPES, ids=str)
@pytest.mark.parametrize("interleaved", [False, True], ids=["halves", "neighbours"])
def test_types(gpu, dtype, out_dtype, interleaved):
    _check(9, 5, 2, 64, 64, dtype, out_dtype, f"{dtype} to {out_dtype}", interleaved)
    _check(9, 5, 2, 42, 30, dtype, out_dtype, f"{dtype} to {out_dtype}, odd", interleaved)


@pytest.mark.parametrize("interleaved", [False, True], ids=["halves", "neighbours"])
@pytest.mark.parametrize("dim,rotated", [(1, 0), (2, 2), (3, 2), (8, 8), (8, 0), (16, 16), (24, 16), (40, 16), (40, 32), (64, 32), (64, 6),
                                         (72, 72), (80, 80), (96, 48), (104, 16), (120, 112), (128, 128), (128, 64), (129, 128), (136, 8),
                                         (200, 130), (248, 240), (255, 254), (256, 256), (256, 16), (256, 0)])
def test_sizes(gpu, dim, rotated, interleaved):
    _check(7, 6, 3, dim, rotated, torch.bfloat16, torch.bfloat16, f"dim {dim} rotated {rotated}", interleaved)


@pytest.mark.parametrize("rows", [1, 2, 3, 63, 500, 9000])
def test_rows(gpu, rows):
    _check(rows, 8, 2, 64, 64, torch.float16, torch.float16, f"{rows} rows", apart=64)
    _check(rows, 3, 1, 20, 20, torch.float16, torch.float16, f"{rows} rows, odd", apart=5)


@pytest.mark.parametrize("heads,kv", [(1, 1), (3, 0), (0, 2), (64, 8), (9, 9), (130, 1)])
def test_heads(gpu, heads, kv):
    _check(5, heads, kv, 128, 128, torch.bfloat16, torch.float16, f"{heads} and {kv} heads")
    _check(5, heads, kv, 12, 8, torch.bfloat16, torch.float16, f"{heads} and {kv} heads, odd")


def test_without_norm_and_without_weights(gpu):
    for dim in (64, 22):
        _check(6, 4, 2, dim, dim, torch.float32, torch.float32, "no norm", weighted=False, eps=None)
        _check(6, 4, 2, dim, dim, torch.float32, torch.float32, "no weights", weighted=False)
        _check(6, 4, 2, dim, dim, torch.bfloat16, torch.bfloat16, "weights of 32 bits", weight_dtype=torch.float32)
        _check(6, 4, 2, dim, dim, torch.float32, torch.bfloat16, "weights of 16 bits", weight_dtype=torch.float16)


def test_far_positions(gpu):
    # angles of two thousand million radians, and negative ones
    for far in (1_000_000, (1 << 31) - 100):
        _check(40, 2, 1, 64, 64, torch.float32, torch.float32, f"positions to {far}", far=far, seed=far % 97)
    say("[rotate] the last positions there are")
    x = _random((4, 1, 32), torch.float32, 3)
    positions = np.array([(1 << 31) - 1, -(1 << 31), -1, 0], np.int32)
    freqs = _freqs(16)
    y, _ = binding.norm_rotate(x.cuda(), x.cuda(), torch.from_numpy(positions).cuda(), torch.from_numpy(freqs).cuda(), eps=None)
    want, bound = bref.turned(x, None, positions, freqs, None, False, torch.float32)
    _close(y, want, bound, "last positions")
    assert torch.equal(y[3].cpu(), x[3])


def test_unaligned_rows(gpu):
    # rows that are not 16-byte aligned go element by element
    room = _random((5 * 4 * 64 + 1,), torch.float16, 4)
    q = room[1:].view(5, 4, 64)
    dq = room.cuda()[1:].view(5, 4, 64)
    say("[rotate] unaligned")
    positions, freqs = np.arange(5, dtype=np.int32), _freqs(32)
    y, _ = binding.norm_rotate(dq, dq, torch.from_numpy(positions).cuda(), torch.from_numpy(freqs).cuda())
    want, bound = bref.turned(q, None, positions, freqs, 1e-6, False, torch.float16)
    _close(y, want, bound, "unaligned")


@pytest.mark.parametrize("dim,rotated,interleaved", [(128, 128, False), (128, 64, True), (50, 34, False)])
def test_in_place(gpu, dim, rotated, interleaved):
    rows, heads, kv = 300, 5, 2
    made = _random((rows, (heads + 2 * kv) * dim), torch.bfloat16, 6).cuda()
    q, k = made[:, : heads * dim].view(rows, heads, dim), made[:, heads * dim: (heads + kv) * dim].view(rows, kv, dim)
    positions = torch.arange(rows, dtype=torch.int32, device="cuda")
    freqs = torch.from_numpy(_freqs(rotated // 2)).cuda()
    rest = made[:, (heads + kv) * dim:].clone()
    say("[rotate] in place")
    want = binding.norm_rotate(q, k, positions, freqs, interleaved=interleaved)
    out = binding.norm_rotate(q, k, positions, freqs, interleaved=interleaved, out=(q, k))
    assert out[0] is q and torch.equal(q, want[0]) and torch.equal(k, want[1])
    assert torch.equal(made[:, (heads + kv) * dim:], rest)


def test_zero_and_special_heads(gpu):
    q = torch.zeros((4, 2, 64), dtype=torch.float16)
    q[1, 0, 3], q[2, 1, 40] = float("nan"), float("inf")
    q[3] = 65504.0
    say("[rotate] special values")
    positions, freqs = torch.arange(4, dtype=torch.int32, device="cuda"), torch.from_numpy(_freqs(32)).cuda()
    y, _ = binding.norm_rotate(q.cuda(), q.cuda(), positions, freqs)
    y = y.cpu()
    assert torch.all(y[0] == 0) and torch.all(y[1, 1] == 0) and torch.all(y[2, 0] == 0)
    assert torch.all(torch.isnan(y[1, 0])) and torch.isnan(y[2, 1, 40]) and torch.isnan(y[2, 1, 8])
    assert torch.all(y[2, 1, :8] == 0) and torch.all(torch.isfinite(y[3]))


# ---------------------------------------------------------------- into the cache
def _cache(pages, page, heads, dim, dtype, layout):
    def make():
        if layout == "heads":
            return torch.full((pages, heads, page, dim), 7.0, dtype=dtype, device="cuda").transpose(1, 2)
        if layout == "padded":
            return torch.full((pages, page + 1, heads + 1, dim + 8), 7.0, dtype=dtype, device="cuda")[:, :page, :heads, :dim]
        return torch.full((pages, page, heads, dim), 7.0, dtype=dtype, device="cuda")
    return binding.PagedCache(make(), make())


@pytest.mark.parametrize("layout", ["slots", "heads", "padded"])
@pytest.mark.parametrize("page", [1, 5, 16])
@pytest.mark.parametrize("dtype,cache_dtype", [(torch.bfloat16, torch.bfloat16), (torch.float32, torch.float16)], ids=str)
@pytest.mark.parametrize("dim,rotated,interleaved", [(64, 64, False), (128, 96, True), (24, 10, False)])
def test_append(gpu, dim, rotated, interleaved, dtype, cache_dtype, page, layout):
    rows, heads, kv, pages = 37, 6, 2, 50
    made = _random((rows, (heads + 2 * kv) * dim), dtype, dim)
    parts = lambda t: (t[:, : heads * dim].view(rows, heads, dim), t[:, heads * dim: (heads + kv) * dim].view(rows, kv, dim),
                       t[:, (heads + kv) * dim:].view(rows, kv, dim))
    q, k, v = parts(made)
    rng = np.random.default_rng(page)
    slots = rng.permutation(pages * page)[:rows] if pages * page >= rows else rng.permutation(rows)
    slots[3], slots[20], slots[30] = -1, pages * page, 1 << 40
    weights = [_random((dim,), dtype, 5 + i, 0.5) for i in range(2)]
    positions, freqs = rng.integers(0, 5000, rows).astype(np.int32), _freqs(rotated // 2)
    cache = _cache(pages, page, kv, dim, cache_dtype, layout)
    say(f"[rotate] append dim {dim} page {page} {layout} {dtype}")
    out = binding.norm_rotate_append(cache, torch.from_numpy(slots.astype(np.int64)).cuda(), *parts(made.cuda()),
                                     torch.from_numpy(positions).cuda(), torch.from_numpy(freqs).cuda(), *[w.cuda() for w in weights],
                                     interleaved=interleaved)
    want, bound = bref.turned(q, weights[0].double().numpy(), positions, freqs, 1e-6, interleaved, cache_dtype)
    _close(out, want, bound, "queries")
    want, bound = bref.turned(k, weights[1].double().numpy(), positions, freqs, 1e-6, interleaved, cache_dtype)
    got_k, got_v = (t.cpu().reshape(pages * page, kv, dim) for t in (cache.k, cache.v))
    here = [i for i in range(rows) if 0 <= slots[i] < pages * page]
    at = slots[here]
    _close(got_k[at], want[here], bound[here], "keys")
    assert torch.equal(got_v[at], v[here].to(cache_dtype))
    rest = np.setdiff1d(np.arange(pages * page), at)
    assert torch.all(got_k[rest] == 7.0) and torch.all(got_v[rest] == 7.0)
    if layout == "padded":
        for t in (cache.k, cache.v):
            whole = t.as_strided((pages, page + 1, kv + 1, dim + 8), (t.stride(0), t.stride(1), t.stride(2), 1))
            assert torch.all(whole[:, page:] == 7.0) and torch.all(whole[:, :, kv:] == 7.0) and torch.all(whole[..., dim:] == 7.0)


def test_append_past_32_bits(gpu):
    pages, page, heads, dim = 8600, 64, 32, 128
    say("[rotate] a pool past 2^31 elements")
    cache = _cache(pages, page, heads, dim, torch.float16, "slots")
    assert cache.k.numel() > 1 << 31
    q, k, v = (_random((2, heads, dim), torch.float16, i).cuda() for i in range(3))
    slots = torch.tensor([pages * page - 1, 5], device="cuda")
    positions, freqs = torch.zeros(2, dtype=torch.int32, device="cuda"), torch.from_numpy(_freqs(64)).cuda()
    binding.norm_rotate_append(cache, slots, q, k, v, positions, freqs, eps=None)
    assert torch.equal(cache.k[-1, -1], k[0]) and torch.equal(cache.v[0, 5], v[1]) and torch.equal(cache.v[-1, -1], v[0])
    # slots past 2^31 of small pages
    small = _cache(1 << 20, 4096, 1, 8, torch.float16, "slots") if torch.cuda.mem_get_info()[0] > 200 << 30 else None
    if small is not None:
        slots = torch.tensor([(1 << 32) - 1, (1 << 31) + 3], device="cuda")
        q, k, v = (t[:, :1, :8].contiguous() for t in (q, k, v))
        binding.norm_rotate_append(small, slots, q, k, v, positions, freqs[:4].contiguous(), eps=None)
        flat = small.v.view(-1, 8)
        assert torch.equal(flat[(1 << 32) - 1], v[0, 0]) and torch.equal(flat[(1 << 31) + 3], v[1, 0])


def test_streams_and_graphs(gpu):
    q, k = _random((70, 8, 128), torch.bfloat16, 1).cuda(), _random((70, 2, 128), torch.bfloat16, 2).cuda()
    positions, freqs = torch.arange(70, dtype=torch.int32, device="cuda"), torch.from_numpy(_freqs(64)).cuda()
    say("[rotate] streams and graphs")
    want = binding.norm_rotate(q, k, positions, freqs)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    other = binding.norm_rotate(q, k, positions, freqs, stream=side)
    side.synchronize()
    assert torch.equal(other[0], want[0]) and torch.equal(other[1], want[1])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = binding.norm_rotate(q, k, positions, freqs)
    base = q.clone()
    for factor in (1.0, -0.5, 2.0):
        q.copy_(base * factor)
        positions.add_(3)
        graph.replay()
        torch.cuda.synchronize()
        again = binding.norm_rotate(q, k, positions, freqs)
        assert torch.equal(out[0], again[0]) and torch.equal(out[1], again[1])
