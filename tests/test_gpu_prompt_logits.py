"""Attention of several new tokens, and behind prefixes, where logits are large: of
one visible key far above the others a row gets the value itself, of equal
ones their mean, whatever the logits' size and however the keys are split."""
import numpy as np
import pytest
import torch

from memory_bound_gemv_row_amd import binding

import prompt_ref as pref
import serving_ref as ref
from gpu_util import say
from test_gpu_prompt import _pools, _starts

pytestmark = pytest.mark.gpu

U32 = ref.U32
# (type, size of queries and keys): logits of 3e7 to 1e10, and of 1e17 to 1e31
LARGE = [(torch.float16, 2000.0), (torch.float16, 6000.0), (torch.float16, 20000.0), (torch.bfloat16, 6000.0), (torch.bfloat16, 1e9),
         (torch.bfloat16, 1e16)]


def _large(pool, size, seed):
    """Keys of the held slots are uniform between -3 and 3 times `size`, which the type holds."""
    g = torch.Generator().manual_seed(seed)
    for b, n in enumerate(pool.lens):
        for j in range(n):
            shape = pool.k[0, 0].shape
            pool.k[pool.table[b, j // pool.page], j % pool.page] = ((torch.rand(shape, generator=g) * 6 - 3) * size).to(pool.k.dtype)
    pool.dk = pool.k.cuda()


def _large_query(rows, heads, dim, dtype, size, seed):
    return ((torch.rand((rows, heads, dim), generator=torch.Generator().manual_seed(seed)) * 6 - 3) * size).to(dtype)


def _winners(k, q, sees, scale):
    """(slot of each row's largest logit, whether it is so far above the others, by
    more than both logits' errors in binary32 and 200, that they weigh nothing)."""
    x = np.where(sees, (q @ k.T) * scale, -np.inf)
    mag = np.abs(q) @ np.abs(k).T * abs(scale)
    e = np.where(sees, 2 * k.shape[1] * U32 * mag + 6 * U32 * np.abs(np.where(sees, x, 0)), 0)
    best = x.argmax(-1)
    at = np.arange(len(best))
    low = x[at, best] - e[at, best]
    others = x + e
    others[at, best] = -np.inf
    return best, low > others.max(-1) + 200


def _expect(got, k, v, q, sees, scale, label):
    best, clear = _winners(k, q, sees, scale)
    assert clear.mean() > 0.9, label
    off = np.flatnonzero(clear & ~(got == v[best]).all(-1))
    assert off.size == 0, (label, off.size, int(clear.sum()), got[off[0], :4], v[best[off[0]], :4])


@pytest.mark.parametrize("dtype,size", LARGE, ids=str)
@pytest.mark.parametrize("lens,news,kv,heads,dim,page,window", [
    ([300, 90], [300, 90], 2, 4, 128, 16, None),
    ([300, 90], [300, 90], 2, 4, 64, 24, 50),
    ([3000], [5], 1, 4, 128, 16, None),
    ([5000, 4097], [7, 2], 1, 4, 64, 16, None),
    ([200, 130], [130, 130], 1, 2, 256, 16, None),
    ([200, 130], [200, 60], 2, 4, 96, 5, None),
], ids=["whole", "window", "split", "shared out", "256", "loose"])
def test_the_largest_logit_has_all_the_weight(gpu, lens, news, kv, heads, dim, page, window, dtype, size):
    label = f"large logits {lens} {news} {dim} {dtype} {size}"
    say(f"[prompt] {label}")
    pool = ref.Pool(lens, kv, dim, page, dtype, seed=41)
    _large(pool, size, 42)
    starts = _starts(news)
    q = _large_query(sum(news), heads, dim, dtype, size, 43)
    scale, G = dim ** -0.5, heads // kv
    out = binding.prompt_attention(binding.PagedCache(pool.dk, pool.dv), pool.dtable, pool.dlens,
                                   torch.tensor(starts, dtype=torch.int32, device="cuda"), q.cuda(), max_new=max(news),
                                   window=window).cpu().double().numpy()
    for b, (L, n) in enumerate(zip(lens, news)):
        k, v = (ref.gathered(pool, p, b, L)[0] for p in (pool.k, pool.v))
        sees = pref.seen(n, L, window)
        for h in range(heads):
            _expect(out[starts[b]: starts[b + 1], h], k[h // G], v[h // G], q[starts[b]: starts[b + 1], h].double().numpy(), sees, scale,
                    label)


@pytest.mark.parametrize("dtype,size", LARGE, ids=str)
@pytest.mark.parametrize("dim,page", [(128, 16), (64, 24), (256, 16)])
def test_the_largest_logit_behind_a_prefix(gpu, dim, page, dtype, size):
    far_lens, groups, lens, kv, heads = [700, 40], [0, 3, 5], [30, 0, 200, 1, 64], 1, 4
    label = f"large logits behind a prefix {dim} {dtype} {size}"
    say(f"[prefix] {label}")
    both, far, near = _pools(far_lens, lens, kv, dim, page, dtype, 44)
    _large(both, size, 45)
    q = _large_query(len(lens), heads, dim, dtype, size, 46)
    out = binding.prefix_attention(binding.PagedCache(both.dk, both.dv), far.dtable, far.dlens,
                                   torch.tensor(groups, dtype=torch.int32, device="cuda"), near.dtable, near.dlens,
                                   q.cuda()).cpu().double().numpy()
    clear = []
    for b, n in enumerate(lens):
        g = 0 if b < groups[1] else 1
        k, v = (np.concatenate([ref.gathered(far, p, g, far_lens[g])[0][0], ref.gathered(near, p, b, n)[0][0]]) for p in (both.k, both.v))
        best, is_clear = _winners(k, q[b].double().numpy(), np.ones((heads, len(k)), bool), dim ** -0.5)
        clear.append(is_clear)
        assert np.array_equal(out[b][is_clear], v[best[is_clear]]), (label, b)
    assert np.mean(clear) > 0.8


@pytest.mark.parametrize("dtype,size", LARGE, ids=str)
def test_equal_large_logits_have_equal_weights(gpu, dtype, size):
    # one key in every slot: the mean of the values, in one part and in several.  The
    # powers are equal numbers p, so a weight is 1 / n but for the sums' 24 units for every
    # sixteen keys, 256 parts, the division's two, and the store's rounding
    for lens, news, heads in (([300], [300], 4), ([3000], [4], 4)):
        say(f"[prompt] equal large logits {lens} {dtype} {size}")
        pool = ref.Pool(lens, 1, 128, 16, dtype, seed=47)
        one = ((torch.rand(128, generator=torch.Generator().manual_seed(48)) + 0.5) * size).to(dtype)
        for j in range(lens[0]):
            pool.k[pool.table[0, j // 16], j % 16, 0] = one
        pool.dk = pool.k.cuda()
        q = one.expand(news[0], heads, 128).contiguous()
        out = binding.prompt_attention(binding.PagedCache(pool.dk, pool.dv), pool.dtable, pool.dlens,
                                       torch.tensor(_starts(news), dtype=torch.int32, device="cuda"), q.cuda()).cpu().double().numpy()
        v = ref.gathered(pool, pool.v, 0, lens[0])[0][0]
        for t in range(news[0]):
            n = lens[0] - news[0] + t + 1
            want, rel = v[:n].mean(0), (24 * -(-n // 16) + 256 + 2) * U32
            bound = pref.stored(want, rel * 2 * np.abs(v[:n]).mean(0), dtype)
            assert np.all(np.abs(out[t] - want) <= bound), (t, dtype, size)


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16], ids=str)
def test_large_logits_that_rise_with_every_key(gpu, dtype):
    # each key's logit is above the last one's by 65536 or more, so every tile moves the
    # maximum and the newest visible token has all the weight; falling, the first one
    n = 120
    pool = ref.Pool([n], 1, 64, 16, dtype, seed=49)
    first = 2048.0 if dtype == torch.float16 else 128.0   # from where the type's steps are 2 and 1
    for j in range(n):
        pool.k[pool.table[0, j // 16], j % 16, 0] = first + j * (2 if dtype == torch.float16 else 1)
    pool.dk = pool.k.cuda()
    say(f"[prompt] rising large logits {dtype}")
    for sign in (1.0, -1.0):
        q = torch.full((n, 2, 64), 8192.0 * sign, dtype=dtype)
        out = binding.prompt_attention(binding.PagedCache(pool.dk, pool.dv), pool.dtable, pool.dlens,
                                       torch.tensor([0, n], dtype=torch.int32, device="cuda"), q.cuda()).cpu().double().numpy()
        v = ref.gathered(pool, pool.v, 0, n)[0][0]
        want = v if sign > 0 else np.repeat(v[:1], n, 0)
        for h in range(2):
            assert np.array_equal(out[:, h], want), (dtype, sign)
