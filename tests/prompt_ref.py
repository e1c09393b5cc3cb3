"""Plain 64-bit forms of attention with several new tokens per sequence, through
a window and behind shared prefixes, and the bounds of their errors."""
import numpy as np
import torch

import serving_ref as ref

U32, HALF_STEP, SMALLEST = ref.U32, ref.HALF_STEP, ref.SMALLEST


def seen(n, length, window=None, sinks=0):
    """bool [n, length]: which slots each of the last n tokens of a sequence sees."""
    p = np.arange(length - n, length)[:, None]
    j = np.arange(length)[None, :]
    sees = j <= p
    if window is not None:
        sees = sees & ((j > p - window) | (j < sinks))
    return sees


def attend(k, v, q, sees, scale, rounding, lowest):
    """(out, bound) in float64 of queries q [R, D] over keys and values [L, D];
    sees bool [R, L].  rounding [L]: the relative error of each power where it
    meets its value; lowest: what a power may be off by when its type cannot
    hold it.

    The logits' errors e are those of ref.attention_by_slot.  A power is off by
    exp(x + e) - exp(x), by four units (exp2, and its argument's sum), by its
    rounding, relative to the power itself or `lowest` of the largest, and in
    binary32 by 2^-126 of that.  All sums of a row run over its keys sixteen at a
    time, each time with 16 additions and at most one rescaling (24 units hold
    them), and over at most 256 parts.  The sum over the powers is that of the
    rounded ones: its error is that of theirs together, S; a probability's then
    (its own + p S) / (1 - S), and the division takes two units."""
    with np.errstate(invalid="ignore"):
        x = np.where(sees, (q @ k.T) * scale, -np.inf)
    counts = x > -np.inf
    live = counts.any(-1)
    top = np.where(live, np.max(np.where(counts, x, -np.inf), -1, initial=-np.inf), 0)[:, None]
    mag = (np.abs(q) @ np.abs(np.where(np.isfinite(k), k, 0)).T) * abs(scale)
    far = np.where(counts, x, 0)
    D, L = q.shape[1], k.shape[0]
    e = np.where(counts, 2 * D * U32 * mag + 6 * U32 * (np.abs(far) + np.abs(top)), 0)
    power = np.exp(np.where(counts, x - top, -np.inf))
    Z = np.where(live, power.sum(-1), 1)[:, None]
    p = power / Z
    sums = (24 * -(-L // 16) + 256) * U32
    diff = (np.exp(np.where(counts, x - top + e, -np.inf)) - power) / Z + p * (4 * U32 + sums) + \
        np.where(counts, np.maximum(p * rounding[None, :], lowest) + 2.0 ** -126, 0)
    S = diff.sum(-1, keepdims=True)
    assert np.all(S < 0.5), "logits too large for this bound"
    off = (diff + p * S) / (1 - S)
    v = np.where(counts.any(0)[:, None], v, 0)   # what no row sees may be anything
    return p @ v, (off + 2 * U32 * p) @ np.abs(v)


def stored(out, bound, dtype):
    half = HALF_STEP[dtype]
    return bound * (1 + half) + half * np.abs(out) + SMALLEST[dtype]


def _power_errors(dtype):
    # relative, and of the largest: a power is below 2^8 times the reference
    # maximum's, whose own power is 1; binary16 has steps of 2^-24 at the least
    return HALF_STEP[dtype], 2.0 ** -25 if dtype == torch.float16 else 2.0 ** -133


def prompt(pool, q, starts, scale, window=None, sinks=0, rounded=True):
    """(out, bound, rows) float64 of q [rows, heads, D]; rows: the rows that belong to a sequence."""
    rows, heads, D = q.shape
    H, G = pool.heads, heads // pool.heads
    slots = pool.width * pool.page
    out, bound, mine = np.zeros((rows, heads, D)), np.zeros((rows, heads, D)), np.zeros(rows, bool)
    half, low = _power_errors(q.dtype) if rounded else (0.0, 0.0)
    qd = q.double().numpy()
    for b, L in enumerate(pool.lens):
        L, n, first = max(0, min(L, slots)), starts[b + 1] - starts[b], starts[b]
        mine[first: first + n] = True
        if n == 0 or L == 0:
            continue
        k, held = ref.gathered(pool, pool.k, b, L)
        v, _ = ref.gathered(pool, pool.v, b, L)
        late = min(n, L)                       # tokens before the first slot see nothing
        sees = np.repeat(seen(late, L, window, sinks) & held[None, :], G, 0)
        for h in range(H):
            rows_of = qd[first + n - late: first + n, h * G: h * G + G].reshape(late * G, D)
            o, e = attend(k[h], v[h], rows_of, sees, scale, np.full(L, half), low)
            out[first + n - late: first + n, h * G: h * G + G] = o.reshape(late, G, D)
            bound[first + n - late: first + n, h * G: h * G + G] = e.reshape(late, G, D)
    return out, stored(out, bound, q.dtype), mine


def prefix(far, near, groups, q, scale):
    """(out, bound) of q [batch, heads, D]: `far` holds the prefixes, `near` the
    sequences' own tokens; groups: starts of each prefix's sequences."""
    B, heads, D = q.shape
    H, G = near.heads, heads // near.heads
    out, bound = np.zeros((B, heads, D)), np.zeros((B, heads, D))
    half, low = _power_errors(q.dtype)
    qd = q.double().numpy()
    for b in range(B):
        parts = []
        for g in range(len(groups) - 1):
            if groups[g] <= b < groups[g + 1]:
                parts.append((far, g, max(0, min(far.lens[g], far.width * far.page)), half, low))
        parts.append((near, b, max(0, min(near.lens[b], near.width * near.page)), 0.0, 0.0))
        k = np.concatenate([ref.gathered(p, p.k, i, n)[0] for p, i, n, _, _ in parts], 1)
        v = np.concatenate([ref.gathered(p, p.v, i, n)[0] for p, i, n, _, _ in parts], 1)
        held = np.concatenate([ref.gathered(p, p.k, i, n)[1] for p, i, n, _, _ in parts])
        rounding = np.concatenate([np.full(n, r) for _, _, n, r, _ in parts])
        lowest = max(r for *_, r in parts)
        if not held.any():
            continue
        for h in range(H):
            o, e = attend(k[h], v[h], qd[b, h * G: h * G + G], np.repeat(held[None], G, 0), scale, rounding, lowest)
            out[b, h * G: h * G + G], bound[b, h * G: h * G + G] = o, e
    return out, stored(out, bound, q.dtype)
