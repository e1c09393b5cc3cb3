"""Plain 64-bit forms of what stands between the projections and attention: norms
and rotation of heads, with their error bounds, and pages for new tokens."""
import numpy as np
import torch

U32 = 2.0 ** -24
HALF_STEP = {torch.float32: 2.0 ** -24, torch.float16: 2.0 ** -11, torch.bfloat16: 2.0 ** -8}
SMALLEST = {torch.float32: 2.0 ** -149, torch.float16: 2.0 ** -25, torch.bfloat16: 2.0 ** -134}


def turned(x, weight, positions, freqs, eps, interleaved, out_dtype):
    """(result, bound) float64 [rows, heads, dim] of x, a tensor on the host; weight
    float64 [dim] or None; eps None: no norm.

    Bound, in units u = 2^-24 of binary32, relative to |a cos| + |b sin| of a
    pair: the squares' sum has `dim` additions of positive numbers (dim + 1 units
    of the sum, half of them of its root); the division by dim and the root's
    reciprocal (v_rsq_f32, one unit in the last place: two u) and the addition of
    eps 4 more; two products with it 2; a cosine or sine is off by 4 u of one
    (its argument's rounding, at most u of pi / 4; the series' end; its sums, and
    its rounding) plus what binary64 leaves of the angle, 2^-52 of it in the
    product and 2^-52 of it in the reduction; a product and a sum 2.  The store
    rounds once more."""
    rows, heads, dim = x.shape
    n = x.double().numpy()
    rel = 0.0
    if eps is not None:
        n = n / np.sqrt((n * n).mean(-1, keepdims=True) + eps)
        if weight is not None:
            n = n * weight
        rel = (dim + 1) / 2 + 4 + 2
    half = len(freqs)
    y, bound = n.copy(), np.abs(n) * rel * U32
    if half:
        a, b = (slice(0, 2 * half, 2), slice(1, 2 * half, 2)) if interleaved else (slice(0, half), slice(half, 2 * half))
        angle = positions.astype(np.float64)[:, None] * freqs[None, :]
        c, s = np.cos(angle)[:, None], np.sin(angle)[:, None]
        off = (4 * U32 + np.abs(angle) * 2.0 ** -51)[:, None]
        p, q = n[..., a], n[..., b]
        y[..., a], y[..., b] = p * c - q * s, q * c + p * s
        bound[..., a] = (np.abs(p * c) + np.abs(q * s)) * (rel + 3) * U32 + (np.abs(p) + np.abs(q)) * off
        bound[..., b] = (np.abs(q * c) + np.abs(p * s)) * (rel + 3) * U32 + (np.abs(p) + np.abs(q)) * off
    step = HALF_STEP[out_dtype]
    return y, bound * (1 + step) + step * np.abs(y) + SMALLEST[out_dtype]


def reserve(free, count, table, lens, added, page_size, rows, pages):
    """(count, lens, starts, positions, slots, table) in whole numbers, row by row."""
    free, table = [int(p) for p in free], np.array(table, np.int64)
    have = max(0, min(int(count), pages))
    stack, missing = free[:have], 0
    starts, out_lens, positions, slots = [0], [], [], []
    for b in range(len(lens)):
        length = max(0, int(lens[b]))
        n = min(max(0, int(added[b])), rows - starts[-1])
        got = min(n, 2 ** 31 - 1 - length)
        held = -(-length // page_size)
        for i in range(n):
            if i >= got:
                positions.append(2 ** 31 - 1), slots.append(-1)
                continue
            p = length + i
            index = p // page_size
            positions.append(p)
            if index >= table.shape[1]:
                slots.append(-1)
                continue
            if index >= held and p % page_size == 0:
                if stack:
                    page = stack.pop()
                else:
                    page, missing = -1, missing + 1
                table[b, index] = page if 0 <= page < pages else -1
            page = int(table[b, index])
            slots.append(page * page_size + p % page_size if 0 <= page < pages else -1)
        starts.append(starts[-1] + n)
        out_lens.append(length + got)
    positions += [0] * (rows - len(positions))
    slots += [-1] * (rows - len(slots))
    return [len(stack), missing], out_lens, starts, positions, slots, table


def release(free, count, table, keep, page_size, pages):
    """(free, count, table) afterwards."""
    free, table = [int(p) for p in free], np.array(table, np.int64)
    at = max(0, min(int(count), pages))
    for b in range(table.shape[0]):
        for i in range(-(-max(0, int(keep[b])) // page_size), table.shape[1]):
            page, table[b, i] = int(table[b, i]), -1
            if 0 <= page < pages and at < pages:
                free[at] = page
                at += 1
    return free, at, table
