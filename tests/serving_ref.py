"""Plain 64-bit forms of the serving operators (numpy, loops over sequences and
heads), their error bounds, and the paged pools that their tests run on."""
import numpy as np
import torch

U32 = 2.0 ** -24                                                     # half a step of binary32
HALF_STEP = {torch.float32: 2.0 ** -24, torch.float16: 2.0 ** -11, torch.bfloat16: 2.0 ** -8}
SMALLEST = {torch.float32: 2.0 ** -149, torch.float16: 2.0 ** -25, torch.bfloat16: 2.0 ** -134}   # half a subnormal step


# ---------------------------------------------------------------- INT8 product
def quantize_tokens(x):
    """x float64 [T, N] -> (codes float64, scales float64 that binary32 holds)."""
    q = np.zeros(x.shape)
    s = np.zeros(x.shape[0])
    for t in range(x.shape[0]):
        if not np.all(np.isfinite(x[t])):
            s[t] = np.nan
            continue
        s[t] = float(np.float32(np.max(np.abs(x[t]), initial=0.0) / 127.0))
        if s[t] > 0:
            q[t] = np.clip(np.rint(x[t] / s[t]), -127, 127)   # rint: ties to even
    return q, s


def product(A, scale, x, x_scale):
    """(float64 result, bound's magnitude |result|) of integer A [M, N], x [T, N]."""
    sums = x.astype(np.int64) @ A.astype(np.int64).T
    return sums.astype(np.float64) * (x_scale.astype(np.float64)[:, None] * scale.astype(np.float64)[None, :])


def product_bound(ref, dtype):
    # the sum's conversion, the scales' product and their product round once
    # each in binary32 (3 u, 4 u holds their compound), the store once more
    return np.abs(ref) * (4 * U32 + HALF_STEP[dtype] * (1 + 4 * U32)) + SMALLEST[dtype] + 2.0 ** -149


# ---------------------------------------------------------------- paged pools
class Pool:
    """A paged cache on the device, made on the host: every slot that no
    sequence holds is filled with NaN and infinities."""

    def __init__(self, lens, heads, dim, page, dtype=torch.float16, width=None, seed=0, layout="slots", extra=3,
                 device="cuda", spread=1.0):
        rng = np.random.default_rng(seed)
        self.lens, self.page, self.heads, self.dim = [int(n) for n in lens], page, heads, dim
        B = len(self.lens)
        self.width = width if width is not None else max([-(-n // page) for n in self.lens] + [1])
        pages = B * self.width + extra
        order = rng.permutation(pages)
        self.table = torch.from_numpy(order[: B * self.width].reshape(B, self.width).astype(np.int32))
        shape = (pages, page, heads, dim)
        junk = torch.tensor([float("nan"), float("inf"), -float("inf")])
        self.k = junk[torch.from_numpy(rng.integers(0, 3, shape))].to(dtype)
        self.v = junk[torch.from_numpy(rng.integers(0, 3, shape))].to(dtype)
        for b, n in enumerate(self.lens):
            for j in range(min(n, self.width * page)):
                p, o = self.table[b, j // page], j % page
                self.k[p, o] = torch.from_numpy(rng.standard_normal((heads, dim)) * spread).to(dtype)
                self.v[p, o] = torch.from_numpy(rng.standard_normal((heads, dim))).to(dtype)
        self.dk, self.dv = (self._lay(t.to(device), layout) for t in (self.k, self.v))
        self.dtable = self.table.to(device)
        self.dlens = torch.tensor(self.lens, dtype=torch.int32, device=device)

    @staticmethod
    def _lay(t, layout):
        if layout == "heads":      # [pages, heads, page_size, dim] in memory
            return t.transpose(1, 2).contiguous().transpose(1, 2)
        if layout == "padded":     # rows with room between them
            pages, page, heads, dim = t.shape
            wide = torch.full((pages, page + 1, heads + 1, dim + 8), float("nan"), dtype=t.dtype, device=t.device)
            wide[:, :page, :heads, :dim] = t
            return wide[:, :page, :heads, :dim]
        return t.contiguous()

    def rows(self, pool, b, h, n):
        """Rows of the first n slots of a head, float64 [n, dim]; holes are left out of `held`."""
        out, held = np.zeros((n, self.dim)), np.zeros(n, bool)
        for j in range(n):
            p = int(self.table[b, j // self.page])
            if 0 <= p < pool.shape[0]:
                out[j] = pool[p, j % self.page, h].double().numpy()
                held[j] = True
        return out, held


def attention(pool, q, scale):
    """(out, its bound, weights, their bound), float64, for q [B, Hq, D] on the host.

    Bound: a logit sums D exact products in some order (2 D u of their
    magnitudes, with room for the sums inside a matrix instruction), is
    multiplied twice and subtracted once; its absolute error e makes the
    power's relative error e, taken twice (numerator and sum).  exp2 is good to
    two units in the last place.  A wave's sums run over at most a quarter of
    the length in tiles of 16, then 4 or 8 waves and at most len / 64 + 1 parts
    are added; the division and the output's rounding come last."""
    B, Hq, D = q.shape
    H, G = pool.heads, Hq // pool.heads
    slots = pool.width * pool.page
    out, bound = np.zeros((B, Hq, D)), np.zeros((B, Hq, D))
    weights, wbound = np.zeros((B, H, slots)), np.zeros((B, H, slots))
    qd = q.double().numpy()
    for b, n in enumerate(pool.lens):
        n = max(0, min(n, slots))
        for h in range(H):
            k, held = pool.rows(pool.k, b, h, n)
            v, _ = pool.rows(pool.v, b, h, n)
            if not held.any():
                continue
            for g in range(G):
                x = (k @ qd[b, h * G + g]) * scale
                mag = (np.abs(k) @ np.abs(qd[b, h * G + g])) * abs(scale)
                x = np.where(held, x, -np.inf)
                p = np.exp(x - x.max())
                p /= p.sum()
                e = (2 * D * U32 * mag + 6 * U32 * (np.abs(np.where(held, x, 0)) + np.abs(x[held]).max()))[held].max()
                sums = (16 * -(-n // 64) + 8 + n // 64 + 1) * U32
                rel = 2 * np.expm1(e) + 8 * U32 + 2 * sums
                o = p @ np.where(held[:, None], v, 0)
                out[b, h * G + g] = o
                bound[b, h * G + g] = rel * (p @ np.abs(np.where(held[:, None], v, 0)))
                weights[b, h, :n] += p
                wbound[b, h, :n] += (rel + G * U32) * p + 2.0 ** -126
    half = HALF_STEP[q.dtype]
    return out, bound * (1 + half) + half * np.abs(out) + SMALLEST[q.dtype], weights, wbound


def evict(lens, seen, weights, positions, budget, recent, slots):
    """(source slot per slot below the budget, weights, positions, lens) afterwards:
    float32 / int32 arrays [B, H, slots]; source[b, h, j] = j where nothing moves."""
    B, H = weights.shape[:2]
    w_out, p_out = np.zeros_like(weights), np.full_like(positions, -1)
    source = np.broadcast_to(np.arange(slots), (B, H, slots)).copy()
    left = np.array([min(max(0, min(n, slots)), budget) for n in lens], np.int32)
    for b in range(B):
        n = max(0, min(int(lens[b]), slots))
        for h in range(H):
            def rank(j):
                w = weights[b, h, j]
                new = int(positions[b, h, j]) >= int(seen[b]) - recent
                return (0 if new else 1, 0.0 if new or np.isnan(w) else 1.0, 0.0 if new or np.isnan(w) else -float(w), j)
            keep = set(sorted(range(n), key=rank)[:budget])
            holes = [j for j in range(min(n, budget)) if j not in keep]
            late = sorted(j for j in keep if j >= budget)
            assert len(holes) == len(late)
            for to, frm in zip(holes, late):
                source[b, h, to] = frm
            for j in range(left[b]):
                w_out[b, h, j] = weights[b, h, source[b, h, j]]
                p_out[b, h, j] = positions[b, h, source[b, h, j]]
    return source, w_out, p_out, left


# ---------------------------------------------------------------- bounds slot by slot
def gathered(pool, t, b, n):
    """Rows of the first n slots of sequence b, float64 [heads, n, dim], and which are held."""
    j = np.arange(n)
    page = pool.table.numpy()[b, j // pool.page].astype(np.int64)
    held = (page >= 0) & (page < t.shape[0])
    rows = t[torch.from_numpy(np.where(held, page, 0)), torch.from_numpy(j % pool.page)].double().numpy()
    return np.where(held[:, None, None], rows, 0).transpose(1, 0, 2), held


def attention_by_slot(pool, q, scale):
    """As `attention`, with the error of every slot's power weighed by its own
    probability, so that a token without weight adds nothing to the bound.

    With x the logits, e_j = 2 D u |k_j| . |q| scale + 6 u (|x_j| + |max x|) is
    the absolute error of x_j - reference (see `attention`; what the reference's
    rises multiply by is counted here too, for their differences add up to at
    most that between the first and the last).  A power is then off by at most
    exp(x_j + e_j) - exp(x_j), by exp2's two units in the last place (4 u) and,
    below 2^-126, by itself.  A wave's sums run over at most a quarter of the
    length in tiles of 16, each with 16 additions and at most one rescaling (an
    exp2 and a product, 5 u; 24 holds them), then 8 waves and len / 64 + 1 parts.
    The normaliser's error S is the sum of those of the powers; a probability's
    is (its own + p S) / (1 - S).  A logit of -inf has probability 0."""
    B, Hq, D = q.shape
    H, G = pool.heads, Hq // pool.heads
    slots = pool.width * pool.page
    out, bound = np.zeros((B, Hq, D)), np.zeros((B, Hq, D))
    weights, wbound = np.zeros((B, H, slots)), np.zeros((B, H, slots))
    for b, n in enumerate(pool.lens):
        n = max(0, min(n, slots))
        if n == 0:
            continue
        k, held = gathered(pool, pool.k, b, n)
        v, _ = gathered(pool, pool.v, b, n)
        qd = q[b].double().numpy().reshape(H, G, D)
        with np.errstate(invalid="ignore"):
            x = np.where(held, (qd @ k.transpose(0, 2, 1)) * scale, -np.inf)
        counts = x > -np.inf
        if not counts.any():
            continue
        top = x.max(-1, keepdims=True)
        k = np.where(np.isfinite(k), k, 0)
        mag = (np.abs(qd) @ np.abs(k).transpose(0, 2, 1)) * abs(scale)
        far = np.where(counts, x, 0)
        e = np.where(counts, 2 * D * U32 * mag + 6 * U32 * (np.abs(far) + np.abs(top)), 0)
        power = np.exp(x - top)
        Z = power.sum(-1, keepdims=True)
        p = power / Z
        sums = (24 * -(-n // 64) + 8 + n // 64 + 1) * U32
        diff = (np.exp(x - top + e) - power) / Z + p * (4 * U32 + sums) + np.where(counts, 2.0 ** -126, 0)
        S = diff.sum(-1, keepdims=True)
        assert np.all(S < 0.5), "logits too large for this bound"
        off = (diff + p * S) / (1 - S)
        out[b] = (p @ v).reshape(Hq, D)
        bound[b] = ((off + 2 * U32 * p) @ np.abs(v)).reshape(Hq, D)
        weights[b, :, :n] = p.sum(1)
        wbound[b, :, :n] = (off + (G + 2) * U32 * p).sum(1)
    half = HALF_STEP[q.dtype]
    return out, bound * (1 + half) + half * np.abs(out) + SMALLEST[q.dtype], weights, wbound
