"""The work of the serving operators, for timing and for comparing them with plain forms.

Four operators: the INT8 product of several tokens (with the activations'
quantiser), attention of one new token per sequence over a paged key-value
cache, the append to that cache, and its eviction by accumulated attention
weight.  `run` makes one pass through one of them: in plain torch operations
where `own` is false, through the framework's entry points where it is true.
"""
import math
import random

import torch

own = False

DTYPES = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32}


# ---------------------------------------------------------------- the cases
def _product(name, tokens, outputs, inner, dtype, quantised):
    c = {"op": "product", "tokens": tokens, "outputs": outputs, "inner": inner, "dtype": dtype, "quantised": quantised}
    return dict(c, name=name) if name else c


def _attention(name, batch, low, high, heads, kv_heads, dim, page, dtype, weighted):
    c = {"op": "attention", "batch": batch, "low": low, "high": high, "heads": heads, "kv_heads": kv_heads, "dim": dim,
         "page": page, "dtype": dtype, "weighted": weighted}
    return dict(c, name=name) if name else c


def _append(name, batch, low, high, new, kv_heads, dim, page, dtype, tracked):
    c = {"op": "append", "batch": batch, "low": low, "high": high, "new": new, "kv_heads": kv_heads, "dim": dim,
         "page": page, "dtype": dtype, "tracked": tracked}
    return dict(c, name=name) if name else c


def _evict(name, batch, low, high, budget, recent, kv_heads, dim, page, dtype, settled):
    c = {"op": "evict", "batch": batch, "low": low, "high": high, "budget": budget, "recent": recent,
         "kv_heads": kv_heads, "dim": dim, "page": page, "dtype": dtype, "settled": settled}
    return dict(c, name=name) if name else c


def listed():
    return [
        # one token through a square projection, activations quantised on the way: the latency of a decode step
        _product("product-1x4096x4096-f16", 1, 4096, 4096, "f16", False),
        # a small decode batch through an up projection
        _product("product-24x14336x4096-bf16", 24, 14336, 4096, "bf16", False),
        # a prompt of odd length through a down projection, kept in 32 bits for the residual
        _product("product-777x4096x14336-f32", 777, 4096, 14336, "f32", False),
        # a long prompt, already quantised (several projections share the quantised activations)
        _product("product-4096x14336x4096-f16", 4096, 14336, 4096, "f16", True),
        # one user, a short conversation: the smallest attention call
        _attention("attention-1x1000-f16", 1, 1000, 1000, 32, 8, 128, 16, "f16", False),
        # a full serving batch of ragged lengths
        _attention("attention-64x8192-bf16", 64, 100, 8192, 32, 8, 128, 16, "bf16", False),
        # every head with keys of its own, small heads, medium lengths
        _attention("attention-16x2047-mha-f16", 16, 301, 2047, 16, 16, 64, 32, "f16", False),
        # a few long documents, the attention weights accumulated for a later eviction
        _attention("attention-4x131072-weights-bf16", 4, 65537, 131072, 64, 8, 128, 64, "bf16", True),
        # the decode step's append: one token for each sequence of a batch
        _append("append-64x1-bf16", 64, 1, 2048, 1, 8, 128, 16, "bf16", True),
        # four prompts written to the cache
        _append("append-4x8191-f16", 4, 8191, 8191, 8191, 8, 128, 64, "f16", False),
        # the decode step's eviction: every sequence one token over its budget
        _evict("evict-32x2049-bf16", 32, 2049, 2049, 2048, 256, 8, 128, 16, "bf16", True),
        # prompts cut down to a budget
        _evict("evict-4x32768-f16", 4, 20000, 32768, 4096, 512, 8, 128, 64, "f16", False),
    ]


def _log(rng, low, high):
    return int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))


def draw(rng):
    op = rng.choice(["product", "product", "attention", "attention", "append", "evict"])
    dtype = rng.choice(["f16", "bf16"])
    kv_heads, dim = rng.choice([1, 2, 4, 5, 8]), rng.choice([64, 80, 96, 128, 128, 256])
    page = rng.choice([8, 16, 24, 32, 64, 128])
    if op == "product":
        inner = _log(rng, 256, 16384)
        if rng.random() < 0.8:
            inner -= inner % 16
        outputs = _log(rng, 256, 16384)
        tokens = _log(rng, 1, max(1, min(4096, 200_000_000_000 // (outputs * inner))))
        return _product(None, tokens, outputs, inner, rng.choice(["f16", "bf16", "f32"]), rng.random() < 0.5)
    if op == "attention":
        high = _log(rng, 1, 65536)
        batch = _log(rng, 1, max(1, min(128, 400_000 // high)))
        return _attention(None, batch, rng.randint(max(1, high // 8), high), high, kv_heads * rng.choice([1, 2, 4, 7, 8, 16]),
                          kv_heads, dim, page, dtype, rng.random() < 0.4)
    if op == "append":
        new = rng.choice([1, 1, _log(rng, 1, 4096)])
        batch = _log(rng, 1, max(1, min(128, 30_000 // new)))
        high = new + _log(rng, 1, 2000)
        return _append(None, batch, rng.randint(new, high), high, new, kv_heads, dim, page, dtype, rng.random() < 0.5)
    high = _log(rng, 64, 32768)
    batch = _log(rng, 1, max(1, min(64, 120_000 // high)))
    budget = max(8, int(high * rng.uniform(0.1, 0.95)))
    return _evict(None, batch, rng.randint(max(1, high // 2), high), high, budget, rng.randint(0, budget // 2), kv_heads, dim,
                  page, dtype, rng.random() < 0.5)


def lengths(case):
    """The sequences' lengths: ragged between `low` and `high`, one of them `high`; the same for every seed."""
    r = random.Random(case["batch"] * 1_000_003 + case["high"])
    return [case["high"]] + [r.randint(case["low"], case["high"]) for _ in range(case["batch"] - 1)]


# ---------------------------------------------------------------- the inputs
def _normal(g, shape, dtype, scale=1.0):
    return (torch.randn(shape, generator=g, device="cuda") * scale).to(dtype)


def _paged(case, g):
    """A pool of pages in use by several sequences, each with its pages anywhere in the pool."""
    dtype, page = DTYPES[case["dtype"]], case["page"]
    width = -(-case["high"] // page)
    pages = case["batch"] * width + 3
    shape = (pages, page, case["kv_heads"], case["dim"])
    table = torch.randperm(pages, generator=g, device="cuda")[: case["batch"] * width].to(torch.int32).view(case["batch"], width)
    k, v = (torch.empty(shape, dtype=dtype, device="cuda") for _ in range(2))
    k.normal_(generator=g)
    v.normal_(generator=g)
    return {"case": case, "k": k, "v": v, "table": table,
            "lens": torch.tensor(lengths(case), dtype=torch.int32, device="cuda"), "slots": width * page}


def _weights(g, shape):
    """Accumulated attention weights: a few tokens draw most of it, the newest have none yet."""
    w = torch.randn(shape, generator=g, device="cuda").mul_(2.0).exp_()
    return w * (torch.rand(shape, generator=g, device="cuda") > 0.05)


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(int(seed))
    if case["op"] == "product":
        T, M, N = case["tokens"], case["outputs"], case["inner"]
        s = {"case": case, "A": torch.randint(-127, 128, (M, N), generator=g, device="cuda", dtype=torch.int8),
             "scale": (torch.rand(M, generator=g, device="cuda") * 1e-3 + 1e-4).to(torch.float16)}
        if case["quantised"]:
            s["q"] = torch.randint(-127, 128, (T, N), generator=g, device="cuda", dtype=torch.int8)
            s["s"] = torch.rand(T, generator=g, device="cuda") * 0.05 + 1e-3
        else:
            s["x"] = _normal(g, (T, N), DTYPES[case["dtype"]], 1.5)
        return s
    s = _paged(case, g)
    B, H, D, C = case["batch"], case["kv_heads"], case["dim"], s["slots"]
    if case["op"] == "attention":
        s["q"] = _normal(g, (B, case["heads"], D), DTYPES[case["dtype"]], 1.5)
        s["scale"] = 1.0 / math.sqrt(D)
        if case["weighted"]:
            s["weights"] = _weights(g, (B, H, C))
    elif case["op"] == "append":
        n = case["new"]
        s["new_k"], s["new_v"] = (_normal(g, (B * n, H, D), DTYPES[case["dtype"]]) for _ in range(2))
        s["starts"] = torch.arange(B + 1, dtype=torch.int32, device="cuda") * n
        s["lens"] = s["lens"].clamp(min=n)
        if case["tracked"]:
            s["weights"] = _weights(g, (B, H, C))
            s["positions"] = torch.arange(C, dtype=torch.int32, device="cuda").expand(B, H, C).contiguous()
            s["seen"] = s["lens"] + 5
    else:
        s["weights"] = _weights(g, (B, H, C))
        s["positions"] = torch.arange(C, dtype=torch.int32, device="cuda").expand(B, H, C).contiguous()
        if case["settled"]:
            # earlier evictions have put the tokens of a head in an order of its own
            dice = torch.rand((B, H, C), generator=g, device="cuda")
            dice = dice.masked_fill(s["positions"] >= s["lens"].view(B, 1, 1), 2.0)
            s["positions"] = dice.argsort(-1).argsort(-1).to(torch.int32)
        s["seen"] = s["lens"].clone()
    if own:
        from memory_bound_gemv_row_amd import PagedCache

        s["cache"] = PagedCache(s["k"], s["v"])
    return s


# ---------------------------------------------------------------- the plain forms
def _plain_product(s):
    A = s["A"].double()
    if s["case"]["quantised"]:
        q, t = s["q"].double(), s["s"].double()[:, None]
    else:
        x = s["x"].double()
        t = (x.abs().amax(1, keepdim=True) / 127).float().double()
        q = torch.where(t > 0, torch.round(x / t), 0.0).clamp(-127, 127)
    # whole numbers below 2^53: the sums are exact
    return ((q @ A.t()) * (t * s["scale"].double())).to(DTYPES[s["case"]["dtype"]])


def _gathered(s, pool, slots):
    """The rows of the first `slots` slots of each sequence, in 32 bits: [batch, kv_heads, slots, dim]."""
    page = s["case"]["page"]
    at = torch.arange(slots, device="cuda")
    rows = pool[s["table"].long()[:, at // page], at % page]
    return rows.permute(0, 2, 1, 3).float().contiguous()


def _plain_attention(s):
    c = s["case"]
    B, H, G, D, L = c["batch"], c["kv_heads"], c["heads"] // c["kv_heads"], c["dim"], c["high"]
    q = s["q"].float().view(B, H, G, D)
    k = _gathered(s, s["k"], L)
    logits = (k @ q.transpose(2, 3).contiguous()).transpose(2, 3).contiguous() * s["scale"]
    del k
    held = torch.arange(L, device="cuda") < s["lens"].view(B, 1, 1, 1)
    logits = torch.where(held, logits, -math.inf)
    p = torch.exp(logits - logits.amax(-1, keepdim=True))
    p = p / p.sum(-1, keepdim=True)
    out = (p @ _gathered(s, s["v"], L)).reshape(B, c["heads"], D).to(s["q"].dtype)
    if not c["weighted"]:
        return out
    s["weights"][:, :, :L] += p.sum(2)
    return out, s["weights"]


def _plain_append(s):
    c = s["case"]
    B, n, page = c["batch"], c["new"], c["page"]
    slot = s["lens"].long()[:, None] - n + torch.arange(n, device="cuda")
    pages = s["table"].long().gather(1, slot // page)
    s["k"][pages, slot % page] = s["new_k"].view(B, n, c["kv_heads"], c["dim"])
    s["v"][pages, slot % page] = s["new_v"].view(B, n, c["kv_heads"], c["dim"])
    if not c["tracked"]:
        return s["k"], s["v"]
    at = slot[:, None, :].expand(B, c["kv_heads"], n)
    s["weights"].scatter_(2, at, 0.0)
    position = (s["seen"][:, None] - n + torch.arange(n, dtype=torch.int32, device="cuda"))[:, None, :]
    s["positions"].scatter_(2, at, position.expand(B, c["kv_heads"], n).contiguous())
    return s["k"], s["v"], s["weights"], s["positions"]


def _plain_evict(s):
    c = s["case"]
    B, H, C, budget, page = c["batch"], c["kv_heads"], s["slots"], c["budget"], c["page"]
    lens, w, pos = s["lens"].view(B, 1, 1), s["weights"], s["positions"]
    at = torch.arange(C, device="cuda").expand(B, H, C)
    held = at < lens
    recent = held & (pos >= s["seen"].view(B, 1, 1) - c["recent"])
    key = torch.where(recent, math.inf, w.double())
    key = torch.where(held, key, -math.inf)
    order = key.sort(dim=-1, descending=True, stable=True).indices
    rank = torch.empty_like(order).scatter_(2, order, at)
    keep = held & (rank < budget)
    hole = held & ~keep & (at < budget)
    mover = keep & (at >= budget)
    movers = torch.zeros((B, H, C + 1), dtype=torch.int64, device="cuda")
    movers.scatter_(2, torch.where(mover, mover.cumsum(-1) - 1, C), at)
    source = torch.where(hole, movers.gather(2, torch.where(hole, hole.cumsum(-1) - 1, C)), at)
    left = s["lens"].clamp(max=budget)
    kept = at < left.view(B, 1, 1)
    new_w = torch.where(kept, w.gather(2, source), 0.0)
    new_pos = torch.where(kept, pos.gather(2, source), -1)
    n = min(budget, C)
    source, head = source[:, :, :n], torch.arange(H, device="cuda").view(1, H, 1)
    table = s["table"].long()
    src = table[torch.arange(B, device="cuda").view(B, 1, 1), source // page], source % page, head
    slot = at[:, :, :n]
    dst = table[torch.arange(B, device="cuda").view(B, 1, 1), slot // page], slot % page, head
    s["k"][dst] = s["k"][src]
    s["v"][dst] = s["v"][src]
    return s["k"], s["v"], new_w, new_pos, left


PLAIN = {"product": _plain_product, "attention": _plain_attention, "append": _plain_append, "evict": _plain_evict}


# ---------------------------------------------------------------- the framework's calls
def _own(s):
    import memory_bound_gemv_row_amd as amd

    c = s["case"]
    if c["op"] == "product":
        q, t = (s["q"], s["s"]) if c["quantised"] else amd.quantize_tokens_q8(s["x"])
        return amd.gemm_q8(s["A"], s["scale"], q, t, out_dtype=DTYPES[c["dtype"]])
    if c["op"] == "attention":
        out = amd.paged_attention(s["cache"], s["table"], s["lens"], s["q"], scale=s["scale"], max_len=c["high"],
                                  weights=s.get("weights"))
        return (out, s["weights"]) if c["weighted"] else out
    if c["op"] == "append":
        if not c["tracked"]:
            amd.kv_append(s["cache"], s["table"], s["lens"], s["starts"], s["new_k"], s["new_v"])
            return s["k"], s["v"]
        amd.kv_append(s["cache"], s["table"], s["lens"], s["starts"], s["new_k"], s["new_v"], weights=s["weights"],
                      positions=s["positions"], seen=s["seen"])
        return s["k"], s["v"], s["weights"], s["positions"]
    w, pos, left = amd.kv_evict(s["cache"], s["table"], s["lens"], s["seen"], s["weights"], s["positions"],
                                budget=c["budget"], recent=c["recent"], max_len=c["high"])
    return s["k"], s["v"], w, pos, left


def run(state):
    return _own(state) if own else PLAIN[state["case"]["op"]](state)


# ---------------------------------------------------------------- work and exact values
def work(case):
    if case["op"] == "product":
        T, M, N = case["tokens"], case["outputs"], case["inner"]
        size = DTYPES[case["dtype"]].itemsize
        x = T * (N + 4) if case["quantised"] else T * N * size
        return {"bytes": M * N + 2 * M + x + T * M * size, "flops": 2 * T * M * N}
    B, H, D, C = case["batch"], case["kv_heads"], case["dim"], -(-case["high"] // case["page"]) * case["page"]
    size, total = 2, sum(lengths(case))
    tables = 4 * sum(-(-n // case["page"]) + 1 for n in lengths(case))
    if case["op"] == "attention":
        moved = 2 * total * H * D * size + 2 * B * case["heads"] * D * size + tables
        return {"bytes": moved + (8 * total * H if case["weighted"] else 0), "flops": 4 * total * case["heads"] * D}
    if case["op"] == "append":
        n = B * case["new"] * H
        return {"bytes": 4 * n * D * size + (8 * n if case["tracked"] else 0) + tables, "flops": 0}
    K, R, moves = case["budget"], case["recent"], 0.0
    for n in lengths(case):
        if n > K:
            # kept slots past the budget: by chance everywhere, or the newest at the end and the others by chance
            spread = (n - K) * K / n
            moves += spread if case["settled"] else min(R, n - K) + max(0, n - R - K) * (K - R) / max(1, n - R)
    return {"bytes": int(moves * H) * 4 * D * size + 8 * total * H + 8 * B * H * C + tables, "flops": 0}


def _exact_product(case, s):
    A, scale = s["A"], s["scale"].double()
    if case["quantised"]:
        q, t = s["q"].float(), s["s"].double()
    else:
        x = s["x"].double()
        t = (x.abs().max(1).values / 127.0).float().double()
        n = x / torch.where(t > 0, t, torch.ones_like(t))[:, None]
        low = torch.floor(n)
        up = (n - low > 0.5) | ((n - low == 0.5) & (low % 2 != 0))
        q = (torch.minimum(torch.maximum(low + up, torch.full_like(n, -127)), torch.full_like(n, 127))).float()
    # sums of whole numbers over pieces that 32 bits hold exactly (1024 * 127 * 128 < 2^24)
    y = torch.zeros((q.shape[0], A.shape[0]), dtype=torch.float64, device="cuda")
    for j in range(0, A.shape[1], 1024):
        y += torch.mm(q[:, j: j + 1024], A[:, j: j + 1024].float().t())
    return y * scale[None, :] * t[:, None]


def _exact_attention(case, s):
    H, G, page = case["kv_heads"], case["heads"] // case["kv_heads"], case["page"]
    out = torch.empty((case["batch"], case["heads"], case["dim"]), dtype=torch.float64, device="cuda")
    weights = s["weights"].double() if case["weighted"] else None
    for b, n in enumerate(lengths(case)):
        rows = s["table"][b, : -(-n // page)].long()
        for h in range(H):
            k, v = (p[rows, :, h].reshape(-1, case["dim"])[:n].double() for p in (s["k"], s["v"]))
            e = (k * s["scale"]) @ s["q"][b, h * G: (h + 1) * G].double().t().contiguous()
            p = torch.exp(e - torch.logsumexp(e, 0))
            out[b, h * G: (h + 1) * G] = p.t().contiguous() @ v
            if weights is not None:
                weights[b, h, :n] += p.sum(1)
    return out if weights is None else (out, weights)


def _exact_evict(case, s):
    """The accumulated weights after the eviction; the rest of what it returns is moved, not computed."""
    w, pos, seen = s["weights"].cpu().tolist(), s["positions"].cpu().tolist(), s["seen"].tolist()
    new, budget = torch.zeros(s["weights"].shape, dtype=torch.float64), case["budget"]
    for b, n in enumerate(lengths(case)):
        for h in range(case["kv_heads"]):
            row, at = w[b][h], pos[b][h]
            best = sorted(range(n), key=lambda j: (at[j] < seen[b] - case["recent"], -row[j], j))[:budget]
            kept = set(best)
            late = iter(sorted(j for j in best if j >= budget))
            for j in range(min(n, budget)):
                new[b, h, j] = row[j] if j in kept else row[next(late)]
    return None, None, new.cuda(), None, None


def exact(case, seed):
    global own
    was, own = own, False
    try:
        s = prepare(case, seed)
    finally:
        own = was
    if case["op"] == "product":
        return _exact_product(case, s)
    if case["op"] == "attention":
        return _exact_attention(case, s)
    return _exact_evict(case, s) if case["op"] == "evict" else None
