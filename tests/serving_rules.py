"""The launch rules of the serving operators in Python, as csrc/tokens_api.hip
and csrc/attention_api.hip state them, so that tests can tell which kernel a
call takes and that their shapes reach every one."""
import math
import os
import re
from collections import namedtuple

from memory_bound_gemv_row_amd import build

Tiling = namedtuple("Tiling", "tokens outputs wt wm wk columns stages rate overhead")


def tilings():
    """{"stream": [...], "any": [...]} as the source lists them."""
    with open(os.path.join(build.SRC_DIR, "tokens_api.hip")) as f:
        text = f.read()
    out = {}
    for kind, macro, n in (("stream", "GTOKENS_STREAM", 9), ("any", "GTOKENS_ANY", 8)):
        rows = []
        for args in re.findall(macro + r"\(([0-9., ]+)\)", text):
            v = [float(a) for a in args.split(",")]
            assert len(v) == n, args
            stages = [int(v[6])] if kind == "stream" else [2]
            rows.append(Tiling(*(int(a) for a in v[:6]), *stages, *v[-2:]))
        assert rows
        out[kind] = rows
    return out


def product_kernel(T, M, N, cus=256, wide=None, _cache={}):
    """("tiles", None), ("stream", Tiling) or ("any", Tiling) of gemv_gemm_q8;
    `wide`: 16-byte-aligned operands (where unset, as N allows)."""
    all_of = _cache.setdefault("all", tilings())
    wide = N >= 16 and N % 16 == 0 if wide is None else wide
    if wide and -(-T // 256) * -(-M // 256) >= cus * 3 // 4:
        return "tiles", None
    kind = "stream" if wide else "any"

    def cost(t):
        tiles = -(-T // t.tokens) * -(-M // t.outputs)
        own = math.ceil(tiles / cus) * ((t.tokens + t.outputs) * N / (t.rate * 1e3) + t.overhead)
        return own * own + (M * N / 6e6) ** 2

    return kind, min(all_of[kind], key=cost)   # the first of equals, as there


def attention_form(batch, limit, kv_heads, q_heads, dim, page, cus=256):
    """(DP, pages hold whole tiles, one eight-wave workgroup, parts) of
    gemv_attention for slots near one another."""
    group = q_heads // kv_heads
    items = batch * kv_heads * -(-group // 16)
    if dim <= 64 and items >= cus and limit > 1024:
        chunk = min((limit * items // (cus * 8) + 63) // 64 * 64, 1024)
    else:
        def cost(c):
            parts = -(-limit // c)
            return -(-items * parts // cus) * (c + 100) + (150 + parts if parts > 1 else 0)
        chunk = min(range(1024, 63, -64), key=cost)
    whole = page % 16 == 0
    lone = whole and chunk < limit and (limit <= 256 or (limit <= 768 and items * 2 >= cus))
    if lone:
        chunk = (limit + 63) // 64 * 64
    return (64 if dim <= 64 else 128 if dim <= 128 else 256), whole, lone, max(1, -(-limit // chunk))


# Shapes (tokens, outputs, columns) of which each tiling is the cheapest for at
# least one, with more columns than twice what its stages hold, columns that end
# inside a stage, and last tiles that are not full.
STREAMED = [(19, 43, 3088), (1400, 40, 3088), (7, 4182, 3088), (45, 5000, 4112), (1400, 40, 4112), (19, 5000, 2064),
            (19, 9001, 1552), (2783, 133, 2512), (45, 9001, 1296), (1402, 730, 1632), (133, 6638, 784), (777, 4091, 2064)]
LOOSE = [(19, 40, 2069), (1400, 40, 1045), (45, 5000, 533), (777, 4091, 1045)]
# 256 x 256 tiles: just above where they are taken, whole rounds, and a rest in
# halves of which the last lies past the outputs
LARGE = [(3830, 3327, 528), (3830, 3327, 1040), (4090, 4000, 4112), (4090, 4300, 1040), (4090, 4200, 1296)]

# (lengths, key-value heads, query heads) by what they are for; the first length
# is the longest.  Pages that are whole tiles and pages that are not, every
# padded head size, exact and not.
LENGTHS = {"one part": ([60, 3], 2, 6), "one workgroup of eight waves": ([250, 17, 0], 2, 4),
           "the same, many heads": ([500, 1, 17] * 11, 4, 8), "split": ([1500, 700], 2, 34)}
DIMS, PAGES = [40, 64, 80, 128, 192, 256], [5, 16, 24]
