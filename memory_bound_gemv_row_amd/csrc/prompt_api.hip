// prompt_api.hip -- C ABI of attention with several new tokens per sequence, with
// a window, and behind shared prefixes (declared in include/gemv_prompt.h):
// validation, workspaces, geometry and launch.
#include "gemv_prompt.h"

#include "attention_host.hpp"
#include "prompt_kernels.hpp"

#include <float.h>
#include <math.h>

namespace gattn {
namespace {

constexpr float kLog2e = 1.44269504088896340736f;

// How query rows and keys are split: places for row tiles of a key-value head,
// parts of the keys and tiles of keys in each.
struct Tiling {
    int64_t tiles;
    TileOrder order;
    int laps, run, parts, chunk;
    int64_t places;          // workgroups of a key-value head
    size_t ms_at, out_at, bytes;
};

// The least estimate, in us.  A workgroup takes a step for each tile of keys and
// kStart for its start and end; a step takes 2.15 us for heads of 128 where a CU
// holds two workgroups (one for heads over 128), less where it holds one.  As
// many as there are places for start together, and where they see alike the next
// ones wait for them: a round that is half empty costs as much as a full one
// (4 x 7 tokens over 65543 keys in parts alike: 16 parts, one round, 149 us; 24
// parts 163, 32 parts 161).  Where a sequence's newest tokens are most of it they see fewer keys
// the earlier they are, and the work spreads evenly but for its end.  A join
// costs a launch, its parts written and read at 6 TB/s, kPart for each of a row's,
// and its waves: 8192 at a time for 3.5 us (7943 rows of 16 heads in two parts: 155
// us, 91 without).  `per_cu`: workgroups that a CU holds (two, for heads up to
// 128, three up to 64), or that it takes of these beside others.
Tiling tile_rows(const gemv_kv_cache* c, int64_t rows, int batch, int group, int limit, int window, int sinks, int max_new,
                 double per_cu, bool shares, int cus)
{
    constexpr double kStart = 1.5, kJoin = 4.0, kMoved = 6e6, kPart = 0.06, kWave = 3.5 / 8192;
    Tiling t{};
    t.tiles = rows * group / kTileRows + batch;
    t.order = kTogether;
    t.laps = 1;
    t.run = (int)t.tiles;
    // Runs of 8 of the last tiles, where sequences have two runs, not much fewer places
    // hold them all and a launch is nowhere near its most: 6 x 1999 tokens, 16 heads
    // of 64, 58 us (68 a sequence after the other, 57 in runs of 1), 4 x 8192 of them
    // 501 (537, 590), 2 x 8192, 32/8 heads of 128, 640 (632, 985: keys of both
    // sequences are more than the L2), 40 x 300 79 (73, 74).
    const int64_t even = ((int64_t)(max_new > 0 ? max_new : rows) * group + kTileRows - 1) / kTileRows;
    if (even == 1) {
        // a tile each: parts of one sequence after another, of which the last are short
        // (20 x 5 tokens through a window of 2000: 35 us, 49 part after part)
        t.order = kSingle;
        t.tiles = batch;
        t.run = 1;
    } else if (even >= 16 && even * batch <= 2 * t.tiles && even * batch * c->heads < 1 << 20) {
        t.order = kLaps;
        t.tiles = even;
        t.laps = batch;
        t.run = 8;
    }
    int64_t keys = ((int64_t)limit + kTileKeys - 1) / kTileKeys;
    if (window > 0) {
        const int64_t near = ((int64_t)window + kTileRows / group + kTileKeys) / kTileKeys + 1;
        const int64_t seen = ((int64_t)sinks + kTileKeys - 1) / kTileKeys + near;
        keys = seen < keys ? seen : keys;
    }
    keys = keys > 0 ? keys : 1;
    const bool uneven = max_new > limit / 2 && window == 0;
    const double mean = uneven ? (double)(limit - max_new / 2) / kTileKeys + 1 : (double)keys;
    const int64_t each = (rows + batch - 1) / (batch > 0 ? batch : 1);   // new tokens of a sequence, about
    const double items = (double)c->heads * batch * (double)((each * group + kTileRows - 1) / kTileRows);
    const double places = cus * per_cu * (c->head_dim > 128 ? 0.5 : waves_of(c->head_dim) / 2.0);
    const double step = 2.15 * (c->head_dim > 64 ? c->head_dim : 64) / 128;
    const double heads = (double)rows * group * c->heads, moved = heads * c->head_dim * 8;   // bytes of each part
    double least = 0;
    for (int64_t parts = 1; parts <= keys && parts <= 256; ++parts) {
        const int64_t chunk = (keys + parts - 1) / parts;
        if ((keys + chunk - 1) / chunk != parts)
            continue;
        const double longest = chunk + kStart, rounds = items * parts / places;
        double steps = rounds <= 1 ? longest : uneven ? items * (mean + kStart * parts) / places + longest / 2 : ceil(rounds) * longest;
        if (items * parts <= cus)
            steps *= 0.75;
        const double cost = steps * step + (parts > 1 ? kJoin + moved * parts / kMoved + kPart * parts + heads * kWave : 0);
        if (t.parts == 0 || cost < least) {
            least = cost;
            t.parts = (int)parts;
            t.chunk = (int)chunk;
        }
    }
    t.places = t.tiles * t.laps * t.parts;
    // A tile each, in several parts: as many places, shared out by the lengths, which
    // only the device knows; a long sequence takes up to four times the parts.
    if (shares && t.order == kSingle && t.parts > 1 && batch > 1 && batch <= 64 && window == 0) {
        t.order = kShares;
        t.tiles = t.places;
        t.parts = (int)(t.places < 4 * t.parts ? t.places : 4 * t.parts);
    }
    return t;
}

void place_parts(Tiling* t, size_t at, int64_t heads, int dim, bool kept)
{
    t->ms_at = at;
    t->out_at = t->bytes = at;
    if (!kept)
        return;
    t->out_at = at + round16((size_t)heads * t->parts * 2 * sizeof(float));
    t->bytes = t->out_at + round16((size_t)heads * t->parts * dim * sizeof(float));
}

// The slots that a single new token sees, in whole tiles of decode attention.
int seen_slots(int limit, int window, int sinks16)
{
    const int64_t seen = (int64_t)sinks16 + window + 15;
    return window > 0 && seen < limit ? (int)seen : limit;
}

// A window that no sequence is longer than hides nothing.
int narrow_window(int window, int limit) { return window < limit ? window : 0; }

int whole_sinks(int sinks, int tile, int limit)
{
    const int64_t n = ((int64_t)sinks + tile - 1) / tile * tile;
    const int64_t most = ((int64_t)limit + tile - 1) / tile * tile;
    return (int)(n < most ? n : most);
}

enum Form { kPrompt, kPrefix };

template <int DT, int DP, int RUN, bool EXACT>
const void* form_of(Form form)
{
    return form == kPrompt ? reinterpret_cast<const void*>(&prompt_kernel<DT, DP, RUN, EXACT>)
                           : reinterpret_cast<const void*>(&prefix_kernel<DT, DP, RUN, EXACT>);
}

template <int DT, int RUN>
const void* tiled_sized(Form form, int dim)
{
    if constexpr (RUN == 16) {
        if (dim == 64)
            return form_of<DT, 64, 16, true>(form);
        if (dim == 96)
            return form_of<DT, 96, 16, true>(form);
        if (dim == 128)
            return form_of<DT, 128, 16, true>(form);
        if (dim == 256)
            return form_of<DT, 256, 16, true>(form);
    }
    return dim <= 64    ? form_of<DT, 64, RUN, false>(form)
           : dim <= 96  ? form_of<DT, 96, RUN, false>(form)
           : dim <= 128 ? form_of<DT, 128, RUN, false>(form) : form_of<DT, 256, RUN, false>(form);
}

template <int DT>
const void* tiled_typed(Form form, const gemv_kv_cache* c)
{
    if (whole_tiles(c))
        return tiled_sized<DT, 16>(form, c->head_dim);
    return c->page_size % 8 == 0 && c->stride_slot < (1 << 26) ? tiled_sized<DT, 8>(form, c->head_dim)
                                                               : tiled_sized<DT, 1>(form, c->head_dim);
}

const void* tiled_for(Form form, const gemv_kv_cache* c)
{
    return c->dtype == GEMV_F16 ? tiled_typed<kF16>(form, c) : tiled_typed<kBF16>(form, c);
}

// Few rows are joined by four waves each, where there are parts enough for them.
int join_parts(const Join& j, int dtype, int cus, hipStream_t stream)
{
    void* args[] = {(void*)&j};
    const int64_t heads = (int64_t)j.rows * j.q_heads;
    const bool spread = heads <= (int64_t)cus * 4 && j.from[0].parts + j.from[1].parts > 8;
    const void* fn = dtype == GEMV_F16 ? spread ? reinterpret_cast<const void*>(&join_parts_kernel<kF16, true>)
                                                : reinterpret_cast<const void*>(&join_parts_kernel<kF16, false>)
                     : spread ? reinterpret_cast<const void*>(&join_parts_kernel<kBF16, true>)
                              : reinterpret_cast<const void*>(&join_parts_kernel<kBF16, false>);
    return launch(fn, spread ? heads : (heads + kJoinWaves - 1) / kJoinWaves, kJoinWaves * 64, args, stream);
}

bool joins_fit(int64_t rows, int q_heads) { return fits((rows * q_heads + kJoinWaves - 1) / kJoinWaves, kJoinWaves * 64); }

// Single new tokens, by the kernel of decode attention.  `at.limit` and
// `split` are for the slots seen.
Attention newest(const gemv_kv_cache* c, const Pages& at, int batch, const Split& split, const void* q, int64_t q_stride,
                 int q_heads, float scale, char* ws, size_t ms_at, size_t out_at, bool kept)
{
    Attention a{};
    a.at = at;
    a.k = static_cast<const uint16_t*>(c->k);
    a.v = static_cast<const uint16_t*>(c->v);
    a.q = static_cast<const uint16_t*>(q);
    a.q_stride = q_stride;
    a.batch = batch;
    a.q_heads = q_heads;
    a.heads = c->heads;
    a.dim = c->head_dim;
    a.group = q_heads / c->heads;
    a.tiles = split.tiles;
    a.parts = split.parts;
    a.chunk = split.chunk;
    a.scale = scale * kLog2e;
    a.part_ms = kept ? reinterpret_cast<float*>(ws + ms_at) : nullptr;
    a.part_out = kept ? reinterpret_cast<float*>(ws + out_at) : nullptr;
    a.partial = kept;
    return a;
}

int64_t newest_grid(const gemv_kv_cache* c, int batch, const Split& p)
{
    const int64_t ranges = (int64_t)batch * p.parts;
    return c->heads * (p.tiles > 1 ? (ranges + 7) / 8 * 8 * p.tiles : ranges);
}

// Rows of several tokens per sequence, or of a group.
Prompt tiled(const gemv_kv_cache* c, const Pages& at, int batch, const int32_t* starts, int rows, const Tiling& t,
             const void* q, int64_t q_stride, int q_heads, float scale, char* ws, bool kept)
{
    Prompt a{};
    a.at = at;
    a.k = static_cast<const uint16_t*>(c->k);
    a.v = static_cast<const uint16_t*>(c->v);
    a.q = static_cast<const uint16_t*>(q);
    a.q_stride = q_stride;
    a.starts = starts;
    a.batch = batch;
    a.rows = rows;
    a.max_new = rows;
    a.q_heads = q_heads;
    a.heads = c->heads;
    a.dim = c->head_dim;
    a.group = q_heads / c->heads;
    a.group_of = divider(a.group);
    a.tiles = (int)t.tiles;
    a.order = t.order;
    a.laps = t.laps;
    a.run = t.run;
    a.stretch = t.run * t.laps;
    a.parts = t.parts;
    a.chunk = t.chunk;
    const float size = fabsf(scale) * kLog2e;
    a.scale = size == 0.0f ? 1.0f : size;
    a.keep = size == 0.0f ? 0u : ~0u;
    a.flip = scale < 0 ? 0x80008000u : 0u;
    a.slack = kSlack / a.scale < FLT_MAX ? kSlack / a.scale : FLT_MAX;
    a.part_ms = kept ? reinterpret_cast<float*>(ws + t.ms_at) : nullptr;
    a.part_out = kept ? reinterpret_cast<float*>(ws + t.out_at) : nullptr;
    return a;
}

struct Plan {
    bool single;        // one new token: the kernel of decode attention
    bool joined;
    int window, sinks;
    Split split;        // single
    Tiling tiling;      // otherwise
    size_t ms_at, out_at, bytes;
};

Plan plan_prompt(const gemv_kv_cache* c, const gemv_kv_batch* s, int limit, int rows, int max_new, int q_heads, int window,
                 int sinks, int cus)
{
    Plan p{};
    p.window = narrow_window(window, limit);
    p.sinks = p.window > 0 ? sinks : 0;
    p.single = max_new == 1;
    const int64_t heads = (int64_t)rows * q_heads;
    if (p.single) {
        p.split = split_for(c, s, seen_slots(limit, p.window, whole_sinks(p.sinks, 16, limit)), q_heads, false, cus);
        p.joined = p.split.parts > 1;
        p.ms_at = 0;
        p.out_at = p.joined ? round16((size_t)heads * p.split.parts * 2 * sizeof(float)) : 0;
        p.bytes = p.joined ? p.out_at + (size_t)heads * p.split.parts * c->head_dim * sizeof(float) : 0;
        return p;
    }
    p.tiling = tile_rows(c, rows, s->batch, q_heads / c->heads, limit, p.window, p.sinks,
                         max_new < rows ? max_new : rows, 2.0, true, cus);
    p.joined = p.tiling.parts > 1;
    place_parts(&p.tiling, 0, heads, c->head_dim, p.joined);
    p.bytes = p.tiling.bytes;
    return p;
}

struct PrefixPlan {
    Tiling shared;
    Split own;
    size_t own_ms_at, own_out_at, bytes;
};

PrefixPlan plan_prefix(const gemv_kv_cache* c, const gemv_kv_batch* prefixes, const gemv_kv_batch* s, int far_limit,
                       int limit, int q_heads, int cus)
{
    PrefixPlan p{};
    const int64_t heads = (int64_t)s->batch * q_heads;
    // one place and a half: the others are for the sequences' own tokens.  Over fourteen
    // shapes (16 to 128 sequences, prefixes of 1000 to 60000, heads of 64 to 256) never
    // more than 9 % above the best of one, one and a quarter, one and a half and two
    // places, which are up to 28, 28, 9 and 23 % above it: 128 behind two of up to 32768 141,
    // 141, 123 and 128 us, 64 behind 8000, 64/8 heads, 48, 47, 47, 54, 128 behind two of
    // 16000, 16/4 heads of 256, 129, 110, 119, 116.
    p.shared = tile_rows(c, s->batch, prefixes->batch, q_heads / c->heads, far_limit, 0, 0, 0, 1.5, false, cus);
    if (prefixes->batch == 0 || far_limit == 0)
        p.shared.parts = 0, p.shared.places = 0;
    place_parts(&p.shared, 0, heads, c->head_dim, true);
    p.own = split_for(c, s, limit, q_heads, false, cus, false);
    if (limit == 0)
        p.own.parts = 0;
    p.own_ms_at = p.shared.bytes;
    p.own_out_at = p.own_ms_at + round16((size_t)heads * p.own.parts * 2 * sizeof(float));
    p.bytes = p.own_out_at + (size_t)heads * p.own.parts * c->head_dim * sizeof(float);
    return p;
}

int check_query(const void* q, int64_t q_stride, const void* out)
{
    if (q == nullptr || out == nullptr)
        return GEMV_E_INVAL;
    return q_stride % 8 != 0 || !aligned(q, 16) || !aligned(out, 16) ? GEMV_E_UNSUPPORTED : GEMV_OK;
}

// Whether out's dense rows of `width` elements are q's own, or share no memory with them:
// otherwise rows are written that other workgroups have yet to read.
bool in_place_or_apart(const void* q, int64_t q_stride, const void* out, int64_t rows, int64_t width)
{
    const uintptr_t from = reinterpret_cast<uintptr_t>(q), to = reinterpret_cast<uintptr_t>(out);
    const uintptr_t row = (uintptr_t)width * 2, step = (uintptr_t)q_stride * 2, bytes = (uintptr_t)rows * row;
    if (to == from)
        return q_stride == width || rows == 1;
    if (to < from)
        return from - to >= bytes;
    const uintptr_t i = (to - from) / step, into = (to - from) % step;   // the last row of q that begins at or before out
    return i >= (uintptr_t)rows || (into >= row && (i + 1 == (uintptr_t)rows || step - into >= bytes));
}

// Rows, and sequences of heads, that no launch has work-items for, whose products
// with what follows could pass 64 bits.
bool countable(int64_t rows, int64_t q_heads, int64_t batch, int64_t heads)
{
    return rows * q_heads <= gemv_device::kMaxWorkItems && batch * heads <= gemv_device::kMaxWorkItems;
}

bool holds(const void* workspace, size_t bytes, size_t need)
{
    return need == 0 || (workspace != nullptr && bytes >= need && aligned(workspace, 16));
}

}  // namespace
}  // namespace gattn

extern "C" {

size_t gemv_prompt_attention_workspace(const gemv_kv_cache* cache, const gemv_kv_batch* batch, int rows, int max_new,
                                       int q_heads, int window, int sinks)
{
    using namespace gattn;
    Pages at{};
    if (check(cache, batch, &at) != GEMV_OK || q_heads < 1 || q_heads % cache->heads != 0 || rows < 1 || max_new < 1 ||
        window < 0 || sinks < 0 || batch->batch == 0 || !countable(rows, q_heads, batch->batch, cache->heads))
        return 0;
    gemv_device::Device dev{};
    if (gemv_device::current(&dev) != GEMV_OK)
        return 0;
    return plan_prompt(cache, batch, at.limit, rows, max_new, q_heads, window, sinks, dev.cus).bytes;
}

int gemv_prompt_attention(const gemv_kv_cache* cache, const gemv_kv_batch* batch, const int32_t* starts, int rows,
                          int max_new, const void* q, int64_t q_stride, int q_heads, float scale, int window, int sinks,
                          void* out, void* workspace, size_t workspace_bytes, hipStream_t stream)
{
    using namespace gattn;
    Pages at{};
    if (int rc = check(cache, batch, &at); rc != GEMV_OK)
        return rc;
    if (rows < 0 || max_new < 0 || window < 0 || sinks < 0 || q_heads < 1 || q_heads % cache->heads != 0 ||
        q_stride < (int64_t)q_heads * cache->head_dim)
        return GEMV_E_INVAL;
    if (starts == nullptr && batch->batch > 0 && (max_new != 1 || rows < batch->batch))
        return GEMV_E_INVAL;
    if (batch->batch == 0 || rows == 0 || max_new == 0)
        return GEMV_OK;
    if (int rc = check_query(q, q_stride, out); rc != GEMV_OK)
        return rc;
    if (!countable(rows, q_heads, batch->batch, cache->heads))
        return GEMV_E_UNSUPPORTED;
    if (!in_place_or_apart(q, q_stride, out, starts != nullptr ? rows : batch->batch, (int64_t)q_heads * cache->head_dim))
        return GEMV_E_INVAL;
    gemv_device::Device dev{};
    if (int rc = gemv_device::current(&dev); rc != GEMV_OK)
        return rc;
    const Plan p = plan_prompt(cache, batch, at.limit, rows, max_new, q_heads, window, sinks, dev.cus);
    if (!holds(workspace, workspace_bytes, p.bytes))
        return GEMV_E_INVAL;
    char* ws = static_cast<char*>(workspace);
    Join j{};
    j.rows = starts != nullptr ? rows : batch->batch;
    j.q_heads = q_heads;
    j.dim = cache->head_dim;
    j.starts = starts;
    j.batch = batch->batch;
    j.max_new = max_new;
    j.out = out;
    if (p.joined && !joins_fit(rows, q_heads))
        return GEMV_E_UNSUPPORTED;
    if (p.single) {
        Attention a = newest(cache, at, batch->batch, p.split, q, q_stride, q_heads, scale, ws, p.ms_at, p.out_at, p.joined);
        a.out = out;
        a.starts = starts;
        a.rows = rows;
        a.window = p.window;
        a.sinks = p.sinks;
        a.sinks16 = whole_sinks(p.sinks, 16, at.limit);
        const int64_t grid = newest_grid(cache, batch->batch, p.split);
        const int block = (p.split.lone ? kLoneWaves : kWaves) * 64;
        if (!fits(grid, block))
            return GEMV_E_UNSUPPORTED;
        void* args[] = {(void*)&a};
        const void* fn = cache->dtype == GEMV_F16 ? attention_for<kF16, true>(cache, p.split.lone)
                                                  : attention_for<kBF16, true>(cache, p.split.lone);
        if (int rc = launch(fn, grid, block, args, stream); rc != GEMV_OK || !p.joined)
            return rc;
        j.from[0] = Source{a.part_ms, a.part_out, a.parts, nullptr, 0};
        return join_parts(j, cache->dtype, dev.cus, stream);
    }
    const int64_t grid = p.tiling.places * cache->heads;
    const int block = 256 * outputs_of(cache->head_dim);
    if (!fits(grid, block))
        return GEMV_E_UNSUPPORTED;
    Prompt a = tiled(cache, at, batch->batch, starts, rows, p.tiling, q, q_stride, q_heads, scale, ws, p.joined);
    a.causal = true;
    a.max_new = max_new < rows ? max_new : rows;
    a.window = p.window;
    a.sinks = p.sinks;
    a.sink_tiles = whole_sinks(p.sinks, kTileKeys, at.limit) / kTileKeys;
    a.out = out;
    void* args[] = {(void*)&a};
    if (int rc = launch(tiled_for(kPrompt, cache), grid, block, args, stream); rc != GEMV_OK || !p.joined)
        return rc;
    j.from[0] = Source{a.part_ms, a.part_out, a.parts, nullptr, 0};
    return join_parts(j, cache->dtype, dev.cus, stream);
}

size_t gemv_prefix_attention_workspace(const gemv_kv_cache* cache, const gemv_kv_batch* prefixes,
                                       const gemv_kv_batch* batch, int q_heads)
{
    using namespace gattn;
    Pages at{}, far{};
    if (check(cache, batch, &at) != GEMV_OK || check(cache, prefixes, &far) != GEMV_OK || q_heads < 1 ||
        q_heads % cache->heads != 0 || batch->batch == 0 ||
        !countable(batch->batch, q_heads, (int64_t)batch->batch + prefixes->batch, cache->heads))
        return 0;
    gemv_device::Device dev{};
    if (gemv_device::current(&dev) != GEMV_OK)
        return 0;
    return plan_prefix(cache, prefixes, batch, far.limit, at.limit, q_heads, dev.cus).bytes;
}

int gemv_prefix_attention(const gemv_kv_cache* cache, const gemv_kv_batch* prefixes, const int32_t* starts,
                          const gemv_kv_batch* batch, const void* q, int64_t q_stride, int q_heads, float scale, void* out,
                          void* workspace, size_t workspace_bytes, hipStream_t stream)
{
    using namespace gattn;
    Pages at{}, far{};
    if (int rc = check(cache, batch, &at); rc != GEMV_OK)
        return rc;
    if (int rc = check(cache, prefixes, &far); rc != GEMV_OK)
        return rc;
    if (q_heads < 1 || q_heads % cache->heads != 0 || q_stride < (int64_t)q_heads * cache->head_dim)
        return GEMV_E_INVAL;
    if (prefixes->batch > 0 && starts == nullptr)
        return GEMV_E_INVAL;
    if (batch->batch == 0)
        return GEMV_OK;
    if (int rc = check_query(q, q_stride, out); rc != GEMV_OK)
        return rc;
    if (!countable(batch->batch, q_heads, (int64_t)batch->batch + prefixes->batch, cache->heads))
        return GEMV_E_UNSUPPORTED;
    if (!in_place_or_apart(q, q_stride, out, batch->batch, (int64_t)q_heads * cache->head_dim))
        return GEMV_E_INVAL;
    gemv_device::Device dev{};
    if (int rc = gemv_device::current(&dev); rc != GEMV_OK)
        return rc;
    const PrefixPlan p = plan_prefix(cache, prefixes, batch, far.limit, at.limit, q_heads, dev.cus);
    if (!holds(workspace, workspace_bytes, p.bytes))
        return GEMV_E_INVAL;
    const int64_t far_count = p.shared.places * cache->heads, far_blocks = (far_count + 7) / 8 * 8;
    const int64_t near_count = p.own.parts > 0 ? newest_grid(cache, batch->batch, p.own) : 0;
    const int block = 256 * outputs_of(cache->head_dim);
    if (!fits(far_blocks + near_count, block) || !joins_fit(batch->batch, q_heads))
        return GEMV_E_UNSUPPORTED;
    char* ws = static_cast<char*>(workspace);
    Join j{};
    j.rows = batch->batch;
    j.q_heads = q_heads;
    j.dim = cache->head_dim;
    j.out = out;
    Prompt f = tiled(cache, far, prefixes->batch, starts, batch->batch, p.shared, q, q_stride, q_heads, scale, ws, true);
    Attention n = newest(cache, at, batch->batch, p.own, q, q_stride, q_heads, scale, ws, p.own_ms_at, p.own_out_at, true);
    n.rows = batch->batch;
    if (far_count > 0)
        j.from[0] = Source{f.part_ms, f.part_out, f.parts, starts, prefixes->batch};
    if (near_count > 0)
        j.from[1] = Source{n.part_ms, n.part_out, n.parts, nullptr, 0};
    if (far_blocks + near_count > 0) {
        int blocks = (int)far_blocks, count = (int)far_count;
        void* args[] = {(void*)&f, (void*)&n, (void*)&blocks, (void*)&count};
        if (int rc = launch(tiled_for(kPrefix, cache), far_blocks + near_count, block, args, stream); rc != GEMV_OK)
            return rc;
    }
    return join_parts(j, cache->dtype, dev.cus, stream);
}

}  // extern "C"
