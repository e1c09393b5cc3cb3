// attention_api.hip -- C ABI of decode attention over a paged key-value cache,
// its append and its eviction (declared in include/gemv_attention.h):
// validation, workspaces, geometry and launch.
#include "gemv_attention.h"
#include "attention_kernels.hpp"
#include "device_info.hpp"

#include <hip/hip_runtime.h>

#include <limits.h>

namespace gattn {
namespace {

bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

size_t round16(size_t n) { return (n + 15) & ~(size_t)15; }

Divider divider(int d)
{
    unsigned shift = 0;
    while (((uint64_t)1 << shift) < (uint64_t)d)
        ++shift;
    const uint64_t over = ((uint64_t)1 << shift) - (uint64_t)d;
    return Divider{(unsigned)((over << 32) / (uint64_t)d + 1), shift};
}

// Checks shared by every entry point; fills the addressing part.
int check(const gemv_kv_cache* c, const gemv_kv_batch* s, Pages* out)
{
    if (c == nullptr || s == nullptr)
        return GEMV_E_INVAL;
    if (s->batch < 0 || s->width < 0 || s->max_len < 0 || s->table_stride < s->width)
        return GEMV_E_INVAL;
    if (c->pages < 0 || c->page_size < 1 || c->heads < 1 || c->head_dim < 1 ||
        (c->dtype != GEMV_F16 && c->dtype != GEMV_BF16))
        return GEMV_E_INVAL;
    if (c->stride_page < c->head_dim || c->stride_slot < c->head_dim || c->stride_head < c->head_dim)
        return GEMV_E_INVAL;
    if (s->batch > 0 && s->lens == nullptr)
        return GEMV_E_INVAL;
    if (s->batch > 0 && s->width > 0 && (s->table == nullptr || (c->pages > 0 && (c->k == nullptr || c->v == nullptr))))
        return GEMV_E_INVAL;
    if (c->head_dim % 8 != 0 || c->head_dim > 256 || c->stride_page % 8 != 0 || c->stride_slot % 8 != 0 ||
        c->stride_head % 8 != 0 || !aligned(c->k, 16) || !aligned(c->v, 16))
        return GEMV_E_UNSUPPORTED;
    // the kernels step past a length by up to a few thousand slots, in int
    const int64_t room = (int64_t)s->width * c->page_size, most = INT_MAX - 4095;
    int64_t limit = room < s->max_len ? room : s->max_len;
    limit = limit < most ? limit : most;
    *out = Pages{s->table, s->table_stride, s->lens, (int)limit, c->pages, c->page_size, divider(c->page_size),
                 c->stride_page, c->stride_slot, c->stride_head};
    return GEMV_OK;
}

int launch(const void* fn, int64_t grid, int block, void** args, hipStream_t stream, int lds = 0)
{
    return hipLaunchKernel(fn, dim3((unsigned)grid), dim3(block), args, lds, stream) == hipSuccess ? GEMV_OK
                                                                                                 : GEMV_E_LAUNCH;
}

bool fits(int64_t grid, int block) { return grid <= gemv_device::kMaxWorkItems / block; }

// How the length is split: workgroups per key-value head and slots of each.
struct Split {
    bool lone;
    int tiles, parts, chunk;
    int64_t logits_stride;
    size_t ms_at, out_at, logits_at, bytes;
};

// Tiles of 16 slots that lie in one page, near enough for 32-bit offsets.
bool whole_tiles(const gemv_kv_cache* c) { return c->page_size % 16 == 0 && c->stride_slot < (1 << 26); }

// Slots of a part, a multiple of 64 (a tile for each wave) up to kMaxChunk: the
// least estimate, in slots, of what the busiest CU reads, with 100 for a
// workgroup's start and end and 150 for a join.  A second round of workgroups
// that is mostly empty costs most.  8 key-value heads of 128, 2 x 8192 slots:
// 19 us, with two workgroups per CU 21.2, with four 24.0; 32 x 1024: 25, 31.1,
// 30.9; 5 heads of 96, 32 x 2000: three parts; one, two and four per CU 41.3,
// 34.8, 37.6.
// Heads of up to 64 have small tiles and wait for them, so where the heads
// alone fill the card and no part holds the whole length they are split into
// eight workgroups per CU: 16 heads of 64, 16 x 301 to 2047 slots 23.8 us, by the
// estimate 26.2; 8 heads, 64 x 100 to 1500 slots 29.8 and 37.3; 32 heads, 8 x 500
// to 4000 slots 38.3 and 49.1.  Fewer heads, or lengths that one part holds, are
// slower so: 4 heads, 1 x 30000 slots 39.9 and 15.5 by the estimate; 8 heads, 2 x
// 8192 23.5 and 13.1; 32 x 1024 21.3 and 15.0.
int chunk_for(int64_t items, int limit, int dim, int cus)
{
    if (dim <= 64 && items >= cus && limit > kMaxChunk) {
        const int64_t chunk = ((int64_t)limit * items / ((int64_t)cus * 8) + 63) / 64 * 64;
        return (int)(chunk < kMaxChunk ? chunk : kMaxChunk);
    }
    int best = kMaxChunk;
    int64_t least = INT64_MAX;
    for (int chunk = kMaxChunk; chunk >= 64; chunk -= 64) {
        const int64_t parts = ((int64_t)limit + chunk - 1) / chunk;
        const int64_t cost = (items * parts + cus - 1) / cus * (chunk + 100) + (parts > 1 ? 150 + parts : 0);
        if (cost < least) {
            best = chunk;
            least = cost;
        }
    }
    return best;
}

Split split_for(const gemv_kv_cache* c, const gemv_kv_batch* s, int limit, int q_heads, bool weighted, int cus)
{
    Split p;
    const int group = q_heads / c->heads;
    p.tiles = (group + 15) / 16;
    const int64_t items = (int64_t)s->batch * c->heads * p.tiles;
    int chunk = chunk_for(items, limit, c->head_dim, cus);
    // Short lengths are not split: eight waves of one workgroup are done before
    // a second launch has joined parts.  Head size 128, in a captured graph: 8
    // key-value heads of 256 slots 7.5 us against 9.5, of 512 slots 11.3 against
    // 8.8; 128 of them, which fill half the card, 512 slots 12.3 against 17.6, 768
    // 15.8 against 16.7.
    p.lone = whole_tiles(c) && chunk < limit && (limit <= 256 || (limit <= 768 && items * 2 >= cus));
    if (p.lone)
        chunk = (limit + 63) / 64 * 64;
    p.chunk = chunk;
    p.parts = (int)(((int64_t)limit + p.chunk - 1) / p.chunk);
    p.parts = p.parts < 1 ? 1 : p.parts;
    const size_t rows = (size_t)s->batch * (size_t)q_heads;
    p.ms_at = 0;
    p.out_at = p.parts > 1 || weighted ? round16(rows * p.parts * 2 * sizeof(float)) : 0;
    p.logits_at = p.out_at + (p.parts > 1 ? round16(rows * p.parts * c->head_dim * sizeof(float)) : 0);
    p.logits_stride = ((int64_t)limit + 15) / 16 * 16;
    p.bytes = p.logits_at + (weighted ? rows * (size_t)p.logits_stride * sizeof(float) : 0);
    return p;
}

template <int DT, bool WHOLE, int WAVES>
const void* attention_sized(int dim)
{
    if constexpr (WHOLE) {
        if (dim == 64)
            return reinterpret_cast<const void*>(&attention_kernel<DT, 64, true, true, WAVES>);
        if (dim == 128)
            return reinterpret_cast<const void*>(&attention_kernel<DT, 128, true, true, WAVES>);
        if (dim == 256)
            return reinterpret_cast<const void*>(&attention_kernel<DT, 256, true, true, WAVES>);
    }
    return dim <= 64    ? reinterpret_cast<const void*>(&attention_kernel<DT, 64, WHOLE, false, WAVES>)
           : dim <= 128 ? reinterpret_cast<const void*>(&attention_kernel<DT, 128, WHOLE, false, WAVES>)
                        : reinterpret_cast<const void*>(&attention_kernel<DT, 256, WHOLE, false, WAVES>);
}

template <int DT>
const void* attention_for(const gemv_kv_cache* c, bool lone)
{
    return lone             ? attention_sized<DT, true, kLoneWaves>(c->head_dim)
           : whole_tiles(c) ? attention_sized<DT, true, kWaves>(c->head_dim)
                            : attention_sized<DT, false, kWaves>(c->head_dim);
}

int evict_moves(int limit, int budget)
{
    const int over = limit > budget ? limit - budget : 0;
    return over < budget ? over : budget;
}

// The workspace of an eviction: what the selection leaves for the launch that
// moves, nothing where it moves by itself.
struct Scratch {
    int words;
    size_t bits_at, moves_at, bytes;
};

Scratch evict_scratch(int batch, int heads, int limit, int budget, int moves)
{
    Scratch s{};
    if (moves <= kFusedMoves)
        return s;
    const size_t bh = (size_t)batch * (size_t)heads;
    s.words = ((budget < limit ? budget : limit) + 63) / 64;
    s.bits_at = round16(bh * sizeof(int32_t));
    s.moves_at = s.bits_at + round16(bh * s.words * sizeof(uint64_t));
    s.bytes = s.moves_at + bh * 2 * (size_t)moves * sizeof(int32_t);
    return s;
}

}  // namespace
}  // namespace gattn

extern "C" {

size_t gemv_attention_workspace(const gemv_kv_cache* cache, const gemv_kv_batch* batch, int q_heads, int weighted)
{
    using namespace gattn;
    Pages at{};
    if (check(cache, batch, &at) != GEMV_OK || q_heads < 1 || q_heads % cache->heads != 0)
        return 0;
    gemv_device::Device dev{};
    if (gemv_device::current(&dev) != GEMV_OK)
        return 0;
    return split_for(cache, batch, at.limit, q_heads, weighted != 0, dev.cus).bytes;
}

int gemv_attention(const gemv_kv_cache* cache, const gemv_kv_batch* batch, const void* q, int64_t q_stride,
                   int q_heads, float scale, void* out, float* weights, int64_t slots, void* workspace,
                   size_t workspace_bytes, hipStream_t stream)
{
    using namespace gattn;
    Attention a{};
    if (int rc = check(cache, batch, &a.at); rc != GEMV_OK)
        return rc;
    if (q_heads < 1 || q_heads % cache->heads != 0 || (weights != nullptr && slots < a.at.limit) ||
        q_stride < (int64_t)q_heads * cache->head_dim)
        return GEMV_E_INVAL;
    if (batch->batch == 0)
        return GEMV_OK;
    if (q == nullptr || out == nullptr)
        return GEMV_E_INVAL;
    if (q_stride % 8 != 0 || !aligned(q, 16) || !aligned(out, 2))
        return GEMV_E_UNSUPPORTED;
    gemv_device::Device dev{};
    if (int rc = gemv_device::current(&dev); rc != GEMV_OK)
        return rc;
    const Split p = split_for(cache, batch, a.at.limit, q_heads, weights != nullptr, dev.cus);
    if (p.bytes > 0 && (workspace == nullptr || workspace_bytes < p.bytes || !aligned(workspace, 16)))
        return GEMV_E_INVAL;
    const int64_t items = (int64_t)batch->batch * cache->heads;
    const int64_t ranges = (int64_t)batch->batch * p.parts;
    const int64_t grid = cache->heads * (p.tiles > 1 ? (ranges + 7) / 8 * 8 * p.tiles : ranges);
    const int64_t joins = p.parts > 1 ? (int64_t)batch->batch * q_heads : 0;
    int blocks = weights != nullptr ? (int)(((int64_t)a.at.limit + 1023) / 1024) : 0;
    const int block = (p.lone ? kLoneWaves : kWaves) * 64;
    if (!fits(grid, block) || !fits(joins + items * blocks, 256))
        return GEMV_E_UNSUPPORTED;
    char* ws = static_cast<char*>(workspace);
    a.k = static_cast<const uint16_t*>(cache->k);
    a.v = static_cast<const uint16_t*>(cache->v);
    a.q = static_cast<const uint16_t*>(q);
    a.q_stride = q_stride;
    a.batch = batch->batch;
    a.q_heads = q_heads;
    a.heads = cache->heads;
    a.dim = cache->head_dim;
    a.group = q_heads / cache->heads;
    a.tiles = p.tiles;
    a.parts = p.parts;
    a.chunk = p.chunk;
    a.scale = scale * 1.44269504088896340736f;
    a.out = out;
    a.part_ms = p.parts > 1 || weights != nullptr ? reinterpret_cast<float*>(ws + p.ms_at) : nullptr;
    a.part_out = p.parts > 1 ? reinterpret_cast<float*>(ws + p.out_at) : nullptr;
    a.logits = weights != nullptr ? reinterpret_cast<float*>(ws + p.logits_at) : nullptr;
    a.logits_stride = p.logits_stride;
    a.weights = weights;
    a.slots = slots;
    a.weights_wide = slots % 4 == 0 && aligned(weights, 16);
    void* args[] = {(void*)&a};
    const void* fn = cache->dtype == GEMV_F16 ? attention_for<kF16>(cache, p.lone) : attention_for<kBF16>(cache, p.lone);
    if (int rc = launch(fn, grid, block, args, stream); rc != GEMV_OK)
        return rc;
    if (joins + items * blocks == 0)
        return GEMV_OK;
    int rows = (int)joins;
    void* jargs[] = {(void*)&a, (void*)&rows, (void*)&blocks};
    return launch(cache->dtype == GEMV_F16 ? reinterpret_cast<const void*>(&join_kernel<kF16>)
                                           : reinterpret_cast<const void*>(&join_kernel<kBF16>),
                  joins + items * blocks, 256, jargs, stream);
}

int gemv_kv_append(const gemv_kv_cache* cache, const gemv_kv_batch* batch, const int32_t* starts, const void* k,
                   int64_t k_stride, const void* v, int64_t v_stride, int rows, float* weights, int32_t* positions,
                   const int32_t* seen, int64_t slots, hipStream_t stream)
{
    using namespace gattn;
    Append a{};
    if (cache == nullptr || batch == nullptr)
        return GEMV_E_INVAL;
    gemv_kv_batch all = *batch;
    all.max_len = INT_MAX;
    if (int rc = check(cache, &all, &a.at); rc != GEMV_OK)
        return rc;
    const int64_t width = (int64_t)cache->heads * cache->head_dim;
    if (rows < 0 || k_stride < width || v_stride < width)
        return GEMV_E_INVAL;
    const int tracked = (weights != nullptr) + (positions != nullptr) + (seen != nullptr);
    if ((tracked != 0 && tracked != 3) || (tracked == 3 && slots < 0))
        return GEMV_E_INVAL;
    if (batch->batch == 0 || rows == 0 || a.at.limit == 0)
        return GEMV_OK;
    if (starts == nullptr || k == nullptr || v == nullptr)
        return GEMV_E_INVAL;
    if (k_stride % 8 != 0 || v_stride % 8 != 0 || !aligned(k, 16) || !aligned(v, 16))
        return GEMV_E_UNSUPPORTED;
    gemv_device::Device dev{};
    if (int rc = gemv_device::current(&dev); rc != GEMV_OK)
        return rc;
    a.k = static_cast<uint16_t*>(cache->k);
    a.v = static_cast<uint16_t*>(cache->v);
    a.starts = starts;
    a.new_k = static_cast<const uint16_t*>(k);
    a.new_v = static_cast<const uint16_t*>(v);
    a.k_stride = k_stride;
    a.v_stride = v_stride;
    a.rows = rows;
    a.batch = batch->batch;
    a.heads = cache->heads;
    a.dim = cache->head_dim;
    a.weights = weights;
    a.positions = positions;
    a.seen = seen;
    a.slots = slots;
    void* args[] = {(void*)&a};
    return launch(reinterpret_cast<const void*>(&append_kernel), gemv_device::capped_grid(((int64_t)rows + 3) / 4, 256),
                  256, args, stream);
}

size_t gemv_kv_evict_workspace(const gemv_kv_cache* cache, const gemv_kv_batch* batch, int budget)
{
    using namespace gattn;
    Pages at{};
    if (check(cache, batch, &at) != GEMV_OK || budget < 0)
        return 0;
    return evict_scratch(batch->batch, cache->heads, at.limit, budget, evict_moves(at.limit, budget)).bytes;
}

int gemv_kv_evict(const gemv_kv_cache* cache, const gemv_kv_batch* batch, const int32_t* seen, const float* weights,
                  const int32_t* positions, int64_t slots, int budget, int recent, float* weights_out,
                  int32_t* positions_out, int32_t* lens_out, void* workspace, size_t workspace_bytes,
                  hipStream_t stream)
{
    using namespace gattn;
    Evict a{};
    if (int rc = check(cache, batch, &a.at); rc != GEMV_OK)
        return rc;
    if (budget < 0 || recent < 0 || slots < a.at.limit)
        return GEMV_E_INVAL;
    if (batch->batch == 0)
        return GEMV_OK;
    if (seen == nullptr || lens_out == nullptr ||
        (slots > 0 && (weights == nullptr || positions == nullptr || weights_out == nullptr || positions_out == nullptr)))
        return GEMV_E_INVAL;
    gemv_device::Device dev{};
    if (int rc = gemv_device::current(&dev); rc != GEMV_OK)
        return rc;
    a.moves_max = evict_moves(a.at.limit, budget);
    const Scratch ws = evict_scratch(batch->batch, cache->heads, a.at.limit, budget, a.moves_max);
    if (ws.bytes > 0 && (workspace == nullptr || workspace_bytes < ws.bytes || !aligned(workspace, 16)))
        return GEMV_E_INVAL;
    const int64_t items = (int64_t)batch->batch * cache->heads;
    // two pieces a thread; a move has head_dim / 4 of them
    int blocks = (int)(((int64_t)a.moves_max * (cache->head_dim / 4) + 511) / 512);
    if (!fits(items, kEvictThreads))
        return GEMV_E_UNSUPPORTED;
    const int64_t most = gemv_device::kMaxWorkItems / 256 / items;   // at least 4; the blocks walk what lies beyond
    blocks = blocks > 1024 ? 1024 : blocks;
    blocks = blocks > most ? (int)most : blocks;
    a.k = static_cast<uint16_t*>(cache->k);
    a.v = static_cast<uint16_t*>(cache->v);
    a.seen = seen;
    a.weights = weights;
    a.positions = positions;
    a.slots = slots;
    a.heads = cache->heads;
    a.dim = cache->head_dim;
    a.budget = budget;
    a.recent = recent;
    a.weights_out = weights_out;
    a.positions_out = positions_out;
    a.lens_out = lens_out;
    char* at = static_cast<char*>(workspace);
    a.words = ws.words;
    a.count = reinterpret_cast<int32_t*>(at);
    a.bits = reinterpret_cast<uint64_t*>(at + ws.bits_at);
    a.moves = reinterpret_cast<int32_t*>(at + ws.moves_at);
    void* args[] = {(void*)&a};
    const bool fused = a.moves_max <= kFusedMoves;
    a.held = a.at.limit < kHeldKeys ? a.at.limit : kHeldKeys;
    if (int rc = launch(fused ? reinterpret_cast<const void*>(&evict_select_kernel<true>)
                              : reinterpret_cast<const void*>(&evict_select_kernel<false>),
                        items, kEvictThreads, args, stream, a.held * (int)sizeof(unsigned));
        rc != GEMV_OK || fused)
        return rc;
    void* margs[] = {(void*)&a, (void*)&blocks};
    return launch(reinterpret_cast<const void*>(&evict_move_kernel), items * blocks, 256, margs, stream);
}

}  // extern "C"
