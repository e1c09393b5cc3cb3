// attention_api.hip -- C ABI of decode attention over a paged key-value cache,
// its append and its eviction (declared in include/gemv_attention.h):
// validation, workspaces, geometry and launch.
#include "attention_host.hpp"
#include "cache_kernels.hpp"

#include <hip/hip_runtime.h>

#include <limits.h>

namespace gattn {
namespace {

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
