// attention_host.hpp -- host code that the entry points over a paged
// key-value cache share: checks, launches, and how decode attention splits a
// length.
#pragma once

#include "gemv_attention.h"
#include "attention_kernels.hpp"
#include "device_info.hpp"

#include <hip/hip_runtime.h>

#include <limits.h>

namespace gattn {

inline bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

inline size_t round16(size_t n) { return (n + 15) & ~(size_t)15; }

inline Divider divider(int d)
{
    unsigned shift = 0;
    while (((uint64_t)1 << shift) < (uint64_t)d)
        ++shift;
    const uint64_t over = ((uint64_t)1 << shift) - (uint64_t)d;
    return Divider{(unsigned)((over << 32) / (uint64_t)d + 1), shift};
}

// Checks shared by every entry point; fills the addressing part.
inline int check(const gemv_kv_cache* c, const gemv_kv_batch* s, Pages* out)
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

inline int launch(const void* fn, int64_t grid, int block, void** args, hipStream_t stream, int lds = 0)
{
    return hipLaunchKernel(fn, dim3((unsigned)grid), dim3(block), args, lds, stream) == hipSuccess ? GEMV_OK
                                                                                                 : GEMV_E_LAUNCH;
}

inline bool fits(int64_t grid, int block) { return grid <= gemv_device::kMaxWorkItems / block; }

// How the length is split: workgroups per key-value head and slots of each.
struct Split {
    bool lone;
    int tiles, parts, chunk;
    int64_t logits_stride;
    size_t ms_at, out_at, logits_at, bytes;
};

// Tiles of 16 slots that lie in one page, near enough for 32-bit offsets.
inline bool whole_tiles(const gemv_kv_cache* c) { return c->page_size % 16 == 0 && c->stride_slot < (1 << 26); }

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
inline int chunk_for(int64_t items, int limit, int dim, int cus)
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

inline Split split_for(const gemv_kv_cache* c, const gemv_kv_batch* s, int limit, int q_heads, bool weighted, int cus,
                       bool may_be_lone = true)
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
    p.lone = may_be_lone && whole_tiles(c) && chunk < limit && (limit <= 256 || (limit <= 768 && items * 2 >= cus));
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

template <int DT, bool WHOLE, int WAVES, bool VIEW>
const void* attention_sized(int dim)
{
    if constexpr (WHOLE) {
        if (dim == 64)
            return reinterpret_cast<const void*>(&attention_kernel<DT, 64, true, true, WAVES, VIEW>);
        if (dim == 128)
            return reinterpret_cast<const void*>(&attention_kernel<DT, 128, true, true, WAVES, VIEW>);
        if (dim == 256)
            return reinterpret_cast<const void*>(&attention_kernel<DT, 256, true, true, WAVES, VIEW>);
    }
    return dim <= 64    ? reinterpret_cast<const void*>(&attention_kernel<DT, 64, WHOLE, false, WAVES, VIEW>)
           : dim <= 128 ? reinterpret_cast<const void*>(&attention_kernel<DT, 128, WHOLE, false, WAVES, VIEW>)
                        : reinterpret_cast<const void*>(&attention_kernel<DT, 256, WHOLE, false, WAVES, VIEW>);
}

template <int DT, bool VIEW = false>
const void* attention_for(const gemv_kv_cache* c, bool lone)
{
    return lone             ? attention_sized<DT, true, kLoneWaves, VIEW>(c->head_dim)
           : whole_tiles(c) ? attention_sized<DT, true, kWaves, VIEW>(c->head_dim)
                            : attention_sized<DT, false, kWaves, VIEW>(c->head_dim);
}

}  // namespace gattn
