// attention_kernels.hpp -- gfx950 (CDNA4) device code for decode attention
// over a paged key-value cache.
//
//   o_h = sum_j p_hj v_j,  p_h = softmax_j(scale * q_h . k_j)
//
// Bound by memory: every key and value is read once for the few operations of
// a group of query heads.  Reached on one MI355X, where a pure read makes 7.1
// TB/s: 5.2 TB/s over 64 sequences of 100 to 8192 slots (8 heads of 128, 222 us;
// 6.0 TB/s where all have 8192).  The same 64 sequences with other heads: 8 of 64
// 127 to 132 us, 80 and 96 195 to 201, 256 460 us (5.1 TB/s).
#pragma once

#include "paged.hpp"

namespace gattn {

// ---------------------------------------------------------------- attention
struct Attention {
    Pages at;
    const uint16_t* k;
    const uint16_t* v;
    const uint16_t* q;
    int64_t q_stride;
    int batch, q_heads, heads, dim;
    int group;        // query heads per key-value head
    int tiles;        // workgroups per key-value head: ceil(group / 16)
    int parts;        // workgroups over the length
    int chunk;        // slots each takes, a multiple of 64
    float scale;      // of the logits, log2(e) included: softmax in powers of two
    void* out;
    float* part_out;  // [batch][q_heads][parts][dim], not divided by the sums
    float* part_ms;   // [batch][q_heads][parts][2]: maximum and sum of powers
    float* logits;    // [batch][q_heads][logits_stride], or null
    int64_t logits_stride;   // the longest length in whole tiles
    float* weights;   // [batch][heads][slots], or null
    int64_t slots;
    bool weights_wide;       // rows of weights are 16-byte aligned
    // VIEW only:
    const int32_t* starts;   // [batch + 1]: a sequence's query is row starts[b + 1] - 1; or null, row b
    int rows;                // of q and out
    int window;              // tokens seen, the newest included; 0: all
    int sinks;               // first tokens seen all the same
    int sinks16;             // in whole tiles
    bool partial;            // parts are kept for a join even where there is one
};

constexpr int kWaves = 4;         // of a workgroup, where the length is split or the card is full
constexpr int kLoneWaves = 8;     // where one workgroup takes a short sequence's whole length
constexpr int kMaxChunk = 1024;  // slots of a part: 16 tiles a wave
constexpr float kSlack = 8.0f;   // powers of two that a logit may pass the reference maximum by

// One workgroup: up to 16 query heads of one key-value head of one sequence,
// over one part of its length.  Its waves take tiles of 16 slots in turn.
//
// Logits: v_mfma_f32_16x16x32 with the tile's keys as rows and the heads'
// queries as columns: lane l loads 16 bytes of key l % 16 and gets, for head
// l % 16, the logits of slots 4 (l / 16) + r, r = 0..3.  These are in place as
// the left operand of v_mfma_f32_16x16x4_f32 (row l % 16, summed index
// l / 16): step r multiplies slot 4 (l / 16) + r of each quarter, whose values lane l
// has loaded 16 bytes of, the elements of column l % 16 of VW tiles.  So neither
// keys, values nor probabilities cross lanes or go through LDS, and the
// probabilities and values are multiplied unrounded in binary32.
//
// The running maximum only moves when a logit passes it by kSlack: the powers
// then stay below 2^kSlack, which binary32 sums hold as exactly as those
// below 1, and the sums are rescaled a few times per sequence instead of
// with each tile.
//
// The binary32 products cost 32 matrix instructions a tile, about 1000 cycles of
// a SIMD; at 7 TB/s a tile's turn on a SIMD is 2900 cycles, so they are hidden.
//
// A wave loads its next tile while it multiplies the current one.  Where
// pages are whole numbers of tiles (WHOLE), a tile has one page and its
// address is the same for all lanes; otherwise each row has an address of its
// own, and its loads wait at a branch (64 sequences of 100 to 8192 slots in pages
// of 5, 8 or 24: 266 to 269 us, where pages of 16 take 223; heads of 256, 659
// against 460).  EXACT: the head's size is DP, so no lane is without an element.
//
// VIEW: the newest token sees a window and the first tokens.  The slots between,
// in whole tiles, are cut out of the length (slot j past the first tokens'
// tiles is slot j + gap of the sequence), so only the window's first tile and the
// first tokens' last hold slots that are not seen; these are not read.
template <int DP, bool WHOLE, int WAVES>
struct AttentionShared {
    float red_m[WAVES][16];
    float red_s[WAVES][16];
    __attribute__((aligned(16))) float red_o[WAVES][16][DP];
    int32_t slot_page[WHOLE ? 1 : kMaxChunk];
};

template <int DT, int DP, bool WHOLE, bool EXACT, int WAVES, bool VIEW>
__device__ __forceinline__ void attention_block(const Attention& a, int block, AttentionShared<DP, WHOLE, WAVES>& shared)
{
    constexpr int kSteps = DP / 32;              // of 32 elements of the dot products
    constexpr int VW = DP == 64 ? 4 : 8;         // elements of a value row per lane and set
    constexpr int kSets = DP / (16 * VW);
    constexpr int kWords = VW / 2;
    auto& red_m = shared.red_m;
    auto& red_s = shared.red_s;
    auto& red_o = shared.red_o;

    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int col = lane & 15, quarter = lane >> 4;
    // Neighbouring workgroups go to the eight XCDs in turn.  Heads vary
    // fastest, so the rows of one token, which lie together, are read at about
    // the same time; each XCD's share moves on by a head from one token range
    // to the next, so that it sees every head's part of the address space; and
    // parts vary slowest, so that the ends that only long sequences reach are
    // spread over all XCDs.
    // Where a head's queries need several workgroups, those that read the same
    // keys are a multiple of eight apart: on one XCD, at about the same time.
    const int turn = block / a.heads;
    const int kv = (block + turn) % a.heads;
    int tile = 0, range = turn;
    if (a.tiles > 1) {
        const int eight = turn / (8 * a.tiles), rest = turn - eight * 8 * a.tiles;
        tile = rest >> 3;
        range = eight * 8 + (rest & 7);
        if (range >= a.batch * a.parts)
            return;
    }
    const int b = range % a.batch;
    const int part = range / a.batch;
    int len = __builtin_amdgcn_readfirstlane(a.at.length(b));
    const int64_t first = (int64_t)part * a.chunk;
    const int head0 = kv * a.group + tile * 16;                          // this workgroup's query heads
    const int nheads = a.group - tile * 16 < 16 ? a.group - tile * 16 : 16;
    int64_t query_row = b;
    int gap = 0, low = 0;                                                // of VIEW: slots cut out, first slot of the window
    if constexpr (VIEW) {
        if (a.starts != nullptr) {
            query_row = row_start(a.starts, b + 1, a.rows) - 1;
            if (row_start(a.starts, b, a.rows) > query_row)
                return;                                                  // no new token
        }
        if (a.window > 0 && len > a.window) {
            low = len - a.window;
            gap = (low & ~15) - a.sinks16;
            gap = gap > 0 ? gap : 0;
            len -= gap;
        }
    }
    if (part > 0 && first >= len) {                                      // the join does not look at it, but of VIEW
        if constexpr (VIEW)
            if ((int)threadIdx.x < nheads) {
                float* ms = a.part_ms + ((query_row * a.q_heads + head0 + threadIdx.x) * a.parts + part) * 2;
                ms[0] = -kInf;
                ms[1] = 0.0f;
            }
        return;
    }
    const int begin = (int)first;
    const int end = first + a.chunk < len ? (int)(first + a.chunk) : len;
    auto seen_at = [&](int j) { return VIEW && j >= a.sinks16 ? j + gap : j; };        // slot of the sequence
    auto is_seen = [&](int j) { return !VIEW || seen_at(j) >= low || j < a.sinks; };

    u32x4 query[kSteps];
#pragma unroll
    for (int s = 0; s < kSteps; ++s) {
        const int d = 32 * s + 8 * quarter;
        query[s] = u32x4{0, 0, 0, 0};
        if (col < nheads && (EXACT || d < a.dim))
            query[s] = *reinterpret_cast<const u32x4*>(a.q + query_row * a.q_stride + (int64_t)(head0 + col) * a.dim + d);
    }

    float m = -kInf, sum = 0.0f;
    f32x4 acc[kSets][VW];
#pragma unroll
    for (int s = 0; s < kSets; ++s)
#pragma unroll
        for (int e = 0; e < VW; ++e)
            acc[s][e] = f32x4{0, 0, 0, 0};

    struct Tile {
        u32x4 key[kSteps];
        unsigned value[4][kSets][kWords];
        unsigned held;   // bit r: slot 4 quarter + r is there
    };
    auto slot_of = [&](int t) { return begin + (wave + t * WAVES) * 16; };   // tile t of this wave
    const uint16_t* k0 = a.k + kv * a.at.stride_head;
    const uint16_t* v0 = a.v + kv * a.at.stride_head;

    // the pages of this part, looked up once so that no tile's loads wait for
    // a page number: WHOLE, tile t of this wave in lane t; otherwise every slot's in LDS
    int pages = -1;
    auto& slot_page = shared.slot_page;
    if constexpr (WHOLE) {
        const int64_t j = (int64_t)begin + (wave + lane * WAVES) * 16;
        if (VIEW ? j < end : j < a.at.limit)
            pages = a.at.table[b * a.at.table_stride + a.at.page_of.by(seen_at((int)j))];
    } else {
        for (int i = threadIdx.x; i < a.chunk; i += WAVES * 64)
            slot_page[i] = begin + i < end && is_seen(begin + i)
                               ? a.at.table[b * a.at.table_stride + a.at.page_of.by(seen_at(begin + i))] : -1;
        __syncthreads();
    }
    auto offset_at = [&](int j) -> int64_t {   // of slot j < end, where !WHOLE
        const int page = slot_page[j - begin];
        if ((unsigned)page >= (unsigned)a.at.pages)
            return -1;
        j = seen_at(j);
        return page * a.at.stride_page + (int64_t)(j - a.at.page_of.by(j) * a.at.page_size) * a.at.stride_slot;
    };
    // byte offsets of this lane's pieces from the tile's first slot (WHOLE;
    // the host has checked that 16 slots span less than 2^31 bytes)
    const unsigned key_lane = (unsigned)(col * (int)a.at.stride_slot + 8 * quarter) * 2;
    const unsigned value_lane = (unsigned)(4 * quarter * (int)a.at.stride_slot + VW * col) * 2;
    const unsigned value_step = (unsigned)a.at.stride_slot * 2;

    auto load = [&](Tile& x, int t) {
        const int j = slot_of(t);
        if constexpr (WHOLE) {
            const int page = __builtin_amdgcn_readlane(pages, t & 63);
            const bool there = j < end && (unsigned)page < (unsigned)a.at.pages;
            const int js = seen_at(j);
            const int i = there ? js - a.at.page_of.by(js) * a.at.page_size : 0;
            const int64_t at = there ? page * a.at.stride_page + (int64_t)i * a.at.stride_slot : 0;
            const Buffer keys = buffer(k0 + at, there ? kNowhere - 1 : 0), values = buffer(v0 + at, there ? kNowhere - 1 : 0);
            const int left = there ? end - j : 0;   // slots of the tile before the end
            const unsigned key_off = col < left && is_seen(j + col) ? key_lane : kNowhere;
#pragma unroll
            for (int s = 0; s < kSteps; ++s)
                x.key[s] = __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(
                    keys, EXACT || 32 * s + 8 * quarter < a.dim ? key_off + 64 * s : kNowhere, 0, 0));
            x.held = 0;
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                const bool mine = 4 * quarter + r < left && is_seen(j + 4 * quarter + r);
                x.held |= (unsigned)mine << r;
                const unsigned off = mine ? value_lane + r * value_step : kNowhere;
#pragma unroll
                for (int s = 0; s < kSets; ++s) {
                    const unsigned o = EXACT || 16 * VW * s + VW * col < a.dim ? off + 32 * VW * s : kNowhere;
                    if constexpr (VW == 8) {
                        const u32x4 w = __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(values, o, 0, kOnce));
                        x.value[r][s][0] = w.x, x.value[r][s][1] = w.y, x.value[r][s][2] = w.z, x.value[r][s][3] = w.w;
                    } else {
                        const u32x2 w = __builtin_bit_cast(u32x2, __builtin_amdgcn_raw_buffer_load_b64(values, o, 0, kOnce));
                        x.value[r][s][0] = w.x, x.value[r][s][1] = w.y;
                    }
                }
            }
        } else {
            const int64_t key_at = j + col < end ? offset_at(j + col) : -1;
#pragma unroll
            for (int s = 0; s < kSteps; ++s) {
                x.key[s] = u32x4{0, 0, 0, 0};
                if (key_at >= 0 && 32 * s + 8 * quarter < a.dim)
                    x.key[s] = *reinterpret_cast<const u32x4*>(k0 + key_at + 32 * s + 8 * quarter);
            }
            x.held = 0;
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                const int64_t at = j + 4 * quarter + r < end ? offset_at(j + 4 * quarter + r) : -1;
                x.held |= (unsigned)(at >= 0) << r;
#pragma unroll
                for (int s = 0; s < kSets; ++s) {
#pragma unroll
                    for (int w = 0; w < kWords; ++w)
                        x.value[r][s][w] = 0;
                    if (at >= 0 && 16 * VW * s + VW * col < a.dim) {
                        const uint16_t* p = v0 + at + 16 * VW * s + VW * col;
                        if constexpr (VW == 8) {
                            const u32x4 w = *reinterpret_cast<const u32x4*>(p);
                            x.value[r][s][0] = w.x, x.value[r][s][1] = w.y, x.value[r][s][2] = w.z, x.value[r][s][3] = w.w;
                        } else {
                            const u32x2 w = *reinterpret_cast<const u32x2*>(p);
                            x.value[r][s][0] = w.x, x.value[r][s][1] = w.y;
                        }
                    }
                }
            }
        }
    };

    auto use = [&](Tile& x, int t) {
        const int j0 = slot_of(t);
        float* logits = nullptr;
        if (a.logits != nullptr)
            logits = a.logits + ((int64_t)b * a.q_heads + head0 + col) * a.logits_stride + j0 + 4 * quarter;
        f32x4 dot = {0, 0, 0, 0};
#pragma unroll
        for (int s = 0; s < kSteps; ++s)
            dot = mfma_dot<DT>(x.key[s], query[s], dot);
        f32x4 p;
#pragma unroll
        for (int r = 0; r < 4; ++r)
            p[r] = x.held >> r & 1 ? dot[r] * a.scale : -kInf;
        if (logits != nullptr && col < nheads && j0 < end)
            *reinterpret_cast<f32x4*>(logits) = p;
        float top = fmaxf(fmaxf(p[0], p[1]), fmaxf(p[2], p[3]));
        if (__any(top > m + kSlack)) {
            top = fmaxf(top, __shfl_xor(top, 16));
            top = fmaxf(top, __shfl_xor(top, 32));
            const float next = fmaxf(m, top);
            const float f = m == -kInf ? 0.0f : exp2_hw(m - next);
            m = next;
            sum *= f;
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                const float fr = __shfl(f, 4 * quarter + r);   // of head 4 (l / 16) + r, whose sums lane l holds
#pragma unroll
                for (int s = 0; s < kSets; ++s)
#pragma unroll
                    for (int e = 0; e < VW; ++e)
                        acc[s][e][r] *= fr;
            }
        }
        const float ref = m == -kInf ? 0.0f : m;
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            p[r] = exp2_hw(p[r] - ref);
            sum += p[r];
        }
#pragma unroll
        for (int r = 0; r < 4; ++r)
#pragma unroll
            for (int s = 0; s < kSets; ++s)
#pragma unroll
                for (int e = 0; e < VW; ++e)
                    acc[s][e] = __builtin_amdgcn_mfma_f32_16x16x4f32(p[r], element<DT>(x.value[r][s], e), acc[s][e], 0, 0, 0);
    };

    // in pairs: a tile past the last has nothing held and adds nothing
    Tile even, odd;
    load(even, 0);
    for (int t = 0; slot_of(t) < end; t += 2) {
        load(odd, t + 1);
        use(even, t);
        load(even, t + 2);
        use(odd, t + 1);
    }

    // the waves' parts meet in LDS
    sum += __shfl_xor(sum, 16);
    sum += __shfl_xor(sum, 32);
    if (quarter == 0) {
        red_m[wave][col] = m;
        red_s[wave][col] = sum;
    }
#pragma unroll
    for (int r = 0; r < 4; ++r)
        if (4 * quarter + r < nheads)
#pragma unroll
            for (int s = 0; s < kSets; ++s)
#pragma unroll
                for (int e = 0; e < VW; ++e)
                    red_o[wave][4 * quarter + r][16 * VW * s + VW * col + e] = acc[s][e][r];
    __syncthreads();
    // a wave's factor for a head, once, then four elements a thread
    if (threadIdx.x < 16) {
        const int h = threadIdx.x;
        float top = -kInf, total = 0.0f;
#pragma unroll
        for (int w = 0; w < WAVES; ++w)
            top = fmaxf(top, red_m[w][h]);
#pragma unroll
        for (int w = 0; w < WAVES; ++w) {
            const float f = part_factor(red_m[w][h], red_s[w][h], top);
            total += f * red_s[w][h];
            red_m[w][h] = f;
        }
        red_s[0][h] = total;
        if (a.part_ms != nullptr && h < nheads) {
            const int64_t row = query_row * a.q_heads + head0 + h;
            a.part_ms[(row * a.parts + part) * 2] = top;
            a.part_ms[(row * a.parts + part) * 2 + 1] = total;
        }
    }
    __syncthreads();
    for (int i = threadIdx.x; i < nheads * (DP / 4); i += WAVES * 64) {
        const int h = i / (DP / 4), d = i % (DP / 4) * 4;
        if (!EXACT && d >= a.dim)
            continue;
        f32x4 o = {0, 0, 0, 0};
#pragma unroll
        for (int w = 0; w < WAVES; ++w)
            o += red_m[w][h] * *reinterpret_cast<const f32x4*>(&red_o[w][h][d]);
        const int64_t row = query_row * a.q_heads + head0 + h;
        if (a.parts > 1 || (VIEW && a.partial)) {
            *reinterpret_cast<f32x4*>(a.part_out + (row * a.parts + part) * a.dim + d) = o;
        } else {
            const float total = red_s[0][h];
#pragma unroll
            for (int k = 0; k < 4; ++k)
                narrow_to<DT>(a.out, row * a.dim + d + k, total == 0.0f ? 0.0f : o[k] / total);
        }
    }
}

template <int DT, int DP, bool WHOLE, bool EXACT, int WAVES, bool VIEW = false>
__global__ void __launch_bounds__(WAVES * 64, DP == 256 ? 1 : 2)
attention_kernel(Attention a)
{
    __shared__ AttentionShared<DP, WHOLE, WAVES> shared;
    attention_block<DT, DP, WHOLE, EXACT, WAVES, VIEW>(a, blockIdx.x, shared);
}

// The maximum and the sum of powers of a query head over the parts that its
// length reaches, by one wave; the same in every lane.  Lane l takes parts l,
// l + 64, ..., and the lanes' sums meet in a fixed order.
struct Whole {
    float top, total;
};

__device__ __forceinline__ Whole whole(const float* ms, int parts, int lane)
{
    Whole w = {-kInf, 0.0f};
    for (int p = lane; p < parts; p += 64)
        w.top = fmaxf(w.top, ms[2 * p]);
#pragma unroll
    for (int d = 1; d < 64; d <<= 1)
        w.top = fmaxf(w.top, __shfl_xor(w.top, d));
    for (int p = lane; p < parts; p += 64)
        w.total += part_factor(ms[2 * p], ms[2 * p + 1], w.top) * ms[2 * p + 1];
#pragma unroll
    for (int d = 1; d < 64; d <<= 1)
        w.total += __shfl_xor(w.total, d);
    return w;
}

constexpr int kJoinHeads = 64;   // query heads whose sums a workgroup keeps at a time

// After the parts: the first `rows` workgroups (none where the length is not
// split) join a query head's parts, in order; the others add 2^(logit -
// maximum) / sum over the heads of a group to the weights of 1024 slots.
template <int DT>
__global__ void __launch_bounds__(256)
join_kernel(Attention a, int rows, int blocks)
{
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    if ((int)blockIdx.x < rows) {
        const int64_t row = blockIdx.x;
        const int b = (int)(row / a.q_heads);
        const int parts = (a.at.length(b) + a.chunk - 1) / a.chunk;
        const float* ms = a.part_ms + row * a.parts * 2;
        const Whole w = whole(ms, parts, lane);
        for (int d = threadIdx.x; d < a.dim; d += 256) {
            float o = 0.0f;
#pragma unroll 8
            for (int p = 0; p < parts; ++p)
                o += part_factor(ms[2 * p], ms[2 * p + 1], w.top) * a.part_out[(row * a.parts + p) * a.dim + d];
            narrow_to<DT>(a.out, row * a.dim + d, w.total == 0.0f ? 0.0f : o / w.total);
        }
        return;
    }
    __shared__ Whole heads[kJoinHeads];
    int item = blockIdx.x - rows;
    const int block = item % blocks;
    item /= blocks;
    const int kv = item % a.heads;
    const int b = item / a.heads;
    const int len = a.at.length(b);
    if (block * 1024 >= len)
        return;
    const int parts = (len + a.chunk - 1) / a.chunk;
    const int j = block * 1024 + (int)threadIdx.x * 4;
    f32x4 total = {0, 0, 0, 0};
    for (int g0 = 0; g0 < a.group; g0 += kJoinHeads) {
        const int n = a.group - g0 < kJoinHeads ? a.group - g0 : kJoinHeads;
        const int64_t row = (int64_t)b * a.q_heads + kv * a.group + g0;
        __syncthreads();
        for (int g = wave; g < n; g += 4) {
            const Whole w = whole(a.part_ms + (row + g) * a.parts * 2, parts, lane);
            if (lane == 0)
                heads[g] = Whole{w.top == -kInf ? 0.0f : w.top, w.total == 0.0f ? 0.0f : 1.0f / w.total};
        }
        __syncthreads();
        if (j < len) {
#pragma unroll 4
            for (int g = 0; g < n; ++g) {
                const f32x4 x = *reinterpret_cast<const f32x4*>(a.logits + (row + g) * a.logits_stride + j);
#pragma unroll
                for (int r = 0; r < 4; ++r)
                    total[r] += exp2_hw(x[r] - heads[g].top) * heads[g].total;
            }
        }
    }
    float* to = a.weights + ((int64_t)b * a.heads + kv) * a.slots + j;
    if (a.weights_wide && j + 4 <= len) {
        *reinterpret_cast<f32x4*>(to) += total;
    } else {
#pragma unroll
        for (int r = 0; r < 4; ++r)
            if (j + r < len)
                to[r] += total[r];
    }
}

}  // namespace gattn
