// attention_kernels.hpp -- gfx950 (CDNA4) device code for decode attention
// over a paged key-value cache, and for the cache's append and eviction.
//
//   o_h = sum_j p_hj v_j,  p_h = softmax_j(scale * q_h . k_j)
//
// All three are bound by memory: attention reads every key and value once for
// the few operations of a group of query heads, append and eviction only move
// rows.  Reached on one MI355X, where a pure read makes 7.1 TB/s and a copy
// 4.95 TB/s of reads and writes: attention 5.2 TB/s over 64 sequences of 100
// to 8192 slots (8 heads of 128, 222 us; 6.0 TB/s where all have 8192), append
// 5.1 to 5.2 TB/s (4 x 8191 tokens, 52 us).  The same 64 sequences with other
// heads: 8 of 64 127 to 132 us, 80 and 96 195 to 201, 256 460 us (5.1 TB/s).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace gattn {

typedef unsigned int u32x2 __attribute__((ext_vector_type(2)));
typedef unsigned int u32x4 __attribute__((ext_vector_type(4)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));

enum Type : int { kF16 = 1, kBF16 = 2 };

constexpr float kInf = __builtin_inff();

__device__ __forceinline__ float exp2_hw(float t) { return __builtin_amdgcn_exp2f(t); }

// n / d for n < 2^31 by a multiplication and a shift (Granlund and
// Montgomery's round-up method): the high half of n * mul, plus n, shifted.
struct Divider {
    unsigned mul, shift;
    __device__ __forceinline__ int by(int n) const
    {
        return (int)((__umulhi((unsigned)n, mul) + (unsigned)n) >> shift);
    }
};

// Where the slots of a sequence lie.
struct Pages {
    const int32_t* table;
    int64_t table_stride;
    const int32_t* lens;
    int limit;        // min(max_len, width * page_size): no slot is at or above it
    int pages;
    int page_size;
    Divider page_of;
    int64_t stride_page, stride_slot, stride_head;

    __device__ __forceinline__ int length(int b) const
    {
        const int n = lens[b];
        return n < 0 ? 0 : (n < limit ? n : limit);
    }
    // element offset of head 0 of slot `j` < limit of sequence `b`; -1 in a hole
    __device__ __forceinline__ int64_t offset(int b, int j) const
    {
        const int i = page_of.by(j);
        const int page = table[b * table_stride + i];
        return (unsigned)page < (unsigned)pages ? page * stride_page + (int64_t)(j - i * page_size) * stride_slot : -1;
    }
};

template <int DT>
__device__ __forceinline__ f32x4 mfma_dot(u32x4 a, u32x4 b, f32x4 c)
{
    if constexpr (DT == kF16)
        return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8, a), __builtin_bit_cast(f16x8, b), c, 0, 0, 0);
    else
        return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b), c, 0, 0, 0);
}

// element e of a run of 16-bit values
template <int DT, int W>
__device__ __forceinline__ float element(const unsigned (&w)[W], int e)
{
    const unsigned pair = w[e >> 1];
    if constexpr (DT == kBF16)
        return __builtin_bit_cast(float, e & 1 ? pair & 0xFFFF0000u : pair << 16);
    else
        return (float)__builtin_bit_cast(_Float16, (unsigned short)(e & 1 ? pair >> 16 : pair));
}

template <int DT>
__device__ __forceinline__ void narrow_to(void* p, int64_t at, float v)
{
    if constexpr (DT == kF16)
        static_cast<_Float16*>(p)[at] = (_Float16)v;
    else
        static_cast<__bf16*>(p)[at] = (__bf16)v;
}

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
};

// What brings a part's sums to the common maximum `top`.  An empty part has
// maximum -inf and sum 0; one whose sum is NaN under a maximum of -inf stays NaN.
__device__ __forceinline__ float part_factor(float m, float s, float top)
{
    return m == -kInf ? (s == 0.0f ? 0.0f : 1.0f) : exp2_hw(m - top);
}

constexpr int kWaves = 4;         // of a workgroup, where the length is split or the card is full
constexpr int kLoneWaves = 8;     // where one workgroup takes a short sequence's whole length
constexpr int kMaxChunk = 1024;  // slots of a part: 16 tiles a wave
constexpr float kSlack = 8.0f;   // powers of two that a logit may pass the reference maximum by

// Loads through a buffer descriptor: an address outside it gives zeros and
// reads nothing, so a lane without an element, a slot past the end and a hole
// need no branch.
typedef __amdgpu_buffer_rsrc_t Buffer;
constexpr int kOnce = 2;                     // cache policy: read once, not to be kept
constexpr unsigned kNowhere = 0x80000000u;   // past every descriptor's end

__device__ __forceinline__ Buffer buffer(const uint16_t* p, unsigned bytes)
{
    return __builtin_amdgcn_make_buffer_rsrc(const_cast<uint16_t*>(p), 0, (int)bytes, 0x00027000);
}

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
template <int DT, int DP, bool WHOLE, bool EXACT, int WAVES>
__global__ void __launch_bounds__(WAVES * 64, DP == 256 ? 1 : 2)
attention_kernel(Attention a)
{
    constexpr int kSteps = DP / 32;              // of 32 elements of the dot products
    constexpr int VW = DP == 64 ? 4 : 8;         // elements of a value row per lane and set
    constexpr int kSets = DP / (16 * VW);
    constexpr int kWords = VW / 2;
    __shared__ float red_m[WAVES][16];
    __shared__ float red_s[WAVES][16];
    __shared__ __attribute__((aligned(16))) float red_o[WAVES][16][DP];

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
    const int turn = (int)blockIdx.x / a.heads;
    const int kv = ((int)blockIdx.x + turn) % a.heads;
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
    const int len = __builtin_amdgcn_readfirstlane(a.at.length(b));
    const int64_t first = (int64_t)part * a.chunk;
    if (part > 0 && first >= len)
        return;                                                          // the join does not look at it
    const int begin = (int)first;
    const int end = first + a.chunk < len ? (int)(first + a.chunk) : len;
    const int head0 = kv * a.group + tile * 16;                          // this workgroup's query heads
    const int nheads = a.group - tile * 16 < 16 ? a.group - tile * 16 : 16;

    u32x4 query[kSteps];
#pragma unroll
    for (int s = 0; s < kSteps; ++s) {
        const int d = 32 * s + 8 * quarter;
        query[s] = u32x4{0, 0, 0, 0};
        if (col < nheads && (EXACT || d < a.dim))
            query[s] = *reinterpret_cast<const u32x4*>(a.q + b * a.q_stride + (int64_t)(head0 + col) * a.dim + d);
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
    __shared__ int32_t slot_page[WHOLE ? 1 : kMaxChunk];
    if constexpr (WHOLE) {
        const int64_t j = (int64_t)begin + (wave + lane * WAVES) * 16;
        if (j < a.at.limit)
            pages = a.at.table[b * a.at.table_stride + a.at.page_of.by((int)j)];
    } else {
        for (int i = threadIdx.x; i < a.chunk; i += WAVES * 64)
            slot_page[i] = begin + i < end ? a.at.table[b * a.at.table_stride + a.at.page_of.by(begin + i)] : -1;
        __syncthreads();
    }
    auto offset_at = [&](int j) -> int64_t {   // of slot j < end, where !WHOLE
        const int page = slot_page[j - begin];
        if ((unsigned)page >= (unsigned)a.at.pages)
            return -1;
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
            const int i = there ? j - a.at.page_of.by(j) * a.at.page_size : 0;
            const int64_t at = there ? page * a.at.stride_page + (int64_t)i * a.at.stride_slot : 0;
            const Buffer keys = buffer(k0 + at, there ? kNowhere - 1 : 0), values = buffer(v0 + at, there ? kNowhere - 1 : 0);
            const int left = there ? end - j : 0;   // slots of the tile before the end
            const unsigned key_off = col < left ? key_lane : kNowhere;
#pragma unroll
            for (int s = 0; s < kSteps; ++s)
                x.key[s] = __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(
                    keys, EXACT || 32 * s + 8 * quarter < a.dim ? key_off + 64 * s : kNowhere, 0, 0));
            x.held = 0;
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                const bool mine = 4 * quarter + r < left;
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
            const int64_t row = (int64_t)b * a.q_heads + head0 + h;
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
        const int64_t row = (int64_t)b * a.q_heads + head0 + h;
        if (a.parts > 1) {
            *reinterpret_cast<f32x4*>(a.part_out + (row * a.parts + part) * a.dim + d) = o;
        } else {
            const float total = red_s[0][h];
#pragma unroll
            for (int k = 0; k < 4; ++k)
                narrow_to<DT>(a.out, row * a.dim + d + k, total == 0.0f ? 0.0f : o[k] / total);
        }
    }
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

// ---------------------------------------------------------------- append
struct Append {
    Pages at;
    uint16_t* k;
    uint16_t* v;
    const int32_t* starts;
    const uint16_t* new_k;
    const uint16_t* new_v;
    int64_t k_stride, v_stride;
    int rows, batch, heads, dim;
    float* weights;
    int32_t* positions;
    const int32_t* seen;
    int64_t slots;
};

// A wave per new token: its sequence is found in `starts`, its slot from the
// length, and its heads' rows are copied 16 bytes per lane.  4 x 8191 tokens of
// 8 heads of 128: 52 us, 5.2 TB/s read and written; 64 tokens: 4 us, the chain
// of loads from `starts` to the page number.
__global__ void __launch_bounds__(256)
append_kernel(Append a)
{
    const int lane = threadIdx.x & 63;
    const int64_t step = (int64_t)gridDim.x * 4;
    for (int64_t row = (int64_t)blockIdx.x * 4 + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6); row < a.rows;
         row += step) {
        // the last sequence that starts at or before this row
        int low = 0, high = a.batch;
        while (low < high) {
            const int mid = (low + high) >> 1;
            if (a.starts[mid] <= row)
                low = mid + 1;
            else
                high = mid;
        }
        const int b = low - 1;
        if (b < 0 || row >= a.starts[b + 1])
            continue;
        const int64_t back = a.starts[b + 1] - row;   // 1 for the newest token
        const int64_t slot = a.at.lens[b] - back;
        if (slot < 0 || slot >= a.at.limit)
            continue;
        const int64_t to = a.at.offset(b, (int)slot);
        if (to < 0)
            continue;
        if (a.weights != nullptr) {
            for (int h = lane; h < a.heads; h += 64) {
                if (slot < a.slots) {
                    const int64_t i = ((int64_t)b * a.heads + h) * a.slots + slot;
                    a.weights[i] = 0.0f;
                    a.positions[i] = (int32_t)(a.seen[b] - back);
                }
            }
        }
        const int per_head = a.dim >> 3, chunks = a.heads * per_head;
        for (int c = lane; c < chunks; c += 64) {
            const int h = c / per_head, d = (c - h * per_head) * 8;
            const int64_t at = to + h * a.at.stride_head + d;
            *reinterpret_cast<u32x4*>(a.k + at) =
                *reinterpret_cast<const u32x4*>(a.new_k + row * a.k_stride + (int64_t)c * 8);
            *reinterpret_cast<u32x4*>(a.v + at) =
                *reinterpret_cast<const u32x4*>(a.new_v + row * a.v_stride + (int64_t)c * 8);
        }
    }
}

// ---------------------------------------------------------------- eviction
struct Evict {
    Pages at;
    uint16_t* k;
    uint16_t* v;
    const int32_t* seen;
    const float* weights;
    const int32_t* positions;
    int64_t slots;
    int heads, dim, budget, recent;
    float* weights_out;
    int32_t* positions_out;
    int32_t* lens_out;
    int moves_max;     // of one head: min(budget, limit - budget), or 0
    int words;         // of 64 slots below the budget
    int held;          // keys that the launch's LDS holds
    int32_t* count;    // [batch][heads]: moves, or -1 where nothing is evicted
    uint64_t* bits;    // [batch][heads][words]: which of those stay
    int32_t* moves;    // [batch][heads][2][moves_max]: to, from
};

// The order of weights as whole numbers: NaN above every number, -0 and 0
// alike.
__device__ __forceinline__ unsigned weight_key(float w)
{
    if (w != w)
        return 0xFF800001u;
    const unsigned u = __builtin_bit_cast(unsigned, w + 0.0f);
    return u & 0x80000000u ? ~u : u | 0x80000000u;
}

constexpr int kEvictThreads = 1024, kEvictWaves = kEvictThreads / 64;
constexpr int kBins = 2048, kCopies = 2;
constexpr int kHeldKeys = 32768;           // in 128 KB of LDS
constexpr unsigned kNewest = 0xFFFFFFFFu;   // the key of the newest tokens, above every weight's
constexpr int kFusedMoves = 64;   // of a head: four for each wave of the selecting workgroup
constexpr int kFewGone = 4;       // tokens that are found one by one

__device__ __forceinline__ int lanes_before(uint64_t mask)
{
    return (int)__builtin_amdgcn_mbcnt_hi((unsigned)(mask >> 32), __builtin_amdgcn_mbcnt_lo((unsigned)mask, 0));
}

// Whether this lane's bit is set in a mask that is the same for all lanes.
__device__ __forceinline__ bool in_mask(uint64_t mask)
{
#ifdef __HIP_DEVICE_COMPILE__
    return __builtin_amdgcn_inverse_ballot_w64(mask);
#else
    return mask != 0;   // not called on the host
#endif
}

// A token's place among all: the least goes first, of equal keys the last slot.
__device__ __forceinline__ uint64_t ranked(unsigned key, int slot)
{
    return (uint64_t)key << 32 | (unsigned)(0x7FFFFFFF - slot);
}

__device__ __forceinline__ int wave_sum(int v)
{
#pragma unroll
    for (int d = 1; d < 64; d <<= 1)
        v += __shfl_xor(v, d);
    return v;
}

// Sum of the waves' counts before this wave, and of all.  `counts` is free
// again after the next barrier.
struct Running {
    int before, all;
};

__device__ __forceinline__ Running over_waves(int mine, int wave, int (&counts)[kEvictWaves])
{
    if ((threadIdx.x & 63) == 0)
        counts[wave] = mine;
    __syncthreads();
    Running r = {0, 0};
#pragma unroll
    for (int w = 0; w < kEvictWaves; ++w) {
        r.before += w < wave ? counts[w] : 0;
        r.all += counts[w];
    }
    return r;
}

// Copies one slot's key and value rows of a head to another slot, by one wave.
__device__ __forceinline__ void move_row(const Evict& a, int b, int h, int from, int to, int lane)
{
    const int per_row = a.dim >> 3;
    const int64_t src = a.at.offset(b, from), dst = a.at.offset(b, to);
    if (src < 0 || dst < 0 || lane >= 2 * per_row)
        return;
    uint16_t* pool = lane < per_row ? a.k : a.v;
    const int64_t d = h * a.at.stride_head + (lane < per_row ? lane : lane - per_row) * 8;
    *reinterpret_cast<u32x4*>(pool + dst + d) = *reinterpret_cast<const u32x4*>(pool + src + d);
}

// One workgroup per head of a sequence.  The weight of the last token kept is
// found digit by digit, in up to three passes over histograms of 11, 11 and 10
// bits of the keys: the first digit is a weight's exponent and two bits more,
// so that weights of like size do not all count in one bin, and lanes count in
// kCopies histograms side by side.  A pass ends the search where a bin is kept
// whole, most often the second.  Where only a few tokens are to go (a decode
// step's eviction), they are found one by one as the least key, of equals the
// last.  Then the slots are walked in order: the kept ones from the budget on
// are matched with the evicted ones below it.
//
// Keys are made once and stay in LDS, up to kHeldKeys; those of longer
// sequences are made anew in each pass, from cache.  (4 x 8 heads of 20000 to
// 32768 slots: 36 to 42 us; with keys in registers, 32 a lane, 45 to 49.  32 x 8
// heads of 2049 slots, one to go: 11 us.  4 x 8 heads of 70000 to 131072 slots, past
// kHeldKeys, and their moves: 376 us.)  A wave takes consecutive groups of 64 slots, one a
// lane, so the order of slots is that of (wave, group, lane), and counts before
// a slot are population counts of lane masks and one sum over the waves.
//
// FUSED: at most kFusedMoves moves, listed in LDS and made here, with the
// weights' and positions' outputs.  Otherwise a second launch makes both, spread
// over the card, from the lists and the kept slots' bits left in the workspace.
template <bool FUSED>
__global__ void __launch_bounds__(kEvictThreads)
evict_select_kernel(Evict a)
{
    extern __shared__ unsigned held_keys[];   // min(limit, kHeldKeys)
    __shared__ unsigned histogram[kCopies][kBins];
    __shared__ unsigned chosen[3];
    __shared__ int counts[3][kEvictWaves];   // of sums that no barrier parts
    __shared__ uint64_t least[kEvictWaves];
    __shared__ int32_t hole_at[FUSED ? kFusedMoves : 1];
    __shared__ int32_t mover_at[FUSED ? kFusedMoves : 1];
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int h = blockIdx.x % a.heads, b = blockIdx.x / a.heads;
    const int64_t bh = (int64_t)b * a.heads + h;
    const int len = __builtin_amdgcn_readfirstlane(a.at.length(b));
    const int kept = len < a.budget ? len : a.budget;
    const float* w = a.weights + bh * a.slots;
    const int32_t* pos = a.positions + bh * a.slots;
    float* w_out = a.weights_out + bh * a.slots;
    int32_t* pos_out = a.positions_out + bh * a.slots;
    if (h == 0 && tid == 0)
        a.lens_out[b] = kept;
    if (len <= a.budget || a.budget == 0) {   // nothing to choose
        if constexpr (FUSED) {
            for (int64_t j = tid; j < a.slots; j += kEvictThreads) {
                w_out[j] = j < kept ? w[j] : 0.0f;
                pos_out[j] = j < kept ? pos[j] : -1;
            }
        } else if (tid == 0) {
            a.count[bh] = -1;
        }
        return;
    }
    const int64_t oldest = (int64_t)a.seen[b] - a.recent;
    const bool held = len <= a.held;
    // this wave's slots: of a length below 2^31, up to 1/16 and a group
    const int per_wave = (int)((((int64_t)len + 63) / 64 + kEvictWaves - 1) / kEvictWaves) * 64;
    const int begin = (int)((int64_t)wave * per_wave < len ? (int64_t)wave * per_wave : len);
    const int end = len - begin < per_wave ? len : begin + per_wave;
    auto made = [&](float weight, int position) { return (int64_t)position >= oldest ? kNewest : weight_key(weight); };
    auto key = [&](int j) { return held ? held_keys[j] : made(w[j], pos[j]); };   // only this wave's: no barrier
    if (held) {
        constexpr int kBatch = 16;
        for (int g = begin; g < end; g += 64 * kBatch) {
            // slots past the end read the last one instead: no branch, so that
            // all loads are on their way before the first is waited for
            float weight[kBatch];
            int position[kBatch];
#pragma unroll
            for (int u = 0; u < kBatch; ++u) {
                const int j = end - g > 64 * u + lane ? g + 64 * u + lane : end - 1;
                weight[u] = w[j];
                position[u] = pos[j];
            }
#pragma unroll
            for (int u = 0; u < kBatch; ++u)
                if (end - g > 64 * u + lane)
                    held_keys[g + 64 * u + lane] = made(weight[u], position[u]);
        }
    }
    if constexpr (FUSED)
        for (int64_t j = kept + tid; j < a.slots; j += kEvictThreads) {
            w_out[j] = 0.0f;
            pos_out[j] = -1;
        }

    // f(slot, its key) for this lane's slots from `from` to before `to`, eight
    // keys read at a time
    auto each = [&](int from, int to, auto f) {
        for (int g = from; g < to; g += 64 * 8) {
            unsigned k[8];
#pragma unroll
            for (int u = 0; u < 8; ++u)
                k[u] = to - g > 64 * u + lane ? key(g + 64 * u + lane) : 0u;
#pragma unroll
            for (int u = 0; u < 8; ++u)
                if (to - g > 64 * u + lane)
                    f(g + 64 * u + lane, k[u]);
        }
    };

    // Tokens with keys above `edge` are kept and the first `ties` of those
    // equal to it, or all but the `few` in `gone`.
    unsigned edge = kNewest;
    int ties = a.budget;
    uint64_t gone[kFewGone];
    const int few = len - a.budget <= kFewGone ? len - a.budget : 0;
    auto is_gone = [&](uint64_t v) {
        bool is = false;
#pragma unroll
        for (int q = 0; q < kFewGone; ++q)
            is = is || v == gone[q];
        return is;
    };
    if (few > 0) {
#pragma unroll
        for (int q = 0; q < kFewGone; ++q)
            gone[q] = ~0ull;
        for (int n = 0; n < few; ++n) {
            uint64_t mine = ~0ull;
            each(begin, end, [&](int j, unsigned k) {
                const uint64_t v = ranked(k, j);
                mine = !is_gone(v) && v < mine ? v : mine;
            });
#pragma unroll
            for (int d = 1; d < 64; d <<= 1) {
                const uint64_t other = (uint64_t)(unsigned)__shfl_xor((int)(mine >> 32), d) << 32 |
                                       (unsigned)__shfl_xor((int)(unsigned)mine, d);
                mine = other < mine ? other : mine;
            }
            __syncthreads();   // `least` is read
            if (lane == 0)
                least[wave] = mine;
            __syncthreads();
#pragma unroll
            for (int v = 0; v < kEvictWaves; ++v)
                mine = least[v] < mine ? least[v] : mine;
#pragma unroll
            for (int q = 0; q < kFewGone; ++q)
                gone[q] = q == n ? mine : gone[q];
        }
    } else {
        unsigned wanted = (unsigned)a.budget, prefix = 0;
        bool found = false;
        for (int pass = 0; pass < 3 && !found; ++pass) {
            const int shift = pass == 0 ? 21 : (pass == 1 ? 10 : 0), bits = pass == 2 ? 10 : 11;
            for (int i = tid; i < kCopies * kBins; i += kEvictThreads)
                (&histogram[0][0])[i] = 0;
            __syncthreads();
            int newest = 0;   // counted apart: they would all wait for one bin
            each(begin, end, [&](int, unsigned k) {
                if (k == kNewest)
                    ++newest;
                else if (pass == 0 || k >> (shift + bits) == prefix >> (shift + bits))
                    atomicAdd(&histogram[lane % kCopies][k >> shift & ((1u << bits) - 1)], 1u);
            });
            if (pass == 0 && newest != 0)
                atomicAdd(&histogram[0][kBins - 1], (unsigned)newest);   // the bin of no other key
            __syncthreads();
            // counts from the highest bin down: thread i has bins 2 i and 2 i + 1 from the top
            unsigned hi = 0, lo = 0;
#pragma unroll
            for (int c = 0; c < kCopies; ++c) {
                hi += histogram[c][kBins - 1 - 2 * tid];
                lo += histogram[c][kBins - 2 - 2 * tid];
            }
            int sum = (int)(hi + lo);
#pragma unroll
            for (int d = 1; d < 64; d <<= 1) {
                const int up = __shfl_up(sum, d);
                sum += lane >= d ? up : 0;
            }
            const Running r = over_waves(__builtin_amdgcn_readlane(sum, 63), wave, counts[1]);
            const unsigned above = (unsigned)(r.before + sum) - hi - lo;
            const bool in_hi = above < wanted && wanted <= above + hi;
            const bool in_lo = above + hi < wanted && wanted <= above + hi + lo;
            if (in_hi || in_lo) {
                chosen[0] = prefix | (unsigned)(kBins - 1 - 2 * tid - (in_lo ? 1 : 0)) << shift;
                chosen[1] = wanted - above - (in_lo ? hi : 0);   // of the bin
                chosen[2] = in_lo ? lo : hi;
            }
            __syncthreads();
            prefix = chosen[0];
            wanted = chosen[1];
            found = true;
            if (pass == 0 && prefix == (unsigned)(kBins - 1) << 21) {
                ;   // the newest alone fill the budget: edge and ties as they are
            } else if (wanted == chosen[2]) {   // the whole bin; it is not the lowest, for not all are kept
                edge = prefix - 1;
                ties = 0;
            } else if (pass == 2) {
                edge = prefix;
                ties = (int)wanted;
            } else {
                found = false;
            }
        }
    }

    const bool tied = few == 0 && ties > 0;
    int before = 0;   // of the slots before: equal to the edge
    if (tied) {
        int n = 0;
        each(begin, end, [&](int, unsigned k) { n += k == edge; });
        before = over_waves(wave_sum(n), wave, counts[2]).before;
    }
    const int first_tie = before;
    auto stays = [&](int j, unsigned k) {   // in the order of the groups, where `tied`
        if (few > 0)
            return !is_gone(ranked(k, j));
        bool is = k > edge;
        if (tied) {
            const uint64_t mask = __ballot(j < end && k == edge);
            is = is || (k == edge && before + lanes_before(mask) < ties);
            before += __popcll(mask);
        }
        return is;
    };
    const int low_end = end < a.budget ? end : a.budget;   // of this wave's slots below the budget, if any
    int n_holes = 0, n_movers = 0;
    if (!tied) {
        each(begin, low_end, [&](int j, unsigned k) { n_holes += !stays(j, k); });
        each(begin > a.budget ? begin : a.budget, end, [&](int j, unsigned k) { n_movers += stays(j, k); });
    } else {
        for (int g = begin; g < end; g += 64) {
            const int j = g + lane;
            const bool is = stays(j, j < end ? key(j) : 0u);
            n_holes += j < low_end && !is;
            n_movers += j >= a.budget && j < end && is;
        }
    }
    const Running holes = over_waves(wave_sum(n_holes), wave, counts[0]);
    const Running movers = over_waves(wave_sum(n_movers), wave, counts[1]);
    int32_t* to = FUSED ? hole_at : a.moves + bh * 2 * a.moves_max;
    int32_t* from = FUSED ? mover_at : to + a.moves_max;
    uint64_t* bits = a.bits + bh * a.words;
    int hole = holes.before, mover = movers.before;
    before = first_tie;
    for (int g = begin; g < end; g += 64) {
        const int j = g + lane;
        const bool is = stays(j, j < end ? key(j) : 0u);
        if (g < a.budget) {
            const uint64_t mask = __ballot(j < low_end && !is);
            if (in_mask(mask)) {
                to[hole + lanes_before(mask)] = j;
            } else if (FUSED && j < low_end) {
                w_out[j] = w[j];
                pos_out[j] = pos[j];
            }
            if (!FUSED && lane == 0)
                bits[g >> 6] = ~mask;
            hole += __popcll(mask);
        }
        if (g + 64 > a.budget) {
            const uint64_t mask = __ballot(j >= a.budget && j < end && is);
            if (in_mask(mask))
                from[mover + lanes_before(mask)] = j;
            mover += __popcll(mask);
        }
    }
    if constexpr (FUSED) {
        __syncthreads();
        if (tid < movers.all) {
            w_out[to[tid]] = w[from[tid]];
            pos_out[to[tid]] = pos[from[tid]];
        }
        for (int i = wave; i < movers.all; i += kEvictWaves)
            move_row(a, b, h, from[i], to[i], lane);
    } else if (tid == 0) {
        a.count[bh] = movers.all;
    }
}

// What the selection leaves to do (4 x 8 heads, 110 MB of rows in pieces of
// 256 bytes anywhere in the pool: 39 us): a thread per slot for the weights and
// positions, then a thread per 16 bytes of the rows that move.
__global__ void __launch_bounds__(256)
evict_move_kernel(Evict a, int blocks)
{
    const int block = blockIdx.x % blocks;
    const int bh = blockIdx.x / blocks;
    const int b = bh / a.heads, h = bh % a.heads;
    const int64_t first = (int64_t)block * 256 + threadIdx.x, step = (int64_t)blocks * 256;
    const int len = a.at.length(b);
    const int kept = len < a.budget ? len : a.budget;
    const int moved = a.count[bh];
    const float* w = a.weights + bh * a.slots;
    const int32_t* pos = a.positions + bh * a.slots;
    float* w_out = a.weights_out + bh * a.slots;
    int32_t* pos_out = a.positions_out + bh * a.slots;
    const uint64_t* bits = a.bits + bh * a.words;
    for (int64_t j = first; j < a.slots; j += step) {
        if (j >= kept) {
            w_out[j] = 0.0f;
            pos_out[j] = -1;
        } else if (moved < 0 || (bits[j >> 6] >> (j & 63) & 1)) {
            w_out[j] = w[j];
            pos_out[j] = pos[j];
        }
    }
    const int per_row = a.dim >> 3, per_move = 2 * per_row;
    const int32_t* to = a.moves + (int64_t)bh * 2 * a.moves_max;
    const int32_t* from = to + a.moves_max;
    for (int64_t i = first; i < (int64_t)moved * per_move; i += step) {
        const int move = (int)(i / per_move), piece = (int)(i - (int64_t)move * per_move);
        const int s = from[move], d = to[move];
        if (piece == 0) {
            w_out[d] = w[s];
            pos_out[d] = pos[s];
        }
        const int64_t src = a.at.offset(b, s), dst = a.at.offset(b, d);
        if (src < 0 || dst < 0)
            continue;
        uint16_t* pool = piece < per_row ? a.k : a.v;
        const int64_t e = h * a.at.stride_head + (piece < per_row ? piece : piece - per_row) * 8;
        *reinterpret_cast<u32x4*>(pool + dst + e) = *reinterpret_cast<const u32x4*>(pool + src + e);
    }
}

}  // namespace gattn
