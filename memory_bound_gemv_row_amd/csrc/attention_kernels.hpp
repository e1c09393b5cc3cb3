// attention_kernels.hpp -- gfx950 (CDNA4) device code for decode attention
// over a paged key-value cache, and for the cache's append and eviction.
//
//   o_h = sum_j p_hj v_j,  p_h = softmax_j(scale * q_h . k_j)
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

constexpr int kWaves = 4;
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
// A wave loads its next tile while it multiplies the current one.  Where
// pages are whole numbers of tiles (WHOLE), a tile has one page and its
// address is the same for all lanes; otherwise each row has an address of its
// own.  EXACT: the head's size is DP, so no lane is without an element.
template <int DT, int DP, bool WHOLE, bool EXACT>
__global__ void __launch_bounds__(kWaves * 64, DP == 256 ? 1 : 2)
attention_kernel(Attention a)
{
    constexpr int kSteps = DP / 32;              // of 32 elements of the dot products
    constexpr int VW = DP == 64 ? 4 : 8;         // elements of a value row per lane and set
    constexpr int kSets = DP / (16 * VW);
    constexpr int kWords = VW / 2;
    __shared__ float red_m[kWaves][16];
    __shared__ float red_s[kWaves][16];
    __shared__ float red_o[kWaves][16][DP];

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
    auto slot_of = [&](int t) { return begin + (wave + t * kWaves) * 16; };   // tile t of this wave
    const uint16_t* k0 = a.k + kv * a.at.stride_head;
    const uint16_t* v0 = a.v + kv * a.at.stride_head;

    // the pages of this part, looked up once so that no tile's loads wait for
    // a page number: WHOLE, tile t of this wave in lane t; otherwise every slot's in LDS
    int pages = -1;
    __shared__ int32_t slot_page[WHOLE ? 1 : kMaxChunk];
    if constexpr (WHOLE) {
        const int64_t j = (int64_t)begin + (wave + lane * kWaves) * 16;
        if (j < a.at.limit)
            pages = a.at.table[b * a.at.table_stride + a.at.page_of.by((int)j)];
    } else {
        for (int i = threadIdx.x; i < a.chunk; i += kWaves * 64)
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
    for (int i = threadIdx.x; i < nheads * DP; i += kWaves * 64) {
        const int h = i / DP, d = i % DP;
        if (!EXACT && d >= a.dim)
            continue;
        float top = -kInf;
#pragma unroll
        for (int w = 0; w < kWaves; ++w)
            top = fmaxf(top, red_m[w][h]);
        float o = 0.0f, total = 0.0f;
#pragma unroll
        for (int w = 0; w < kWaves; ++w) {
            const float f = part_factor(red_m[w][h], red_s[w][h], top);
            o += f * red_o[w][h][d];
            total += f * red_s[w][h];
        }
        const int64_t row = (int64_t)b * a.q_heads + head0 + h;
        if (a.part_ms != nullptr && d == 0) {
            a.part_ms[(row * a.parts + part) * 2] = top;
            a.part_ms[(row * a.parts + part) * 2 + 1] = total;
        }
        if (a.parts > 1)
            a.part_out[(row * a.parts + part) * a.dim + d] = o;
        else
            narrow_to<DT>(a.out, row * a.dim + d, total == 0.0f ? 0.0f : o / total);
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
// length, and its heads' rows are copied 16 bytes per lane.
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
        if (a.weights != nullptr) {
            for (int h = lane; h < a.heads; h += 64) {
                if (slot < a.slots) {
                    const int64_t i = ((int64_t)b * a.heads + h) * a.slots + slot;
                    a.weights[i] = 0.0f;
                    a.positions[i] = (int32_t)(a.seen[b] - back);
                }
            }
        }
        if (to < 0)
            continue;
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
    int32_t* count;    // [batch][heads]: moves
    int32_t* moves;    // [batch][heads][2][moves_max]: to, from
};

// The order in which tokens are kept, as whole numbers: recent ones above
// all, then NaN, then numbers by value (-0 and 0 alike).
__device__ __forceinline__ unsigned rank_key(float w, bool recent)
{
    if (recent)
        return 0xFFFFFFFFu;
    if (w != w)
        return 0xFF800001u;
    const unsigned u = __builtin_bit_cast(unsigned, w + 0.0f);
    return u & 0x80000000u ? ~u : u | 0x80000000u;
}

constexpr int kEvictThreads = 1024;

// Exclusive sums of two counts over the workgroup, and the totals.
struct Pair {
    int a, b;
};

__device__ __forceinline__ Pair block_scan(Pair v, Pair* totals, Pair (&waves)[kEvictThreads / 64])
{
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    Pair s = v;
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
        const int ua = __shfl_up(s.a, d), ub = __shfl_up(s.b, d);
        if (lane >= d) {
            s.a += ua;
            s.b += ub;
        }
    }
    __syncthreads();   // `waves` may still be read from the scan before
    if (lane == 63)
        waves[wave] = s;
    __syncthreads();
    Pair before = {0, 0}, all = {0, 0};
#pragma unroll
    for (int w = 0; w < kEvictThreads / 64; ++w) {
        if (w < wave) {
            before.a += waves[w].a;
            before.b += waves[w].b;
        }
        all.a += waves[w].a;
        all.b += waves[w].b;
    }
    *totals = all;
    return Pair{before.a + s.a - v.a, before.b + s.b - v.b};
}

// One workgroup per head of a sequence: finds the budget-th largest key in four
// passes over histograms of its bytes, then walks the slots in order, matching
// the kept ones past the budget with the evicted ones before it.
__global__ void __launch_bounds__(kEvictThreads)
evict_select_kernel(Evict a)
{
    __shared__ unsigned histogram[256];
    __shared__ unsigned chosen[2];
    __shared__ Pair waves[kEvictThreads / 64];
    const int tid = threadIdx.x;
    const int h = blockIdx.x % a.heads, b = blockIdx.x / a.heads;
    const int64_t bh = (int64_t)b * a.heads + h;
    const int len = a.at.length(b);
    const int kept = len < a.budget ? len : a.budget;
    const float* w = a.weights + bh * a.slots;
    const int32_t* pos = a.positions + bh * a.slots;
    float* w_out = a.weights_out + bh * a.slots;
    int32_t* pos_out = a.positions_out + bh * a.slots;
    const int64_t oldest = (int64_t)a.seen[b] - a.recent;
    if (h == 0 && tid == 0)
        a.lens_out[b] = kept;
    auto key = [&](int j) { return rank_key(w[j], (int64_t)pos[j] >= oldest); };

    int moved = 0;
    if (len > a.budget && a.budget > 0) {
        // the key of the last token kept, and how many of that key are kept
        unsigned prefix = 0;
        unsigned wanted = (unsigned)a.budget;
        for (int shift = 24; shift >= 0; shift -= 8) {
            if (tid < 256)
                histogram[tid] = 0;
            __syncthreads();
            for (int j = tid; j < len; j += kEvictThreads) {
                const unsigned u = key(j);
                if (shift == 24 || (u >> (shift + 8)) == (prefix >> (shift + 8)))
                    atomicAdd(&histogram[(u >> shift) & 255u], 1u);
            }
            __syncthreads();
            if (tid == 0) {
                unsigned left = wanted;
                int d = 255;
                while (d > 0 && histogram[d] < left) {
                    left -= histogram[d];
                    --d;
                }
                chosen[0] = prefix | ((unsigned)d << shift);
                chosen[1] = left;
            }
            __syncthreads();
            prefix = chosen[0];
            wanted = chosen[1];
            __syncthreads();
        }
        int32_t* to = a.moves + bh * 2 * a.moves_max;
        int32_t* from = to + a.moves_max;
        int equal = 0, holes = 0, movers = 0;   // found in the slots before this round of the walk
        for (int j0 = 0; j0 < len; j0 += kEvictThreads) {
            const int j = j0 + tid;
            const unsigned u = j < len ? key(j) : 0u;
            const bool same = j < len && u == prefix;
            Pair all;
            const int before = block_scan(Pair{same, 0}, &all, waves).a;
            const bool keep = j < len && (u > prefix || (same && (unsigned)(equal + before) < wanted));
            equal += all.a;
            const bool hole = j < a.budget && j < len && !keep, mover = j >= a.budget && keep;
            const Pair at = block_scan(Pair{hole, mover}, &all, waves);
            if (hole)
                to[holes + at.a] = j;
            if (mover)
                from[movers + at.b] = j;
            holes += all.a;
            movers += all.b;
        }
        moved = movers;
        __syncthreads();
    }
    if (tid == 0)
        a.count[bh] = moved;
    for (int64_t j = tid; j < a.slots; j += kEvictThreads) {
        w_out[j] = j < kept ? w[j] : 0.0f;
        pos_out[j] = j < kept ? pos[j] : -1;
    }
    __syncthreads();
    const int32_t* to = a.moves + bh * 2 * a.moves_max;
    const int32_t* from = to + a.moves_max;
    for (int i = tid; i < moved; i += kEvictThreads) {
        w_out[to[i]] = w[from[i]];
        pos_out[to[i]] = pos[from[i]];
    }
}

// A wave per move: one key row and one value row.
__global__ void __launch_bounds__(256)
evict_move_kernel(Evict a, int blocks)
{
    const int lane = threadIdx.x & 63;
    const int block = blockIdx.x % blocks;
    const int bh = blockIdx.x / blocks;
    const int h = bh % a.heads, b = bh / a.heads;
    const int moved = a.count[bh];
    const int32_t* to = a.moves + (int64_t)bh * 2 * a.moves_max;
    const int32_t* from = to + a.moves_max;
    const int per_row = a.dim >> 3;
    for (int i = block * 4 + (threadIdx.x >> 6); i < moved; i += blocks * 4) {
        const int64_t src = a.at.offset(b, from[i]), dst = a.at.offset(b, to[i]);
        if (src < 0 || dst < 0 || lane >= 2 * per_row)
            continue;
        uint16_t* pool = lane < per_row ? a.k : a.v;
        const int64_t d = h * a.at.stride_head + (lane < per_row ? lane : lane - per_row) * 8;
        *reinterpret_cast<u32x4*>(pool + dst + d) = *reinterpret_cast<const u32x4*>(pool + src + d);
    }
}

}  // namespace gattn
