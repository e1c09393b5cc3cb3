// cache_kernels.hpp -- gfx950 (CDNA4) device code for the append to a paged
// key-value cache and the eviction from it.
//
// Both only move rows and are bound by memory: append 5.1 to 5.2 TB/s read and
// written (4 x 8191 tokens, 52 us) where a copy makes 4.95 TB/s.
#pragma once

#include "paged.hpp"

namespace gattn {

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
