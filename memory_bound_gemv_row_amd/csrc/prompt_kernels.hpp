// prompt_kernels.hpp -- gfx950 (CDNA4) device code for attention of many query
// rows over a paged key-value cache: several new tokens per sequence, and the
// shared prefix of a group of sequences.
//
//   o_r = sum_j p_rj v_j,  p_r = softmax_j(scale * q_r . k_j),  j visible to r
//
// Both products are matrix products with the keys read once for 128 rows, so
// long prompts are bound by the matrix units and the exponentials between the
// two products, few rows by memory.
#pragma once

#include "attention_kernels.hpp"

#include <type_traits>

namespace gattn {

typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef float f32x2 __attribute__((ext_vector_type(2)));
typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef _Float16 f16x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));

constexpr int kTileRows = 128;   // query rows of a workgroup, 32 a wave
constexpr int kTileKeys = 64;    // keys of a step, 16 loaded by each wave
constexpr int kEverySlot = 0x7FFFFFFE;

// The power of two that a row's largest power has where its logit is the running
// maximum.  binary16 has room for 2^15, of which the slack takes eight, and loses
// what is below 2^-14 bit by bit: so raised, a power is rounded by half a step down
// to 2^-21 of the largest, and by 2^-32 of the largest below that.
constexpr float raised_of(int type) { return type == kF16 ? 7.0f : 0.0f; }
constexpr float lowered_of(int type) { return type == kF16 ? 0x1p-7f : 1.0f; }
constexpr float kFar = 1 << 20;  // of scaled logits: half their step there, 2^-4, is little beside the slack

// Waves that have the same 32 rows, and share out the output's elements: heads of
// over 128 need two, for the sums of 256 elements leave no registers to work with.
constexpr int outputs_of(int dim) { return dim > 128 ? 2 : 1; }

// Waves of a SIMD that registers are shared out for.  Heads of 64 have as many
// exponentials for half the matrix products and gain by a third wave (6 x 1999
// tokens of 16 heads, one sequence's tiles after another's: 79.9 -> 69.1 us; a
// fourth leaves too few registers, 83.2).
constexpr int waves_of(int dim) { return dim > 64 ? 2 : 3; }

// Where the row tiles stand among a head's places.
enum TileOrder {
    kTogether,               // rows * group / 128 + batch places for all sequences' tiles in turn
    kSingle,                 // no sequence has more than one: place i is sequence i's
    kLaps,                   // as many places for each sequence, `run` of one before the next one's
    kShares,                 // none has more than one: `tiles` places for the parts of all, shared out by their lengths
};

struct Prompt {
    Pages at;
    const uint16_t* k;
    const uint16_t* v;
    const uint16_t* q;
    int64_t q_stride;
    const int32_t* starts;   // [batch + 1]: rows of q of each sequence
    int batch, rows, max_new;
    int q_heads, heads, dim;
    int group;               // query heads per key-value head
    Divider group_of;
    bool causal;
    int window;              // tokens seen, the row's own included; 0: all
    int sinks, sink_tiles;   // first tokens seen all the same, and the tiles that hold them
    TileOrder order;
    int tiles;               // places for row tiles per key-value head: of all sequences, or kLaps of each
    int laps;                // 1, kLaps: batch
    int run, stretch;        // places that follow each other, and of all laps: run * laps
    int parts, chunk;        // workgroups over the keys, and tiles of keys of each; kShares: parts at the most
    float scale;             // of the logits, above zero, log2(e) included
    float slack;             // kSlack / scale
    unsigned keep, flip;     // bits of q: none where the scale is zero; the signs flipped where it is negative
    void* out;
    float* part_out;         // [rows][q_heads][parts][dim], not divided by the sums, or null
    float* part_ms;          // [rows][q_heads][parts][2]: maximum and sum of powers
};

template <int DT>
__device__ __forceinline__ f32x16 mfma_wide(u32x4 a, u32x4 b, f32x16 c)
{
    if constexpr (DT == kF16)
        return __builtin_amdgcn_mfma_f32_32x32x16_f16(__builtin_bit_cast(f16x8, a), __builtin_bit_cast(f16x8, b), c, 0, 0, 0);
    else
        return __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b), c, 0, 0, 0);
}

template <int DT>
__device__ __forceinline__ unsigned narrow_pair(float x, float y)
{
    const f32x2 v = {x, y};
    if constexpr (DT == kF16)
        return __builtin_bit_cast(unsigned, __builtin_convertvector(v, f16x2));
    else
        return __builtin_bit_cast(unsigned, __builtin_convertvector(v, bf16x2));
}

// sum + both elements of a pair
template <int DT>
__device__ __forceinline__ float add_pair([[maybe_unused]] unsigned pair, float sum)
{
#ifdef __HIP_DEVICE_COMPILE__
    if constexpr (DT == kF16)
        return __builtin_amdgcn_fdot2(__builtin_bit_cast(f16x2, pair), f16x2{(_Float16)1.0f, (_Float16)1.0f}, sum, false);
    else
        return __builtin_amdgcn_fdot2_f32_bf16(__builtin_bit_cast(bf16x2, pair), bf16x2{(__bf16)1.0f, (__bf16)1.0f}, sum, false);
#else
    return sum;
#endif
}

// Sixteen bytes of each lane straight to LDS, to its place behind byte `to` (the
// same for all lanes).  Written out, for the compiler would make every read of
// LDS wait for such loads, those into the other buffer too; the kernel waits for
// them itself, before the barrier that hands a buffer over.  s_nop: five steps
// between a vector instruction that writes a scalar register and its use as a
// descriptor, and one after m0 is set.  (m0 cannot be named as changed: it is reserved,
// and the compiler sets it right before each use of its own.)
__device__ __forceinline__ void piece_to_lds([[maybe_unused]] u32x4 from, [[maybe_unused]] unsigned offset,
                                             [[maybe_unused]] unsigned to)
{
#ifdef __HIP_DEVICE_COMPILE__
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 4\n\tbuffer_load_dwordx4 %1, %2, 0 offen lds"
                 :: "s"(to), "v"(offset), "s"(from) : "memory");
#endif
}

__device__ __forceinline__ void piece_to_lds([[maybe_unused]] const void* from, [[maybe_unused]] unsigned to)
{
#ifdef __HIP_DEVICE_COMPILE__
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 4\n\tglobal_load_lds_dwordx4 %1, off" :: "s"(to), "v"(from) : "memory");
#endif
}

// Byte address of LDS memory.
__device__ __forceinline__ unsigned lds_byte([[maybe_unused]] const void* p)
{
#ifdef __HIP_DEVICE_COMPILE__
    return (unsigned)(uintptr_t)(__attribute__((address_space(3))) const char*)p;
#else
    return 0;
#endif
}

// A buffer descriptor as four words, the same for all lanes.
__device__ __forceinline__ u32x4 descriptor(const uint16_t* p, unsigned bytes)
{
    const uint64_t at = reinterpret_cast<uint64_t>(p);
    return u32x4{(unsigned)at, (unsigned)(at >> 32) & 0xFFFFu, bytes, 0x00027000u};
}

// A word that no kernel running at the same time writes, at an address that
// all lanes share.
__device__ __forceinline__ int shared_word(const int32_t* p)
{
    return *(const __attribute__((address_space(4))) int32_t*)(uintptr_t)p;
}

// Four keys of one column: within 16 lanes, lane i points at four elements of
// row i / 4, columns 4 (i % 4) on, and gets column i of the four rows.
__device__ __forceinline__ u32x2 column_of_four([[maybe_unused]] const u32x4* base, [[maybe_unused]] unsigned byte)
{
#ifdef __HIP_DEVICE_COMPILE__
    auto p = (__attribute__((address_space(3))) const char*)base + byte;
    return __builtin_bit_cast(u32x2, __builtin_amdgcn_ds_read_tr16_b64_v4i16((__attribute__((address_space(3))) s16x4*)p));
#else
    return u32x2{0, 0};
#endif
}

__device__ __forceinline__ unsigned bits_below(int64_t n) { return n <= 0 ? 0u : n >= 32 ? ~0u : (1u << n) - 1u; }

// The sequence whose row tiles hold place `u`, of places that a sequence b has
// from floor(starts[b] * group / 128) + b on: as many as it can need, none
// twice.  A wave looks at 64 sequences at a time; what it has to know of the last
// 64 is loaded at once, for each load that waits for another is half a
// microsecond of a workgroup's start.
struct Sequence {
    int b, len, from, to;   // its rows
};

__device__ __forceinline__ Sequence sequence_at(const Pages& at, const int32_t* starts, int batch, int rows, int group, int64_t u)
{
    const int lane = threadIdx.x & 63;
    int low = 0, count = batch;   // the answer is in [low, low + count)
    while (count > 64) {
        const int step = (count + 63) / 64;
        const int i = lane * step;
        const bool below = i < count && row_start(starts, low + i, rows) * group / kTileRows + low + i <= u;
        const int n = __popcll(__ballot(below));   // the places rise with the sequence
        const int first = n > 0 ? (n - 1) * step : 0;
        low += first;
        count = count - first < step ? count - first : step;
    }
    const int b = low + (lane < count ? lane : count - 1);
    const int from = (int)row_start(starts, b, rows), to = (int)row_start(starts, b + 1, rows), len = at.length(b);
    const int n = __popcll(__ballot(lane < count && (int64_t)from * group / kTileRows + b <= u));
    const int it = n > 0 ? n - 1 : 0;
    return Sequence{low + it, __builtin_amdgcn_readlane(len, it), __builtin_amdgcn_readlane(from, it),
                    __builtin_amdgcn_readlane(to, it)};
}

// Place `w` of kShares: every part is of `chunk` tiles of keys, about the fewest
// with which the places hold all sequences' parts, so that short sequences leave
// no place idle (4 x 6 tokens behind up to 20000, 16/4 heads of 256: 74 -> 65 us;
// 4 x 7 behind up to 65536, 32/8 heads of 128: 149 -> 136).  Lane b counts for
// sequence b.
struct Share {
    Sequence sequence;
    int part, parts, chunk;   // parts: of this sequence; 0: nobody's place
};

__device__ __forceinline__ Share share_at(const Prompt& a, int w)
{
    const int lane = threadIdx.x & 63;
    const int b = lane < a.batch ? lane : a.batch - 1;
    const int from = (int)row_start(a.starts, b, a.rows), to = (int)row_start(a.starts, b + 1, a.rows), len = a.at.length(b);
    const bool any = lane < a.batch && to > from;
    const int count = any && len > 0 ? (len - 1) / kTileKeys + 1 : any;   // a sequence without keys has its rows cleared
    int most = count;
    unsigned all = count;   // no more than 64 times 2^25
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
        const int other = __shfl_xor(most, d);
        most = most > other ? most : other;
        all += (unsigned)__shfl_xor((int)all, d);
    }
    // with fewer neither the places nor the room for parts would do
    int chunk = (int)((all + a.tiles - 1) / a.tiles);
    const int for_room = (most + a.parts - 1) / a.parts;
    chunk = chunk > for_room ? chunk : for_room;
    chunk = chunk > 1 ? chunk : 1;
    int parts, upto, held;
    for (;; chunk += (chunk + 7) / 8) {   // ends: there is a place for each sequence
        parts = (count + chunk - 1) / chunk;
        upto = parts;
#pragma unroll
        for (int d = 1; d < 64; d <<= 1) {
            const int up = __shfl_up(upto, d);
            upto += lane >= d ? up : 0;
        }
        held = __builtin_amdgcn_readlane(upto, 63);
        if (held <= a.tiles || chunk >= most)
            break;
    }
    if (w >= held)
        return Share{};
    const int it = __popcll(__ballot(upto <= w)), own = __builtin_amdgcn_readlane(parts, it);
    return Share{Sequence{it, __builtin_amdgcn_readlane(len, it), __builtin_amdgcn_readlane(from, it),
                          __builtin_amdgcn_readlane(to, it)},
                 w - __builtin_amdgcn_readlane(upto, it) + own, own, chunk};
}

// The key-value head, the part of the keys, and the place among the head's row tiles
// (of sequence `lap`, where a.order is kLaps) of a workgroup, for all orders but
// kShares.
//
// Workgroups go to the eight XCDs in turn.  Those that read the same keys
// (a head's, of a part) are on one XCD where such sets are a multiple of
// eight, and the last parts, which only long sequences have, come first.  From
// part to part an XCD moves on by a head, so that it sees every head's part of
// the address space.  Of the row tiles the last, which see most, come first, a run
// of them from one sequence before the next one's, so that they find its keys
// in the L2, and all sequences' and sets' last run before the one before it, so that
// what is started last is short.
//
// `quotient` divides two numbers that are the same for all lanes.
struct Spot {
    int kv, part, place, lap;
};

template <class Quotient>
__host__ __device__ __forceinline__ Spot spot_of(const Prompt& a, int block, Quotient quotient)
{
    const int sets = a.heads * a.parts;
    const bool eight = sets % 8 == 0;
    const int each = eight ? sets >> 3 : 1;                                 // sets of an XCD
    int j = eight ? block >> 3 : quotient(block, sets);
    const int first = quotient(j, each * a.stretch);
    j -= first * each * a.stretch;
    const int left = a.tiles - first * a.run;
    const int run = left < a.run ? left : a.run;
    const int lap = quotient(j, run), set_of = quotient(lap, a.laps);
    const int set = eight ? set_of * 8 + (block & 7) : block - quotient(block, sets) * sets;
    const int part_back = quotient(set, a.heads), part = a.parts - 1 - part_back;
    const int kv_at = set - part_back * a.heads + part;
    return Spot{kv_at - quotient(kv_at, a.heads) * a.heads, part, a.tiles - 1 - first * a.run - (j - lap * run), lap - set_of * a.laps};
}

// 16 zeros that slots without a page are read from
__device__ const u32x4 kZeros[1] = {{0, 0, 0, 0}};

// One workgroup: 128 query rows (tokens times the query heads of one key-value
// head, a token's heads together) of one sequence, over one part of the keys
// that any of them sees.  Each wave has 32 rows (heads of over 128: two waves
// have the same, take the same logits, and half of the output each); they load
// 64 keys and values at a time straight to LDS, into one of two buffers while the
// other is multiplied.
//
// Logits: v_mfma_f32_32x32x16 with keys as rows and queries, which stay in
// registers, as columns: lane l gets, for query row l % 32, the logits of keys
// 8 (i / 4) + 4 (l / 32) + i % 4, i = 0..15.  A lane so has one query row: its
// maximum and sum need no other lane but l ^ 32's, and that only when the
// maximum moves (past it by kSlack, as in decode attention) and at the end.
// The powers, in pairs rounded to 16 bits, are in place as the right operand of
// the product with the values, if that takes its summed index in the same
// order of keys; the left operand, columns of four values, comes out of LDS
// turned by ds_read_b64_tr_b16.  The powers' rounding is half a step, 2^-11 or 2^-8
// relative each (see raised_of), which adds about as much to the output's error as its
// own rounding does (1.2 to 1.4 times that alone); the sum is taken over the rounded
// powers, so the weights still add up to one.  A second number for what the first
// rounds off would leave 2^-22 or 2^-16, and takes as many products with the values
// again: 2 x 16384 tokens through a window of 4096 2340 us for 1790, 4 x 8192, 16 heads
// of 64, 670 for 500, 128 sequences behind prefixes of 32768 149 for 127, 4 x 7
// tokens behind 65536 142 for 137.  Its products with an infinite value are
// NaN besides, for it is zero or below as often as above.
//
// RUN: slots that lie in one page from their first multiple on, 16 or 8, whose
// address is the same for all lanes; 1: each row has an address of its own (4 x
// 8192 tokens, 16 heads of 64: 513 us in pages of 16, 517 in pages of 24, 562 in
// pages of 5; 2 x 8192, 32/8 heads of 128: 610, 633, 736).
//
// Bound, where prompts are long, by the matrix and the vector units in turn: both
// are busy 45 % of the time, for a wave takes its products, maximum, powers and
// products one after another, and that a SIMD's other wave does something else meanwhile is
// left to chance.  (Up to 128 that one is of another workgroup, with a barrier of its
// own; over 128 both wait at one.)  2 x 16384 tokens through a window of
// 4096, 32/8 heads of 128: 1710 to 1850 us by card, 886 to 957 TFLOP/s; the products and
// barriers alone take 64 % of a long prompt's time, exponentials 10 %, reads of
// LDS 16 %, loads 17 %, the maximum 3 %, each taken out by itself.  Heads of 64 have half
// the products for as many powers, whose 26 cycles for 64 of them are more than
// the products' 16: 4 x 8192 tokens of 16 heads 260 us of vector instructions alone.
// Where rows are few, by memory: 4 x 7 tokens behind up to 65536 read 715 MB in 131 us.
// Of a few hundred rows, by the 1.1 to 2 us that a step takes however few waves
// there are.  Heads of over 128 keep 22 to 132 registers in scratch memory, most of
// them read outside of the loop over whole tiles, and take their logits twice.
//
// Places in LDS: piece c (16 bytes) of key row r lies at c ^ swizzle(r), such
// that the 16 rows that a read of keys takes at a time, and the four rows of
// 64 bytes that a read of values does, are in different banks.
//
// Masks are looked at in tiles that some row of the wave does not see whole, each
// wave for itself, 32 keys at a time, and those that none of its rows sees left
// out (8 x 4000 tokens through a window of 512: 294 us where a tile is whole or
// masked for all waves, 272; 300 tokens 14.3 and 13.3).  There the values may
// hold NaN or infinities in slots that only some rows see; 0 * NaN would bring
// them to the others, so where there are any such a tile is multiplied key by
// key, and rows that do not see the key keep their sums.
template <int DP>
struct PromptShared {
    u32x4 buffers[2][2][kTileKeys * DP / 8];                    // keys and values of a step, and of the next
    __attribute__((aligned(8))) uint16_t held_bits[2][4];       // bit per key: its slot is there
};

template <int DT, int DP, int RUN, bool EXACT>
__device__ __forceinline__ void prompt_block(const Prompt& a, int block, PromptShared<DP>& shared)
{
    constexpr int CH = DP / 8;        // pieces of a row
    constexpr int kLoads = CH / 4;    // 64 pieces each of the 16 rows that a wave loads
    constexpr int kSteps = DP / 16;   // of 16 elements of the dot products
    constexpr int kOutputs = outputs_of(DP);
    constexpr int kBlocks = DP / 32 / kOutputs;   // of 32 elements of the output
    auto& buffers = shared.buffers;
    auto& held_bits = shared.held_bits;

    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6 & 3);
    const int output = kOutputs == 1 ? 0 : __builtin_amdgcn_readfirstlane(threadIdx.x >> 8);
    const int half = lane >> 5;

    // `one`: the same for all lanes, and known to be where the vector unit has computed it
    auto one = [](int x) { return __builtin_amdgcn_readfirstlane(x); };
    auto quotient = [&](int x, int y) { return one((int)((unsigned)x / (unsigned)y)); };
    Sequence sequence;
    int kv, tile, part, parts = a.parts, chunk = a.chunk;
    if (a.order == kShares) {
        const int w = quotient(block, a.heads);
        const Share share = share_at(a, w);
        if (share.parts == 0)
            return;
        sequence = share.sequence;
        tile = 0;
        part = share.part;
        parts = share.parts;
        chunk = share.chunk;
        const int kv_at = block - w * a.heads + part;
        kv = kv_at - quotient(kv_at, a.heads) * a.heads;
    } else {
        const Spot spot = spot_of(a, block, quotient);
        part = spot.part;
        kv = spot.kv;
        tile = spot.place;
        if (a.order != kTogether) {
            const int at = a.order == kSingle ? spot.place : spot.lap;
            tile = a.order == kSingle ? 0 : spot.place;
            sequence = Sequence{at, a.at.length(at), (int)row_start(a.starts, at, a.rows), (int)row_start(a.starts, at + 1, a.rows)};
        } else {
            sequence = sequence_at(a.at, a.starts, a.batch, a.rows, a.group, spot.place);
            tile = spot.place - (int)((int64_t)sequence.from * a.group / kTileRows) - sequence.b;
        }
    }
    kv = one(kv);
    part = one(part);
    parts = one(parts);
    chunk = one(chunk);
    const int b = one(sequence.b), len = one(sequence.len), to = one(sequence.to);
    int n = to - one(sequence.from);                                            // new tokens
    n = n < a.max_new ? n : a.max_new;
    const int64_t row0 = to - n;                                                // the first of them
    // this tile's first row; rows times the group are below 2^30, as the launch's work-items are
    const int r0 = one(tile * kTileRows);
    if (n <= 0 || r0 < 0 || r0 >= n * a.group)
        return;
    const int rows = n * a.group - r0 < kTileRows ? n * a.group - r0 : kTileRows;

    // tokens of the tile and of this wave, and the slots they see
    auto token_of = [&](int r) { return a.group_of.by(r0 + r); };
    // position of a row's token, the last slot that it sees; -1: none
    auto position_of = [&](int r) {
        const int p = len - n + token_of(r);
        return !a.causal ? kEverySlot : p > -1 ? p : -1;
    };
    const int tile_min = one(position_of(0)), tile_max = one(position_of(rows - 1));
    const bool mine = 32 * wave < rows;
    const int last = rows - 1 < 32 * wave + 31 ? rows - 1 : 32 * wave + 31;
    const int wave_min = one(position_of(mine ? 32 * wave : 0)), wave_max = one(position_of(last));
    const int top_slot = tile_max + 1 < len ? tile_max + 1 : len;               // no row sees this or beyond
    const int tiles_all = top_slot > 0 ? (top_slot + kTileKeys - 1) / kTileKeys : 0;
    int jump = 0;                                                               // tiles cut out after the first tokens'
    if (a.window > 0 && tile_min >= a.window) {
        jump = (tile_min - a.window + 1) / kTileKeys - a.sink_tiles;
        jump = jump > 0 ? jump : 0;
    }
    const int count = tiles_all - jump;
    const int begin = part * chunk, end = count < begin + chunk ? count : begin + chunk;
    auto slot_of = [&](int u) { return (u < a.sink_tiles ? u : u + jump) * kTileKeys; };

    // this lane's query row
    const int r = 32 * wave + (lane & 31);
    const bool there = r < rows;
    const int safe = there ? r : 0;                                             // no lane's address needs a branch
    const int token = token_of(safe);
    const int head = kv * a.group + (r0 + safe - token * a.group);
    const int64_t row = row0 + token;
    const int position = there ? position_of(r) : -1;
    u32x4 query[kSteps];   // loaded behind the first keys
    const uint16_t* const query_at = a.q + row * a.q_stride + (int64_t)head * a.dim;

    float m = -kInf, sum = 0.0f;
    f32x16 acc[kBlocks];
#pragma unroll
    for (int k = 0; k < kBlocks; ++k)
        acc[k] = f32x16{};

    // ---- loads: this lane's pieces of the wave's 16 rows
    auto key_swizzle = [](int row) {
        return DP == 64 ? (row >> 1) & 7 : DP == 96 ? (row >> 2) & 3 : row & 15;
    };
    auto value_swizzle = [](int row) {
        return DP == 64 ? (row >> 1 & 1) << 2 : DP == 96 ? 0 : (row & 3) << 2;
    };
    // of keys and of values, or where two waves have the same rows, of one of them
    constexpr int kKinds = 2 / kOutputs;
    const uint16_t* pool[kKinds];
    int load_row[kLoads];
    unsigned piece[kKinds][kLoads];   // bytes from the row's start; of runs: from the run's first row's
    constexpr bool kRun = RUN > 1;
    constexpr int kRuns = kRun ? 16 / RUN : 1;
    // the run of a load's first piece, and the lane from which on its pieces are of the
    // next one: none, but of heads of 96 in runs of eight the second load's middle
    auto run_of = [](int i) { return kRun ? i * 64 / CH / RUN : 0; };
    auto next_from = [run_of](int i) { return kRun ? (run_of(i) + 1) * RUN * CH - i * 64 : 64; };
#pragma unroll
    for (int x = 0; x < kKinds; ++x)
        pool[x] = (x + output == 0 ? a.k : a.v) + kv * a.at.stride_head;
#pragma unroll
    for (int i = 0; i < kLoads; ++i) {
        const int p = i * 64 + lane, rw = p / CH, c = p - rw * CH;
        load_row[i] = rw - (kRun ? run_of(i) * RUN + (lane < next_from(i) ? 0 : RUN) : 0);
#pragma unroll
        for (int x = 0; x < kKinds; ++x) {
            const int at = c ^ (x + output == 0 ? key_swizzle(rw) : value_swizzle(rw));
            const unsigned first = kRun ? (unsigned)(load_row[i] * (int)a.at.stride_slot) * 2 : 0u;
            piece[x][i] = EXACT || at * 8 < a.dim ? first + at * 16 : kNowhere;
        }
    }
    struct Place {
        int page[kRun ? kRuns : kLoads];
    };
    // the pages of step u, looked up a step before its loads
    auto look = [&](int u) {
        Place w;
        const int j = slot_of(u) + 16 * wave;
        if constexpr (kRun) {
#pragma unroll
            for (int g = 0; g < kRuns; ++g) {
                w.page[g] = -1;
                if (u < end && j + g * RUN < len)
                    w.page[g] = shared_word(a.at.table + b * a.at.table_stride + a.at.page_of.by(j + g * RUN));
            }
        } else {
#pragma unroll
            for (int i = 0; i < kLoads; ++i) {
                w.page[i] = -1;
                if (u < end && j + load_row[i] < len)
                    w.page[i] = a.at.table[b * a.at.table_stride + a.at.page_of.by(j + load_row[i])];
            }
        }
        return w;
    };
    constexpr unsigned kHalfBytes = kTileKeys * CH * 16;
    const unsigned wave_byte = __builtin_amdgcn_readfirstlane(lds_byte(&buffers[0][output][0])) + wave * 16 * CH * 16;
    auto fetch = [&](int which, int u, const Place& w) {
        const int j = slot_of(u) + 16 * wave;
        const unsigned to = wave_byte + which * 2 * kHalfBytes;
        unsigned bits;
        if constexpr (kRun) {
            bits = 0;
            u32x4 from[kRuns][kKinds];
            int left[kRuns];   // slots of the run before the end
#pragma unroll
            for (int g = 0; g < kRuns; ++g) {
                const int jg = j + g * RUN;
                const bool is = (unsigned)w.page[g] < (unsigned)a.at.pages;
                left[g] = is ? len - jg : 0;
                const int64_t at = is ? w.page[g] * a.at.stride_page + (int64_t)(jg - a.at.page_of.by(jg) * a.at.page_size) * a.at.stride_slot : 0;
#pragma unroll
                for (int x = 0; x < kKinds; ++x)
                    from[g][x] = descriptor(pool[x] + at, is ? kNowhere - 1 : 0);
                bits |= (left[g] >= RUN ? (1u << RUN) - 1u : (1u << (left[g] > 0 ? left[g] : 0)) - 1u) << (g * RUN);
            }
#pragma unroll
            for (int i = 0; i < kLoads; ++i)
#pragma unroll
                for (int x = 0; x < kKinds; ++x) {
                    const unsigned at = to + x * kHalfBytes + i * 1024;
                    const int run = run_of(i);
                    if (lane < next_from(i))
                        piece_to_lds(from[run][x], load_row[i] < left[run] ? piece[x][i] : kNowhere, at);
                    else if (run + 1 < kRuns)
                        piece_to_lds(from[run + 1][x], load_row[i] < left[run + 1] ? piece[x][i] : kNowhere, at);
                }
        } else {
            bits = 0;
#pragma unroll
            for (int i = 0; i < kLoads; ++i) {
                const int s = j + load_row[i];
                const bool is = s < len && (unsigned)w.page[i] < (unsigned)a.at.pages;
                const int64_t at = is ? w.page[i] * a.at.stride_page + (int64_t)(s - a.at.page_of.by(s) * a.at.page_size) * a.at.stride_slot : 0;
#pragma unroll
                for (int x = 0; x < kKinds; ++x)
                    piece_to_lds(is && piece[x][i] != kNowhere ? reinterpret_cast<const char*>(pool[x] + at) + piece[x][i]
                                                               : reinterpret_cast<const char*>(kZeros),
                                 to + x * kHalfBytes + i * 1024);
                // a row's first piece speaks for it
                const uint64_t lanes = __ballot(is);
#pragma unroll
                for (int rw = 0; rw < 16; ++rw)
                    if (rw * CH >= i * 64 && rw * CH < i * 64 + 64)
                        bits |= (unsigned)(lanes >> (rw * CH - i * 64) & 1) << rw;
            }
        }
        if (lane == 0 && output == 0)
            held_bits[which][wave] = (uint16_t)bits;
    };

    // ---- products
    const int key_row = lane & 31;
    const int key_base = key_swizzle(key_row & 15) ^ half;                       // piece 2 s + half lies at 2 s ^ key_base
    const int i16 = lane & 15, value_row = 4 * half + (i16 >> 2);                // and 8, 16, ... rows on
    const unsigned value_byte = (unsigned)(value_row * CH * 16 + (i16 & 1) * 8);
    const int value_base = value_swizzle(value_row & 15);
    const int value_col = 2 * (lane >> 4 & 1) + (i16 >> 1 & 1);                  // piece 4 block + this

    auto key_piece_at = [&](int t, int e) { return (32 * t + key_row) * CH + ((2 * e) ^ key_base); };
    // four and four keys of step `step` (16 keys), 32 columns from 32 `block` on
    auto value = [&](const u32x4* values, int step, int block) {
        const unsigned byte = value_byte + (unsigned)((4 * (kBlocks * output + block) + value_col) ^ value_base) * 16;
        const u32x2 x = column_of_four(values, byte + (unsigned)(16 * step) * CH * 16);
        const u32x2 y = column_of_four(values, byte + (unsigned)(16 * step + 8) * CH * 16);
        return u32x4{x.x, x.y, y.x, y.y};
    };
    // the running maximum and all sums, where some logit passes it by kSlack
    auto raise = [&](float top) {
        if (__any(top - m > a.slack)) {
            top = fmaxf(top, __shfl_xor(top, 32));
            const float next = fmaxf(m, top);
            const float f = m == -kInf ? 0.0f : exp2_hw((m - next) * a.scale);
            m = next;
            sum *= f;
#pragma unroll
            for (int k = 0; k < kBlocks; ++k)
                acc[k] *= f;
        }
        return m == -kInf ? 0.0f : m;
    };
    // Two powers, times 2^raised.  A logit is subtracted from before it is scaled, so
    // that the largest has power 1 and equal ones equal powers, however large they
    // are.  Fused: in one operation, from a product that is rounded already; what that
    // left off multiplies all powers of a row alike, up to 2^(half a step of the product).
    constexpr bool kFused = kOutputs == 1;
    constexpr float kRaised = raised_of(DT), kLowered = lowered_of(DT);
    auto power_pair = [&](auto fused, float x, float y, float from) {
        auto power = [&](float z) {
            return exp2_hw(decltype(fused)::value ? __builtin_fmaf(z, a.scale, -from) : __builtin_fmaf(z - from, a.scale, kRaised));
        };
        const unsigned pair = narrow_pair<DT>(power(x), power(y));
        sum = add_pair<DT>(pair, sum);
        return pair;
    };

    // A tile that every row sees whole; or false, and nothing summed, where powers are
    // fused and some logits are too far from zero for that.  (Not fused at all: 4 x 8192
    // tokens, 16 heads of 64, 520 us for 494, 2 x 8192, 32/8 of 128, 642 for 629.  Heads of
    // over 128 have no registers for the other way out: 329 us to 489 by it, 332 without.)
    auto use = [&](const u32x4* keys, const u32x4* values) {
        f32x16 s[2];
#pragma unroll
        for (int t = 0; t < 2; ++t) {
            s[t] = f32x16{};
#pragma unroll
            for (int e = 0; e < kSteps; ++e)
                s[t] = mfma_wide<DT>(keys[key_piece_at(t, e)], query[e], s[t]);
        }
        float top = s[0][0];
#pragma unroll
        for (int i = 1; i < 32; ++i)
            top = fmaxf(top, s[i / 16][i % 16]);
        float from = raise(top);
        if constexpr (kFused) {
            from = __builtin_fmaf(from, a.scale, -kRaised);
            if (__any(fabsf(from) > kFar))
                return false;
        }
        u32x4 p[4];
#pragma unroll
        for (int i = 0; i < 32; i += 2)
            p[i / 8][i % 8 / 2] = power_pair(std::bool_constant<kFused>{}, s[i / 16][i % 16], s[i / 16][i % 16 + 1], from);
#pragma unroll
        for (int e = 0; e < 4; ++e)
#pragma unroll
            for (int k = 0; k < kBlocks; ++k)
                acc[k] = mfma_wide<DT>(value(values, e, k), p[e], acc[k]);
        return true;
    };

    // any other tile, 32 keys at a time
    auto use_masked = [&](const u32x4* keys, const u32x4* values, uint64_t held, int j0) {
#pragma unroll 1
        for (int t = 0; t < 2; ++t, keys += 32 * CH, values += 32 * CH, held >>= 32, j0 += 32) {
            // bit j: this lane's row sees slot j0 + j
            auto look_at = [&] {
                unsigned seen = bits_below((int64_t)position + 1 - j0);
                if (a.window > 0)
                    seen &= ~bits_below((int64_t)position + 1 - a.window - j0) | bits_below((int64_t)a.sinks - j0);
                return seen & (unsigned)held;
            };
            unsigned visible = 0;
            if constexpr (kOutputs == 1) {
                visible = look_at();
                if (!__any(visible != 0))
                    continue;
            }
            f32x16 s = f32x16{};
#pragma unroll
            for (int e = 0; e < kSteps; ++e)
                s = mfma_wide<DT>(keys[key_piece_at(0, e)], query[e], s);
            if constexpr (kOutputs > 1)   // there registers are short: 332 us against 486 for 2 x 4096 tokens, 16/4 heads of 256
                visible = look_at();
            const unsigned seen = visible >> (4 * half);   // element i is bit 8 (i / 4) + i % 4
            float top = -kInf;
#pragma unroll
            for (int i = 0; i < 16; ++i) {
                s[i] = seen >> (8 * (i / 4) + i % 4) & 1 ? s[i] : -kInf;
                top = fmaxf(top, s[i]);
            }
            const float from = raise(top);
            u32x4 p[2];
#pragma unroll
            for (int i = 0; i < 16; i += 2)
                p[i / 8][i % 8 / 2] = power_pair(std::false_type{}, s[i], s[i + 1], from);
            constexpr unsigned kExp = DT == kF16 ? 0x7C007C00u : 0x7F807F80u, kLow = DT == kF16 ? 0x04000400u : 0x00800080u;
            unsigned over = 0;
            if (__any(there && visible != ~0u)) {
#pragma unroll
                for (int k = 0; k < kBlocks; ++k)
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        const u32x4 x = value(values, e, k);
#pragma unroll
                        for (int w = 0; w < 4; ++w)
                            over |= (x[w] & kExp) + kLow;
                    }
            }
            if (!__any((over & 0x80008000u) != 0)) {
#pragma unroll
                for (int e = 0; e < 2; ++e)
#pragma unroll
                    for (int k = 0; k < kBlocks; ++k)
                        acc[k] = mfma_wide<DT>(value(values, e, k), p[e], acc[k]);
                continue;
            }
            // one key at a time, kept by the rows that see it
#pragma unroll 1
            for (int c = 0; c < 32; ++c) {
                const bool sees = visible >> c & 1;
#pragma unroll
                for (int k = 0; k < kBlocks; ++k) {
                    f32x16 next = acc[k];
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        u32x4 x = value(values, e, k), w = p[e];
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            const int first = 16 * e + 8 * (i / 2) + 2 * (i % 2) + 4 * half;   // key of the pair's lower half
                            const unsigned only = c == first ? 0xFFFFu : c == first + 1 ? 0xFFFF0000u : 0u;
                            x[i] &= only;
                            w[i] &= only;
                        }
                        next = mfma_wide<DT>(x, w, next);
                    }
#pragma unroll
                    for (int i = 0; i < 16; ++i)
                        acc[k][i] = sees ? next[i] : acc[k][i];
                }
            }
        }
    };

    // All of this wave's reads of the current buffers are done and its pieces of
    // the next ones in LDS; after the barrier every wave's are.
    auto turn = [] {
        __builtin_amdgcn_s_waitcnt(0x0070);   // vmcnt(0) and lgkmcnt(0)
        __syncthreads();
    };
    auto held_of = [](const uint16_t* at) {
        uint64_t h;
        __builtin_memcpy(&h, at, sizeof h);
        return (uint64_t)(unsigned)__builtin_amdgcn_readfirstlane((int)(h >> 32)) << 32 |
               (unsigned)__builtin_amdgcn_readfirstlane((int)h);
    };
    if (begin < end) {
        Place next = look(begin);
        fetch(0, begin, next);
        next = look(begin + 1);
#pragma unroll
        for (int s = 0; s < kSteps; ++s) {
            const int d = 16 * s + 8 * half;
            query[s] = *reinterpret_cast<const u32x4*>(query_at + (EXACT || d < a.dim ? d : 0));
        }
#pragma unroll
        for (int s = 0; s < kSteps; ++s)
            query[s] = there && (EXACT || 16 * s + 8 * half < a.dim) ? (query[s] & a.keep) ^ a.flip : u32x4{0, 0, 0, 0};
        int u = begin, which = 0;
        // the buffers of step u are there, and the loads of the next one on their way
        auto step = [&] {
            turn();
            if (u + 1 < end)
                fetch(which ^ 1, u + 1, next);
            next = look(u + 2);
        };
        // this wave has rows, and each sees all of step u
        auto whole = [&] {
            const int j0 = slot_of(u);
            return mine && j0 + kTileKeys - 1 <= wave_min &&
                   (a.window == 0 || j0 > wave_max - a.window || j0 + kTileKeys - 1 < a.sinks) &&
                   held_of(held_bits[which]) == ~0ull;
        };
        step();
        for (;;) {
            // most steps: a loop of its own, so that what the others need costs it no registers
            while (whole() && use(buffers[which][0], buffers[which][1])) {
                if (++u >= end)
                    break;
                which ^= 1;
                step();
            }
            if (u >= end)
                break;
            const int j0 = slot_of(u);
            const bool unseen = j0 > wave_max || (a.window > 0 && j0 >= a.sinks && j0 + kTileKeys - 1 <= wave_min - a.window);
            if (mine && !unseen)
                use_masked(buffers[which][0], buffers[which][1], held_of(held_bits[which]), j0);
            if (++u >= end)
                break;
            which ^= 1;
            step();
        }
    }

    sum += __shfl_xor(sum, 32);
    if (!there)
        return;
    const int64_t at = row * a.q_heads + head;
    if (a.part_out != nullptr) {
        const int64_t to_part = at * a.parts + part;
        if (half == 0 && output == 0) {
            a.part_ms[to_part * 2] = m == -kInf ? -kInf : m * a.scale;
            a.part_ms[to_part * 2 + 1] = sum * kLowered;
            // parts that this sequence does not have saw nothing
            if (a.order == kShares)
                for (int p = parts + part; p < a.parts; p += parts) {
                    a.part_ms[(at * a.parts + p) * 2] = -kInf;
                    a.part_ms[(at * a.parts + p) * 2 + 1] = 0.0f;
                }
        }
        if (begin < end)
#pragma unroll
            for (int k = 0; k < kBlocks; ++k)
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int d = 32 * (kBlocks * output + k) + 8 * i + 4 * half;
                    if (EXACT || d < a.dim)
                        *reinterpret_cast<f32x4*>(a.part_out + to_part * a.dim + d) =
                            f32x4{acc[k][4 * i], acc[k][4 * i + 1], acc[k][4 * i + 2], acc[k][4 * i + 3]} * kLowered;
                }
        return;
    }
    const float by = sum == 0.0f ? 0.0f : 1.0f / sum;
    uint16_t* const out = static_cast<uint16_t*>(a.out) + at * a.dim;
#pragma unroll
    for (int k = 0; k < kBlocks; ++k)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int d = 32 * (kBlocks * output + k) + 8 * i + 4 * half;
            u32x2 w = {0, 0};
            if (sum != 0.0f) {
                w.x = narrow_pair<DT>(acc[k][4 * i] * by, acc[k][4 * i + 1] * by);
                w.y = narrow_pair<DT>(acc[k][4 * i + 2] * by, acc[k][4 * i + 3] * by);
            }
            if (EXACT || d < a.dim)
                *reinterpret_cast<u32x2*>(out + d) = w;
        }
}

template <int DT, int DP, int RUN, bool EXACT>
__global__ void __launch_bounds__(256 * outputs_of(DP), waves_of(DP))
prompt_kernel(Prompt a)
{
    __shared__ PromptShared<DP> shared;
    prompt_block<DT, DP, RUN, EXACT>(a, blockIdx.x, shared);
}

// Shared prefixes and the sequences' own tokens in one launch: the first
// `far_blocks` workgroups (a multiple of eight, so that the others too keep to
// their XCDs) take the prefixes, which the matrix units bound, the others the
// rest, which memory does; a CU that holds one of each is slowed by neither (128
// sequences behind two prefixes of up to 32768, 32/8 heads of 128: 146 us in two
// launches, 110 in one, and 9 for the join).
template <int DT, int DP, int RUN, bool EXACT>
__global__ void __launch_bounds__(256 * outputs_of(DP), waves_of(DP))
prefix_kernel(Prompt far, Attention near, int far_blocks, int far_count)
{
    constexpr int NP = DP == 96 ? 128 : DP, kNearWaves = 4 * outputs_of(DP);
    __shared__ union {
        PromptShared<DP> far;
        AttentionShared<NP, RUN == 16, kNearWaves> near;
    } shared;
    const int block = blockIdx.x;
    if (block >= far_blocks)
        attention_block<DT, NP, RUN == 16, RUN == 16 && EXACT && DP == NP, kNearWaves, true>(near, block - far_blocks, shared.near);
    else if (block < far_count)
        prompt_block<DT, DP, RUN, EXACT>(far, block, shared.far);
}
// Parts of the same rows: of `parts` each, in the layout of part_out and
// part_ms.  `starts`: the groups whose rows the parts are of (a row outside
// them has none), or null: every row.
struct Source {
    const float* ms;
    const float* out;
    int parts;
    const int32_t* starts;
    int batch;
};

struct Join {
    Source from[2];
    int rows, q_heads, dim;
    const int32_t* starts;   // rows to write: the last max_new of each sequence; null: every row
    int batch, max_new;
    void* out;
};

// The sequence that holds a row, as [first, last) of its rows; false where none does.
__device__ __forceinline__ bool sequence_of(const int32_t* starts, int batch, int rows, int64_t row, int64_t* first,
                                            int64_t* last)
{
    const int lane = threadIdx.x & 63;
    int low = 0, count = batch;
    while (count > 1) {
        const int step = (count + 63) / 64;
        const int at = lane * step;
        const int n = __popcll(__ballot(at < count && row_start(starts, low + at, rows) <= row));
        const int skip = n > 0 ? (n - 1) * step : 0;
        low += skip;
        count = count - skip < step ? count - skip : step;
    }
    *first = row_start(starts, low, rows);
    *last = row_start(starts, low + 1, rows);
    return row >= *first && row < *last;
}

// WAVES waves join the parts of one row's head: parts 64 at a time, an eighth or a
// quarter of those a wave where there are several, in a fixed order.  Lane p has
// part p's maximum and sum, and so its weight; then every lane adds up its E
// elements over the parts that saw anything, whose loads do not wait for each
// other.
template <int DT, int E, int WAVES>
__device__ __forceinline__ void join_row(const Join& a, int64_t at, const int (&parts)[2])
{
    typedef float f32xE __attribute__((ext_vector_type(E)));
    __shared__ float red_o[WAVES > 1 ? WAVES : 1][WAVES > 1 ? 64 * E : 1];
    __shared__ float red_t[WAVES];
    const int lane = threadIdx.x & 63;
    const int wave = WAVES > 1 ? __builtin_amdgcn_readfirstlane(threadIdx.x >> 6) : 0;
    float top = -kInf;
    for (int s = 0; s < 2; ++s)
        for (int p = lane; p < parts[s]; p += 64)
            top = fmaxf(top, a.from[s].ms[(at * a.from[s].parts + p) * 2]);
#pragma unroll
    for (int d = 1; d < 64; d <<= 1)
        top = fmaxf(top, __shfl_xor(top, d));
    const bool mine = lane * E < a.dim;
    float total = 0.0f;
    f32xE o = {};
    for (int s = 0; s < 2; ++s) {
        const Source& f = a.from[s];
        for (int base = 0; base < parts[s]; base += 64) {
            float w = 0.0f, ps = 0.0f;
            if (base + lane < parts[s] && (WAVES == 1 || lane % WAVES == wave)) {
                const float* ms = f.ms + (at * f.parts + base + lane) * 2;
                ps = ms[1];
                w = part_factor(ms[0], ps, top);
            }
            uint64_t live = __ballot(!(ps == 0.0f));    // the others saw nothing: their sums were not written
            total += w * ps;
            const float* out = f.out + (at * f.parts + base) * a.dim + lane * E;
            while (live != 0) {
                f32xE x[8];
                float wp[8];
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const int p = live != 0 ? __builtin_ctzll(live) : 0;
                    wp[i] = live != 0 ? __builtin_bit_cast(float, __builtin_amdgcn_readlane(__builtin_bit_cast(int, w), p)) : 0.0f;
                    x[i] = f32xE{};
                    if (live != 0 && mine)
                        x[i] = *reinterpret_cast<const f32xE*>(out + (int64_t)p * a.dim);
                    live &= live - 1;
                }
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    o += wp[i] * x[i];
            }
        }
    }
#pragma unroll
    for (int d = 1; d < 64; d <<= 1)
        total += __shfl_xor(total, d);
    if constexpr (WAVES > 1) {
        *reinterpret_cast<f32xE*>(&red_o[wave][lane * E]) = o;
        if (lane == 0)
            red_t[wave] = total;
        __syncthreads();
        if (wave > 0)
            return;
        for (int w = 1; w < WAVES; ++w) {
            o += *reinterpret_cast<const f32xE*>(&red_o[w][lane * E]);
            total += red_t[w];
        }
    }
    if (!mine)
        return;
    uint16_t* const to = static_cast<uint16_t*>(a.out) + at * a.dim + lane * E;
    if constexpr (E == 1) {
        narrow_to<DT>(to, 0, total == 0.0f ? 0.0f : o[0] / total);
    } else {
#pragma unroll
        for (int e = 0; e < E; e += 2)
            reinterpret_cast<unsigned*>(to)[e / 2] = total == 0.0f ? 0u : narrow_pair<DT>(o[e] / total, o[e + 1] / total);
    }
}

constexpr int kJoinWaves = 4;

// A wave for each row's head, or (SPREAD) all four where there are few rows.  Bound
// by latency: 4 to 6 us for up to a thousand rows' heads, 9 for 4096 of a dozen parts.
template <int DT, bool SPREAD>
__global__ void __launch_bounds__(kJoinWaves * 64)
join_parts_kernel(Join a)
{
    const int64_t at = SPREAD ? (int64_t)blockIdx.x
                              : (int64_t)blockIdx.x * kJoinWaves + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    if (at >= (int64_t)a.rows * a.q_heads)
        return;
    const int64_t row = at / a.q_heads;
    int64_t first = 0, last = 0;
    if (a.starts != nullptr && (!sequence_of(a.starts, a.batch, a.rows, row, &first, &last) || row < last - a.max_new))
        return;
    int parts[2];
#pragma unroll
    for (int s = 0; s < 2; ++s) {
        const Source& f = a.from[s];
        parts[s] = f.parts;
        if (f.parts > 0 && f.starts != nullptr && !sequence_of(f.starts, f.batch, a.rows, row, &first, &last))
            parts[s] = 0;
    }
    constexpr int W = SPREAD ? kJoinWaves : 1;
    if (a.dim <= 64)
        join_row<DT, 1, W>(a, at, parts);
    else if (a.dim <= 128)
        join_row<DT, 2, W>(a, at, parts);
    else
        join_row<DT, 4, W>(a, at, parts);
}

}  // namespace gattn
