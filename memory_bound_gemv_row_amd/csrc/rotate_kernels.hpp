// rotate_kernels.hpp -- gfx950 (CDNA4) device code for the norms of queries and
// keys and their rotation by position, into tensors or into a paged cache.
//
// A head is read and written once, about ten operations for an element: bound
// by memory for a prompt, by the launch for a token.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace grot {

typedef unsigned int u32x4 __attribute__((ext_vector_type(4)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef float f32x8 __attribute__((ext_vector_type(8), aligned(16)));
typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));

enum Type : int { kF32 = 0, kF16 = 1, kBF16 = 2 };

template <int T>
struct Elem;
template <>
struct Elem<kF32> {
    typedef float type;
    typedef f32x8 wide;
};
template <>
struct Elem<kF16> {
    typedef _Float16 type;
    typedef f16x8 wide;
};
template <>
struct Elem<kBF16> {
    typedef __bf16 type;
    typedef bf16x8 wide;
};

constexpr int kMaxDim = 256;
constexpr int kWaves = 4;

// How the pairs of a head lie to the pieces of eight elements: halves of whole
// pieces, neighbours, and halves that end inside a piece.
enum Pairing : int { kHalves = 0, kNeighbours = 1, kLoose = 2 };

enum Kind : int { kQuery = 0, kKey = 1, kValue = 2 };

struct Heads {
    const void* x;
    int64_t stride;
    int heads;
    const void* weight;
    void* out;
    int64_t out_stride;
    int turns;   // steps of a wave that its heads take
};

struct Rotate {
    Heads of[3];             // queries, keys, values
    const int32_t* positions;
    int rows, dim, rotated;
    float per_element;       // 1 / dim
    bool interleaved, norm;
    float eps;
    const double* freqs;
    int weight_dtype;
    int units;               // pairs of pieces of a head
    int lanes;               // of a head: units, rounded up to a power of two
    int turns, span;         // steps of a row, and how many of them a wave takes
    // into a cache, where slots is not null:
    const int64_t* slots;
    int64_t pages, stride_page, stride_slot, stride_head;
    int page_size;
};

// cos and sin of position * freq.  The product and what is left of it past the
// nearest multiple of pi / 2 are formed in binary64 (pi / 2 in two parts); on
// [-pi/4, pi/4] the power series to r^9 and r^8 end below 2^-24.
__device__ __forceinline__ float2 turn_of(int position, double freq)
{
    const double t = (double)position * freq;
    const double n = rint(t * 0.63661977236758134308);
    const double left = fma(-n, 6.123233995736766e-17, fma(-n, 1.5707963267948966, t));
    const int quadrant = (int)(int64_t)n & 3;
    const float r = (float)left, z = r * r;
    const float s = r + r * z * (-1.0f / 6 + z * (1.0f / 120 + z * (-1.0f / 5040 + z * (1.0f / 362880))));
    const float c = 1.0f - 0.5f * z + z * z * (1.0f / 24 + z * (-1.0f / 720 + z * (1.0f / 40320)));
    const float x = quadrant & 1 ? s : c, y = quadrant & 1 ? c : s;
    return float2{quadrant == 1 || quadrant == 2 ? -x : x, quadrant >= 2 ? -y : y};
}

// sum over groups of `lanes` neighbouring lanes, 1 to 16, in every lane
__device__ __forceinline__ float group_sum(float v, int lanes)
{
    if (lanes > 1)
        v += __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, v), 0xB1, 0xF, 0xF, true));    // lane ^ 1
    if (lanes > 2)
        v += __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, v), 0x4E, 0xF, 0xF, true));    // lane ^ 2
    if (lanes > 4)
        v += __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, v), 0x141, 0xF, 0xF, true));   // 8 lanes mirrored
    if (lanes > 8)
        v += __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, v), 0x140, 0xF, 0xF, true));   // 16 lanes mirrored
    return v;
}

__device__ __forceinline__ float wave_sum(float v)
{
    const int s = __builtin_bit_cast(int, group_sum(v, 16));
    float total = 0.0f;
#pragma unroll
    for (int i = 0; i < 64; i += 16)
        total += __builtin_bit_cast(float, __builtin_amdgcn_readlane(s, i));
    return total;
}

__device__ __forceinline__ float weight_at(const void* w, int dtype, int d)
{
    return dtype == kF32 ? static_cast<const float*>(w)[d]
           : dtype == kF16 ? (float)static_cast<const _Float16*>(w)[d] : (float)static_cast<const __bf16*>(w)[d];
}

__device__ __forceinline__ f32x8 weights_at(const void* w, int dtype, int d)
{
    if (dtype == kF32)
        return *reinterpret_cast<const f32x8*>(static_cast<const float*>(w) + d);
    if (dtype == kF16)
        return __builtin_convertvector(*reinterpret_cast<const f16x8*>(static_cast<const _Float16*>(w) + d), f32x8);
    return __builtin_convertvector(*reinterpret_cast<const bf16x8*>(static_cast<const __bf16*>(w) + d), f32x8);
}

// Where a row's results of a kind begin; null where its slot is not in the cache.
template <int OUT>
__device__ __forceinline__ typename Elem<OUT>::type* row_out(const Rotate& a, int kind, int64_t row, int64_t* head_stride)
{
    typedef typename Elem<OUT>::type E;
    E* const out = static_cast<E*>(a.of[kind].out);
    *head_stride = a.dim;
    if (kind == kQuery || a.slots == nullptr)
        return out + row * a.of[kind].out_stride;
    *head_stride = a.stride_head;
    const int64_t slot = a.slots[row];
    if (slot < 0)
        return nullptr;
    const int64_t page = slot <= 0x7FFFFFFF ? (int64_t)((unsigned)slot / (unsigned)a.page_size) : slot / a.page_size;
    return page < a.pages ? out + page * a.stride_page + (slot - page * a.page_size) * a.stride_slot : nullptr;
}

// The heads' kind and first head at step `turn` of a row, `per` heads a step.
__device__ __forceinline__ int kind_at(const Rotate& a, int turn, int per, int* head)
{
    int kind = kQuery;
    if (turn >= a.of[kQuery].turns) {
        turn -= a.of[kQuery].turns;
        kind = kKey;
        if (turn >= a.of[kKey].turns) {
            turn -= a.of[kKey].turns;
            kind = kValue;
        }
    }
    *head = turn * per;
    return kind;
}

// A wave per row (or per `span` of its steps where there are few rows).  A lane
// holds two pieces of eight elements of a head.  With halves of whole pieces they
// are those at 8 u and rotated / 2 + 8 u, with neighbours as pairs those at 16 u
// and 16 u + 8: a lane's pairs are its own, and both times its angles are 8 u ..
// 8 u + 7.  Loose halves are held like neighbours, and each element's other half
// comes over LDS, with angles by element (3001 tokens of 40 + 8 + 8 heads of 80,
// 70 rotated: 19 us; with angles by pair, chosen per element, 37, for that leaves
// registers for two waves a SIMD).  A head takes 1 to 16 lanes, a step 64 / lanes
// heads of a kind.  The angles of a row are taken once, one a lane, and meet the
// heads over LDS.
//
// 8191 tokens of 32 + 8 + 8 heads of 128 (bfloat16) into a cache: 43.5 us, 4.6
// TB/s read and written, where a copy makes 4.95; one token 3.7 us.
template <int IN, int OUT, int PAIRING>
__global__ void __launch_bounds__(kWaves * 64)
rotate_kernel(Rotate a)
{
    typedef typename Elem<IN>::wide In;
    typedef typename Elem<OUT>::wide Out;
    // of loose halves, for each rotated element its pair's cosine and sine, with its own
    // sign, and each step's elements; a lane's sixteen words are followed by one more,
    // so that lanes meet in no bank
    constexpr int kApart = 17;
    constexpr int kAngles = PAIRING == kLoose ? kMaxDim / 16 * kApart : kMaxDim / 2;
    __shared__ __attribute__((aligned(16))) float cosines[kWaves][kAngles], sines[kWaves][kAngles];
    __shared__ float others[PAIRING == kLoose ? kWaves : 1][PAIRING == kLoose ? 64 * kApart : 1];
    auto word = [](int d) { return d / 16 * kApart + d % 16; };
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int spans = (a.turns + a.span - 1) / a.span;
    const int64_t items = (int64_t)a.rows * spans;
    const int per = 64 / a.lanes;
    const int group = lane / a.lanes, unit = lane - group * a.lanes;
    const bool live = unit < a.units;

    // this lane's two pieces: elements first and second on
    const int half = a.rotated / 2;
    int first = 16 * unit, second = first + 8;
    bool turned = PAIRING == kNeighbours && first < a.rotated;
    if constexpr (PAIRING == kHalves) {
        turned = 8 * unit < half;
        first = turned ? 8 * unit : a.rotated + 16 * (unit - half / 8);
        second = turned ? half + first : first + 8;
    }
    const bool both = live && second < a.dim;
    int other[PAIRING == kLoose ? 16 : 1];   // where each element's other half lies among the lane's head's
    unsigned rotates = 0;                    // bit per element
    if constexpr (PAIRING == kLoose) {
#pragma unroll
        for (int e = 0; e < 16; ++e) {
            const int d = first + e;
            other[e] = word(d < half ? d + half : d < a.rotated ? d - half : d);
            rotates |= (unsigned)(d < a.rotated) << e;
        }
    }

    f32x8 weight_first, weight_second;
    int weights_of = -1;
    for (int64_t item = (int64_t)blockIdx.x * kWaves + wave; item < items; item += (int64_t)gridDim.x * kWaves) {
        const int64_t row = spans == 1 ? item : item / spans;
        const int begin = (int)(item - row * spans) * a.span, end = begin + a.span < a.turns ? begin + a.span : a.turns;
        // a step's pieces are loaded while the step before is turned, the first ones behind the angles
        auto load = [&](int turn, In& x, In& y) {
            int head;
            const int kind = __builtin_amdgcn_readfirstlane(kind_at(a, turn, per, &head));
            head += group;
            const Heads& h = a.of[kind];
            const typename Elem<IN>::type* from = static_cast<const typename Elem<IN>::type*>(h.x) + row * h.stride + (int64_t)head * a.dim;
            x = y = In{};
            if (live && head < h.heads)
                x = *reinterpret_cast<const In*>(from + first);
            if (both && head < h.heads)
                y = *reinterpret_cast<const In*>(from + second);
        };
        In next_x, next_y;
        load(begin, next_x, next_y);
        const int position = a.positions[row];
        for (int i = lane; i < half; i += 64) {
            const float2 t = turn_of(position, a.freqs[i]);
            if constexpr (PAIRING == kLoose) {
                cosines[wave][word(i)] = cosines[wave][word(i + half)] = t.x;
                sines[wave][word(i)] = -t.y;
                sines[wave][word(i + half)] = t.y;
            } else {
                cosines[wave][i] = t.x;
                sines[wave][i] = t.y;
            }
        }
        // a wave reads what it wrote itself, and LDS takes its accesses in order
        __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
        __builtin_amdgcn_wave_barrier();
        f32x8 c = {}, s = {}, c_second = {}, s_second = {};
        if constexpr (PAIRING == kLoose) {
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                c[e] = cosines[wave][unit * kApart + e];
                s[e] = sines[wave][unit * kApart + e];
                c_second[e] = cosines[wave][unit * kApart + 8 + e];
                s_second[e] = sines[wave][unit * kApart + 8 + e];
            }
        } else if (live && turned) {
            c = *reinterpret_cast<const f32x8*>(&cosines[wave][8 * unit]);
            s = *reinterpret_cast<const f32x8*>(&sines[wave][8 * unit]);
        }
        for (int turn = begin; turn < end; ++turn) {
            int head;
            const int kind = __builtin_amdgcn_readfirstlane(kind_at(a, turn, per, &head));
            head += group;
            const Heads& h = a.of[kind];
            const bool mine = live && head < h.heads, mine_too = both && head < h.heads;
            f32x8 x = __builtin_convertvector(next_x, f32x8), y = __builtin_convertvector(next_y, f32x8);
            if (turn + 1 < end)
                load(turn + 1, next_x, next_y);
            if (kind != kValue) {
                if (a.norm) {
                    if (weights_of != kind) {
                        weights_of = kind;
                        weight_first = weight_second = f32x8{1, 1, 1, 1, 1, 1, 1, 1};
                        if (h.weight != nullptr && live)
                            weight_first = weights_at(h.weight, a.weight_dtype, first);
                        if (h.weight != nullptr && both)
                            weight_second = weights_at(h.weight, a.weight_dtype, second);
                    }
                    float sum = 0.0f;
#pragma unroll
                    for (int e = 0; e < 8; ++e)
                        sum += x[e] * x[e] + y[e] * y[e];
                    sum = group_sum(sum, a.lanes);
                    const float by = __builtin_amdgcn_rsqf(__builtin_fmaf(sum, a.per_element, a.eps));
                    x = x * by * weight_first;
                    y = y * by * weight_second;
                }
                if constexpr (PAIRING == kNeighbours) {
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        if (first + 2 * e < a.rotated) {
                            const float p = x[2 * e], q = x[2 * e + 1];
                            x[2 * e] = p * c[e] - q * s[e];
                            x[2 * e + 1] = q * c[e] + p * s[e];
                        }
                        if (second + 2 * e < a.rotated) {
                            const float p = y[2 * e], q = y[2 * e + 1];
                            y[2 * e] = p * c[4 + e] - q * s[4 + e];
                            y[2 * e + 1] = q * c[4 + e] + p * s[4 + e];
                        }
                    }
                } else if constexpr (PAIRING == kHalves) {
                    if (turned) {
                        const f32x8 p = x, q = y;
                        x = p * c - q * s;
                        y = q * c + p * s;
                    }
                } else {
                    float* const mine_all = &others[wave][group * a.lanes * kApart];
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        mine_all[unit * kApart + e] = x[e];
                        mine_all[unit * kApart + 8 + e] = y[e];
                    }
                    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
                    __builtin_amdgcn_wave_barrier();
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        const float p = mine_all[other[e]], q = mine_all[other[8 + e]];
                        x[e] = rotates >> e & 1 ? x[e] * c[e] + p * s[e] : x[e];
                        y[e] = rotates >> (8 + e) & 1 ? y[e] * c_second[e] + q * s_second[e] : y[e];
                    }
                    __builtin_amdgcn_wave_barrier();   // the next step's writes come after these reads
                }
            }
            int64_t head_stride;
            typename Elem<OUT>::type* to = row_out<OUT>(a, kind, row, &head_stride);
            if (to != nullptr) {
                to += head * head_stride;
                if (mine)
                    *reinterpret_cast<Out*>(to + first) = __builtin_convertvector(x, Out);
                if (mine_too)
                    *reinterpret_cast<Out*>(to + second) = __builtin_convertvector(y, Out);
            }
        }
        __builtin_amdgcn_wave_barrier();   // the next row's angles come after this row's reads
    }
}

// Any size and alignment: a wave takes one head after the other, a pair (or an
// element past the rotated ones) a lane at a time, so that a lane's angles are
// those of every head of the row.
template <int IN, int OUT>
__global__ void __launch_bounds__(kWaves * 64)
rotate_elementwise(Rotate a)
{
    typedef typename Elem<IN>::type E;
    typedef typename Elem<OUT>::type O;
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int spans = (a.turns + a.span - 1) / a.span;
    const int64_t items = (int64_t)a.rows * spans;
    const int half = a.rotated / 2, singles = a.dim - a.rotated;
    // elements of this lane: pairs lane and lane + 64, singles lane, lane + 64, ... : 256 in all
    int at[2][2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const int n = lane + 64 * i;
        at[i][0] = a.interleaved ? 2 * n : n;
        at[i][1] = a.interleaved ? 2 * n + 1 : n + half;
    }
    struct Head {
        E pair[2][2], single[4];
    };
    for (int64_t item = (int64_t)blockIdx.x * kWaves + wave; item < items; item += (int64_t)gridDim.x * kWaves) {
        const int64_t row = spans == 1 ? item : item / spans;
        const int begin = (int)(item - row * spans) * a.span, end = begin + a.span < a.turns ? begin + a.span : a.turns;
        auto load = [&](int turn, Head& x) {
            int head;
            const int kind = __builtin_amdgcn_readfirstlane(kind_at(a, turn, 1, &head));
            const Heads& h = a.of[kind];
            const E* from = static_cast<const E*>(h.x) + row * h.stride + (int64_t)head * a.dim;
#pragma unroll
            for (int i = 0; i < 2; ++i)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    x.pair[i][e] = E(0);
                    if (lane + 64 * i < half)
                        x.pair[i][e] = from[at[i][e]];
                }
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                x.single[i] = E(0);
                if (lane + 64 * i < singles)
                    x.single[i] = from[a.rotated + lane + 64 * i];
            }
        };
        Head next;
        load(begin, next);
        const int position = a.positions[row];
        float2 t[2] = {};
#pragma unroll
        for (int i = 0; i < 2; ++i)
            if (lane + 64 * i < half)
                t[i] = turn_of(position, a.freqs[lane + 64 * i]);
        for (int turn = begin; turn < end; ++turn) {
            int head;
            const int kind = __builtin_amdgcn_readfirstlane(kind_at(a, turn, 1, &head));
            const Heads& h = a.of[kind];
            const Head x = next;
            if (turn + 1 < end)
                load(turn + 1, next);
            const bool normed = kind != kValue && a.norm;
            float by = 1.0f;
            if (normed) {
                float sum = 0.0f;
#pragma unroll
                for (int i = 0; i < 2; ++i)
                    sum += (float)x.pair[i][0] * (float)x.pair[i][0] + (float)x.pair[i][1] * (float)x.pair[i][1];
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    sum += (float)x.single[i] * (float)x.single[i];
                sum = wave_sum(sum);
                by = __builtin_amdgcn_rsqf(__builtin_fmaf(sum, a.per_element, a.eps));
            }
            auto scaled = [&](E e, int d) {
                const float v = (float)e;
                return !normed ? v : h.weight != nullptr ? v * by * weight_at(h.weight, a.weight_dtype, d) : v * by;
            };
            int64_t head_stride;
            O* to = row_out<OUT>(a, kind, row, &head_stride);
            if (to == nullptr)
                continue;
            to += head * head_stride;
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                if (lane + 64 * i >= half)
                    continue;
                float p = scaled(x.pair[i][0], at[i][0]), q = scaled(x.pair[i][1], at[i][1]);
                if (kind != kValue) {
                    const float u = p * t[i].x - q * t[i].y;
                    q = q * t[i].x + p * t[i].y;
                    p = u;
                }
                to[at[i][0]] = (O)p;
                to[at[i][1]] = (O)q;
            }
#pragma unroll
            for (int i = 0; i < 4; ++i)
                if (lane + 64 * i < singles)
                    to[a.rotated + lane + 64 * i] = (O)scaled(x.single[i], a.rotated + lane + 64 * i);
        }
    }
}

}  // namespace grot
