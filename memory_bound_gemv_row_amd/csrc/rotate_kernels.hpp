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
// holds two pieces of eight elements of a head, such that its pairs are its own:
// the pieces at 8 u and rotated / 2 + 8 u, or at 16 u and 16 u + 8 where pairs
// are neighbours; both times its angles are 8 u .. 8 u + 7.  A head takes 1 to
// 16 lanes, a step 64 / lanes heads of a kind.  The angles of a row are taken
// once, one a lane, and meet the heads over LDS.
template <int IN, int OUT>
__global__ void __launch_bounds__(kWaves * 64)
rotate_kernel(Rotate a)
{
    typedef typename Elem<IN>::wide In;
    typedef typename Elem<OUT>::wide Out;
    __shared__ __attribute__((aligned(16))) float cosines[kWaves][kMaxDim / 2], sines[kWaves][kMaxDim / 2];
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int spans = (a.turns + a.span - 1) / a.span;
    const int64_t items = (int64_t)a.rows * spans;
    const int per = 64 / a.lanes;
    const int group = lane / a.lanes, unit = lane - group * a.lanes;
    const bool live = unit < a.units;

    // this lane's two pieces: elements first and second on, with angles or without
    int first, second;
    bool turned, second_turned;
    const int half = a.rotated / 2;
    if (a.interleaved) {
        first = 16 * unit;
        second = first + 8;
        turned = first < a.rotated;
        second_turned = second < a.rotated;
    } else if (8 * unit < half) {
        first = 8 * unit;
        second = half + first;
        turned = second_turned = true;
    } else {
        first = a.rotated + 16 * (unit - half / 8);
        second = first + 8;
        turned = second_turned = false;
    }
    const bool both = live && second < a.dim;

    f32x8 weight_first, weight_second;
    int weights_of = -1;
    for (int64_t item = (int64_t)blockIdx.x * kWaves + wave; item < items; item += (int64_t)gridDim.x * kWaves) {
        const int64_t row = spans == 1 ? item : item / spans;
        const int begin = (int)(item - row * spans) * a.span, end = begin + a.span < a.turns ? begin + a.span : a.turns;
        // a step's pieces are loaded while the step before is turned, the first ones behind the angles
        auto load = [&](int turn, f32x8& x, f32x8& y) {
            int head;
            const int kind = __builtin_amdgcn_readfirstlane(kind_at(a, turn, per, &head));
            head += group;
            const Heads& h = a.of[kind];
            const typename Elem<IN>::type* from = static_cast<const typename Elem<IN>::type*>(h.x) + row * h.stride + (int64_t)head * a.dim;
            x = y = f32x8{};
            if (live && head < h.heads)
                x = __builtin_convertvector(*reinterpret_cast<const In*>(from + first), f32x8);
            if (both && head < h.heads)
                y = __builtin_convertvector(*reinterpret_cast<const In*>(from + second), f32x8);
        };
        f32x8 x, y, next_x = {}, next_y = {};
        load(begin, x, y);
        const int position = a.positions[row];
        for (int i = lane; i < half; i += 64) {
            const float2 t = turn_of(position, a.freqs[i]);
            cosines[wave][i] = t.x;
            sines[wave][i] = t.y;
        }
        // a wave reads what it wrote itself: its writes are done once they are waited for
        __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
        __builtin_amdgcn_wave_barrier();
        f32x8 c = {}, s = {};
        if (live && turned) {
            c = *reinterpret_cast<const f32x8*>(&cosines[wave][8 * unit]);
            s = *reinterpret_cast<const f32x8*>(&sines[wave][8 * unit]);
        }
        for (int turn = begin; turn < end; ++turn) {
            int head;
            const int kind = __builtin_amdgcn_readfirstlane(kind_at(a, turn, per, &head));
            head += group;
            const Heads& h = a.of[kind];
            const bool mine = live && head < h.heads, mine_too = both && head < h.heads;
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
                    const float by = __builtin_amdgcn_rsqf(sum / (float)a.dim + a.eps);
                    x = x * by * weight_first;
                    y = y * by * weight_second;
                }
                if (a.interleaved) {
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        if (turned) {
                            const float p = x[2 * e], q = x[2 * e + 1];
                            x[2 * e] = p * c[e] - q * s[e];
                            x[2 * e + 1] = q * c[e] + p * s[e];
                        }
                        if (second_turned) {
                            const float p = y[2 * e], q = y[2 * e + 1];
                            y[2 * e] = p * c[4 + e] - q * s[4 + e];
                            y[2 * e + 1] = q * c[4 + e] + p * s[4 + e];
                        }
                    }
                } else if (turned) {
                    const f32x8 p = x, q = y;
                    x = p * c - q * s;
                    y = q * c + p * s;
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
            x = next_x;
            y = next_y;
        }
        __builtin_amdgcn_wave_barrier();   // the next row's angles come after this row's reads
    }
}

// Any size and alignment: a wave per head, a pair (or an element past the
// rotated ones) a lane at a time.
template <int IN, int OUT>
__global__ void __launch_bounds__(kWaves * 64)
rotate_elementwise(Rotate a)
{
    typedef typename Elem<IN>::type E;
    typedef typename Elem<OUT>::type O;
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int half = a.rotated / 2, singles = a.dim - a.rotated;
    for (int64_t item = (int64_t)blockIdx.x * kWaves + wave; item < (int64_t)a.rows * a.turns; item += (int64_t)gridDim.x * kWaves) {
        const int64_t row = item / a.turns;
        int head;
        const int kind = __builtin_amdgcn_readfirstlane(kind_at(a, (int)(item - row * a.turns), 1, &head));
        const Heads& h = a.of[kind];
        const E* from = static_cast<const E*>(h.x) + row * h.stride + (int64_t)head * a.dim;
        // pairs lane and lane + 64, singles lane, lane + 64, ... : at most 256 elements
        float p[2][2] = {}, single[4] = {};
        int at[2][2] = {};
        float sum = 0.0f;
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int n = lane + 64 * i;
            at[i][0] = a.interleaved ? 2 * n : n;
            at[i][1] = a.interleaved ? 2 * n + 1 : n + half;
            if (n < half)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    p[i][e] = (float)from[at[i][e]];
                    sum += p[i][e] * p[i][e];
                }
        }
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if (lane + 64 * i < singles) {
                single[i] = (float)from[a.rotated + lane + 64 * i];
                sum += single[i] * single[i];
            }
        float by = 1.0f;
        const bool normed = kind != kValue && a.norm;
        if (normed) {
#pragma unroll
            for (int d = 1; d < 64; d <<= 1)
                sum += __shfl_xor(sum, d);
            by = __builtin_amdgcn_rsqf(sum / (float)a.dim + a.eps);
        }
        auto scaled = [&](float x, int d) {
            return !normed ? x : h.weight != nullptr ? x * by * weight_at(h.weight, a.weight_dtype, d) : x * by;
        };
        int64_t head_stride;
        O* to = row_out<OUT>(a, kind, row, &head_stride);
        if (to == nullptr)
            continue;
        to += head * head_stride;
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int n = lane + 64 * i;
            if (n >= half)
                continue;
            float x = scaled(p[i][0], at[i][0]), y = scaled(p[i][1], at[i][1]);
            if (kind != kValue) {
                const float2 t = turn_of(a.positions[row], a.freqs[n]);
                const float u = x * t.x - y * t.y;
                y = y * t.x + x * t.y;
                x = u;
            }
            to[at[i][0]] = (O)x;
            to[at[i][1]] = (O)y;
        }
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if (lane + 64 * i < singles)
                to[a.rotated + lane + 64 * i] = (O)scaled(single[i], a.rotated + lane + 64 * i);
    }
}

}  // namespace grot
