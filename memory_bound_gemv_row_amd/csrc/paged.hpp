// paged.hpp -- device code that the kernels over a paged key-value cache share:
// where slots lie, loads that need no branch, and 16-bit elements.
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

// Where the rows of sequence b begin, of `rows` in all.
__device__ __forceinline__ int64_t row_start(const int32_t* starts, int b, int rows)
{
    const int s = starts[b];
    return s < 0 ? 0 : (s < rows ? s : rows);
}

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

// What brings a part's sums to the common maximum `top`.  An empty part has
// maximum -inf and sum 0; one whose sum is NaN under a maximum of -inf stays NaN.
__device__ __forceinline__ float part_factor(float m, float s, float top)
{
    return m == -kInf ? (s == 0.0f ? 0.0f : 1.0f) : exp2_hw(m - top);
}

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

}  // namespace gattn
