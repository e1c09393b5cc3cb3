// tokens_kernels.hpp -- gfx950 (CDNA4) device code for the INT8 product of
// several tokens and the quantiser of its activations.
//
//   s_t = max_j |x_tj| / 127,  q_tj = round(x_tj / s_t)
//   y_ti = (sum_j q_tj A_ij) * (s_t * scale_i)
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace gtokens {

typedef unsigned int u32x2 __attribute__((ext_vector_type(2)));
typedef unsigned int u32x4 __attribute__((ext_vector_type(4)));
typedef int i32x4 __attribute__((ext_vector_type(4)));
typedef int i32x16 __attribute__((ext_vector_type(16)));

enum Type : int { kF32 = 0, kF16 = 1, kBF16 = 2 };

template <int DT> struct Elem;
template <> struct Elem<kF32> {
    typedef float type;
    static __device__ __forceinline__ float widen(float v) { return v; }
    static __device__ __forceinline__ float narrow(float v) { return v; }
};
template <> struct Elem<kF16> {
    typedef _Float16 type;
    static __device__ __forceinline__ float widen(_Float16 v) { return (float)v; }
    static __device__ __forceinline__ _Float16 narrow(float v) { return (_Float16)v; }
};
template <> struct Elem<kBF16> {
    typedef __bf16 type;
    static __device__ __forceinline__ float widen(__bf16 v) { return (float)v; }
    static __device__ __forceinline__ __bf16 narrow(float v) { return (__bf16)v; }
};

__device__ __forceinline__ unsigned bits(float v) { return __builtin_bit_cast(unsigned, v); }
__device__ __forceinline__ float from_bits(unsigned v) { return __builtin_bit_cast(float, v); }

// ---------------------------------------------------------------- quantiser
// The bits of |v| order finite magnitudes as whole numbers, with infinities
// and NaNs above all of them, so one integer maximum finds the row's largest
// magnitude and whether the row has a scale at all.
__device__ __forceinline__ unsigned magnitude(float v) { return bits(v) & 0x7FFFFFFFu; }

template <int CTRL>
__device__ __forceinline__ unsigned dpp_max(unsigned a)
{
    const unsigned b = (unsigned)__builtin_amdgcn_update_dpp(0, (int)a, CTRL, 0xF, 0xF, false);
    return a > b ? a : b;
}

__device__ __forceinline__ unsigned umax(unsigned a, unsigned b) { return a > b ? a : b; }

// Maximum over the 64 lanes, the same in each.
__device__ __forceinline__ unsigned wave_max(unsigned v)
{
    v = dpp_max<0xB1>(v);    // lane ^ 1
    v = dpp_max<0x4E>(v);    // lane ^ 2
    v = dpp_max<0x141>(v);   // other quad of the 8-lane half row
    v = dpp_max<0x140>(v);   // other half of the 16-lane row
    v = umax(v, (unsigned)__builtin_amdgcn_ds_swizzle((int)v, 0x401F));   // lane ^ 16 within 32
    return umax((unsigned)__builtin_amdgcn_readlane((int)v, 0), (unsigned)__builtin_amdgcn_readlane((int)v, 32));
}

// What a row's codes are made with: x * lift is compared with the grid of
// step `step` = scale * lift.  lift is 1 except for scales so small that
// their reciprocal is no finite binary32, where it is 2^64 (exact for both).
struct Grid {
    float scale, step, inverse, lift;
};

__device__ __forceinline__ Grid grid_for(unsigned top)
{
    Grid g;
    if (top >= 0x7F800000u) {
        g.scale = __builtin_nanf("");
        g.step = 0.0f;
        g.inverse = 0.0f;
        g.lift = 0.0f;
        return g;
    }
    g.scale = from_bits(top) / 127.0f;
    g.lift = g.scale < 0x1p-100f ? 0x1p64f : 1.0f;
    g.step = g.scale * g.lift;
    g.inverse = g.step > 0.0f ? 1.0f / g.step : 0.0f;
    return g;
}

// The nearest whole number to the exact quotient v / step, ties to even.  The
// reciprocal's product is off by a few parts in 2^24, so its rounding k is
// right or one off beside a tie; the remainder v - k step, in one fma, is
// exact wherever it is compared with half a step (both are whole multiples
// of step's last place, halved, and of at most 25 bits), and says which.
__device__ __forceinline__ int code(float v, const Grid& g)
{
    const float x = v * g.lift;
    const float k = __builtin_rintf(x * g.inverse);
    const float r = __builtin_fmaf(-k, g.step, x);
    const float half = 0.5f * g.step;
    int c = (int)k;
    if (__builtin_fabsf(r) >= half && g.step > 0.0f) {
        const int toward = r > 0.0f ? 1 : -1;
        if (__builtin_fabsf(r) > half || (c & 1))
            c += toward;
    }
    c = c > 127 ? 127 : c;
    return c < -127 ? -127 : c;
}

template <int DT>
struct Eight {   // eight consecutive elements as loaded
    u32x4 w[DT == kF32 ? 2 : 1];

    __device__ __forceinline__ void load(const void* p)
    {
        const u32x4* q = reinterpret_cast<const u32x4*>(p);
        w[0] = q[0];
        if constexpr (DT == kF32)
            w[1] = q[1];
    }
    __device__ __forceinline__ void clear()
    {
        w[0] = u32x4{0, 0, 0, 0};
        if constexpr (DT == kF32)
            w[1] = u32x4{0, 0, 0, 0};
    }
    __device__ __forceinline__ float at(int k) const
    {
        if constexpr (DT == kF32)
            return from_bits(w[k >> 2][k & 3]);
        const unsigned pair = w[0][k >> 1];
        if constexpr (DT == kBF16)
            return from_bits(k & 1 ? pair & 0xFFFF0000u : pair << 16);
        return (float)__builtin_bit_cast(_Float16, (unsigned short)(k & 1 ? pair >> 16 : pair));
    }
};

// Preconditions (host): N % 8 == 0, N >= 8, rows of x 16-byte aligned, rows
// of q 8-byte aligned.  A workgroup of W waves owns a row and walks the grid;
// rows of up to W * CH * 512 elements stay in registers between the maximum
// and the codes, longer ones are read twice (the second time from cache).
template <int DT, int W, int CH>
__global__ void __launch_bounds__(W * 64)
quantize_tokens_kernel(const void* __restrict__ x, int64_t stride, int8_t* __restrict__ q, float* __restrict__ scale,
                       int T, int N)
{
    typedef typename Elem<DT>::type E;
    __shared__ unsigned tops[W];
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int chunks = N >> 3;
    const bool resident = chunks <= W * 64 * CH;
    for (int64_t t = blockIdx.x; t < T; t += gridDim.x) {
        const E* row = static_cast<const E*>(x) + t * stride;
        Eight<DT> held[CH];
        unsigned top = 0;
        for (int base = 0; base < chunks; base += W * 64 * CH) {
#pragma unroll
            for (int k = 0; k < CH; ++k) {
                const int c = base + k * W * 64 + (int)threadIdx.x;
                if (c < chunks)
                    held[k].load(row + (int64_t)c * 8);
                else
                    held[k].clear();
            }
#pragma unroll
            for (int k = 0; k < CH; ++k)
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    top = umax(top, magnitude(held[k].at(e)));
        }
        top = wave_max(top);
        if constexpr (W > 1) {
            if ((threadIdx.x & 63) == 0)
                tops[wave] = top;
            __syncthreads();
            top = tops[0];
#pragma unroll
            for (int w = 1; w < W; ++w)
                top = umax(top, tops[w]);
            __syncthreads();   // the next row rewrites tops
        }
        const Grid g = grid_for(top);
        const bool zero = !(g.step > 0.0f);
        if (threadIdx.x == 0)
            scale[t] = g.scale;
        u32x2* out = reinterpret_cast<u32x2*>(q + t * N);
        for (int base = 0; base < chunks; base += W * 64 * CH) {
#pragma unroll
            for (int k = 0; k < CH; ++k) {
                const int c = base + k * W * 64 + (int)threadIdx.x;
                if (c >= chunks)
                    break;
                if (!resident)
                    held[k].load(row + (int64_t)c * 8);
                unsigned w[2] = {0, 0};
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    w[e >> 2] |= ((unsigned)code(held[k].at(e), g) & 0xFFu) << (8 * (e & 3));
                out[c] = zero ? u32x2{0, 0} : u32x2{w[0], w[1]};
            }
        }
    }
}

// Any N and alignment: a workgroup per row, element by element.
template <int DT>
__global__ void __launch_bounds__(256)
quantize_tokens_elementwise(const void* __restrict__ x, int64_t stride, int8_t* __restrict__ q,
                            float* __restrict__ scale, int T, int N)
{
    typedef typename Elem<DT>::type E;
    __shared__ unsigned tops[4];
    for (int64_t t = blockIdx.x; t < T; t += gridDim.x) {
        const E* row = static_cast<const E*>(x) + t * stride;
        unsigned top = 0;
        for (int64_t j = threadIdx.x; j < N; j += 256)
            top = umax(top, magnitude(Elem<DT>::widen(row[j])));
        top = wave_max(top);
        if ((threadIdx.x & 63) == 0)
            tops[threadIdx.x >> 6] = top;
        __syncthreads();
        top = umax(umax(tops[0], tops[1]), umax(tops[2], tops[3]));
        __syncthreads();
        const Grid g = grid_for(top);
        const bool zero = !(g.step > 0.0f);
        if (threadIdx.x == 0)
            scale[t] = g.scale;
        for (int64_t j = threadIdx.x; j < N; j += 256)
            q[t * N + j] = zero ? (int8_t)0 : (int8_t)code(Elem<DT>::widen(row[j]), g);
    }
}

// ---------------------------------------------------------------- product
// y = rn(float(sum) * (x_scale * scale)): the whole-number sum is exact, its
// conversion, the scales' product and their product each round once in
// binary32, the store once more to the output's type.
template <int DT>
__device__ __forceinline__ void store(void* y, int64_t at, int sum, float xs, float s)
{
    static_cast<typename Elem<DT>::type*>(y)[at] = Elem<DT>::narrow((float)sum * (xs * s));
}

__device__ __forceinline__ float half_value(uint16_t h) { return (float)__builtin_bit_cast(_Float16, h); }

// Sixteen bytes of row `row`, from column `col` on; zeros outside the matrix.
__device__ __forceinline__ i32x4 load16(const int8_t* p, int row, int rows, int col, int N)
{
    i32x4 v = {0, 0, 0, 0};
    if (row >= rows)
        return v;
    const int8_t* at = p + (int64_t)row * N + col;
    if (col + 16 <= N) {
        __builtin_memcpy(&v, at, 16);   // any alignment
    } else {
#pragma unroll
        for (int w = 0; w < 4; ++w) {
            unsigned u = 0;
#pragma unroll
            for (int b = 0; b < 4; ++b)
                if (col + 4 * w + b < N)
                    u |= ((unsigned)at[4 * w + b] & 0xFFu) << (8 * b);
            v[w] = (int)u;
        }
    }
    return v;
}

// Any size and alignment.  A workgroup of four waves owns 64 tokens by 64
// outputs, each wave a 32 x 32 quarter of it; 128 columns of both operands
// go through LDS at a time, loaded into registers while the step before is
// multiplied.  v_mfma_i32_32x32x32_i8: lane l holds row (column) l % 32 and 16
// of the 32 summed values; register r of its result is row
// 8 (r / 4) + 4 (l / 32) + r % 4, column l % 32.  A 16-byte chunk c of row r
// is kept at c ^ (r / 2 % 8), so that the 16 rows that one read phase takes
// lie in 16 different 16-byte columns of LDS.
template <int DT>
__global__ void __launch_bounds__(256)
gemm_q8_any(const int8_t* __restrict__ A, const uint16_t* __restrict__ scale, const int8_t* __restrict__ x,
            const float* __restrict__ x_scale, void* __restrict__ y, int T, int M, int N, int tiles_m)
{
    __shared__ i32x4 lx[64 * 8];
    __shared__ i32x4 la[64 * 8];
    const int lane = threadIdx.x & 63;
    const int wave = threadIdx.x >> 6;
    const int t0 = (int)(blockIdx.x / tiles_m) * 64;
    const int m0 = (int)(blockIdx.x % tiles_m) * 64;
    const int wt = (wave >> 1) * 32, wm = (wave & 1) * 32;
    i32x16 acc = {};
    i32x4 vx[2], va[2];
    auto fetch = [&](int k0) {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int s = (int)threadIdx.x + 256 * i;
            const int col = k0 + (s & 7) * 16;
            vx[i] = col < N ? load16(x, t0 + (s >> 3), T, col, N) : i32x4{0, 0, 0, 0};
            va[i] = col < N ? load16(A, m0 + (s >> 3), M, col, N) : i32x4{0, 0, 0, 0};
        }
    };
    fetch(0);
    for (int k0 = 0; k0 < N; k0 += 128) {
        __syncthreads();
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int s = (int)threadIdx.x + 256 * i;
            const int r = s >> 3, c = s & 7;
            lx[r * 8 + (c ^ ((r >> 1) & 7))] = vx[i];
            la[r * 8 + (c ^ ((r >> 1) & 7))] = va[i];
        }
        __syncthreads();
        if (k0 + 128 < N)
            fetch(k0 + 128);
        const int rx = wt + (lane & 31), ra = wm + (lane & 31);
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const int c = 2 * k + (lane >> 5);
            acc = __builtin_amdgcn_mfma_i32_32x32x32_i8(lx[rx * 8 + (c ^ ((rx >> 1) & 7))],
                                                        la[ra * 8 + (c ^ ((ra >> 1) & 7))], acc, 0, 0, 0);
        }
    }
    const int m = m0 + wm + (lane & 31);
    if (m >= M)
        return;
    const float s = half_value(scale[m]);
#pragma unroll
    for (int r = 0; r < 16; ++r) {
        const int t = t0 + wt + 8 * (r >> 2) + 4 * (lane >> 5) + (r & 3);
        if (t < T)
            store<DT>(y, (int64_t)t * M + m, acc[r], x_scale[t], s);
    }
}

}  // namespace gtokens
