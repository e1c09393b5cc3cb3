// tokens_kernels.hpp -- gfx950 (CDNA4) device code for the INT8 product of
// several tokens and the quantiser of its activations.
//
//   s_t = max_j |x_tj| / 127,  q_tj = round(x_tj / s_t)
//   y_ti = (sum_j q_tj A_ij) * (s_t * scale_i)
//
// Up to some hundred tokens the product is bound by reading A, beyond by the
// matrix units, which this card feeds at a clock that falls with their load
// (1.45 to 1.55 GHz at 8192 x 8192 x 8192, by the card; the matrix units busy
// 64 % of it).  Reached back to back in a captured graph, where two figures
// stand on two cards (tokens x outputs x inner): 1 x 4096 x 4096 5.1 us; 24 x 14336
// x 4096 11.7 us, 5.1 TB/s; 777 x 4096 x 14336 60 and 66 us, 1535 and 1380 TOP/s;
// 4096 x 14336 x 4096 240 and 259 us, 2000 and 1860 TOP/s; 4096 x 4096 x 14336 212
// and 226 us, 2270 and 2130 TOP/s.
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

// Eight codes as bytes.  In the common case, that of an ordinary scale and no
// quotient at or beside a tie, x / step + 1.5 * 2^23 holds the rounded quotient
// in its low byte; the same remainders as above say whether this is the case,
// for all eight at once (one code at a time: 45 us for 8192 x 8192 of binary16,
// 13.8 for 777 x 14336).
__device__ __forceinline__ u32x2 codes8(const float (&v)[8], const Grid& g)
{
    constexpr float kMagic = 12582912.0f;
    unsigned t[8];
    float worst = 0.0f;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        const float sum = __builtin_fmaf(v[e], g.inverse, kMagic);
        const float r = __builtin_fmaf(kMagic - sum, g.step, v[e]);
        worst = fmaxf(worst, __builtin_fabsf(r));
        t[e] = bits(sum);
    }
    if (g.lift != 1.0f || worst >= 0.5f * g.step) {
#pragma unroll
        for (int e = 0; e < 8; ++e)
            t[e] = g.step > 0.0f ? (unsigned)code(v[e], g) : 0u;
    }
    // the low bytes of four, by byte selection: 0 to 3 from the second operand, 4 to 7 from the first
    auto four = [](unsigned a, unsigned b, unsigned c, unsigned d) {
        return __builtin_amdgcn_perm(__builtin_amdgcn_perm(d, c, 0x0C0C0400u), __builtin_amdgcn_perm(b, a, 0x0C0C0400u),
                                     0x05040100u);
    };
    return u32x2{four(t[0], t[1], t[2], t[3]), four(t[4], t[5], t[6], t[7])};
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

// Bound by memory (8192 x 8192 of binary16: 37 us, 5.4 TB/s read and written;
// 777 x 14336 of binary32: 11.2 us, 5.0 TB/s, 13 under a kernel trace), a single
// row by latency (4096 of binary16: 2.6 us).
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
                float v[8];
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    v[e] = held[k].at(e);
                out[c] = codes8(v, g);
            }
        }
    }
}

// Any N and alignment: a workgroup per row, element by element, read twice
// (8192 x 8191 of binary16: 123 us; 777 x 14335 of binary32: 40; a row of 4095: 6.0).
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

// ---------------------------------------------------------------- product, large
typedef __amdgpu_buffer_rsrc_t Buffer;
constexpr unsigned kNowhere = 0xFFFFFF00u;   // past every descriptor's end: such loads give zeros

__device__ __forceinline__ Buffer rows_buffer(const int8_t* p, int row, int rows, int tile, int N)
{
    const int64_t n = rows - row < tile ? rows - row : tile;
    return __builtin_amdgcn_make_buffer_rsrc(const_cast<int8_t*>(p) + (int64_t)row * N, 0, (int)(n > 0 ? n * N : 0),
                                             0x00027000);
}

// Sixteen bytes of each lane, from its offset in the descriptor to its place
// behind `to` (the same address for all lanes): straight to LDS.
__device__ __forceinline__ void load_to_lds([[maybe_unused]] Buffer from, [[maybe_unused]] unsigned offset,
                                            [[maybe_unused]] i32x4* to)
{
#ifdef __HIP_DEVICE_COMPILE__   // the host pass does not know this size
    __builtin_amdgcn_raw_ptr_buffer_load_lds(from, (__attribute__((address_space(3))) void*)to, 16, offset, 0, 0, 0);
#endif
}

// Workgroups k, k + 8, ... run on XCD k: the tile of workgroup i of n, such
// that each XCD takes a run of neighbouring ones.
__device__ __forceinline__ int tile_of(int i, int n)
{
    const int xcd = i & 7, share = n >> 3, more = n & 7;
    return xcd * share + (xcd < more ? xcd : more) + (i >> 3);
}

// One tile of BT tokens by BM outputs, from t0 and m0, by TW x MW waves, each
// a BT / TW by BM / MW part of it in 32 x 32 products.  128 columns of both
// operands at a time go straight from memory to LDS, 16 bytes a lane, into one
// of two buffers while the other is multiplied.  The memory pipe writes a
// wave's 64 pieces one after the other, so the pieces are put in their
// swizzled order (piece c of row r at c ^ (r / 2 % 8)) by choosing which piece a
// lane reads; rows past the end and columns past N read as zeros.
template <int DT, int BT, int BM, int TW, int MW>
__device__ __forceinline__ void
gemm_tile(const int8_t* __restrict__ A, const uint16_t* __restrict__ scale, const int8_t* __restrict__ x,
          const float* __restrict__ x_scale, void* __restrict__ y, int T, int M, int N, int t0, int m0,
          i32x4* even_x, i32x4* even_a, i32x4* odd_x, i32x4* odd_a)
{
    constexpr int kThreads = TW * MW * 64;
    constexpr int FT = BT / TW / 32, FM = BM / MW / 32;   // products of a wave
    constexpr int LX = BT * 8 / kThreads, LA = BM * 8 / kThreads;
    static_assert(LX > 0 && LA > 0 && FT > 0 && FM > 0, "every wave loads and multiplies");
    static_assert(kThreads / 8 % 16 == 0, "the swizzle repeats over the rounds of loads");
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const Buffer from_x = rows_buffer(x, t0, T, BT, N), from_a = rows_buffer(A, m0, M, BM, N);
    // piece s = i * kThreads + thread of a buffer: row s / 8, place s % 8
    unsigned off_x[LX], off_a[LA];
    const int row = threadIdx.x >> 3, piece = (threadIdx.x & 7) ^ ((row >> 1) & 7);
#pragma unroll
    for (int i = 0; i < LX; ++i)
        off_x[i] = (unsigned)((row + i * (kThreads / 8)) * N + piece * 16);
#pragma unroll
    for (int i = 0; i < LA; ++i)
        off_a[i] = (unsigned)((row + i * (kThreads / 8)) * N + piece * 16);

    auto fetch = [&](i32x4* to_x, i32x4* to_a, int k0) {
        const bool in = k0 + piece * 16 < N;
#pragma unroll
        for (int i = 0; i < LX; ++i)
            load_to_lds(from_x, in ? off_x[i] + k0 : kNowhere, to_x + i * kThreads + wave * 64);
#pragma unroll
        for (int i = 0; i < LA; ++i)
            load_to_lds(from_a, in ? off_a[i] + k0 : kNowhere, to_a + i * kThreads + wave * 64);
    };

    i32x16 acc[FT][FM];
#pragma unroll
    for (int i = 0; i < FT; ++i)
#pragma unroll
        for (int j = 0; j < FM; ++j)
            acc[i][j] = i32x16{};
    const int rx = (wave / MW) * (BT / TW) + (lane & 31), ra = (wave % MW) * (BM / MW) + (lane & 31);
    const int swizzle = ((lane & 31) >> 1) & 7;   // the same for every product: rows differ by multiples of 32

    // One step of 32 columns: its pieces are read while the step before is
    // multiplied.
    struct Step {
        i32x4 x[FT], a[FM];
    };
    auto read = [&](Step& f, const i32x4* lx, const i32x4* la, int k) {
        const int c = (2 * k + (lane >> 5)) ^ swizzle;
#pragma unroll
        for (int i = 0; i < FT; ++i)
            f.x[i] = lx[(rx + 32 * i) * 8 + c];
#pragma unroll
        for (int j = 0; j < FM; ++j)
            f.a[j] = la[(ra + 32 * j) * 8 + c];
        __builtin_amdgcn_sched_barrier(0);
    };
    auto multiply = [&](const Step& f) {
#pragma unroll
        for (int i = 0; i < FT; ++i)
#pragma unroll
            for (int j = 0; j < FM; ++j)
                acc[i][j] = __builtin_amdgcn_mfma_i32_32x32x32_i8(f.x[i], f.a[j], acc[i][j], 0, 0, 0);
        __builtin_amdgcn_sched_barrier(0);
    };
    // All of this wave's reads of the current buffer are in registers and its
    // pieces of the next one in LDS; after the barrier every wave's are.
    auto turn = [&] {
        __builtin_amdgcn_s_waitcnt(0x0070);   // vmcnt(0) and lgkmcnt(0)
        __syncthreads();
        __builtin_amdgcn_sched_barrier(0);
    };
    Step f, g;
    auto stage = [&](const i32x4* lx, const i32x4* la, i32x4* next_x, i32x4* next_a, int k0) {
        fetch(next_x, next_a, k0);
        __builtin_amdgcn_sched_barrier(0);
        read(g, lx, la, 1);
        multiply(f);
        read(f, lx, la, 2);
        multiply(g);
        read(g, lx, la, 3);
        multiply(f);
        turn();
        read(f, next_x, next_a, 0);
        multiply(g);
    };
    fetch(even_x, even_a, 0);
    turn();
    read(f, even_x, even_a, 0);
    for (int k0 = 0; k0 < N; k0 += 256) {
        stage(even_x, even_a, odd_x, odd_a, k0 + 128);
        stage(odd_x, odd_a, even_x, even_a, k0 + 256);
    }

#pragma unroll
    for (int j = 0; j < FM; ++j) {
        const int m = m0 + ra + 32 * j;
        if (m >= M)
            continue;
        const float s = half_value(scale[m]);
#pragma unroll
        for (int i = 0; i < FT; ++i)
#pragma unroll
            for (int r = 0; r < 16; ++r) {
                const int t = t0 + (wave / MW) * (BT / TW) + 32 * i + 8 * (r >> 2) + 4 * (lane >> 5) + (r & 3);
                if (t < T)
                    store<DT>(y, (int64_t)t * M + m, acc[i][j][r], x_scale[t], s);
            }
    }
}

// Preconditions (host): N % 16 == 0, N >= 16, A and x 16-byte aligned.
//
// Tiles of 256 x 256, one to a CU, by 16 waves of 64 x 64 (8 waves of 128 x 64
// read a quarter less LDS but were slower: 8192 x 8192 x 8192 in 507 against
// 482 us).  The first `whole` tiles are done so; the rest, where they are too
// few to fill the CUs once more, in halves of 128 outputs.  Each XCD takes its
// run of tiles in bands of four rows of tiles, so that what it has in flight
// at a time reads few different rows of either operand.
template <int DT>
__global__ void __launch_bounds__(1024)
gemm_q8_tiles(const int8_t* __restrict__ A, const uint16_t* __restrict__ scale, const int8_t* __restrict__ x,
              const float* __restrict__ x_scale, void* __restrict__ y, int T, int M, int N, int tiles_t, int tiles_m,
              int whole)
{
    __shared__ i32x4 even_x[256 * 8];
    __shared__ i32x4 even_a[256 * 8];
    __shared__ i32x4 odd_x[256 * 8];
    __shared__ i32x4 odd_a[256 * 8];
    const int i = blockIdx.x;
    const bool half = i >= whole;
    const int rest = half ? tile_of(i - whole, 2 * (tiles_t * tiles_m - whole)) : 0;
    const int at = half ? whole + (rest >> 1) : tile_of(i, whole);
    const int band = at / (4 * tiles_m), in_band = at - band * 4 * tiles_m;
    const int band_rows = tiles_t - band * 4 < 4 ? tiles_t - band * 4 : 4;
    const int t0 = (band * 4 + in_band % band_rows) * 256, m0 = in_band / band_rows * 256;
    if (!half)
        gemm_tile<DT, 256, 256, 4, 4>(A, scale, x, x_scale, y, T, M, N, t0, m0, even_x, even_a, odd_x, odd_a);
    else if (m0 + (rest & 1) * 128 < M)
        gemm_tile<DT, 256, 128, 4, 4>(A, scale, x, x_scale, y, T, M, N, t0, m0 + (rest & 1) * 128, even_x, even_a, odd_x,
                                      odd_a);
}

// ---------------------------------------------------------------- product, few tokens
// Waits until this wave's reads of LDS are in registers and all but its LEFT
// newest loads have come, then for the workgroup's other waves.  A barrier of
// its own kind: __syncthreads() would wait for every load.
template <int LEFT>
__device__ __forceinline__ void wait_and_meet()
{
    static_assert(LEFT >= 0 && LEFT < 64, "the counter has six bits");
    __builtin_amdgcn_sched_barrier(0);
    asm volatile("" ::: "memory");
    __builtin_amdgcn_s_waitcnt((LEFT & 15) | (LEFT >> 4) << 14 | 0x0070);   // vmcnt, lgkmcnt(0)
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
    __builtin_amdgcn_sched_barrier(0);
}

// Stores a tile's products, register r of acc[i][j] being token
// 4 (l / 16) + r and output l % 16 of its 16 x 16.  Where the waves along WK
// hold parts of the sums, they first meet in `sums` by integer atomics, whose
// order does not matter; no wave may still need that part of LDS.
template <int DT, int BT, int BM, int WT, int WM, int WK>
__device__ __forceinline__ void
store_tile(const i32x4 (&acc)[BT / WT / 16][BM / WM / 16], [[maybe_unused]] int* sums, const uint16_t* __restrict__ scale,
           const float* __restrict__ x_scale, void* __restrict__ y, int T, int M, int t0, int m0)
{
    constexpr int kThreads = WT * WM * WK * 64;
    constexpr int FT = BT / WT / 16, FM = BM / WM / 16;
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, low = lane & 15;
    const int wm = wave / WK % WM, wt = wave / WK / WM;
    if constexpr (WK == 1) {
#pragma unroll
        for (int j = 0; j < FM; ++j) {
            const int m = m0 + (wm * FM + j) * 16 + low;
            if (m >= M)
                continue;
            const float s = half_value(scale[m]);
#pragma unroll
            for (int i = 0; i < FT; ++i)
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    const int t = t0 + (wt * FT + i) * 16 + 4 * (lane >> 4) + r;
                    if (t < T)
                        store<DT>(y, (int64_t)t * M + m, acc[i][j][r], x_scale[t], s);
                }
        }
    } else {
        for (int i = threadIdx.x; i < BT * BM; i += kThreads)
            sums[i] = 0;
        __syncthreads();
#pragma unroll
        for (int i = 0; i < FT; ++i)
#pragma unroll
            for (int j = 0; j < FM; ++j)
#pragma unroll
                for (int r = 0; r < 4; ++r)
                    atomicAdd(&sums[((wt * FT + i) * 16 + 4 * (lane >> 4) + r) * BM + (wm * FM + j) * 16 + low],
                              acc[i][j][r]);
        __syncthreads();
        for (int i = threadIdx.x; i < BT * BM; i += kThreads) {
            const int t = t0 + i / BM, m = m0 + i % BM;
            if (t < T && m < M)
                store<DT>(y, (int64_t)t * M + m, sums[i], x_scale[t], half_value(scale[m]));
        }
    }
}

// Preconditions (host): N % 16 == 0, N >= 16, A and x 16-byte aligned.
//
// For products whose time is that of reading A: a workgroup of WT x WM x WK
// waves owns BT tokens by BM outputs, chosen so that the outputs fill the card,
// and keeps S - 1 stages of C columns of both operands on their way to LDS,
// whose S buffers it goes round.  Waves along WK take every WK-th step of 64
// columns.  Direct loads of the operands into registers, without LDS, read x as
// often as A: 24 x 14336 x 4096 in 16.4 us against 11.2.  v_mfma_i32_16x16x64_i8: lane l holds row (column) l % 16
// and columns 16 (l / 16) .. + 15 of the 64 summed; register r of its result
// is row 4 (l / 16) + r, column l % 16.
template <int DT, int BT, int BM, int WT, int WM, int WK, int C, int S>
__global__ void __launch_bounds__(WT * WM * WK * 64)
gemm_q8_stream(const int8_t* __restrict__ A, const uint16_t* __restrict__ scale, const int8_t* __restrict__ x,
               const float* __restrict__ x_scale, void* __restrict__ y, int T, int M, int N, int tiles_t)
{
    constexpr int kThreads = WT * WM * WK * 64;
    constexpr int FT = BT / WT / 16, FM = BM / WM / 16;
    constexpr int kRow = C / 16;                          // pieces of a row
    constexpr int kPieces = (BT + BM) * kRow, L = kPieces / kThreads;
    static_assert(kPieces % kThreads == 0 && kThreads % kRow == 0, "whole rounds of loads");
    static_assert(S >= 3 && S <= 5, "stages that there are buffers for");
    static_assert((kThreads / kRow) % 16 == 0, "the swizzle repeats over the rounds of loads");
    static_assert(BT % (kThreads / kRow) == 0, "a round loads rows of one operand");
    static_assert(WK == 1 || BT * BM * 4 <= kPieces * 16, "the sums fit one buffer");
    constexpr int kSteps = C / 64 / WK;
    // a buffer each, so that the compiler knows which of them a load fills
    __shared__ i32x4 b0[kPieces];
    __shared__ i32x4 b1[kPieces];
    __shared__ i32x4 b2[kPieces];
    __shared__ i32x4 b3[S > 3 ? kPieces : 1];
    __shared__ i32x4 b4[S > 4 ? kPieces : 1];
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int wk = wave % WK, wm = wave / WK % WM, wt = wave / WK / WM;
    const int at = tile_of(blockIdx.x, gridDim.x);
    const int t0 = at % tiles_t * BT, m0 = at / tiles_t * BM;
    const Buffer from_x = rows_buffer(x, t0, T, BT, N), from_a = rows_buffer(A, m0, M, BM, N);
    auto turned = [](int r) { return kRow >= 16 ? r & 15 : (r >> 1) & 7; };
    const int row = threadIdx.x / kRow, piece = (threadIdx.x % kRow) ^ turned(row);

    auto fetch = [&](i32x4* to, int k0) {
        const int k = k0 + piece * 16;
#pragma unroll
        for (int i = 0; i < L; ++i) {
            const int r = row + i * (kThreads / kRow);
            const bool of_x = i * (kThreads / kRow) < BT;
            const unsigned off = k < N ? (unsigned)((of_x ? r : r - BT) * N + k) : kNowhere;
            load_to_lds(of_x ? from_x : from_a, off, to + i * kThreads + wave * 64);
        }
        __builtin_amdgcn_sched_barrier(0);
    };
    i32x4 acc[FT][FM];
#pragma unroll
    for (int i = 0; i < FT; ++i)
#pragma unroll
        for (int j = 0; j < FM; ++j)
            acc[i][j] = i32x4{0, 0, 0, 0};
    const int low = lane & 15;
    auto multiply = [&](const i32x4* b) {
#pragma unroll
        for (int k = 0; k < kSteps; ++k) {
            const int c = (4 * (k * WK + wk) + (lane >> 4)) ^ turned(low);
            i32x4 vx[FT], va[FM];
#pragma unroll
            for (int j = 0; j < FM; ++j)
                va[j] = b[(BT + (wm * FM + j) * 16 + low) * kRow + c];
#pragma unroll
            for (int i = 0; i < FT; ++i)
                vx[i] = b[((wt * FT + i) * 16 + low) * kRow + c];
#pragma unroll
            for (int i = 0; i < FT; ++i)
#pragma unroll
                for (int j = 0; j < FM; ++j)
                    acc[i][j] = __builtin_amdgcn_mfma_i32_16x16x64_i8(vx[i], va[j], acc[i][j], 0, 0, 0);
        }
    };
    // this wave's pieces of the stage have come, then every wave's, and every
    // wave is done with the buffer that is filled next
    auto stage = [&](const i32x4* now, i32x4* next, int k0) {
        wait_and_meet<L * (S - 2)>();
        fetch(next, k0 + (S - 1) * C);
        multiply(now);
    };
    fetch(b0, 0);
    fetch(b1, C);
    if constexpr (S > 3) fetch(b2, 2 * C);
    if constexpr (S > 4) fetch(b3, 3 * C);
    i32x4* const last = S == 3 ? b2 : S == 4 ? b3 : b4;
    for (int k0 = 0; k0 < N; k0 += S * C) {
        stage(b0, last, k0);
        if (k0 + C >= N) break;
        stage(b1, b0, k0 + C);
        if (k0 + 2 * C >= N) break;
        stage(b2, b1, k0 + 2 * C);
        if constexpr (S > 3) { if (k0 + 3 * C >= N) break; stage(b3, b2, k0 + 3 * C); }
        if constexpr (S > 4) { if (k0 + 4 * C >= N) break; stage(b4, b3, k0 + 4 * C); }
    }
    // no load may still be on its way to LDS that is reused below, or by the
    // next workgroup
    wait_and_meet<0>();
    store_tile<DT, BT, BM, WT, WM, WK>(acc, reinterpret_cast<int*>(b0), scale, x_scale, y, T, M, t0, m0);
}

// Any size and alignment.  The same tiles, but rows of any alignment come
// through registers, two stages of C columns ahead, and are written to one of
// two buffers; columns past N are zeros there.  1 x 4096 x 4095: 8.4 us; 777 x
// 4096 x 14335: 114 us; 4096 x 4096 x 4095: 163 us, where the large tiles take 70 to
// 77 for 4096 columns: pieces of any alignment cannot go straight to LDS.
template <int DT, int BT, int BM, int WT, int WM, int WK, int C>
__global__ void __launch_bounds__(WT * WM * WK * 64)
gemm_q8_any(const int8_t* __restrict__ A, const uint16_t* __restrict__ scale, const int8_t* __restrict__ x,
            const float* __restrict__ x_scale, void* __restrict__ y, int T, int M, int N, int tiles_t)
{
    constexpr int kThreads = WT * WM * WK * 64;
    constexpr int FT = BT / WT / 16, FM = BM / WM / 16;
    constexpr int kRow = C / 16;
    constexpr int kPieces = (BT + BM) * kRow, L = kPieces / kThreads;
    static_assert(kPieces % kThreads == 0 && BT * kRow % kThreads == 0, "whole rounds of loads, each of one operand");
    static_assert(WK == 1 || BT * BM * 4 <= kPieces * 16, "the sums fit one buffer");
    constexpr int kSteps = C / 64 / WK;
    __shared__ i32x4 buffers[2][kPieces];
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int wk = wave % WK, wm = wave / WK % WM, wt = wave / WK / WM;
    const int at = tile_of(blockIdx.x, gridDim.x);
    const int t0 = at % tiles_t * BT, m0 = at / tiles_t * BM;
    auto turned = [](int r) { return kRow >= 16 ? r & 15 : (r >> 1) & 7; };

    struct Stage {
        i32x4 v[L];
    };
    auto fetch = [&](Stage& s, int k0) {
#pragma unroll
        for (int i = 0; i < L; ++i) {
            const int piece = i * kThreads + (int)threadIdx.x, r = piece / kRow, col = k0 + piece % kRow * 16;
            const bool of_x = i * kThreads < BT * kRow;
            s.v[i] = i32x4{0, 0, 0, 0};
            if (col < N)
                s.v[i] = of_x ? load16(x, t0 + r, T, col, N) : load16(A, m0 + r - BT, M, col, N);
        }
    };
    i32x4 acc[FT][FM];
#pragma unroll
    for (int i = 0; i < FT; ++i)
#pragma unroll
        for (int j = 0; j < FM; ++j)
            acc[i][j] = i32x4{0, 0, 0, 0};
    const int low = lane & 15;
    auto stage = [&](Stage& s, i32x4* b, int k0) {
#pragma unroll
        for (int i = 0; i < L; ++i) {
            const int piece = i * kThreads + (int)threadIdx.x, r = piece / kRow;
            b[r * kRow + ((piece % kRow) ^ turned(r))] = s.v[i];
        }
        __syncthreads();   // the other buffer was read before the barrier before this
        fetch(s, k0 + 2 * C);
#pragma unroll
        for (int k = 0; k < kSteps; ++k) {
            const int c = (4 * (k * WK + wk) + (lane >> 4)) ^ turned(low);
            i32x4 vx[FT], va[FM];
#pragma unroll
            for (int j = 0; j < FM; ++j)
                va[j] = b[(BT + (wm * FM + j) * 16 + low) * kRow + c];
#pragma unroll
            for (int i = 0; i < FT; ++i)
                vx[i] = b[((wt * FT + i) * 16 + low) * kRow + c];
#pragma unroll
            for (int i = 0; i < FT; ++i)
#pragma unroll
                for (int j = 0; j < FM; ++j)
                    acc[i][j] = __builtin_amdgcn_mfma_i32_16x16x64_i8(vx[i], va[j], acc[i][j], 0, 0, 0);
        }
    };
    Stage even, odd;
    fetch(even, 0);
    fetch(odd, C);
    for (int k0 = 0; k0 < N; k0 += 2 * C) {
        stage(even, buffers[0], k0);
        stage(odd, buffers[1], k0 + C);   // past N: zeros
    }
    __syncthreads();
    store_tile<DT, BT, BM, WT, WM, WK>(acc, reinterpret_cast<int*>(buffers[0]), scale, x_scale, y, T, M, t0, m0);
}

}  // namespace gtokens
