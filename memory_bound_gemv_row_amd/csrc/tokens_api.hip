// tokens_api.hip -- C ABI of the INT8 product of several tokens and of its
// activations' quantiser (declared in include/gemv_tokens.h): validation,
// geometry and launch.
#include "gemv_tokens.h"
#include "device_info.hpp"
#include "tokens_kernels.hpp"

#include <hip/hip_runtime.h>

#include <math.h>

namespace gtokens {
namespace {

bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

int element_bytes(int dtype) { return dtype == GEMV_F32 ? 4 : 2; }

// Waves and chunks per lane so that rows of up to 16384 elements stay in
// registers; a wave per row for the shortest, where a workgroup of four would
// leave most lanes without a chunk.
template <int DT>
const void* quantize_kernel(int N, int* waves)
{
    if (N <= 1024) {
        *waves = 1;
        return reinterpret_cast<const void*>(&quantize_tokens_kernel<DT, 1, 2>);
    }
    if (N <= 8192) {
        *waves = 4;
        return N <= 4096 ? reinterpret_cast<const void*>(&quantize_tokens_kernel<DT, 4, 2>)
                         : reinterpret_cast<const void*>(&quantize_tokens_kernel<DT, 4, 4>);
    }
    *waves = 8;
    return reinterpret_cast<const void*>(&quantize_tokens_kernel<DT, 8, 4>);
}

const void* quantize_kernel(int dtype, int N, int* waves)
{
    return dtype == GEMV_F32 ? quantize_kernel<kF32>(N, waves)
         : dtype == GEMV_F16 ? quantize_kernel<kF16>(N, waves)
                             : quantize_kernel<kBF16>(N, waves);
}

const void* quantize_elementwise(int dtype)
{
    return dtype == GEMV_F32 ? reinterpret_cast<const void*>(&quantize_tokens_elementwise<kF32>)
         : dtype == GEMV_F16 ? reinterpret_cast<const void*>(&quantize_tokens_elementwise<kF16>)
                             : reinterpret_cast<const void*>(&quantize_tokens_elementwise<kBF16>);
}

// ---- product
// A kernel for products of moderate size: its tile, its threads, and what a CU
// was measured to do with one of its workgroups (bytes of both operands per
// us, and us besides).
struct Tiling {
    int tokens, outputs, threads;
    double rate, overhead;
    const void* fn[3];   // by gemv_dtype
};

#define GTOKENS_STREAM(BT, BM, WT, WM, WK, C, S, RATE, OVERHEAD)                     \
    {BT, BM, WT * WM * WK * 64, RATE * 1e3, OVERHEAD,                                \
     {reinterpret_cast<const void*>(&gemm_q8_stream<kF32, BT, BM, WT, WM, WK, C, S>), \
      reinterpret_cast<const void*>(&gemm_q8_stream<kF16, BT, BM, WT, WM, WK, C, S>), \
      reinterpret_cast<const void*>(&gemm_q8_stream<kBF16, BT, BM, WT, WM, WK, C, S>)}}

#define GTOKENS_ANY(BT, BM, WT, WM, WK, C, RATE, OVERHEAD)                         \
    {BT, BM, WT * WM * WK * 64, RATE * 1e3, OVERHEAD,                              \
     {reinterpret_cast<const void*>(&gemm_q8_any<kF32, BT, BM, WT, WM, WK, C>),     \
      reinterpret_cast<const void*>(&gemm_q8_any<kF16, BT, BM, WT, WM, WK, C>),     \
      reinterpret_cast<const void*>(&gemm_q8_any<kBF16, BT, BM, WT, WM, WK, C>)}}

// Rates and overheads fitted to 28 shapes (1 to 3000 tokens, 1000 to 14336
// outputs, 1000 to 14336 columns) timed with each of these.
const Tiling kStream[] = {
    GTOKENS_STREAM(16, 16, 1, 1, 8, 512, 3, 126, 0.4), GTOKENS_STREAM(16, 32, 1, 2, 4, 512, 3, 112, 0.6),
    GTOKENS_STREAM(16, 64, 1, 4, 2, 512, 3, 116, 1.7), GTOKENS_STREAM(32, 16, 1, 1, 8, 512, 3, 128, 0.8),
    GTOKENS_STREAM(32, 32, 1, 2, 4, 256, 4, 99, 0.6),  GTOKENS_STREAM(32, 64, 1, 4, 2, 256, 3, 92, 0.6),
    GTOKENS_STREAM(64, 32, 2, 2, 2, 256, 4, 103, 2.1), GTOKENS_STREAM(64, 64, 2, 4, 1, 128, 5, 82, 0.9),
    GTOKENS_STREAM(128, 32, 4, 1, 2, 256, 3, 123, 3.3), GTOKENS_STREAM(128, 64, 4, 2, 1, 128, 3, 87, 2.5),
    GTOKENS_STREAM(128, 128, 4, 4, 1, 128, 4, 90, 4.3),
};

const Tiling kAny[] = {
    GTOKENS_ANY(16, 16, 1, 1, 8, 512, 126, 0.4),
    GTOKENS_ANY(32, 32, 1, 2, 4, 256, 99, 0.6),
    GTOKENS_ANY(64, 64, 2, 4, 1, 128, 82, 0.9),
    GTOKENS_ANY(128, 128, 4, 4, 1, 128, 90, 4.3),
};

// The tiling whose estimate is least: what the busiest CU moves at its rate,
// or reading A once from memory at 6 TB/s, joined as a root of squares since
// neither hides the other fully.  Within 1.9 % of the fastest on average over
// the shapes above.
template <int K>
const Tiling* pick(const Tiling (&all)[K], int T, int M, int N, int cus)
{
    const Tiling* best = nullptr;
    double least = 0.0;
    for (const Tiling& t : all) {
        const double tiles = ceil((double)T / t.tokens) * ceil((double)M / t.outputs);
        const double own = ceil(tiles / cus) * ((double)(t.tokens + t.outputs) * N / t.rate + t.overhead);
        const double memory = (double)M * N / 6e6, us2 = own * own + memory * memory;
        if (best == nullptr || us2 < least) {
            best = &t;
            least = us2;
        }
    }
    return best;
}

template <int DT>
const void* tiles_kernel() { return reinterpret_cast<const void*>(&gemm_q8_tiles<DT>); }

bool known(int dtype) { return dtype == GEMV_F32 || dtype == GEMV_F16 || dtype == GEMV_BF16; }

}  // namespace
}  // namespace gtokens

extern "C" {

int gemv_quantize_tokens_q8(const void* x, int dtype, int64_t stride, int8_t* q, float* scale, int T, int N,
                            hipStream_t stream)
{
    using namespace gtokens;
    if (T < 0 || N < 0 || stride < N || !known(dtype))
        return GEMV_E_INVAL;
    if (T == 0)
        return GEMV_OK;
    if (scale == nullptr || (N > 0 && (x == nullptr || q == nullptr)))
        return GEMV_E_INVAL;
    gemv_device::Device dev{};
    if (int rc = gemv_device::current(&dev); rc != GEMV_OK)
        return rc;
    const int per16 = 16 / element_bytes(dtype);
    const bool wide = N >= 8 && N % 8 == 0 && aligned(x, 16) && stride % per16 == 0 && aligned(q, 8);
    int waves = 4;
    const void* fn = wide ? quantize_kernel(dtype, N, &waves) : quantize_elementwise(dtype);
    void* args[] = {(void*)&x, (void*)&stride, (void*)&q, (void*)&scale, (void*)&T, (void*)&N};
    const int grid = gemv_device::capped_grid(T, waves * 64);
    return hipLaunchKernel(fn, dim3(grid), dim3(waves * 64), args, 0, stream) == hipSuccess ? GEMV_OK : GEMV_E_LAUNCH;
}

int gemv_gemm_q8(const int8_t* A, const uint16_t* scale, const int8_t* x, const float* x_scale, void* y, int dtype,
                 int T, int M, int N, hipStream_t stream)
{
    using namespace gtokens;
    if (T < 0 || M < 0 || N < 0 || !known(dtype))
        return GEMV_E_INVAL;
    if (N > 131071)
        return GEMV_E_UNSUPPORTED;
    if (T == 0 || M == 0)
        return GEMV_OK;
    if (scale == nullptr || x_scale == nullptr || y == nullptr || (N > 0 && (A == nullptr || x == nullptr)))
        return GEMV_E_INVAL;
    gemv_device::Device dev{};
    if (int rc = gemv_device::current(&dev); rc != GEMV_OK)
        return rc;
    auto launch = [&](const void* fn, int64_t grid, int block, void** args) {
        if (grid > gemv_device::kMaxWorkItems / block)
            return (int)GEMV_E_UNSUPPORTED;
        return (int)(hipLaunchKernel(fn, dim3((unsigned)grid), dim3(block), args, 0, stream) == hipSuccess
                         ? GEMV_OK
                         : GEMV_E_LAUNCH);
    };
    auto tiles = [](int n, int size) { return ((int64_t)n + size - 1) / size; };
    const bool wide = N >= 16 && N % 16 == 0 && aligned(A, 16) && aligned(x, 16);
    int tiles_t = (int)tiles(T, 256), tiles_m = (int)tiles(M, 256);
    const int64_t large = (int64_t)tiles_t * tiles_m;
    // tiles of 256 x 256 once they occupy three quarters of the CUs (192 of
    // them, 1500 x 8192 x 2048: 38.3 us against 41.3 in tiles of 128 x 128; 128 of
    // them, 2048 x 4096 x 4096: 52 against 45)
    if (wide && large >= dev.cus * 3 / 4) {
        // what is left after whole rounds of the CUs, if at most half a round, in halves
        const int64_t left = large % dev.cus;
        const int64_t halved = large > dev.cus && left <= dev.cus / 2 ? left : 0;
        if (large > gemv_device::kMaxWorkItems / 2048)
            return GEMV_E_UNSUPPORTED;
        int whole = (int)(large - halved);
        void* args[] = {(void*)&A, (void*)&scale, (void*)&x, (void*)&x_scale, (void*)&y, (void*)&T, (void*)&M, (void*)&N,
                        (void*)&tiles_t, (void*)&tiles_m, (void*)&whole};
        static const void* const fn[] = {tiles_kernel<kF32>(), tiles_kernel<kF16>(), tiles_kernel<kBF16>()};
        return launch(fn[dtype], whole + 2 * halved, 1024, args);
    }
    const Tiling* t = wide ? pick(kStream, T, M, N, dev.cus) : pick(kAny, T, M, N, dev.cus);
    tiles_t = (int)tiles(T, t->tokens);
    void* args[] = {(void*)&A, (void*)&scale, (void*)&x, (void*)&x_scale, (void*)&y, (void*)&T, (void*)&M, (void*)&N,
                    (void*)&tiles_t};
    return launch(t->fn[dtype], tiles_t * tiles(M, t->outputs), t->threads, args);
}

}  // extern "C"
