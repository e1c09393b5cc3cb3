// tokens_api.hip -- C ABI of the INT8 product of several tokens and of its
// activations' quantiser (declared in include/gemv_tokens.h): validation,
// geometry and launch.
#include "gemv_tokens.h"
#include "device_info.hpp"
#include "tokens_kernels.hpp"

#include <hip/hip_runtime.h>

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
    const int64_t tiles_t = ((int64_t)T + 63) / 64, wide = ((int64_t)M + 63) / 64;
    if (tiles_t * wide > gemv_device::kMaxWorkItems / 256)
        return GEMV_E_UNSUPPORTED;
    int tiles_m = (int)wide;
    const void* fn = dtype == GEMV_F32 ? reinterpret_cast<const void*>(&gemm_q8_any<kF32>)
                   : dtype == GEMV_F16 ? reinterpret_cast<const void*>(&gemm_q8_any<kF16>)
                                       : reinterpret_cast<const void*>(&gemm_q8_any<kBF16>);
    void* args[] = {(void*)&A, (void*)&scale, (void*)&x, (void*)&x_scale, (void*)&y, (void*)&T, (void*)&M, (void*)&N,
                    (void*)&tiles_m};
    return hipLaunchKernel(fn, dim3((unsigned)(tiles_t * wide)), dim3(256), args, 0, stream) == hipSuccess
               ? GEMV_OK
               : GEMV_E_LAUNCH;
}

}  // extern "C"
