// common.cuh -- small device helpers shared by the libssd kernels.
#pragma once

#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

namespace ssd {

// Device status word values (the first int32 of the workspace).
enum : int { kDevOk = 0, kDevTimeout = 5 };

// Lets `kernel` be launched with as much dynamic shared memory as a block can have
// beside `fixed` bytes of its own.  The limit is one number per kernel and device for
// the whole process, so it is the same number whatever a call needs: with each call's
// own size, another thread's smaller one could come between setting and launching.
template <typename... P>
inline cudaError_t allow_smem(void (*kernel)(P...), int fixed) {
    constexpr int block = 227 * 1024;
    return cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, block - fixed);
}

// Element loads/stores: every kernel computes in fp32.
__device__ __forceinline__ float to_f32(float v) { return v; }
__device__ __forceinline__ float to_f32(__nv_bfloat16 v) { return __bfloat162float(v); }
template <typename T> __device__ __forceinline__ T from_f32(float v);
template <> __device__ __forceinline__ float from_f32<float>(float v) { return v; }
template <> __device__ __forceinline__ __nv_bfloat16 from_f32<__nv_bfloat16>(float v) {
    return __float2bfloat16_rn(v);
}

// 2^x on the special-function unit (the hardware instruction, ~2^-22
// relative error; denormal results flush to zero)
__device__ __forceinline__ float ex2_approx(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// sum over the 32 lanes, returned in every lane
__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}

__device__ __forceinline__ float warp_inclusive_scan(float v) {
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        float u = __shfl_up_sync(0xffffffffu, v, o);
        if (lane >= o) v += u;
    }
    return v;
}

}  // namespace ssd
