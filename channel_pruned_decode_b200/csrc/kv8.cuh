// Conversions of the paged 8-bit cache's codes.
#pragma once

#include <cuda_fp16.h>

#include "spark_internal.cuh"

namespace spark {

// Largest code value: 448 = 1.75 * 2^8, 127 = 1.984375 * 2^6.
template <int kType> struct Kv8;
template <> struct Kv8<SPARK_KV8_E4M3> {
    static constexpr int kTopExp = 8;
    static constexpr uint32_t kTopMant = 0x600000u;  // mantissa bits of 1.75f
};
template <> struct Kv8<SPARK_KV8_I8> {
    static constexpr int kTopExp = 6;
    static constexpr uint32_t kTopMant = 0x7e0000u;  // mantissa bits of 1.984375f
};

constexpr int kKv8MinExp = -126, kKv8MaxExp = 120;

// Smallest E in range with a <= M 2^E, from a's bits: a = m 2^e with m in
// [1, 2), so E = e - kTopExp, one more where m is above M's own mantissa.
template <int kType> __device__ __forceinline__ int kv8_exponent(float a) {
    const uint32_t u = __float_as_uint(a);
    const int e = (int)(u >> 23) - 127 - Kv8<kType>::kTopExp + ((u & 0x7fffffu) > Kv8<kType>::kTopMant ? 1 : 0);
    return min(max(e, kKv8MinExp), kKv8MaxExp);  // subnormal a (and 0) are below the range
}

__device__ __forceinline__ float exp2_int(int e) { return __int_as_float((e + 127) << 23); }  // -126 <= e <= 127

// Two codes (a in the low byte): round to nearest even, largest code beyond the range.
template <int kType> __device__ __forceinline__ uint32_t kv8_encode2(float a, float b) {
    if (kType == SPARK_KV8_E4M3) {
        uint16_t r;
        asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(b), "f"(a));
        return r;
    }
    const int x = min(max(__float2int_rn(a), -127), 127), y = min(max(__float2int_rn(b), -127), 127);
    return (uint32_t)(x & 0xff) | ((uint32_t)(y & 0xff) << 8);
}

// The values of two codes (low byte first), exact in fp16.
template <int kType> __device__ __forceinline__ __half2 kv8_decode2(uint32_t two) {
    uint32_t r;
    if (kType == SPARK_KV8_E4M3) {
        asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"((uint16_t)two));
        return *reinterpret_cast<__half2 *>(&r);
    }
    return __floats2half2_rn((float)(int8_t)(two & 0xff), (float)(int8_t)((two >> 8) & 0xff));
}

// ---------------------------------------------------- programmatic launches
// The calls of a serving step follow one another on a stream, and the smaller
// ones take less time than a launch.  These kernels are launched so that one may
// be set up while the one ahead of it ends; each touches no global memory before
// wait_for_prior_kernel().  What it then reads may have been written while it was
// already resident, so such data is read with plain loads, never as read-only
// (no __ldg, no const __restrict__).
__device__ __forceinline__ void wait_for_prior_kernel() {
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    asm volatile("griddepcontrol.wait;" ::: "memory");
}

template <typename... K, typename... A>
inline cudaError_t launch_after_prior(void (*kernel)(K...), unsigned grid, unsigned block, size_t smem,
                                      cudaStream_t st, A... args) {
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(grid);
    cfg.blockDim = dim3(block);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, static_cast<K>(args)...);
}

}  // namespace spark
