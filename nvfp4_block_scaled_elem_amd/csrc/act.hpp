// Device-side helpers that the kernels share: barriers that order LDS alone, sums over a wave, and activations.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "launch.hpp"

namespace nvfp4 {

// A barrier that orders LDS alone: __syncthreads also waits until the work-group's stores to global memory have
// been acknowledged, which nothing here depends on.
__device__ __forceinline__ void lds_barrier() {
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "workgroup", "local");
    __builtin_amdgcn_s_barrier();
    __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "workgroup", "local");
}

// Between what a wave's lanes store in LDS and what other lanes of it load there, or store over it: the hardware keeps a
// wave's LDS accesses in order, this keeps the compiler from reordering them. No instruction.
__device__ __forceinline__ void wave_handover() {
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront", "local");
    __builtin_amdgcn_wave_barrier();
    __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront", "local");
}

// ------------------------------------------------------------------------------------- sums over a wave

// row_shr and row_bcast of the rows in MASK; 0 where there is no source.
template <int CTRL, int MASK>
__device__ __forceinline__ uint32_t shifted(uint32_t v) {
    return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, CTRL, MASK, 0xF, false);
}

// Inclusive sums over a wave: within rows of 16 lanes, then row 0's over row 1 and row 2's over row 3, then the first
// half's over the second.
template <typename T>
__device__ __forceinline__ T sums_to(T v) {
    v += __builtin_bit_cast(T, shifted<0x111, 0xF>(__builtin_bit_cast(uint32_t, v)));
    v += __builtin_bit_cast(T, shifted<0x112, 0xF>(__builtin_bit_cast(uint32_t, v)));
    v += __builtin_bit_cast(T, shifted<0x114, 0xF>(__builtin_bit_cast(uint32_t, v)));
    v += __builtin_bit_cast(T, shifted<0x118, 0xF>(__builtin_bit_cast(uint32_t, v)));
    v += __builtin_bit_cast(T, shifted<0x142, 0xA>(__builtin_bit_cast(uint32_t, v)));
    v += __builtin_bit_cast(T, shifted<0x143, 0xC>(__builtin_bit_cast(uint32_t, v)));
    return v;
}
template <typename T>
__device__ __forceinline__ T wave_sum(T v) {
    return __builtin_bit_cast(T, __builtin_amdgcn_readlane(__builtin_bit_cast(int, sums_to(v)), 63));
}

// ------------------------------------------------------------------------------------- activations

constexpr float kGelu2C = 1.5957691216057308f;  // 2 sqrt(2 / pi)
constexpr float kGeluA = 0.044715f;

// 1 / (1 + e^-v): the hardware exp2 and reciprocal, each within about one unit in the last place; v itself
// is rounded once more in v log2(e), a relative error of |v| 2^-24 in e^-v.
__device__ __forceinline__ float logistic(float v) {
    return __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(v * -1.4426950408889634f));
}

__device__ __forceinline__ float act_value(float z, int act) {
    if (act == kActSilu) return z * logistic(z);
    if (act == kActGelu) return z * logistic(kGelu2C * __builtin_fmaf(kGeluA * z * z, z, z));
    return z;
}

// act(z) and act'(z). The gelu's derivative is 0 or 1 to fp32 beyond |z| = 30; the clamp keeps z^2 finite. The clamp
// would take a NaN or an infinity for a number: z - z, 0 for every finite z, makes its slope the NaN that the formulas
// give (an infinity's is inf * 0).
__device__ __forceinline__ float2 act_both(float z, int act) {
    if (act == kActSilu) {
        const float s = logistic(z);
        return make_float2(z * s, s * __builtin_fmaf(z, 1.0f - s, 1.0f));
    }
    const float c = fminf(fmaxf(z, -30.0f), 30.0f);
    const float c2 = c * c;
    const float s = logistic(kGelu2C * __builtin_fmaf(kGeluA * c2, c, c));
    const float slope = __builtin_fmaf(c * s * (1.0f - s), kGelu2C * __builtin_fmaf(3.0f * kGeluA, c2, 1.0f), s);
    return make_float2(z * s, slope + (z - z));
}

}  // namespace nvfp4
