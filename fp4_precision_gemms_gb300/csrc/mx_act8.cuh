// mx_act8.cuh -- device pieces shared by the norm and activation kernels:
// element access in bf16 / fp32, and the 8-bit checkpoint's group codec.
#pragma once
#include <cstdint>
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "mx_codec.cuh"

namespace mx {

constexpr int kAct8Group = 32;  // columns that share one scale byte
__host__ __device__ inline int64_t act8_groups(int64_t cols) { return (cols + kAct8Group - 1) / kAct8Group; }

__device__ __forceinline__ float load_f(const float* p) { return *p; }
__device__ __forceinline__ float load_f(const __nv_bfloat16* p) { return __bfloat162float(*p); }
__device__ __forceinline__ void store_f(float* p, float v) { *p = v; }
__device__ __forceinline__ void store_f(__nv_bfloat16* p, float v) { *p = __float2bfloat16_rn(v); }
// v as it reads back from a T
template <typename T>
__device__ __forceinline__ float as_stored(float v)
{
    if constexpr (sizeof(T) == 2)
        return __bfloat162float(__float2bfloat16_rn(v));
    return v;
}

// x where it is finite, NaN elsewhere (Inf * 0 is NaN); the sign of zero stays.
// fmaxf skips the NaN, so a group's maximum is that of its finite values, and
// the conversion turns it into the NaN code.
__device__ __forceinline__ float finite_or_nan(float x) { return fmaf(x, 0.0f, x); }

// Exponent of a group whose largest finite |x| is b, and 2^-e.
__device__ __forceinline__ int act8_exponent(float b) { return pow2_exponent<kElemE4M3>(b, MX_SCALE_CEIL); }

// Two E4M3 codes (low byte first) as floats; both conversions are exact.
__device__ __forceinline__ float2 dec_e4m3x2(uint32_t two)
{
    uint32_t h;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"(static_cast<uint16_t>(two)));
    return __half22float2(*reinterpret_cast<const __half2*>(&h));
}

// 2^(byte - 127)
__device__ __forceinline__ float act8_scale(uint32_t byte) { return exp2_neg(127 - static_cast<int>(byte)); }

// |v| as the bits that a maximum over unsigned words orders (NaN above all).
__device__ __forceinline__ uint32_t abs_bits(float v) { return __float_as_uint(v) & 0x7FFFFFFFu; }

}  // namespace mx
