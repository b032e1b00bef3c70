// mx_act8.cuh -- device pieces shared by the norm and activation kernels:
// element access in bf16 / fp32, and the 8-bit checkpoint's group codec.
#pragma once
#include <cstdint>
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "mx_codec.cuh"
#include "mx_internal.cuh"

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

// Division of n < 2^31 by a d >= 1 known before the launch, by a multiplication
// (Granlund and Montgomery, "Division by Invariant Integers using
// Multiplication", 1994): with 2^s >= d and m = floor(2^32 (2^s - d) / d) + 1,
// n / d = (mulhi(n, m) + n) >> s; the sum stays below 2^32.
struct FastDiv {
    uint32_t d, m, s;
};
inline FastDiv fast_div(uint32_t d)
{
    uint32_t s = 0;
    while ((uint64_t{1} << s) < d)
        ++s;
    return {d, static_cast<uint32_t>((((uint64_t{1} << s) - d) << 32) / d + 1), s};
}
__device__ __forceinline__ uint32_t div_by(uint32_t n, const FastDiv& f) { return (__umulhi(n, f.m) + n) >> f.s; }

// ------------------------------------------------------ eight columns a thread
// 16 bytes of bf16 or 32 bytes of fp32, 16-byte aligned.  The loads stay before
// the stores that follow them in the source: an output may be an input's memory.
struct Oct {
    float v[8];
};

__device__ __forceinline__ void unpack_bf16x2(uint32_t w, float& lo, float& hi)
{
    lo = __uint_as_float(w << 16);
    hi = __uint_as_float(w & 0xFFFF0000u);
}
__device__ __forceinline__ void unpack_oct(uint4 w, Oct& o)
{
    unpack_bf16x2(w.x, o.v[0], o.v[1]);
    unpack_bf16x2(w.y, o.v[2], o.v[3]);
    unpack_bf16x2(w.z, o.v[4], o.v[5]);
    unpack_bf16x2(w.w, o.v[6], o.v[7]);
}
__device__ __forceinline__ uint32_t pack_bf16x2(float lo, float hi)
{
    const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&h);
}
__device__ __forceinline__ uint4 pack_oct(const Oct& o)
{
    return make_uint4(pack_bf16x2(o.v[0], o.v[1]), pack_bf16x2(o.v[2], o.v[3]), pack_bf16x2(o.v[4], o.v[5]),
                      pack_bf16x2(o.v[6], o.v[7]));
}

// The words of an oct as loaded, so that several loads can be in flight.
template <typename T>
struct RawOct;
template <>
struct RawOct<__nv_bfloat16> {
    uint4 w;
    __device__ __forceinline__ void load(const __nv_bfloat16* p)
    {
        asm volatile("ld.global.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
                     : "=r"(w.x), "=r"(w.y), "=r"(w.z), "=r"(w.w)
                     : "l"(p)
                     : "memory");
    }
    __device__ __forceinline__ void clear() { w = make_uint4(0, 0, 0, 0); }
    __device__ __forceinline__ void get(Oct& o) const { unpack_oct(w, o); }
};
template <>
struct RawOct<float> {
    float4 a, b;
    __device__ __forceinline__ void load(const float* p)
    {
        asm volatile("ld.global.L1::no_allocate.v4.f32 {%0, %1, %2, %3}, [%4];"
                     : "=f"(a.x), "=f"(a.y), "=f"(a.z), "=f"(a.w)
                     : "l"(p)
                     : "memory");
        asm volatile("ld.global.L1::no_allocate.v4.f32 {%0, %1, %2, %3}, [%4];"
                     : "=f"(b.x), "=f"(b.y), "=f"(b.z), "=f"(b.w)
                     : "l"(p + 4)
                     : "memory");
    }
    __device__ __forceinline__ void clear() { a = b = make_float4(0.0f, 0.0f, 0.0f, 0.0f); }
    __device__ __forceinline__ void get(Oct& o) const
    {
        o.v[0] = a.x, o.v[1] = a.y, o.v[2] = a.z, o.v[3] = a.w;
        o.v[4] = b.x, o.v[5] = b.y, o.v[6] = b.z, o.v[7] = b.w;
    }
};
__device__ __forceinline__ void decode_oct(uint2 w, float s, Oct& o)
{
    const float2 p = dec_e4m3x2(w.x & 0xFFFFu), q = dec_e4m3x2(w.x >> 16);
    const float2 t = dec_e4m3x2(w.y & 0xFFFFu), u = dec_e4m3x2(w.y >> 16);
    o.v[0] = p.x * s, o.v[1] = p.y * s, o.v[2] = q.x * s, o.v[3] = q.y * s;
    o.v[4] = t.x * s, o.v[5] = t.y * s, o.v[6] = u.x * s, o.v[7] = u.y * s;
}
// Eight checkpoint codes and their group's exponent byte.
struct RawCodes {
    uint2 w;
    uint32_t e;
    __device__ __forceinline__ void load(const Act8View& a, int64_t unit)  // unit: 8 columns
    {
        asm volatile("ld.global.L1::no_allocate.v2.u32 {%0, %1}, [%2];" : "=r"(w.x), "=r"(w.y) : "l"(a.codes + unit * 8) : "memory");
        e = a.sf[unit >> 2];
    }
    __device__ __forceinline__ void clear() { w = make_uint2(0, 0), e = 127; }
    __device__ __forceinline__ void get(Oct& o) const { decode_oct(w, act8_scale(e), o); }
};

// Asynchronous copies into a thread's own shared-memory words: no other thread
// reads them, so the thread's own wait is all the synchronisation they need.
__device__ __forceinline__ void copy_async16(uint32_t dst, const void* src)
{
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void copy_async8(uint32_t dst, const void* src)
{
    asm volatile("cp.async.ca.shared.global [%0], [%1], 8;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void copy_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
// All but the newest `pending` (0, 1 or 2) groups have arrived.
__device__ __forceinline__ void copy_wait(int pending)
{
    if (pending == 2)
        asm volatile("cp.async.wait_group 2;" ::: "memory");
    else if (pending == 1)
        asm volatile("cp.async.wait_group 1;" ::: "memory");
    else
        asm volatile("cp.async.wait_group 0;" ::: "memory");
}

// Writes an oct rounded to its type and folds |written values| into `top`:
// packed bf16 maxima (finish with oct_top), or fp32 bits.
__device__ __forceinline__ void store_oct(__nv_bfloat16* p, const Oct& o, uint32_t& top)
{
    const uint4 w = pack_oct(o);
    *reinterpret_cast<uint4*>(p) = w;
    top = __vmaxu2(top, w.x & 0x7FFF7FFFu);
    top = __vmaxu2(top, w.y & 0x7FFF7FFFu);
    top = __vmaxu2(top, w.z & 0x7FFF7FFFu);
    top = __vmaxu2(top, w.w & 0x7FFF7FFFu);
}
__device__ __forceinline__ void store_oct(float* p, const Oct& o, uint32_t& top)
{
    *reinterpret_cast<float4*>(p) = make_float4(o.v[0], o.v[1], o.v[2], o.v[3]);
    *reinterpret_cast<float4*>(p + 4) = make_float4(o.v[4], o.v[5], o.v[6], o.v[7]);
#pragma unroll
    for (int i = 0; i < 8; ++i)
        top = max(top, __float_as_uint(o.v[i]) & 0x7FFFFFFFu);
}
// One value of type T folded the same way.
template <typename T>
__device__ __forceinline__ void fold_top(uint32_t& top, float v)
{
    const uint32_t u = __float_as_uint(as_stored<T>(v)) & 0x7FFFFFFFu;
    top = sizeof(T) == 2 ? __vmaxu2(top, u >> 16) : max(top, u);
}
// The folded maximum as fp32 bits.
template <typename T>
__device__ __forceinline__ uint32_t oct_top(uint32_t top)
{
    return sizeof(T) == 2 ? max(top & 0xFFFFu, top >> 16) << 16 : top;
}

__device__ __forceinline__ float max_nan(float a, float b)
{
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
    return r;
}
__device__ __forceinline__ bool non_finite(float v) { return (__float_as_uint(v) & 0x7F800000u) == 0x7F800000u; }

// The checkpoint of a group that four consecutive lanes hold, eight columns
// each (0 past the row's end).  Executed by whole warps.  Groups without Inf
// and NaN take one maximum and one product per value; a warp that has one of
// the others repeats the maximum over the finite values.
__device__ __forceinline__ uint2 encode_oct(const Oct& o, int& e)
{
    float z[8], m = 0.0f;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        z[i] = o.v[i];
        m = max_nan(m, fabsf(z[i]));
    }
    m = max_nan(m, __shfl_xor_sync(0xFFFFFFFFu, m, 1));
    m = max_nan(m, __shfl_xor_sync(0xFFFFFFFFu, m, 2));
    if (__any_sync(0xFFFFFFFFu, non_finite(m))) {
        m = 0.0f;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            z[i] = finite_or_nan(z[i]);
            m = fmaxf(m, fabsf(z[i]));
        }
        m = fmaxf(m, __shfl_xor_sync(0xFFFFFFFFu, m, 1));
        m = fmaxf(m, __shfl_xor_sync(0xFFFFFFFFu, m, 2));
    }
    e = act8_exponent(m);
    const float s = exp2_neg(e);
    return make_uint2(cvt_e4m3x2(z[0] * s, z[1] * s) | cvt_e4m3x2(z[2] * s, z[3] * s) << 16,
                      cvt_e4m3x2(z[4] * s, z[5] * s) | cvt_e4m3x2(z[6] * s, z[7] * s) << 16);
}

// |v| as the bits that a maximum over unsigned words orders (NaN above all).
__device__ __forceinline__ uint32_t abs_bits(float v) { return __float_as_uint(v) & 0x7FFFFFFFu; }

}  // namespace mx
