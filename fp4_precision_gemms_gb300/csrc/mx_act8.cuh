// mx_act8.cuh -- device pieces shared by the norm and activation kernels:
// element access in bf16 / fp32, and the 8-bit checkpoint's group codec.
#pragma once
#include <algorithm>
#include <cstdint>
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "mx_codec.cuh"
#include "mx_internal.cuh"

namespace mx {

// Programmatic dependent launch: a kernel launched early may start while the
// kernel before it in the stream still runs, and waits here for that kernel's
// end and its writes (nothing to wait for in an ordinary launch).  The kernel
// before says at its start that this may happen.
__device__ __forceinline__ void wait_for_launch_before() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
__device__ __forceinline__ void let_next_launch_start() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }

// `early`: the launch may overlap the end of the one before.
template <typename... P, typename... A>
int launch_kernel(void (*kernel)(P...), unsigned grid_x, unsigned grid_y, int threads, size_t smem, bool early, cudaStream_t s,
                  A... args)
{
    cudaLaunchConfig_t c = {};
    c.gridDim = dim3(grid_x, grid_y);
    c.blockDim = dim3(threads);
    c.dynamicSmemBytes = smem;
    c.stream = s;
    cudaLaunchAttribute attr;
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    c.attrs = &attr;
    c.numAttrs = early ? 1 : 0;
    count_launch();
    if (cudaLaunchKernelEx(&c, kernel, static_cast<P>(args)...) == cudaSuccess)
        return MX_OK;
    (void)cudaGetLastError();
    return MX_ERR_CUDA;
}
// Registers a thread of a kernel, and the CTAs of an SM that they allow.
template <auto KERNEL>
int registers_of()
{
    static const int n = [] {
        cudaFuncAttributes f = {};
        return cudaFuncGetAttributes(&f, KERNEL) == cudaSuccess ? f.numRegs : 128;
    }();
    return n;
}
template <auto KERNEL>
int resident_ctas(int threads)
{
    const int n = std::min(65536 / ((registers_of<KERNEL>() + 7) / 8 * 8 * threads), 2048 / threads);
    return std::max(1, std::min(32, n));
}

// Sets the word that flush_top folds into to zero (none: nothing is launched).
int launch_zero(unsigned* word, cudaStream_t s);

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

// Exponent byte e + 127 of a group whose largest finite |x| is b, the CEIL rule
// in four integer operations: 448 = 1.75 * 2^8, so e + 127 is b's exponent field
// less 8, and one more when its fraction is above 0.75, which is when adding
// 2^21 - 1 to it carries.  Subnormal b fall below the byte's lower end like the
// smallest normal ones; b = 0 has e = 0.
__device__ __forceinline__ uint32_t act8_byte(float b)
{
    const uint32_t u = __float_as_uint(b);
    const int byte = max(static_cast<int>((u + 0x1FFFFFu) >> 23) - 8, 0);
    return u == 0 ? 127u : static_cast<uint32_t>(byte);
}
// 2^-e = 2^(127 - byte), for the bytes that act8_byte gives (0 to 247)
__device__ __forceinline__ float act8_inverse(uint32_t byte) { return __uint_as_float((254u - byte) << 23); }

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
    float2 p[4];  // pairs, as the two-wide fp32 instructions take them
    __device__ __forceinline__ float& operator[](int i) { return i & 1 ? p[i >> 1].y : p[i >> 1].x; }
    __device__ __forceinline__ float operator[](int i) const { return i & 1 ? p[i >> 1].y : p[i >> 1].x; }
    __device__ __forceinline__ void fill(float v)
    {
#pragma unroll
        for (int k = 0; k < 4; ++k)
            p[k] = make_float2(v, v);
    }
};

__device__ __forceinline__ float2 unpack_bf16x2(uint32_t w)
{
    return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xFFFF0000u));
}
__device__ __forceinline__ void unpack_oct(uint4 w, Oct& o)
{
    o.p[0] = unpack_bf16x2(w.x);
    o.p[1] = unpack_bf16x2(w.y);
    o.p[2] = unpack_bf16x2(w.z);
    o.p[3] = unpack_bf16x2(w.w);
}
__device__ __forceinline__ uint32_t pack_bf16x2(float2 v)
{
    const __nv_bfloat162 h = __float22bfloat162_rn(v);
    return *reinterpret_cast<const uint32_t*>(&h);
}
__device__ __forceinline__ uint4 pack_oct(const Oct& o)
{
    return make_uint4(pack_bf16x2(o.p[0]), pack_bf16x2(o.p[1]), pack_bf16x2(o.p[2]), pack_bf16x2(o.p[3]));
}
__device__ __forceinline__ float2 both(float v) { return make_float2(v, v); }

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
        o.p[0] = make_float2(a.x, a.y), o.p[1] = make_float2(a.z, a.w);
        o.p[2] = make_float2(b.x, b.y), o.p[3] = make_float2(b.z, b.w);
    }
};
// The codes' own values; times 2^e they are the checkpoint's.
__device__ __forceinline__ void decode_oct(uint2 w, Oct& o)
{
    o.p[0] = dec_e4m3x2(w.x & 0xFFFFu), o.p[1] = dec_e4m3x2(w.x >> 16);
    o.p[2] = dec_e4m3x2(w.y & 0xFFFFu), o.p[3] = dec_e4m3x2(w.y >> 16);
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
    __device__ __forceinline__ void get(Oct& o, int = 8) const
    {
        decode_oct(w, o);
        const float2 s = both(act8_scale(e));
#pragma unroll
        for (int k = 0; k < 4; ++k)
            o.p[k] = __fmul2_rn(o.p[k], s);
    }
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

__device__ __forceinline__ float max_nan(float a, float b)
{
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
    return r;
}
__device__ __forceinline__ float max_nan(float a, float b, float c)
{
    float r;
    asm("max.NaN.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
    return r;
}
__device__ __forceinline__ float max_abs(float m, float2 v) { return max_nan(m, fabsf(v.x), fabsf(v.y)); }

// Running maximum of |written value|, NaN once there was one: two packed bf16
// maxima, or one of fp32.
template <typename T>
struct Top;
template <>
struct Top<__nv_bfloat16> {
    __nv_bfloat162 m = __float2bfloat162_rn(0.0f);
    __device__ __forceinline__ void word(uint32_t w)
    {
        m = __hmax2_nan(m, __habs2(*reinterpret_cast<const __nv_bfloat162*>(&w)));
    }
    __device__ __forceinline__ void value(float v) { word(pack_bf16x2(make_float2(v, 0.0f))); }
    __device__ __forceinline__ uint32_t bits() const
    {
        const uint32_t w = *reinterpret_cast<const uint32_t*>(&m) & 0x7FFF7FFFu;
        return max(w & 0xFFFFu, w >> 16) << 16;
    }
};
template <>
struct Top<float> {
    float m = 0.0f;
    __device__ __forceinline__ void pair(float2 v) { m = max_abs(m, v); }
    __device__ __forceinline__ void value(float v) { m = max_nan(m, fabsf(v)); }
    __device__ __forceinline__ uint32_t bits() const { return __float_as_uint(m) & 0x7FFFFFFFu; }
};
// Folds the CTA's maxima into *out, which the launch before this one sets to zero
// (launch_zero); a maximum does not depend on the order, and most warps find
// theirs already covered.
template <typename T>
__device__ __forceinline__ void flush_top(unsigned* out, const Top<T>& top)
{
    wait_for_launch_before();
    const uint32_t m = __reduce_max_sync(0xFFFFFFFFu, top.bits());
    if ((threadIdx.x & 31) == 0 && m > *static_cast<volatile unsigned*>(out))
        atomicMax(out, m);
}

// Writes an oct rounded to its type.
__device__ __forceinline__ void store_oct(__nv_bfloat16* p, const Oct& o, Top<__nv_bfloat16>& top)
{
    const uint4 w = pack_oct(o);
    *reinterpret_cast<uint4*>(p) = w;
    top.word(w.x), top.word(w.y), top.word(w.z), top.word(w.w);
}
__device__ __forceinline__ void store_oct(float* p, const Oct& o, Top<float>& top)
{
    *reinterpret_cast<float4*>(p) = make_float4(o.p[0].x, o.p[0].y, o.p[1].x, o.p[1].y);
    *reinterpret_cast<float4*>(p + 4) = make_float4(o.p[2].x, o.p[2].y, o.p[3].x, o.p[3].y);
    top.pair(o.p[0]), top.pair(o.p[1]), top.pair(o.p[2]), top.pair(o.p[3]);
}

// ------------------------------------------------------ rows at any address
// A row that does not start on a 16-byte boundary is still read and written in
// aligned 16-byte words: an oct lies in two of them (three of fp32) and is
// shifted into place, and on the way out each lane joins its neighbour's last
// values to its own.  Elements that share an aligned word with another warp's,
// and the row's ragged end, go one by one.
__device__ __forceinline__ int misaligned(const void* p, int bytes)  // elements past the boundary
{
    return static_cast<int>(reinterpret_cast<uintptr_t>(p) & 15) / bytes;
}

// Elements s .. s + 7 of the 16 bf16 in (lo, hi), s <= 7.
__device__ __forceinline__ uint4 shifted(uint4 lo, uint4 hi, int s)
{
    const uint32_t w[8] = {lo.x, lo.y, lo.z, lo.w, hi.x, hi.y, hi.z, hi.w};
    uint32_t a[6], b[5];
#pragma unroll
    for (int i = 0; i < 6; ++i)
        a[i] = s & 4 ? w[i + 2] : w[i];
#pragma unroll
    for (int i = 0; i < 5; ++i)
        b[i] = s & 2 ? a[i + 1] : a[i];
    const int bits = (s & 1) * 16;
    return make_uint4(__funnelshift_r(b[0], b[1], bits), __funnelshift_r(b[1], b[2], bits),
                      __funnelshift_r(b[2], b[3], bits), __funnelshift_r(b[3], b[4], bits));
}
// Words s .. s + 7 of the twelve in (x, y, z), s <= 3.
__device__ __forceinline__ void shifted(uint4 x, uint4 y, uint4 z, int s, uint4& lo, uint4& hi)
{
    const uint32_t w[12] = {x.x, x.y, x.z, x.w, y.x, y.y, y.z, y.w, z.x, z.y, z.z, z.w};
    uint32_t a[9], b[8];
#pragma unroll
    for (int i = 0; i < 9; ++i)
        a[i] = s & 2 ? w[i + 2] : w[i];
#pragma unroll
    for (int i = 0; i < 8; ++i)
        b[i] = s & 1 ? a[i + 1] : a[i];
    lo = make_uint4(b[0], b[1], b[2], b[3]);
    hi = make_uint4(b[4], b[5], b[6], b[7]);
}
__device__ __forceinline__ void words_to_oct(uint4 a, uint4 b, Oct& o)
{
    o.p[0] = make_float2(__uint_as_float(a.x), __uint_as_float(a.y));
    o.p[1] = make_float2(__uint_as_float(a.z), __uint_as_float(a.w));
    o.p[2] = make_float2(__uint_as_float(b.x), __uint_as_float(b.y));
    o.p[3] = make_float2(__uint_as_float(b.z), __uint_as_float(b.w));
}
// Zeros in place of what lies past the first n values.
__device__ __forceinline__ void keep_first(Oct& o, int n)
{
#pragma unroll
    for (int i = 0; i < 8; ++i)
        if (i >= n)
            o[i] = 0.0f;
}
__device__ __forceinline__ uint4 shfl_up1(uint4 v)
{
    return make_uint4(__shfl_up_sync(0xFFFFFFFFu, v.x, 1), __shfl_up_sync(0xFFFFFFFFu, v.y, 1),
                      __shfl_up_sync(0xFFFFFFFFu, v.z, 1), __shfl_up_sync(0xFFFFFFFFu, v.w, 1));
}

// Writes an oct (its first n values, n may be <= 0) at any address p; executed
// by whole warps.  prev / next: the neighbouring lane holds the oct before /
// after this one in the same row, the latter with at least one value.  With s
// elements between the aligned word and p, a lane's word holds the s last values
// of the lane before it and its own first 8 - s.
template <typename T, typename W>
__device__ __forceinline__ void store_rest(T* p, const W (&own)[8], const W (&left)[8], int n, int s, bool whole,
                                           bool prev, bool next)
{
    W* const to = reinterpret_cast<W*>(p);
    // one by one: the first 8 - s where no lane's word takes them, the last s
    // where the next lane does not
    const int from = whole ? 8 - s : 0, end = next ? min(n, 8 - s) : n;
#pragma unroll
    for (int i = 0; i < 8; ++i)
        if (i >= from && i < end)
            to[i] = own[i];
    if (!whole && prev && n > 0)  // a row's end that does not fill its word: the lane before leaves it its last s
#pragma unroll
        for (int i = 1; i < 8; ++i)
            if (i >= 8 - s)
                to[i - 8] = left[i];
}
// A warp whose 32 octs are whole and follow one another: every lane but the
// first writes its word, and eight lanes write the first lane's values before
// its word and the last lane's after it.
__device__ __forceinline__ bool whole_warp(int n, bool prev)
{
    return __all_sync(0xFFFFFFFFu, n == 8 && (prev || (threadIdx.x & 31) == 0));
}
__device__ __forceinline__ void store_ragged(__nv_bfloat16* p, Oct o, int n, bool prev, bool next, Top<__nv_bfloat16>& top)
{
    if (n < 8)
        keep_first(o, n);
    const uint4 own = pack_oct(o), left = shfl_up1(own);
    const int s = misaligned(p, 2);
    top.word(own.x), top.word(own.y), top.word(own.z), top.word(own.w);
    if (whole_warp(n, prev)) {
        const int lane = threadIdx.x & 31;
        if (s == 0) {
            *reinterpret_cast<uint4*>(p) = own;
            return;
        }
        if (lane > 0)
            *reinterpret_cast<uint4*>(p - s) = shifted(left, own, 8 - s);
        const int from = lane < 8 - s ? 0 : 31;  // lane i < 8: value i of lane 0, or of lane 31
        const uint32_t a = __shfl_sync(0xFFFFFFFFu, own.x, from), b = __shfl_sync(0xFFFFFFFFu, own.y, from);
        const uint32_t c = __shfl_sync(0xFFFFFFFFu, own.z, from), d = __shfl_sync(0xFFFFFFFFu, own.w, from);
        const uint32_t w = lane & 4 ? (lane & 2 ? d : c) : (lane & 2 ? b : a);
        if (lane < 8)
            reinterpret_cast<uint16_t*>(p - 8 * lane)[8 * from + lane] = static_cast<uint16_t>(w >> ((lane & 1) * 16));
        return;
    }
    const bool whole = n == 8 && (prev || s == 0);
    if (whole)
        *reinterpret_cast<uint4*>(p - s) = s == 0 ? own : shifted(left, own, 8 - s);
    if (!whole || (!next && s != 0)) {
        const uint32_t a[4] = {own.x, own.y, own.z, own.w}, b[4] = {left.x, left.y, left.z, left.w};
        uint16_t v[8], l[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            v[i] = static_cast<uint16_t>(a[i >> 1] >> ((i & 1) * 16));
            l[i] = static_cast<uint16_t>(b[i >> 1] >> ((i & 1) * 16));
        }
        store_rest(p, v, l, n, s, whole, prev, next);
    }
}
__device__ __forceinline__ void store_ragged(float* p, Oct o, int n, bool prev, bool next, Top<float>& top)
{
    if (n < 8)
        keep_first(o, n);
    const uint4 a = make_uint4(__float_as_uint(o.p[0].x), __float_as_uint(o.p[0].y), __float_as_uint(o.p[1].x),
                               __float_as_uint(o.p[1].y));
    const uint4 b = make_uint4(__float_as_uint(o.p[2].x), __float_as_uint(o.p[2].y), __float_as_uint(o.p[3].x),
                               __float_as_uint(o.p[3].y));
    const uint4 left = shfl_up1(b);
    const int s = misaligned(p, 4);
    top.pair(o.p[0]), top.pair(o.p[1]), top.pair(o.p[2]), top.pair(o.p[3]);
    if (whole_warp(n, prev)) {
        const int lane = threadIdx.x & 31;
        uint4 lo = a, hi = b;
        if (s != 0)
            shifted(left, a, b, 4 - s, lo, hi);
        if (lane > 0 || s == 0)
            reinterpret_cast<uint4*>(p - s)[0] = lo;
        reinterpret_cast<uint4*>(p - s)[1] = hi;
        if (s != 0) {  // lane i < 4: value i of lane 0, or value 4 + i of lane 31
            const bool head = lane < 4 - s;
            const uint32_t x = __shfl_sync(0xFFFFFFFFu, a.x, 0), y = __shfl_sync(0xFFFFFFFFu, a.y, 0);
            const uint32_t z = __shfl_sync(0xFFFFFFFFu, a.z, 0);
            const uint32_t u = __shfl_sync(0xFFFFFFFFu, b.y, 31), v = __shfl_sync(0xFFFFFFFFu, b.z, 31);
            const uint32_t w = __shfl_sync(0xFFFFFFFFu, b.w, 31);
            const uint32_t first = lane == 0 ? x : lane == 1 ? y : z, last = lane == 1 ? u : lane == 2 ? v : w;
            if (lane < 4)
                reinterpret_cast<uint32_t*>(p - 8 * lane)[head ? lane : 31 * 8 + 4 + lane] = head ? first : last;
        }
        return;
    }
    const bool whole = n == 8 && (prev || s == 0);
    if (whole) {
        uint4 lo = a, hi = b;
        if (s != 0)
            shifted(left, a, b, 4 - s, lo, hi);
        reinterpret_cast<uint4*>(p - s)[0] = lo;
        reinterpret_cast<uint4*>(p - s)[1] = hi;
    }
    if (!whole || (!next && s != 0)) {
        const uint32_t v[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w}, l[8] = {0, 0, 0, 0, left.x, left.y, left.z, left.w};
        store_rest(p, v, l, n, s, whole, prev, next);
    }
}

// 32 bytes at a multiple of 32: a whole sector in one access.
__device__ __forceinline__ void store_sector(uint8_t* to, const uint32_t (&w)[8])
{
    asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(to), "r"(w[0]), "r"(w[1]), "r"(w[2]), "r"(w[3]),
                 "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7])
                 : "memory");
}

__device__ __forceinline__ bool non_finite(float v) { return (__float_as_uint(v) & 0x7F800000u) == 0x7F800000u; }

// The checkpoint of a group that four consecutive lanes hold, eight columns
// each (0 past the row's end).  Executed by whole warps.  Groups without Inf
// and NaN take one maximum and one product per value; a warp that has one of
// the others repeats the maximum over the finite values.
__device__ __forceinline__ uint2 encode_oct(Oct z, uint8_t& byte)
{
    float m = max_abs(max_abs(max_abs(max_abs(0.0f, z.p[0]), z.p[1]), z.p[2]), z.p[3]);
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
    const uint32_t e = act8_byte(m);
    byte = static_cast<uint8_t>(e);
    const float2 s = both(act8_inverse(e));
#pragma unroll
    for (int k = 0; k < 4; ++k)
        z.p[k] = __fmul2_rn(z.p[k], s);
    return make_uint2(cvt_e4m3x2(z.p[0].x, z.p[0].y) | cvt_e4m3x2(z.p[1].x, z.p[1].y) << 16,
                      cvt_e4m3x2(z.p[2].x, z.p[2].y) | cvt_e4m3x2(z.p[3].x, z.p[3].y) << 16);
}

// |v| as the bits that a maximum over unsigned words orders (NaN above all).
__device__ __forceinline__ uint32_t abs_bits(float v) { return __float_as_uint(v) & 0x7FFFFFFFu; }

}  // namespace mx
