// act.cu -- the MLP's activation, forward and backward, and the 8-bit
// activation checkpoints on their own.
#include <algorithm>
#include <cstring>
#include <type_traits>

#include "mx_act8.cuh"
#include "mx_internal.cuh"

namespace mx {
namespace {

constexpr int kThreads = 256;

// Of two arguments.
struct ValueSlope {
    float2 value, slope;
};

// FAST: results that are rounded to bf16.  The value and the slope are off by less
// than 2^-20 of their terms for the arguments that matter.  Beside half a bf16 place,
// 2^-9, that is nothing but where a slope's terms cancel: at the bf16 argument next to
// a slope's zero, 1/200 to 1/360 of a term remains, and the error is up to a fifth of
// half a place there.
//
// exp(x), x <= 0: the approximate exponential is off by 2 + 1.2 |x| last places,
// so by 2^-22 of the result for the arguments that matter and below 2^-16 for all.
template <bool FAST>
__device__ __forceinline__ float exponential(float x)
{
    return FAST ? __expf(x) : expf(x);
}
// 1 / d for 1 <= d <= 2.  FAST: within 2 last places.  fp32: one step of Newton's
// iteration from there, r + r (1 - d r), whose error is the square of r's, so that its
// own rounding is what is left.  (The operator's division takes care of every d, in a
// subroutine: 3x192 forward 3.4 us in place of 2.4, 1023x11009 32.6 in place of 30.9.)
template <bool FAST>
__device__ __forceinline__ float reciprocal(float d)
{
    const float r = __fdividef(1.0f, d);
    return FAST ? r : fmaf(r, fmaf(-d, r, 1.0f), r);
}

// p = 1 / (1 + exp(-t)) and its slope q = p (1 - p).  From exp(-|t|) nothing
// overflows, and the smaller of p and 1 - p keeps its precision down to the last
// subnormal exponential (|t| = 103); from that one nothing cancels in q.
struct Logistic {
    float p, q;
};
template <bool FAST>
__device__ __forceinline__ Logistic logistic(float t)
{
    const float e = exponential<FAST>(-fabsf(t)), r = reciprocal<FAST>(1.0f + e), least = e * r;
    return {t < 0.0f ? least : r, fmaf(-least, least, least)};
}

struct NormalTail {
    float2 tail, gauss;  // Phi(-y) and exp(-y^2 / 2)
};
// The normal distribution's tail at y >= 0 in the form of Hastings, "Approximations
// for Digital Computers" (1955; Abramowitz and Stegun 26.2.17): exp(-y^2 / 2) times
// a polynomial in t = 1 / (1 + k y).  One exponential serves the value and the
// slope; with the library's erfc and a second one the bf16 backward pass of
// 8192x14336 took 287 us.
//
// It is t (1/2 + w Q(w)), w = k y t = 1 - t: near y = 0, where most arguments lie, w
// is small and Q's rounding with it, and on the far side the tail keeps its
// precision.  Q is a least squares fit, reweighted to an even relative error over 0 <=
// y <= 14.5 (tests/test_normal_tail_fit.py has the fit): 2e-8, 4e-8 with its
// coefficients rounded; FAST two degrees less and 3e-7, 3e-7.
//
// fp32: what y^2 loses to rounding goes into the exponential as a factor.  With every
// operation rounded the tail is off by 4e-7 of itself at most, and the slope's root
// mean square error is that of its plain form by erf.  Of t's two last places (a
// division to nearest: 33 us in place of 29.7 for 1023x11009 backward) that shows
// nothing.
template <bool FAST>
__device__ __forceinline__ NormalTail normal_tail(float2 y)
{
    constexpr float k = FAST ? 0.42f : 0.4f;
    constexpr float fast[] = {-0.449849814f, 0.0171071552f, 0.111512974f, 0.0109572522f,
                              0.0409163237f, -0.107324116f, 0.0442672148f};
    constexpr float full[] = {-0.497356862f,  0.0678424835f, 0.116752833f, 0.0223698318f, -0.0597253218f,
                              0.0548196249f, -0.12487451f,   0.11158748f,  -0.0318392329f};
    const float2 ky = __fmul2_rn(y, both(k)), d = __fadd2_rn(ky, both(1.0f));
    const float2 t = make_float2(__fdividef(1.0f, d.x), __fdividef(1.0f, d.y));
    // k y t is the more precise; 1 - t holds for infinite y too
    const float2 w = FAST ? __ffma2_rn(t, both(-1.0f), both(1.0f)) : __fmul2_rn(ky, t);
    float2 q = both(FAST ? fast[6] : full[8]);
#pragma unroll
    for (int i = FAST ? 5 : 7; i >= 0; --i)
        q = __ffma2_rn(q, w, both(FAST ? fast[i] : full[i]));
    const float2 half = __fmul2_rn(y, both(-0.5f)), a = __fmul2_rn(half, y);
    float2 e = make_float2(exponential<FAST>(a.x), exponential<FAST>(a.y));
    if constexpr (!FAST)
        e = __ffma2_rn(e, __ffma2_rn(half, y, make_float2(-a.x, -a.y)), e);
    return {__fmul2_rn(e, __fmul2_rn(t, __ffma2_rn(w, q, both(0.5f)))), e};
}

// a(z) and a'(z).
template <int ACT, bool FAST>
__device__ __forceinline__ ValueSlope activate(float2 z)
{
    if constexpr (ACT == MX_ACT_SILU) {
        const Logistic f = logistic<FAST>(z.x), g = logistic<FAST>(z.y);
        return {make_float2(z.x * f.p, z.y * g.p), make_float2(f.p + z.x * f.q, g.p + z.y * g.q)};
    } else if constexpr (ACT == MX_ACT_GELU) {
        float2 y = make_float2(fabsf(z.x), fabsf(z.y));
        if constexpr (!FAST)  // the tail is 0 from 14.5 on, and y^2 stays finite
            y = make_float2(fminf(y.x, 16.0f), fminf(y.y, 16.0f));
        const NormalTail n = normal_tail<FAST>(y);
        const float2 p = make_float2(z.x > 0.0f ? 1.0f - n.tail.x : n.tail.x, z.y > 0.0f ? 1.0f - n.tail.y : n.tail.y);
        return {__fmul2_rn(z, p), __ffma2_rn(z, __fmul2_rn(n.gauss, both(0.39894228040143268f)), p)};
    } else {  // (1 + tanh t) / 2 = 1 / (1 + exp(-2 t))
        constexpr float k = 0.79788456080286536f;
        auto one = [](float v, float& value, float& slope) {
            const float vv = v * v;
            const Logistic f = logistic<FAST>(2.0f * k * (v + 0.044715f * v * vv));
            value = v * f.p;
            // q is 0 where v^2 may have overflowed: the slope is p there
            slope = f.q == 0.0f ? f.p : f.p + v * f.q * (2.0f * k) * (1.0f + 0.134145f * vv);
        };
        ValueSlope r;
        one(z.x, r.value.x, r.slope.x);
        one(z.y, r.value.y, r.slope.y);
        return r;
    }
}

// A unit is eight columns of a row, a row has 4 G units (whole groups, so that
// the four lanes of a group always work together; those past the row's end hold
// zeros).  A thread keeps units_in_flight() units' loads in flight, and a grid of
// kFwdCtas, kBwdCtas (from the kept inputs), kBwd8Ctas (from checkpoints) or k8Ctas
// CTAs an SM strides over the units, or as many as registers allow.  8192x14336
// bf16 gated SiLU measured, in us, at 3 / 4 / 5 / 6 CTAs: forward with checkpoints
// 161 / 150 and no more fit, backward from the kept inputs 194 / 179 / 181 / 187 (GELU
// 196 / 185 at 4 / 5), from checkpoints 179 / 163 / 151 / 148; 4096x11008 saved and
// restored at 3 / 4 / 5 / 8 50 / 46 / 44 / 42.  One unit in place of two: 170, 149 and
// 45, but at any address, where the shifts take the registers, 1023x11009 fp32 32.5
// -> 29.7, 8192x14335 248 -> 243, 4096x11007 saved and restored 67.5 -> 64.7.
// ANY: rows of any address and length; else they start on 16-byte boundaries and their
// length is a multiple of eight.
constexpr int kFwdCtas = 4, kBwdCtas = 5, kBwd8Ctas = 6, k8Ctas = 8;
__host__ __device__ constexpr int units_in_flight(bool any) { return any ? 1 : 2; }

struct UnitMap {
    FastDiv per_row;
    uint32_t total;  // < 2^31
};
struct Place {
    int64_t row;
    uint32_t unit;  // in the row
    int32_t cols;   // columns of the unit inside the row: 8, fewer at its end, <= 0 past it
};
__device__ __forceinline__ Place place(uint32_t i, const UnitMap& m, int64_t cols)
{
    const uint32_t r = div_by(i, m.per_row), u = i - r * m.per_row.d;
    Place p = {r, u, static_cast<int32_t>(min(cols - static_cast<int64_t>(u) * 8, int64_t{8}))};
    if (i >= m.total)
        p.cols = 0;
    return p;
}

// A unit's words.  ANY: the aligned words that it lies in; they may hold a
// neighbouring row's elements, but nothing before the matrix's first element or
// after its last one is touched.
template <typename T, bool ANY>
struct Unit {
    RawOct<T> w;
    uint4 more;
    int s;

    __device__ __forceinline__ void load(const void* base, int64_t ld, const Place& p, int64_t rows, int64_t cols)
    {
        const T* src = static_cast<const T*>(base) + p.row * ld + static_cast<int64_t>(p.unit) * 8;
        if constexpr (!ANY) {
            if (p.cols > 0)
                w.load(src);
            else
                w.clear();
        } else {
            s = misaligned(src, sizeof(T));
            const int64_t at = p.row * ld + static_cast<int64_t>(p.unit) * 8, end = (rows - 1) * ld + cols;
            w.clear();
            more = make_uint4(0, 0, 0, 0);
            if (p.cols <= 0)
                return;
            if (at < 8 || at + 16 > end) {  // the aligned words may reach past the matrix
                T v[8];
#pragma unroll
                for (int c = 0; c < 8; ++c)
                    v[c] = c < p.cols ? src[c] : T(0.0f);
                memcpy(&w, v, sizeof v);
                s = 0;
                return;
            }
            w.load(src - s);
            if (s + p.cols > 8) {
                RawOct<__nv_bfloat16> m;
                m.load(reinterpret_cast<const __nv_bfloat16*>(src - s + 8));
                more = m.w;
            }
        }
    }
    __device__ __forceinline__ void get(Oct& o, int n) const
    {
        if constexpr (!ANY) {
            w.get(o);
        } else {
            if constexpr (sizeof(T) == 2) {
                unpack_oct(shifted(w.w, more, s), o);
            } else {
                uint4 a, b, lo, hi;
                memcpy(&a, &w.a, 16);
                memcpy(&b, &w.b, 16);
                shifted(a, b, more, s, lo, hi);
                words_to_oct(lo, hi, o);
            }
            if (n < 8)
                keep_first(o, n);
        }
    }
};

template <typename T, bool ANY>
__device__ __forceinline__ void store_unit(void* base, int64_t ld, const Place& p, const Oct& o, int64_t cols, Top<T>& top)
{
    T* dst = static_cast<T*>(base) + p.row * ld + static_cast<int64_t>(p.unit) * 8;
    if constexpr (!ANY) {
        if (p.cols > 0)
            store_oct(dst, o, top);
    } else {
        const int lane = threadIdx.x & 31;
        store_ragged(dst, o, p.cols, lane > 0 && p.unit > 0, lane < 31 && static_cast<int64_t>(p.unit) * 8 + 8 < cols, top);
    }
}

__device__ __forceinline__ void save_unit(const Act8View& out, int64_t unit, bool in, const Oct& o)
{
    uint8_t e;
    const uint2 codes = encode_oct(o, e);
    if (in) {
        *reinterpret_cast<uint2*>(out.codes + unit * 8) = codes;
        if ((threadIdx.x & 3) == 0)
            out.sf[unit >> 2] = e;
    }
}

// h = a(gate) up, the checkpoints of both inputs and the maximum from one reading.
// Bound by DRAM: 8192x14336 bf16 SiLU with checkpoints 150 us (946 MB, 6.3 TB/s);
// GELU 173 us, where the instructions show; fp32 279 us (1651 MB, 5.9 TB/s); 14335
// columns 243 us.
template <typename T, int ACT, bool GATED, bool ANY>
__global__ void __launch_bounds__(kThreads) act_fwd_kernel(ActArgs a, UnitMap m)
{
    constexpr int kUnits = units_in_flight(ANY);
    Top<T> top;
    for (uint32_t base = blockIdx.x * (kThreads * kUnits); base < m.total; base += gridDim.x * (kThreads * kUnits)) {
        Unit<T, ANY> g[kUnits], u[kUnits];
        Place p[kUnits];
#pragma unroll
        for (int k = 0; k < kUnits; ++k) {
            const uint32_t i = base + k * kThreads + threadIdx.x;
            p[k] = place(i, m, a.cols);
            g[k].load(a.gate, a.ldg, p[k], a.rows, a.cols);
            if constexpr (GATED)
                u[k].load(a.up, a.ldu, p[k], a.rows, a.cols);
        }
#pragma unroll
        for (int k = 0; k < kUnits; ++k) {
            const uint32_t i = base + k * kThreads + threadIdx.x;
            Oct gv, uv, h;
            g[k].get(gv, p[k].cols);
            if constexpr (GATED)
                u[k].get(uv, p[k].cols);
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                h.p[j] = activate<ACT, sizeof(T) == 2>(gv.p[j]).value;
                if constexpr (GATED)
                    h.p[j].x *= uv.p[j].x, h.p[j].y *= uv.p[j].y;
            }
            store_unit<T, ANY>(a.h, a.ldh, p[k], h, a.cols, top);
            if (a.gate8.codes)
                save_unit(a.gate8, i, i < m.total, gv);
            if constexpr (GATED)
                if (a.up8.codes)
                    save_unit(a.up8, i, i < m.total, uv);
        }
    }
    if (a.amax)
        flush_top(a.amax, top);
}

// dgate = dh up a'(gate), dup = dh a(gate): one exponential gives value and slope.
// Bound by DRAM: 8192x14336 bf16 SiLU from checkpoints 148 us (946 MB, 6.4 TB/s),
// from the kept inputs 181 us (1175 MB, 6.5 TB/s); GELU 181 and 185 us, where the
// registers are held to what lets its CTAs be resident (without: 188 and 200 us; 0
// leaves them to the compiler); 14335 columns, SiLU, 238 us.
template <typename T, int ACT, bool GATED, bool FROM8, bool ANY>
__global__ void __launch_bounds__(kThreads, !ANY && sizeof(T) == 2 && ACT == MX_ACT_GELU ? (FROM8 ? kBwd8Ctas : kBwdCtas) : 0)
    act_bwd_kernel(ActArgs a, UnitMap m)
{
    constexpr int kUnits = units_in_flight(ANY);
    using Raw = std::conditional_t<FROM8, RawCodes, Unit<T, ANY>>;
    Top<T> top;
    for (uint32_t base = blockIdx.x * (kThreads * kUnits); base < m.total; base += gridDim.x * (kThreads * kUnits)) {
        Raw g[kUnits], u[kUnits];
        Unit<T, ANY> d[kUnits];
        Place p[kUnits];
#pragma unroll
        for (int k = 0; k < kUnits; ++k) {
            const uint32_t i = base + k * kThreads + threadIdx.x;
            p[k] = place(i, m, a.cols);
            d[k].load(a.h, a.ldh, p[k], a.rows, a.cols);
            if constexpr (FROM8) {
                g[k].clear();
                u[k].clear();
                if (p[k].cols > 0) {
                    g[k].load(a.gate8, i);
                    if constexpr (GATED)
                        u[k].load(a.up8, i);
                }
            } else {
                g[k].load(a.gate, a.ldg, p[k], a.rows, a.cols);
                if constexpr (GATED)
                    u[k].load(a.up, a.ldu, p[k], a.rows, a.cols);
            }
        }
#pragma unroll
        for (int k = 0; k < kUnits; ++k) {
            Oct gv, uv, dv, dg;
            d[k].get(dv, p[k].cols);
            g[k].get(gv, p[k].cols);
            if constexpr (GATED)
                u[k].get(uv, p[k].cols);
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const ValueSlope f = activate<ACT, sizeof(T) == 2>(gv.p[j]);
                dg.p[j].x = dv.p[j].x * f.slope.x, dg.p[j].y = dv.p[j].y * f.slope.y;
                if constexpr (GATED) {
                    dg.p[j].x *= uv.p[j].x, dg.p[j].y *= uv.p[j].y;
                    dv.p[j].x *= f.value.x, dv.p[j].y *= f.value.y;
                }
            }
            store_unit<T, ANY>(a.dgate, a.lddg, p[k], dg, a.cols, top);
            if constexpr (GATED)
                store_unit<T, ANY>(a.dup, a.lddu, p[k], dv, a.cols, top);
        }
    }
    if (a.amax)
        flush_top(a.amax, top);
}

// A checkpoint on its own, both ways, bound by DRAM: 4096x11008 bf16 saved and
// restored 42 us (273 MB, 6.6 TB/s), 11007 columns 65 us.
template <typename T, bool ANY>
__global__ void __launch_bounds__(kThreads) act8_save_kernel(const void* __restrict__ x, int64_t ldx, int64_t rows,
                                                             int64_t cols, Act8View out, UnitMap m)
{
    constexpr int kUnits = units_in_flight(ANY);
    for (uint32_t base = blockIdx.x * (kThreads * kUnits); base < m.total; base += gridDim.x * (kThreads * kUnits)) {
        Unit<T, ANY> w[kUnits];
        Place p[kUnits];
#pragma unroll
        for (int k = 0; k < kUnits; ++k) {
            p[k] = place(base + k * kThreads + threadIdx.x, m, cols);
            w[k].load(x, ldx, p[k], rows, cols);
        }
#pragma unroll
        for (int k = 0; k < kUnits; ++k) {
            const uint32_t i = base + k * kThreads + threadIdx.x;
            Oct v;
            w[k].get(v, p[k].cols);
            save_unit(out, i, i < m.total, v);
        }
    }
}

template <typename T, bool ANY>
__global__ void __launch_bounds__(kThreads) act8_restore_kernel(Act8View a, int64_t cols, void* __restrict__ out,
                                                                int64_t ldo, UnitMap m)
{
    constexpr int kUnits = units_in_flight(ANY);
    Top<T> unused;
    for (uint32_t base = blockIdx.x * (kThreads * kUnits); base < m.total; base += gridDim.x * (kThreads * kUnits)) {
        RawCodes w[kUnits];
        Place p[kUnits];
#pragma unroll
        for (int k = 0; k < kUnits; ++k) {
            const uint32_t i = base + k * kThreads + threadIdx.x;
            p[k] = place(i, m, cols);
            w[k].clear();
            if (p[k].cols > 0)
                w[k].load(a, i);
        }
#pragma unroll
        for (int k = 0; k < kUnits; ++k) {
            Oct v;
            w[k].get(v, p[k].cols);
            store_unit<T, ANY>(out, ldo, p[k], v, cols, unused);
        }
    }
}

// Rows that one launch can take (its unit count is 31 bits).
int64_t slab_rows(int64_t cols) { return std::max<int64_t>(1, ((int64_t{1} << 31) - (1 << 22)) / (act8_groups(cols) * 4)); }
UnitMap unit_map(int64_t rows, int64_t cols)
{
    const int64_t per_row = act8_groups(cols) * 4;
    return {fast_div(static_cast<uint32_t>(per_row)), static_cast<uint32_t>(rows * per_row)};
}
// A grid of at most per_sm CTAs an SM, all of them resident.
template <auto KERNEL, typename... A>
int launch_units(const UnitMap& m, bool any, int per_sm, bool early, const Device& d, cudaStream_t s, A... args)
{
    const int64_t per_cta = int64_t{kThreads} * units_in_flight(any);
    const int64_t most = int64_t{d.sms} * std::min(per_sm, resident_ctas<KERNEL>(kThreads));
    return launch_kernel(KERNEL, static_cast<unsigned>(std::min((m.total + per_cta - 1) / per_cta, most)), 1, kThreads, 0,
                         early, s, args..., m);
}

// Whether every row of a matrix starts on a 16-byte boundary.
bool wide(const void* p, int64_t ld, int dtype)
{
    return (reinterpret_cast<uintptr_t>(p) & 15) == 0 && (ld * (dtype == MX_OUT_BF16 ? 2 : 4)) % 16 == 0;
}

// p moved on by `rows` rows of a matrix (null stays null).
template <typename P>
P* ahead(P* p, int64_t rows, int64_t ld, int dtype)
{
    using B = std::conditional_t<std::is_const_v<P>, const char, char>;
    return p ? static_cast<P*>(static_cast<B*>(p) + rows * ld * (dtype == MX_OUT_BF16 ? 2 : 4)) : p;
}
Act8View ahead(Act8View v, int64_t rows, int64_t cols)
{
    if (v.codes) {
        v.codes += rows * act8_groups(cols) * kAct8Group;
        v.sf += rows * act8_groups(cols);
    }
    return v;
}

template <typename T, int ACT>
int fwd(const ActArgs& a, const Device& d, cudaStream_t s)
{
    const bool aligned = a.cols % 8 == 0 && wide(a.gate, a.ldg, a.dtype) && wide(a.h, a.ldh, a.dtype) && wide(a.up, a.ldu, a.dtype);
    const int64_t slab = slab_rows(a.cols);
    int rc = launch_zero(a.amax, s);
    if (rc != MX_OK)
        return rc;
    for (int64_t r = 0; r < a.rows; r += slab) {
        const bool early = a.amax && r == 0;
        ActArgs b = a;
        b.rows = std::min(slab, a.rows - r);
        b.gate = ahead(a.gate, r, a.ldg, a.dtype);
        b.up = ahead(a.up, r, a.ldu, a.dtype);
        b.h = ahead(a.h, r, a.ldh, a.dtype);
        b.gate8 = ahead(a.gate8, r, a.cols);
        b.up8 = ahead(a.up8, r, a.cols);
        const UnitMap m = unit_map(b.rows, a.cols);
        if (aligned && a.gated)
            rc = launch_units<act_fwd_kernel<T, ACT, true, false>>(m, !aligned, kFwdCtas, early, d, s, b);
        else if (aligned)
            rc = launch_units<act_fwd_kernel<T, ACT, false, false>>(m, !aligned, kFwdCtas, early, d, s, b);
        else if (a.gated)
            rc = launch_units<act_fwd_kernel<T, ACT, true, true>>(m, !aligned, kFwdCtas, early, d, s, b);
        else
            rc = launch_units<act_fwd_kernel<T, ACT, false, true>>(m, !aligned, kFwdCtas, early, d, s, b);
        if (rc != MX_OK)
            return rc;
    }
    return MX_OK;
}

template <typename T, int ACT, bool FROM8>
int bwd(const ActArgs& a, const Device& d, cudaStream_t s)
{
    const bool aligned = a.cols % 8 == 0 && wide(a.h, a.ldh, a.dtype) && wide(a.dgate, a.lddg, a.dtype) && wide(a.dup, a.lddu, a.dtype) &&
                         wide(a.gate, a.ldg, a.dtype) && wide(a.up, a.ldu, a.dtype);
    const int64_t slab = slab_rows(a.cols);
    int rc = launch_zero(a.amax, s);
    if (rc != MX_OK)
        return rc;
    for (int64_t r = 0; r < a.rows; r += slab) {
        const bool early = a.amax && r == 0;
        ActArgs b = a;
        b.rows = std::min(slab, a.rows - r);
        b.gate = ahead(a.gate, r, a.ldg, a.dtype);
        b.up = ahead(a.up, r, a.ldu, a.dtype);
        b.h = ahead(a.h, r, a.ldh, a.dtype);
        b.dgate = ahead(a.dgate, r, a.lddg, a.dtype);
        b.dup = ahead(a.dup, r, a.lddu, a.dtype);
        b.gate8 = ahead(a.gate8, r, a.cols);
        b.up8 = ahead(a.up8, r, a.cols);
        const UnitMap m = unit_map(b.rows, a.cols);
        if (aligned && a.gated)
            rc = launch_units<act_bwd_kernel<T, ACT, true, FROM8, false>>(m, !aligned, FROM8 ? kBwd8Ctas : kBwdCtas, early, d, s, b);
        else if (aligned)
            rc = launch_units<act_bwd_kernel<T, ACT, false, FROM8, false>>(m, !aligned, FROM8 ? kBwd8Ctas : kBwdCtas, early, d, s, b);
        else if (a.gated)
            rc = launch_units<act_bwd_kernel<T, ACT, true, FROM8, true>>(m, !aligned, FROM8 ? kBwd8Ctas : kBwdCtas, early, d, s, b);
        else
            rc = launch_units<act_bwd_kernel<T, ACT, false, FROM8, true>>(m, !aligned, FROM8 ? kBwd8Ctas : kBwdCtas, early, d, s, b);
        if (rc != MX_OK)
            return rc;
    }
    return MX_OK;
}

template <typename T>
int save(const void* x, int64_t ldx, int dtype, int64_t rows, int64_t cols, Act8View out, const Device& d,
         cudaStream_t s)
{
    const bool aligned = cols % 8 == 0 && wide(x, ldx, dtype);
    const int64_t slab = slab_rows(cols);
    int rc = MX_OK;
    for (int64_t r = 0; r < rows; r += slab) {
        const int64_t n = std::min(slab, rows - r);
        const UnitMap m = unit_map(n, cols);
        const void* from = ahead(x, r, ldx, dtype);
        if (aligned)
            rc = launch_units<act8_save_kernel<T, false>>(m, !aligned, k8Ctas, false, d, s, from, ldx, n, cols, ahead(out, r, cols));
        else
            rc = launch_units<act8_save_kernel<T, true>>(m, !aligned, k8Ctas, false, d, s, from, ldx, n, cols, ahead(out, r, cols));
        if (rc != MX_OK)
            return rc;
    }
    return MX_OK;
}

template <typename T>
int restore(Act8View a, int64_t rows, int64_t cols, void* out, int64_t ldo, int dtype, const Device& d, cudaStream_t s)
{
    const bool aligned = cols % 8 == 0 && wide(out, ldo, dtype);
    const int64_t slab = slab_rows(cols);
    int rc = MX_OK;
    for (int64_t r = 0; r < rows; r += slab) {
        const int64_t n = std::min(slab, rows - r);
        const UnitMap m = unit_map(n, cols);
        void* to = ahead(out, r, ldo, dtype);
        if (aligned)
            rc = launch_units<act8_restore_kernel<T, false>>(m, !aligned, k8Ctas, false, d, s, ahead(a, r, cols), cols, to, ldo);
        else
            rc = launch_units<act8_restore_kernel<T, true>>(m, !aligned, k8Ctas, false, d, s, ahead(a, r, cols), cols, to, ldo);
        if (rc != MX_OK)
            return rc;
    }
    return MX_OK;
}

template <typename T>
int fwd_by_act(const ActArgs& a, const Device& d, cudaStream_t s)
{
    switch (a.act) {
    case MX_ACT_SILU: return fwd<T, MX_ACT_SILU>(a, d, s);
    case MX_ACT_GELU: return fwd<T, MX_ACT_GELU>(a, d, s);
    default: return fwd<T, MX_ACT_GELU_TANH>(a, d, s);
    }
}

template <typename T, bool FROM8>
int bwd_by_act(const ActArgs& a, const Device& d, cudaStream_t s)
{
    switch (a.act) {
    case MX_ACT_SILU: return bwd<T, MX_ACT_SILU, FROM8>(a, d, s);
    case MX_ACT_GELU: return bwd<T, MX_ACT_GELU, FROM8>(a, d, s);
    default: return bwd<T, MX_ACT_GELU_TANH, FROM8>(a, d, s);
    }
}

__global__ void zero_word_kernel(unsigned* word)
{
    let_next_launch_start();
    *word = 0;
}

}  // namespace

int launch_zero(unsigned* word, cudaStream_t s)
{
    return word ? launch_kernel(zero_word_kernel, 1, 1, 1, 0, false, s, word) : MX_OK;
}

int launch_act_fwd(const ActArgs& a, const Device& d, cudaStream_t s)
{
    return a.dtype == MX_OUT_BF16 ? fwd_by_act<__nv_bfloat16>(a, d, s) : fwd_by_act<float>(a, d, s);
}

int launch_act_bwd(const ActArgs& a, const Device& d, cudaStream_t s)
{
    if (a.gate8.codes)
        return a.dtype == MX_OUT_BF16 ? bwd_by_act<__nv_bfloat16, true>(a, d, s) : bwd_by_act<float, true>(a, d, s);
    return a.dtype == MX_OUT_BF16 ? bwd_by_act<__nv_bfloat16, false>(a, d, s) : bwd_by_act<float, false>(a, d, s);
}

int launch_act8_save(const void* x, int64_t ldx, int dtype, int64_t rows, int64_t cols, Act8View out, const Device& d,
                     cudaStream_t s)
{
    return dtype == MX_OUT_BF16 ? save<__nv_bfloat16>(x, ldx, dtype, rows, cols, out, d, s)
                                : save<float>(x, ldx, dtype, rows, cols, out, d, s);
}

int launch_act8_restore(Act8View a, int64_t rows, int64_t cols, void* out, int64_t ldo, int dtype, const Device& d,
                        cudaStream_t s)
{
    return dtype == MX_OUT_BF16 ? restore<__nv_bfloat16>(a, rows, cols, out, ldo, dtype, d, s)
                                : restore<float>(a, rows, cols, out, ldo, dtype, d, s);
}

}  // namespace mx
