// mx_activate.cuh -- the MLP's activations and their slopes.
#pragma once
#include "mx_act8.cuh"

namespace mx {

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

}  // namespace mx
