// act.cu -- the MLP's activation, forward and backward, and the 8-bit
// activation checkpoints on their own.
#include <algorithm>

#include "mx_act8.cuh"
#include "mx_internal.cuh"

namespace mx {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;

struct ValueSlope {
    float value, slope;
};

// a(z) and a'(z).
template <int ACT>
__device__ __forceinline__ ValueSlope activate(float z)
{
    if constexpr (ACT == MX_ACT_SILU) {
        const float p = 1.0f / (1.0f + expf(-z));
        return {z * p, p + z * p * (1.0f - p)};
    } else if constexpr (ACT == MX_ACT_GELU) {
        const float p = 0.5f * erfcf(z * -0.70710678118654752f);
        return {z * p, p + z * (0.39894228040143268f * expf(-0.5f * z * z))};
    } else {  // (1 + tanh t) / 2 = 1 / (1 + exp(-2 t))
        constexpr float k = 0.79788456080286536f;
        const float zz = z * z, p = 1.0f / (1.0f + expf(-2.0f * k * (z + 0.044715f * z * zz)));
        const float q = p * (1.0f - p);  // 0 where z^2 may have overflowed: the slope is p there
        return {z * p, q == 0.0f ? p : p + z * q * (2.0f * k) * (1.0f + 0.134145f * zz)};
    }
}

__device__ __forceinline__ void flush_amax(unsigned* out, uint32_t top)
{
    top = __reduce_max_sync(0xFFFFFFFFu, top);
    if ((threadIdx.x & 31) == 0)
        atomicMax(out, top);  // a maximum does not depend on the order
}

// The warp's 32 lanes hold one group (0 past the row's end).
__device__ __forceinline__ void save_group(float v, const Act8View& out, int64_t group)
{
    const int lane = threadIdx.x & 31;
    const float z = finite_or_nan(v);
    const float b = __uint_as_float(__reduce_max_sync(0xFFFFFFFFu, abs_bits(fmaxf(fabsf(z), 0.0f))));
    const int e = act8_exponent(b);
    out.codes[group * kAct8Group + lane] = static_cast<uint8_t>(cvt_e4m3x2(z * exp2_neg(e), 0.0f));
    if (lane == 0)
        out.sf[group] = static_cast<uint8_t>(e + 127);
}

__device__ __forceinline__ float restored(const Act8View& a, int64_t group, int lane)
{
    return dec_e4m3x2(a.codes[group * kAct8Group + lane]).x * act8_scale(a.sf[group]);
}

// ------------------------------------------------------------------ any width
// A warp per group of 32 columns of a row, one column a lane.  Serves every
// width and alignment.

template <typename T, int ACT, bool GATED>
__global__ void __launch_bounds__(kThreads) act_fwd_any_kernel(ActArgs a)
{
    const int lane = threadIdx.x & 31;
    const int64_t G = act8_groups(a.cols), total = a.rows * G;
    uint32_t top = 0;
    for (int64_t i = blockIdx.x * static_cast<int64_t>(kWarps) + (threadIdx.x >> 5); i < total;
         i += static_cast<int64_t>(gridDim.x) * kWarps) {
        const int64_t r = i / G, c = (i - r * G) * kAct8Group + lane;
        const bool in = c < a.cols;
        const float g = in ? load_f(static_cast<const T*>(a.gate) + r * a.ldg + c) : 0.0f;
        float h = activate<ACT>(g).value, u = 0.0f;
        if constexpr (GATED) {
            u = in ? load_f(static_cast<const T*>(a.up) + r * a.ldu + c) : 0.0f;
            h *= u;
        }
        if (in) {
            h = as_stored<T>(h);
            store_f(static_cast<T*>(a.h) + r * a.ldh + c, h);
            top = max(top, abs_bits(h));
        }
        if (a.gate8.codes)
            save_group(g, a.gate8, i);
        if (GATED && a.up8.codes)
            save_group(u, a.up8, i);
    }
    if (a.amax)
        flush_amax(a.amax, top);
}

template <typename T, int ACT, bool GATED, bool FROM8>
__global__ void __launch_bounds__(kThreads) act_bwd_any_kernel(ActArgs a)
{
    const int lane = threadIdx.x & 31;
    const int64_t G = act8_groups(a.cols), total = a.rows * G;
    uint32_t top = 0;
    for (int64_t i = blockIdx.x * static_cast<int64_t>(kWarps) + (threadIdx.x >> 5); i < total;
         i += static_cast<int64_t>(gridDim.x) * kWarps) {
        const int64_t r = i / G, c = (i - r * G) * kAct8Group + lane;
        if (c >= a.cols)
            continue;
        const float g = FROM8 ? restored(a.gate8, i, lane) : load_f(static_cast<const T*>(a.gate) + r * a.ldg + c);
        const float dh = load_f(static_cast<const T*>(a.h) + r * a.ldh + c);
        const ValueSlope f = activate<ACT>(g);
        float dg = dh * f.slope;
        if constexpr (GATED) {
            const float u = FROM8 ? restored(a.up8, i, lane) : load_f(static_cast<const T*>(a.up) + r * a.ldu + c);
            dg *= u;
            const float du = as_stored<T>(dh * f.value);
            store_f(static_cast<T*>(a.dup) + r * a.lddu + c, du);
            top = max(top, abs_bits(du));
        }
        dg = as_stored<T>(dg);
        store_f(static_cast<T*>(a.dgate) + r * a.lddg + c, dg);
        top = max(top, abs_bits(dg));
    }
    if (a.amax)
        flush_amax(a.amax, top);
}

template <typename T>
__global__ void __launch_bounds__(kThreads) act8_save_any_kernel(const T* __restrict__ x, int64_t ldx, int64_t rows,
                                                                 int64_t cols, Act8View out)
{
    const int64_t G = act8_groups(cols), total = rows * G;
    for (int64_t i = blockIdx.x * static_cast<int64_t>(kWarps) + (threadIdx.x >> 5); i < total;
         i += static_cast<int64_t>(gridDim.x) * kWarps) {
        const int64_t r = i / G, c = (i - r * G) * kAct8Group + (threadIdx.x & 31);
        save_group(c < cols ? load_f(x + r * ldx + c) : 0.0f, out, i);
    }
}

template <typename T>
__global__ void __launch_bounds__(kThreads) act8_restore_any_kernel(Act8View a, int64_t rows, int64_t cols,
                                                                    T* __restrict__ out, int64_t ldo)
{
    const int lane = threadIdx.x & 31;
    const int64_t G = act8_groups(cols), total = rows * G;
    for (int64_t i = blockIdx.x * static_cast<int64_t>(kWarps) + (threadIdx.x >> 5); i < total;
         i += static_cast<int64_t>(gridDim.x) * kWarps) {
        const int64_t r = i / G, c = (i - r * G) * kAct8Group + lane;
        if (c < cols)
            store_f(out + r * ldo + c, restored(a, i, lane));
    }
}

unsigned any_grid(int64_t rows, int64_t cols, const Device& d)
{
    const int64_t ctas = (rows * act8_groups(cols) + kWarps - 1) / kWarps;
    return static_cast<unsigned>(std::min<int64_t>(ctas, d.sms * 8));
}

int launched()
{
    count_launch();
    return cudaGetLastError() == cudaSuccess ? MX_OK : MX_ERR_CUDA;
}

template <typename T, int ACT>
int fwd(const ActArgs& a, const Device& d, cudaStream_t s)
{
    const unsigned grid = any_grid(a.rows, a.cols, d);
    if (a.gated)
        act_fwd_any_kernel<T, ACT, true><<<grid, kThreads, 0, s>>>(a);
    else
        act_fwd_any_kernel<T, ACT, false><<<grid, kThreads, 0, s>>>(a);
    return launched();
}

template <typename T, int ACT, bool FROM8>
int bwd(const ActArgs& a, const Device& d, cudaStream_t s)
{
    const unsigned grid = any_grid(a.rows, a.cols, d);
    if (a.gated)
        act_bwd_any_kernel<T, ACT, true, FROM8><<<grid, kThreads, 0, s>>>(a);
    else
        act_bwd_any_kernel<T, ACT, false, FROM8><<<grid, kThreads, 0, s>>>(a);
    return launched();
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

}  // namespace

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
    const unsigned grid = any_grid(rows, cols, d);
    if (dtype == MX_OUT_BF16)
        act8_save_any_kernel<<<grid, kThreads, 0, s>>>(static_cast<const __nv_bfloat16*>(x), ldx, rows, cols, out);
    else
        act8_save_any_kernel<<<grid, kThreads, 0, s>>>(static_cast<const float*>(x), ldx, rows, cols, out);
    return launched();
}

int launch_act8_restore(Act8View a, int64_t rows, int64_t cols, void* out, int64_t ldo, int dtype, const Device& d,
                        cudaStream_t s)
{
    const unsigned grid = any_grid(rows, cols, d);
    if (dtype == MX_OUT_BF16)
        act8_restore_any_kernel<<<grid, kThreads, 0, s>>>(a, rows, cols, static_cast<__nv_bfloat16*>(out), ldo);
    else
        act8_restore_any_kernel<<<grid, kThreads, 0, s>>>(a, rows, cols, static_cast<float*>(out), ldo);
    return launched();
}

}  // namespace mx
