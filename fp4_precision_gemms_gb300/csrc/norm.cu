// norm.cu -- layer norm and RMS norm over the rows of a residual stream,
// forward and backward.
#include <algorithm>

#include "mx_act8.cuh"
#include "mx_internal.cuh"

namespace mx {
namespace {

constexpr int kRowThreads = 256;
constexpr int kRowWarps = kRowThreads / 32;

__device__ __forceinline__ float warp_sum(float v)
{
#pragma unroll
    for (int o = 16; o > 0; o >>= 1)
        v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
    return v;
}

// Sum over the CTA in a fixed order, known to every thread.
__device__ __forceinline__ float cta_sum(float v, float* part)
{
    v = warp_sum(v);
    __syncthreads();  // the previous sum's words have been read
    if ((threadIdx.x & 31) == 0)
        part[threadIdx.x >> 5] = v;
    __syncthreads();
    v = 0.0f;
#pragma unroll
    for (int w = 0; w < kRowWarps; ++w)
        v += part[w];
    return v;
}

__device__ __forceinline__ float param(const void* p, int dtype, int64_t c, float absent)
{
    if (!p)
        return absent;
    return dtype == MX_OUT_BF16 ? load_f(static_cast<const __nv_bfloat16*>(p) + c) : static_cast<const float*>(p)[c];
}

// ------------------------------------------------------------------ any width
// One CTA per row, a warp per 32 columns at a time, the row read once per sum.
// Serves every width and alignment.

template <typename T, typename TY>
__global__ void __launch_bounds__(kRowThreads) norm_fwd_any_kernel(NormFwdArgs a)
{
    __shared__ float part[kRowWarps];
    const int lane = threadIdx.x & 31;
    const int64_t C = a.cols, G = act8_groups(C);
    const float inv_c = 1.0f / static_cast<float>(C);
    uint32_t top = 0;
    for (int64_t r = blockIdx.x; r < a.rows; r += gridDim.x) {
        const T* x = static_cast<const T*>(a.x) + r * a.ldx;
        float sum = 0.0f;
        if (a.residual) {
            const T* res = static_cast<const T*>(a.residual) + r * a.ldr;
            T* so = static_cast<T*>(a.sum_out) + r * a.lds;
            for (int64_t c = threadIdx.x; c < C; c += kRowThreads) {
                const float v = as_stored<T>(load_f(x + c) + load_f(res + c));
                store_f(so + c, v);
                sum += v;
            }
            x = so;  // each thread reads back what it wrote
        } else {
            for (int64_t c = threadIdx.x; c < C; c += kRowThreads)
                sum += load_f(x + c);
        }
        const float mean = a.kind == MX_NORM_LAYER ? cta_sum(sum, part) * inv_c : 0.0f;
        float sq = 0.0f;
        for (int64_t c = threadIdx.x; c < C; c += kRowThreads) {
            const float d = load_f(x + c) - mean;
            sq += d * d;
        }
        const float rstd = 1.0f / sqrtf(cta_sum(sq, part) * inv_c + a.eps);
        if (threadIdx.x == 0) {
            if (a.mean && a.kind == MX_NORM_LAYER)
                a.mean[r] = mean;
            if (a.rstd)
                a.rstd[r] = rstd;
        }
        TY* y = static_cast<TY*>(a.y) + r * a.ldy;
        for (int64_t g = threadIdx.x >> 5; g < G; g += kRowWarps) {  // warp-uniform
            const int64_t c = g * kAct8Group + lane;
            const float v = c < C ? load_f(x + c) : 0.0f;
            if (c < C) {
                const float o = as_stored<TY>((v - mean) * rstd * param(a.weight, a.w_dtype, c, 1.0f) +
                                              param(a.bias, a.w_dtype, c, 0.0f));
                store_f(y + c, o);
                top = max(top, abs_bits(o));
            }
            if (a.save.codes) {
                const float z = finite_or_nan(v);
                const float b = __uint_as_float(__reduce_max_sync(0xFFFFFFFFu, abs_bits(fmaxf(fabsf(z), 0.0f))));
                const int e = act8_exponent(b);
                a.save.codes[(r * G + g) * kAct8Group + lane] =
                    static_cast<uint8_t>(cvt_e4m3x2(z * exp2_neg(e), 0.0f));
                if (lane == 0)
                    a.save.sf[r * G + g] = static_cast<uint8_t>(e + 127);
            }
        }
    }
    if (a.amax) {
        top = __reduce_max_sync(0xFFFFFFFFu, top);
        if (lane == 0)
            atomicMax(a.amax, top);  // a maximum does not depend on the order
    }
}

// s of row r, column c: the kept tensor or the checkpoint.
template <typename T>
__device__ __forceinline__ float kept(const NormBwdArgs& a, int64_t r, int64_t c, int64_t G)
{
    if (a.x8.codes)
        return dec_e4m3x2(a.x8.codes[r * G * kAct8Group + c]).x * act8_scale(a.x8.sf[r * G + c / kAct8Group]);
    return load_f(static_cast<const T*>(a.x) + r * a.ldx + c);
}

template <typename T, typename TY>
__global__ void __launch_bounds__(kRowThreads) norm_dx_any_kernel(NormBwdArgs a)
{
    __shared__ float part[kRowWarps];
    const int64_t C = a.cols, G = act8_groups(C);
    const float inv_c = 1.0f / static_cast<float>(C);
    uint32_t top = 0;
    for (int64_t r = blockIdx.x; r < a.rows; r += gridDim.x) {
        const TY* dy = static_cast<const TY*>(a.dy) + r * a.ldy;
        const float rstd = a.rstd[r], mean = a.kind == MX_NORM_LAYER ? a.mean[r] : 0.0f;
        float sgh = 0.0f, sg = 0.0f;
        for (int64_t c = threadIdx.x; c < C; c += kRowThreads) {
            const float g = load_f(dy + c) * param(a.weight, a.w_dtype, c, 1.0f);
            sgh += g * ((kept<T>(a, r, c, G) - mean) * rstd);
            sg += g;
        }
        const float c1 = cta_sum(sgh, part) * inv_c;
        const float c2 = a.kind == MX_NORM_LAYER ? cta_sum(sg, part) * inv_c : 0.0f;
        const T* dres = static_cast<const T*>(a.dres) + r * a.ldres;
        T* dx = static_cast<T*>(a.dx) + r * a.lddx;
        for (int64_t c = threadIdx.x; c < C; c += kRowThreads) {
            const float g = load_f(dy + c) * param(a.weight, a.w_dtype, c, 1.0f);
            const float h = (kept<T>(a, r, c, G) - mean) * rstd;
            float v = (g - h * c1 - c2) * rstd;
            if (a.dres)
                v += load_f(dres + c);
            v = as_stored<T>(v);
            store_f(dx + c, v);
            top = max(top, abs_bits(v));
        }
    }
    if (a.amax) {
        top = __reduce_max_sync(0xFFFFFFFFu, top);
        if ((threadIdx.x & 31) == 0)
            atomicMax(a.amax, top);
    }
}

// Partial column sums: CTA (x, y) adds 32 columns of every gridDim.y-th row.
template <typename T, typename TY>
__global__ void __launch_bounds__(kRowThreads) norm_dw_any_kernel(NormBwdArgs a)
{
    __shared__ float pw[kRowWarps][32], pb[kRowWarps][32];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int64_t C = a.cols, G = act8_groups(C), c = blockIdx.x * 32ll + lane;
    float w = 0.0f, b = 0.0f;
    if (c < C) {
        for (int64_t r = blockIdx.y * kRowWarps + warp; r < a.rows; r += static_cast<int64_t>(gridDim.y) * kRowWarps) {
            const float dy = load_f(static_cast<const TY*>(a.dy) + r * a.ldy + c);
            const float mean = a.kind == MX_NORM_LAYER ? a.mean[r] : 0.0f;
            w += dy * ((kept<T>(a, r, c, G) - mean) * a.rstd[r]);
            b += dy;
        }
    }
    pw[warp][lane] = w;
    pb[warp][lane] = b;
    __syncthreads();
    if (warp == 0 && c < C) {
#pragma unroll
        for (int i = 1; i < kRowWarps; ++i) {
            w += pw[i][lane];
            b += pb[i][lane];
        }
        a.parts[blockIdx.y * C + c] = w;
        a.parts[(gridDim.y + blockIdx.y) * C + c] = b;
    }
}

// dw and db from `parts` partial sums of each column (rows of parts: dw's, then db's).
__global__ void __launch_bounds__(kRowThreads) norm_dw_join_kernel(const float* __restrict__ src, int64_t C, int parts,
                                                                   float* __restrict__ dw, float* __restrict__ db)
{
    __shared__ float p[kRowWarps][32];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int64_t c = blockIdx.x * 32ll + lane;
    float* out = blockIdx.y ? db : dw;
    if (!out)
        return;
    float v = 0.0f;
    if (c < C)
        for (int i = warp; i < parts; i += kRowWarps)
            v += src[(static_cast<int64_t>(blockIdx.y) * parts + i) * C + c];
    p[warp][lane] = v;
    __syncthreads();
    if (warp == 0 && c < C) {
#pragma unroll
        for (int i = 1; i < kRowWarps; ++i)
            v += p[i][lane];
        out[c] = v;
    }
}

template <typename T, typename TY>
int fwd(const NormFwdArgs& a, const Device& d, cudaStream_t s)
{
    const unsigned grid = static_cast<unsigned>(std::min<int64_t>(a.rows, d.sms * 8));
    norm_fwd_any_kernel<T, TY><<<grid, kRowThreads, 0, s>>>(a);
    count_launch();
    return cudaGetLastError() == cudaSuccess ? MX_OK : MX_ERR_CUDA;
}

template <typename T, typename TY>
int bwd(const NormBwdArgs& a, const Device& d, cudaStream_t s)
{
    if (a.dw || a.db) {  // before dx, which may be dy's memory
        const int parts = static_cast<int>(norm_bwd_parts(a.rows, a.cols));
        const unsigned cols32 = static_cast<unsigned>((a.cols + 31) / 32);
        norm_dw_any_kernel<T, TY><<<dim3(cols32, parts), kRowThreads, 0, s>>>(a);
        norm_dw_join_kernel<<<dim3(cols32, 2), kRowThreads, 0, s>>>(a.parts, a.cols, parts, a.dw, a.db);
        count_launch();
        count_launch();
    }
    const unsigned grid = static_cast<unsigned>(std::min<int64_t>(a.rows, d.sms * 8));
    norm_dx_any_kernel<T, TY><<<grid, kRowThreads, 0, s>>>(a);
    count_launch();
    return cudaGetLastError() == cudaSuccess ? MX_OK : MX_ERR_CUDA;
}

}  // namespace

int64_t norm_bwd_parts(int64_t rows, int64_t cols)
{
    (void)cols;
    return std::max<int64_t>(1, std::min<int64_t>((rows + kRowWarps - 1) / kRowWarps, 64));
}

int launch_norm_fwd(const NormFwdArgs& a, const Device& d, cudaStream_t s)
{
    using bf = __nv_bfloat16;
    if (a.x_dtype == MX_OUT_BF16)
        return a.y_dtype == MX_OUT_BF16 ? fwd<bf, bf>(a, d, s) : fwd<bf, float>(a, d, s);
    return a.y_dtype == MX_OUT_BF16 ? fwd<float, bf>(a, d, s) : fwd<float, float>(a, d, s);
}

int launch_norm_bwd(const NormBwdArgs& a, const Device& d, cudaStream_t s)
{
    using bf = __nv_bfloat16;
    if (a.dx_dtype == MX_OUT_BF16)
        return a.dy_dtype == MX_OUT_BF16 ? bwd<bf, bf>(a, d, s) : bwd<bf, float>(a, d, s);
    return a.dy_dtype == MX_OUT_BF16 ? bwd<float, bf>(a, d, s) : bwd<float, float>(a, d, s);
}

}  // namespace mx
