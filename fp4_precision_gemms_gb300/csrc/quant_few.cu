// quant_few.cu -- the rowwise quantization of a few rows in one short launch, for
// the serving path, where the producer's passes over a small tensor cost more in
// latency than in work.  Codes, scale bytes and tensor scales are those of
// quantize.cu's producers for round to nearest and the formats' default rules.
//
// Formats with a tensor scale need the tensor's maximum before the first code: one
// cluster of sixteen CTAs holds the whole tensor in registers, exchanges its maxima
// through distributed shared memory and encodes.  (152 SMs in ten groups or fewer: one group
// has the sixteen.)  The others need no exchange and take plain CTAs.  48 x 4096 NVFP4: 2 us
// in front of the product that it overlaps (eight CTAs: 4), in place of two launches of 8.3;
// bound by the latencies of the load, the exchange and the encoding.
#include <cuda_bf16.h>

#include "mx_act8.cuh"
#include "mx_codec.cuh"
#include "mx_internal.cuh"
#include "mx_ptx.cuh"

namespace mx {
namespace {

constexpr int kCluster = 16;
constexpr int kMaxOcts = 4;  // of a thread

// A thread's eight values, as loaded.
__device__ __forceinline__ uint4 load_words(const void* x, int64_t ld, int64_t oct, int per_row)
{
    const int64_t row = oct / per_row, col = (oct - row * per_row) * 8;
    return *reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(x) + row * ld + col);
}

__device__ __forceinline__ float top_of(const Oct& o)
{
    float m = fabsf(o[0]);
#pragma unroll
    for (int i = 1; i < 8; ++i)
        m = fmaxf(m, fabsf(o[i]));
    return m;  // NaN where all are
}
// The maximum over the lanes that share a block of 16 or 32 values.
template <int BLOCK>
__device__ __forceinline__ float block_top(float m)
{
    m = fmaxf(m, __shfl_xor_sync(0xFFFFFFFFu, m, 1));
    return BLOCK == 32 ? fmaxf(m, __shfl_xor_sync(0xFFFFFFFFu, m, 2)) : m;
}

// Whole warps; in: the oct exists.
template <int FMT>
__device__ __forceinline__ void encode(Oct o, float ts, bool in, int64_t oct, int per_row, int64_t kgroups, uint8_t* codes,
                                       uint8_t* sf)
{
    constexpr int BLOCK = fmt_block(FMT);
    constexpr int ELEM = elem_of(FMT);
    if constexpr (FMT == MX_FMT_MOSS_FP8)
#pragma unroll
        for (int i = 0; i < 8; ++i)
            o[i] = __fdiv_rn(o[i], ts);
    const float b = block_top<BLOCK>(top_of(o));
    uint32_t byte;
    float q[8];
    if constexpr (fmt_is_nvfp4(FMT)) {
        byte = cvt_e4m3x2(__fdiv_rn(b, __fmul_rn(6.0f, ts)), 0.0f) & 0x7Fu;
        const float d = __fmul_rn(dec_e4m3_pos(byte), ts);
        if (d > 0x1p-90f && d < 0x1p90f) {
            // the quotient to nearest from the reciprocal to nearest and one residual (Markstein,
            // "Computation of elementary functions on the IBM RISC System/6000 processor", 1990);
            // where x is so small that the residual is not exact the code is 0 either way
            const float r = __frcp_rn(d);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const float a = __fmul_rn(o[i], r);
                q[i] = fmaf(fmaf(-a, d, o[i]), r, a);
            }
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i)  // a block whose scale decodes to 0 holds zeros that keep their signs
                q[i] = d == 0.0f ? copysignf(0.0f, o[i]) : __fdiv_rn(o[i], d);
        }
    } else {
        const int e = pow2_exponent<ELEM>(b, FMT == MX_FMT_MOSS_FP8 ? MX_SCALE_CEIL : MX_SCALE_FLOOR);
        byte = static_cast<uint32_t>(e + 127);
        const float s = exp2_neg(e);
#pragma unroll
        for (int i = 0; i < 8; ++i)
            q[i] = __fmul_rn(o[i], s);
    }
    if (!in)
        return;
    if constexpr (ELEM == kElemE2M1)
        *reinterpret_cast<uint32_t*>(codes + oct * 4) = cvt_e2m1x8(q);
    else
        *reinterpret_cast<uint2*>(codes + oct * 8) = make_uint2(cvt_e4m3x2(q[0], q[1]) | cvt_e4m3x2(q[2], q[3]) << 16,
                                                                cvt_e4m3x2(q[4], q[5]) | cvt_e4m3x2(q[6], q[7]) << 16);
    const int64_t row = oct / per_row, kb = (oct - row * per_row) / (BLOCK / 8);
    if (oct % (BLOCK / 8) == 0)
        sf[sf_offset(row, kb, kgroups)] = static_cast<uint8_t>(byte);
}

template <int FMT>
__global__ void __launch_bounds__(256) quantize_few_kernel(const void* x, int64_t ld, int per_row, int octs, int64_t kgroups,
                                                           uint8_t* codes, uint8_t* sf, unsigned* zero, int zeros)
{
    wait_for_launch_before();  // everything before has finished when the next launch starts
    let_next_launch_start();
    const int oct = blockIdx.x * 256 + threadIdx.x;
    for (int i = oct; i < zeros; i += gridDim.x * 256)
        zero[i] = 0;
    const bool in = oct < octs;
    Oct o;
    unpack_oct(in ? load_words(x, ld, oct, per_row) : make_uint4(0, 0, 0, 0), o);
    encode<FMT>(o, 1.0f, in, oct, per_row, kgroups, codes, sf);
}

// Thread t of the cluster holds octs t, t + 16384, ...
template <int FMT>
__global__ void __cluster_dims__(kCluster, 1, 1) __launch_bounds__(1024)
    quantize_few_cluster_kernel(const void* x, int64_t ld, int per_row, int octs, int64_t kgroups, uint8_t* codes, uint8_t* sf,
                                float* amax, float* tensor_scale, unsigned* zero, int zeros)
{
    asm volatile("barrier.cluster.arrive.relaxed.aligned;");
    wait_for_launch_before();
    let_next_launch_start();
    for (int i = blockIdx.x * 1024 + threadIdx.x; i < zeros; i += kCluster * 1024)
        zero[i] = 0;
    __shared__ uint32_t of_warp[32];
    __shared__ uint32_t of_cta[kCluster];
    const int first = blockIdx.x * 1024 + threadIdx.x;
    uint4 w[kMaxOcts];
    uint32_t top = 0;
#pragma unroll
    for (int k = 0; k < kMaxOcts; ++k) {
        const int oct = first + k * (kCluster * 1024);
        w[k] = oct < octs ? load_words(x, ld, oct, per_row) : make_uint4(0, 0, 0, 0);
    }
#pragma unroll
    for (int k = 0; k < kMaxOcts; ++k)  // magnitudes by their bits, in pairs; a NaN is the largest
        top = __vmaxu2(top, __vmaxu2(__vmaxu2(w[k].x & 0x7FFF7FFFu, w[k].y & 0x7FFF7FFFu),
                                     __vmaxu2(w[k].z & 0x7FFF7FFFu, w[k].w & 0x7FFF7FFFu)));
    top = max(top << 16, top & 0xFFFF0000u);
    top = __reduce_max_sync(0xFFFFFFFFu, top);
    if ((threadIdx.x & 31) == 0)
        of_warp[threadIdx.x >> 5] = top;
    asm volatile("barrier.cluster.wait.aligned;" ::: "memory");  // every CTA has started: its shared memory may be written
    __syncthreads();
    if (threadIdx.x < 32) {
        top = __reduce_max_sync(0xFFFFFFFFu, of_warp[threadIdx.x]);
        if (threadIdx.x < kCluster)  // lane r tells CTA r
            asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(mapa_shared(smem_u32(&of_cta[cluster_ctarank()]), threadIdx.x)),
                         "r"(top)
                         : "memory");
    }
    cluster_sync();
    top = 0;
#pragma unroll
    for (int r = 0; r < kCluster; ++r)
        top = max(top, of_cta[r]);
    const float b = __uint_as_float(top);
    const float ts = b == 0.0f ? 1.0f : __fdiv_rn(b, fmt_is_nvfp4(FMT) ? 2688.0f : 448.0f);
    if (first == 0) {
        *amax = b;
        *tensor_scale = ts;
    }
#pragma unroll
    for (int k = 0; k < kMaxOcts; ++k) {
        if (k * (kCluster * 1024) >= octs)
            break;
        const int oct = first + k * (kCluster * 1024);
        Oct o;
        unpack_oct(w[k], o);
        encode<FMT>(o, ts, oct < octs, oct, per_row, kgroups, codes, sf);
    }
}

template <int FMT>
int launch_few(const void* x, int64_t ld, const mx_tensor* out, unsigned* zero, int zeros, const Device& d, cudaStream_t s)
{
    const int per_row = static_cast<int>(out->k / 8), octs = static_cast<int>(out->rows) * per_row;
    const int64_t kgroups = sf_kgroups(out->k / fmt_block(FMT));
    uint8_t* codes = static_cast<uint8_t*>(out->codes);
    if constexpr (fmt_has_tensor_scale(FMT)) {
        static int configured_device = -1;
        if (configured_device != d.id) {
            if (cudaFuncSetAttribute(quantize_few_cluster_kernel<FMT>, cudaFuncAttributeNonPortableClusterSizeAllowed, 1) !=
                cudaSuccess)
                return MX_ERR_CUDA;
            configured_device = d.id;
        }
        return launch_kernel(quantize_few_cluster_kernel<FMT>, kCluster, 1, 1024, 0, true, s, x, ld, per_row, octs, kgroups,
                             codes, out->sf, out->amax, out->tensor_scale, zero, zeros);
    } else {
        return launch_kernel(quantize_few_kernel<FMT>, static_cast<unsigned>((octs + 255) / 256), 1, 256, 0, true, s, x, ld,
                             per_row, octs, kgroups, codes, out->sf, zero, zeros);
    }
}

}  // namespace

// With a tensor scale as many values as the cluster's registers hold; else any number that
// its 32-bit indexes reach.
bool quantize_few_takes(int fmt, int64_t rows, int64_t k)
{
    const int64_t most = fmt_has_tensor_scale(fmt) ? int64_t{kCluster} * 1024 * kMaxOcts * 8 : int64_t{1} << 33;
    return rows > 0 && rows <= kGatedFewTokens && k % 32 == 0 && rows * k <= most;
}

int launch_quantize_few(const void* x, int64_t ld, const mx_tensor* out, unsigned* zero, int zeros, const Device& d, cudaStream_t s)
{
    switch (out->fmt) {
    case MX_FMT_MXFP8_E4M3: return launch_few<MX_FMT_MXFP8_E4M3>(x, ld, out, zero, zeros, d, s);
    case MX_FMT_MXFP4_E2M1: return launch_few<MX_FMT_MXFP4_E2M1>(x, ld, out, zero, zeros, d, s);
    case MX_FMT_MOSS_FP8: return launch_few<MX_FMT_MOSS_FP8>(x, ld, out, zero, zeros, d, s);
    default: return launch_few<MX_FMT_NVFP4>(x, ld, out, zero, zeros, d, s);  // one region at most: the local scale is the tensor's
    }
}

}  // namespace mx
