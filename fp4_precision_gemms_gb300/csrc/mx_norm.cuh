// mx_norm.cuh -- what the norm's translation units share.
#pragma once
#include <atomic>

#include "mx_act8.cuh"
#include "mx_internal.cuh"

namespace mx {

// Weight or bias c (`absent` without one).
__device__ __forceinline__ float param(const void* p, int dtype, int64_t c, float absent)
{
    if (!p)
        return absent;
    return dtype == MX_OUT_BF16 ? load_f(static_cast<const __nv_bfloat16*>(p) + c) : static_cast<const float*>(p)[c];
}
// Eight of them, from a 16-byte boundary.
__device__ __forceinline__ void param_oct(const void* p, int dtype, int c, float absent, Oct& o)
{
    if (!p) {
        o.fill(absent);
    } else if (dtype == MX_OUT_BF16) {
        unpack_oct(__ldg(reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(p) + c)), o);
    } else {
        const uint4* q = reinterpret_cast<const uint4*>(static_cast<const float*>(p) + c);
        words_to_oct(__ldg(q), __ldg(q + 1), o);
    }
}

// Floats from one row of partial sums to the next: rows of any width are written
// eight columns at a time.
__host__ __device__ inline int64_t part_stride(int64_t cols) { return (cols + 7) / 8 * 8; }

// The rings of rows in flight: bytes of an SM's shared memory that they take, all
// its CTAs together, and the words beside one.
constexpr int64_t kRingBytes = 220 * 1024;
constexpr int kRingExtra = 64;

// Lets KERNEL be launched with `bytes` of dynamic shared memory.  The limit is one
// of the kernel, not of the launch, and other host threads launch it with rings of
// other sizes: it is set once on a device, to the most that a ring can be.  Two
// threads that both come first set the same value.
template <auto KERNEL>
int allow_ring(size_t bytes, const Device& d)
{
    static std::atomic<uint64_t> set{0};  // a bit for each of the first 64 devices
    const uint64_t bit = d.id < 64 ? uint64_t{1} << d.id : 0;
    if (bytes <= 40 * 1024 || (set.load(std::memory_order_acquire) & bit))  // 48 KiB without asking, static words included
        return MX_OK;
    if (cudaFuncSetAttribute(KERNEL, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(kRingBytes) + kRingExtra) !=
        cudaSuccess) {
        (void)cudaGetLastError();
        return MX_ERR_CUDA;
    }
    set.fetch_or(bit, std::memory_order_release);
    return MX_OK;
}

// The kernels of norm_cta_fwd.cu and norm_cta_bwd.cu: columns they take, and a CTA's threads, two octs
// each up to kCtaTwoOcts columns and four above, whole checkpoint groups.
constexpr int64_t kCtaMinCols = 513, kCtaTwoOcts = 8192, kCtaMaxCols = 16384;
inline int cta_threads(int64_t cols)
{
    const int64_t octs = act8_groups(cols) * 4, nv = cols <= kCtaTwoOcts ? 2 : 4;
    return static_cast<int>(((octs + nv - 1) / nv + 31) / 32 * 32);
}
// aligned: rows on 16-byte boundaries of a multiple of eight columns.
int launch_norm_fwd_cta(const NormFwdArgs& a, bool aligned, const Device& d, cudaStream_t s);
// At most `most` CTAs; *grid returns their number, each of which leaves a row of
// partial sums.
int launch_norm_bwd_cta(const NormBwdArgs& a, bool aligned, int most, const Device& d, cudaStream_t s, unsigned* grid);

}  // namespace mx
