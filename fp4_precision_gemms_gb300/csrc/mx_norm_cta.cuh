// mx_norm_cta.cuh -- what the norm's kernels for rows of 513 to 16384 columns
// share (norm_cta_fwd.cu, norm_cta_bwd.cu).
//
// A CTA takes a row at a time (forward without a residual: two), NV octs (eight
// columns) a thread, with the column sums of the backward pass in registers over
// all of its rows.  Two octs up to 8192 columns: the weights, the biases and a
// row's g and h stay in registers too.  Four above: those are read again.  One
// thread copies the rows to come into a ring of shared-memory stages by bulk
// copies, an mbarrier says when a stage is there, and the row sums' barrier that
// the stage before it may be filled again.
//
// What bounds them: with the ring the memory system is never idle, and what is
// left is the number of instructions a row takes.  The options are therefore
// compile-time and fp32 arithmetic is two-wide; two rows of the forward kernel
// share one barrier and one exchange per sum.  8192x4096 bf16 measured: forward
// with residual, checkpoint and maximum 52 us (303 MB, 5.9 TB/s; 65536 rows 6.6),
// backward from the checkpoint with the residual's gradient 45.5 us (236 MB, 5.2
// TB/s; 65536 rows 6.8), of which the partial sums and their join take 5; layer
// norm alone at 32768 rows 90 us (537 MB, 5.9 TB/s).  At odd addresses the
// shifts double the instructions: 8192x4099 fp32 in, bf16 out 61 us, where
// 8192x4096 takes 34.
#pragma once
#include <algorithm>

#include "mx_act8.cuh"
#include "mx_internal.cuh"
#include "mx_norm.cuh"
#include "mx_ptx.cuh"

namespace mx {
namespace {

constexpr int kMaxThreads = 512;  // 128 registers each
constexpr int kMaxStages = 6;
constexpr int kBarBytes = kRingExtra;
constexpr int kWarps = kMaxThreads / 32;

// The ring: PARTS matrices, R rows of each in a stage.  ANY: rows at any address,
// one to a stage.  A stage then holds the aligned 16-byte words that a row lies
// in, and an oct is shifted into place when it is read.  The words may hold a
// neighbouring row's elements; the first and the last rows, whose words would
// reach past the matrix, are not copied but read where they are.
template <int PARTS, int R, bool ANY>
struct Pipe {
    static_assert(!ANY || R == 1, "rows at any address come one at a time");
    const char* src[PARTS];     // row 0
    int64_t next_row[PARTS];    // bytes
    uint32_t row_bytes[PARTS];  // of a row, or of its words' room (ANY)
    uint32_t length[PARTS];     // ANY: bytes of a row
    uint32_t at[PARTS];         // in a stage
    uint32_t shift[PARTS], shift_step[PARTS];  // ANY: the row's bytes past a boundary; what a step adds
    uint32_t bars, base, stage_bytes, here;    // here: the current stage
    int stages, stage = 0, skip;               // skip: test hook, a tile that is never copied
    uint32_t phase = 0;
    int64_t edge = 1;     // ANY: rows at either end that are not copied
    bool direct = false;  // ANY: this row is one of them

    // A matrix of rows of n bytes; words: they start on 16-byte boundaries.
    __device__ __forceinline__ void matrix(int m, const void* p, int64_t row, uint32_t n, bool words)
    {
        src[m] = static_cast<const char*>(p);
        next_row[m] = row;
        length[m] = n;
        row_bytes[m] = room(n, ANY && !words);
        if (ANY && row < 16)
            edge = 16;
    }
    __host__ __device__ static constexpr uint32_t room(uint32_t n, bool any) { return any ? (n + 15) / 16 * 16 + 32 : n; }
    __device__ __forceinline__ uint32_t shift_of(int m, int64_t r) const
    {
        return static_cast<uint32_t>(reinterpret_cast<uintptr_t>(src[m]) + r * next_row[m]) & 15u;
    }
    __device__ __forceinline__ bool at_edge(int64_t r, int64_t rows) const { return ANY && (r < edge || r >= rows - edge); }

    __device__ __forceinline__ void layout(uint8_t* smem, int stages_, int skip_, int64_t rows)
    {
        stages = stages_;
        skip = skip_;
        bars = smem_u32(smem);
        here = base = bars + kBarBytes;
        uint32_t n = 0;
#pragma unroll
        for (int m = 0; m < PARTS; ++m) {
            at[m] = n;
            n += R * row_bytes[m];
            if constexpr (ANY) {
                shift[m] = shift_of(m, blockIdx.x);
                shift_step[m] = static_cast<uint32_t>(gridDim.x * next_row[m]) & 15u;
            }
        }
        stage_bytes = n;
        direct = at_edge(blockIdx.x, rows);
    }
    // Tile `it` (rows r, r + 1 ..) of the CTA into stage st (one thread).
    __device__ __forceinline__ void fill(int it, int64_t rows, int st)
    {
        if (it == skip)
            return;
        const int64_t r = (blockIdx.x + static_cast<int64_t>(it) * gridDim.x) * R;
        const uint32_t bar = bars + st * 8, to = base + st * stage_bytes;
        if constexpr (ANY) {
            if (at_edge(r, rows)) {
                mbar_arrive(bar);
                return;
            }
            uint32_t bytes = 0;
#pragma unroll
            for (int m = 0; m < PARTS; ++m)
                bytes += (shift_of(m, r) + length[m] + 15) / 16 * 16;
            mbar_arrive_expect_tx(bar, bytes);
#pragma unroll
            for (int m = 0; m < PARTS; ++m)
                bulk_load(to + at[m], src[m] + r * next_row[m] - shift_of(m, r), (shift_of(m, r) + length[m] + 15) / 16 * 16, bar);
        } else {
            const int n = static_cast<int>(min(static_cast<int64_t>(R), rows - r));
            uint32_t bytes = 0;
#pragma unroll
            for (int m = 0; m < PARTS; ++m)
                bytes += n * row_bytes[m];
            mbar_arrive_expect_tx(bar, bytes);
#pragma unroll
            for (int m = 0; m < PARTS; ++m)
                for (int i = 0; i < n; ++i)
                    bulk_load(to + at[m] + i * row_bytes[m], src[m] + (r + i) * next_row[m], row_bytes[m], bar);
        }
    }
    // Barriers and the first tiles; ends with a CTA barrier.
    __device__ __forceinline__ void start(int64_t rows, int tiles)
    {
        if (threadIdx.x == 0) {
            for (int i = 0; i < stages; ++i)
                mbar_init(bars + i * 8, 1);
            fence_mbar_init();
            for (int i = 0; i < stages && i < tiles; ++i)
                fill(i, rows, i);
        }
        __syncthreads();
    }
    __device__ __forceinline__ bool wait(uint64_t limit_ns) { return mbar_wait_bounded(bars + stage * 8, phase, limit_ns); }
    // After a barrier that follows every thread's last reading of tile it's stage.
    __device__ __forceinline__ void refill(int it, int64_t rows, int tiles, int st)
    {
        if (threadIdx.x == 0 && it >= 0 && it + stages < tiles)
            fill(it + stages, rows, st);
    }
    __device__ __forceinline__ int before() const { return stage == 0 ? stages - 1 : stage - 1; }
    // On to the tile that begins with row r.
    __device__ __forceinline__ void next(int64_t r, int64_t rows)
    {
        if constexpr (ANY) {
#pragma unroll
            for (int m = 0; m < PARTS; ++m)
                shift[m] = (shift[m] + shift_step[m]) & 15u;
            direct = at_edge(r, rows);
        }
        here += stage_bytes;
        if (++stage == stages) {
            stage = 0;
            here = base;
            phase ^= 1;
        }
    }
    // A wait of tile `it` ran out: those in flight (the newest is tile
    // last - 1) are waited for before the CTA's memory goes back.
    __device__ __forceinline__ void abandon(int it, int last, uint64_t limit_ns, int* status)
    {
        if (threadIdx.x != 0)
            return;
        atomicExch(status, MX_ERR_TIMEOUT);
        for (; it < last; ++it) {
            wait(limit_ns);
            next(0, 0);
        }
    }

    // Oct j of row r (number q of its tile) of matrix m, whose first n values
    // (n > 0) are inside the row.
    template <typename T>
    __device__ __forceinline__ void oct(int m, int q, int j, int64_t r, int n, Oct& o) const
    {
        const uint32_t from = here + at[m] + q * row_bytes[m] + (threadIdx.x + j * blockDim.x) * (8 * sizeof(T));
        if constexpr (!ANY) {
            if constexpr (sizeof(T) == 2)
                unpack_oct(lds128(from), o);
            else
                words_to_oct(lds128(from), lds128(from + 16), o);
        } else {
            if (direct) {
                const T* p = reinterpret_cast<const T*>(src[m] + r * next_row[m]) + (threadIdx.x + j * blockDim.x) * 8;
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    o[i] = i < n ? load_f(p + i) : 0.0f;
                return;
            }
            const int s = static_cast<int>(shift[m] / sizeof(T));
            if constexpr (sizeof(T) == 2) {
                unpack_oct(shifted(lds128(from), lds128(from + 16), s), o);
            } else {
                uint4 lo, hi;
                shifted(lds128(from), lds128(from + 16), lds128(from + 32), s, lo, hi);
                words_to_oct(lo, hi, o);
            }
            if (n < 8)
                keep_first(o, n);
        }
    }
    // Oct j of a checkpoint's codes, as their own values.
    __device__ __forceinline__ void codes(int m, int j, int64_t r, Oct& o) const
    {
        const uint32_t c = (threadIdx.x + j * blockDim.x) * 8;
        uint2 w;
        if (ANY && direct)
            w = *reinterpret_cast<const uint2*>(src[m] + r * next_row[m] + c);
        else
            asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];" : "=r"(w.x), "=r"(w.y) : "r"(here + at[m] + c) : "memory");
        decode_oct(w, o);
    }
};

// Writes n values of an oct (ANY: by whole warps).
template <bool ANY, typename T>
__device__ __forceinline__ void put(T* p, const Oct& o, int n, int c, int C, Top<T>& top)
{
    if constexpr (ANY) {
        const int lane = threadIdx.x & 31;
        store_ragged(p, o, n, lane > 0, lane < 31 && c + 8 < C, top);
    } else if (n > 0) {
        store_oct(p, o, top);
    }
}
template <bool ANY>
__device__ __forceinline__ void params(const void* p, int dtype, int c, int n, float absent, Oct& o)
{
    o.fill(0.0f);
    if (ANY && (n < 8 || (reinterpret_cast<uintptr_t>(p) & 15) != 0)) {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (i < n)
                o[i] = param(p, dtype, c + i, absent);
    } else if (n > 0) {
        param_oct(p, dtype, c, absent, o);
    }
}

// Two sums over the CTA, in a fixed order, known to every thread.  The halves of
// a warp exchange them, so that each half finishes one; `part` has an entry a
// warp, zero past the CTA's.  The barrier also collects `bad`.
__device__ __forceinline__ float2 cta_sum2(float x, float y, float2* part, bool& bad)
{
    const bool second = threadIdx.x & 16;
    float s = second ? y : x;
    s += __shfl_xor_sync(0xFFFFFFFFu, second ? x : y, 16);
#pragma unroll
    for (int o = 8; o > 0; o >>= 1)
        s += __shfl_xor_sync(0xFFFFFFFFu, s, o);
    if ((threadIdx.x & 15) == 0)
        reinterpret_cast<float*>(part)[threadIdx.x >> 4] = s;
    bad = __syncthreads_or(bad);
    const float4* p = reinterpret_cast<const float4*>(part);
    float2 sum = make_float2(0.0f, 0.0f);
#pragma unroll
    for (int w = 0; w < 4; ++w)
        sum = __fadd2_rn(sum, __fadd2_rn(make_float2(p[w].x, p[w].y), make_float2(p[w].z, p[w].w)));
    if (blockDim.x > 256)
#pragma unroll
        for (int w = 4; w < 8; ++w)
            sum = __fadd2_rn(sum, __fadd2_rn(make_float2(p[w].x, p[w].y), make_float2(p[w].z, p[w].w)));
    return sum;
}

// CTAs an SM that registers allow, with at least two stages each where that can be.
template <auto KERNEL>
int ctas_per_sm(int threads, int64_t stage_bytes)
{
    int n = resident_ctas<KERNEL>(threads);
    while (n > 1 && n * 2 * stage_bytes > kRingBytes)
        --n;
    return n;
}
template <auto KERNEL, typename A>
int launch(const A& a, int threads, int64_t stage_bytes, int per_sm, unsigned grid, const Device& d, cudaStream_t s)
{
    const int stages =
        static_cast<int>(std::max<int64_t>(1, std::min<int64_t>(kMaxStages, kRingBytes / (per_sm * stage_bytes))));
    const size_t smem = static_cast<size_t>(stage_bytes) * stages + kBarBytes;
    if (const int rc = allow_ring<KERNEL>(smem, d); rc != MX_OK)
        return rc;
    return launch_kernel(KERNEL, grid, 1, threads, smem, a.amax != nullptr, s, a, stages);
}

// How the rows of a call lie: every thread's octs inside the row, some past it,
// or rows at any address.
enum Rows { kFull, kPart, kAny };

// Above 8192 columns the rows may always end before a thread's octs do (as
// kPart), which halves the kernels there.
inline bool full_rows(int64_t cols) { return cols == 16 * cta_threads(cols); }

}  // namespace
}  // namespace mx
