// norm.cu -- layer norm and RMS norm over the rows of a residual stream,
// forward and backward.
#include <algorithm>
#include <type_traits>

#include "mx_act8.cuh"
#include "mx_internal.cuh"
#include "mx_norm.cuh"
#include "mx_ptx.cuh"

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
    Top<TY> top;
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
        const float rstd = rsqrtf(cta_sum(sq, part) * inv_c + a.eps);
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
                top.value(o);
            }
            if (a.save.codes) {
                const float z = finite_or_nan(v);
                const float b = __uint_as_float(__reduce_max_sync(0xFFFFFFFFu, abs_bits(fmaxf(fabsf(z), 0.0f))));
                const uint32_t e = act8_byte(b);
                a.save.codes[(r * G + g) * kAct8Group + lane] =
                    static_cast<uint8_t>(cvt_e4m3x2(z * act8_inverse(e), 0.0f));
                if (lane == 0)
                    a.save.sf[r * G + g] = static_cast<uint8_t>(e);
            }
        }
    }
    if (a.amax)
        flush_top(a.amax, top);
}

// s of row r, column c: the kept tensor or the checkpoint.
template <typename T>
__device__ __forceinline__ float kept(const NormBwdArgs& a, int64_t r, int64_t c, int64_t G)
{
    if (a.x8.codes)
        return dec_e4m3x2(a.x8.codes[r * G * kAct8Group + c]).x * act8_scale(a.x8.sf[r * G + c / kAct8Group]);
    return load_f(static_cast<const T*>(a.x) + r * a.ldx + c);
}

// dx of row r.
template <typename T, typename TY>
__device__ __forceinline__ void dx_row(const NormBwdArgs& a, int64_t r, float* part, Top<T>& top)
{
    const int64_t C = a.cols, G = act8_groups(C);
    const float inv_c = 1.0f / static_cast<float>(C);
    const TY* dy = static_cast<const TY*>(a.dy) + r * a.ldy;
    const float rstd = a.rstd[r], mean = a.kind == MX_NORM_LAYER ? a.mean[r] : 0.0f;
    float sgh = 0.0f, sg = 0.0f;
#pragma unroll 4
    for (int64_t c = threadIdx.x; c < C; c += kRowThreads) {
        const float g = load_f(dy + c) * param(a.weight, a.w_dtype, c, 1.0f);
        sgh += g * ((kept<T>(a, r, c, G) - mean) * rstd);
        sg += g;
    }
    const float c1 = cta_sum(sgh, part) * inv_c;
    const float c2 = a.kind == MX_NORM_LAYER ? cta_sum(sg, part) * inv_c : 0.0f;
    const T* dres = static_cast<const T*>(a.dres) + r * a.ldres;
    T* dx = static_cast<T*>(a.dx) + r * a.lddx;
#pragma unroll 4
    for (int64_t c = threadIdx.x; c < C; c += kRowThreads) {
        const float g = load_f(dy + c) * param(a.weight, a.w_dtype, c, 1.0f);
        const float h = (kept<T>(a, r, c, G) - mean) * rstd;
        float v = (g - h * c1 - c2) * rstd;
        if (a.dres)
            v += load_f(dres + c);
        v = as_stored<T>(v);
        store_f(dx + c, v);
        top.value(v);
    }
}

// Sums over rows first, first + step .. of column c of the lane, this warp's
// share of them joined with the other warps' (in warp 0).
struct ColumnSums {
    float w, b;
};
template <typename T, typename TY>
__device__ __forceinline__ ColumnSums column_sums(const NormBwdArgs& a, int64_t c, int64_t first, int64_t step)
{
    __shared__ float pw[kRowWarps][32], pb[kRowWarps][32];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int64_t G = act8_groups(a.cols);
    ColumnSums s = {0.0f, 0.0f};
    if (c < a.cols)
#pragma unroll 4
        for (int64_t r = first + warp; r < a.rows; r += step) {
            const float dy = load_f(static_cast<const TY*>(a.dy) + r * a.ldy + c);
            const float mean = a.kind == MX_NORM_LAYER ? a.mean[r] : 0.0f;
            s.w += dy * ((kept<T>(a, r, c, G) - mean) * a.rstd[r]);
            s.b += dy;
        }
    pw[warp][lane] = s.w;
    pb[warp][lane] = s.b;
    __syncthreads();
    if (warp == 0)
#pragma unroll
        for (int i = 1; i < kRowWarps; ++i) {
            s.w += pw[i][lane];
            s.b += pb[i][lane];
        }
    return s;
}

template <typename T, typename TY>
__global__ void __launch_bounds__(kRowThreads) norm_dx_any_kernel(NormBwdArgs a)
{
    __shared__ float part[kRowWarps];
    Top<T> top;
    for (int64_t r = blockIdx.x; r < a.rows; r += gridDim.x)
        dx_row<T, TY>(a, r, part, top);
    if (a.amax)
        flush_top(a.amax, top);
}

// Partial column sums: CTA (x, y) adds 32 columns of every gridDim.y-th eight rows.
template <typename T, typename TY>
__global__ void __launch_bounds__(kRowThreads) norm_dw_any_kernel(NormBwdArgs a)
{
    let_next_launch_start();  // the join
    const int64_t C = a.cols, c = blockIdx.x * 32ll + (threadIdx.x & 31);
    const ColumnSums s = column_sums<T, TY>(a, c, blockIdx.y * kRowWarps, static_cast<int64_t>(gridDim.y) * kRowWarps);
    if (threadIdx.x < 32 && c < C) {
        a.parts[blockIdx.y * C + c] = s.w;
        a.parts[(gridDim.y + blockIdx.y) * C + c] = s.b;
    }
}

// Few short rows: dx by the CTAs first_cta .. a.rows - 1 and the finished column
// sums by those from a.rows on, without a workspace and, unless dx is the memory
// of dy or x, which both read, in one launch.
template <typename T, typename TY>
__global__ void __launch_bounds__(kRowThreads) norm_bwd_few_kernel(NormBwdArgs a, unsigned first_cta)
{
    __shared__ float part[kRowWarps];
    const int64_t cta = static_cast<int64_t>(blockIdx.x) + first_cta;
    if (cta < a.rows) {
        Top<T> top;
        dx_row<T, TY>(a, cta, part, top);
        if (a.amax)
            flush_top(a.amax, top);
        return;
    }
    const int64_t c = (cta - a.rows) * 32 + (threadIdx.x & 31);
    const ColumnSums s = column_sums<T, TY>(a, c, 0, kRowWarps);
    if (threadIdx.x < 32 && c < a.cols) {
        if (a.dw)
            a.dw[c] = s.w;
        if (a.db)
            a.db[c] = s.b;
    }
}

// dw and db from `parts` partial sums of each column (rows of parts: dw's, then
// db's), 32 columns and up to 32 runs of parts a CTA.
constexpr int kJoinWarps = 32;
__global__ void __launch_bounds__(kJoinWarps * 32) norm_dw_join_kernel(const float* __restrict__ src, int64_t C,
                                                                       int parts, float* __restrict__ dw,
                                                                       float* __restrict__ db)
{
    __shared__ float p[kJoinWarps][32];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int64_t c = blockIdx.x * 32ll + lane;
    float* out = blockIdx.y ? db : dw;
    wait_for_launch_before();
    if (!out)
        return;
    float v = 0.0f;
    if (c < C) {
        const float* from = src + (static_cast<int64_t>(blockIdx.y) * parts + warp) * C + c;
#pragma unroll 8
        for (int i = warp; i < parts; i += kJoinWarps, from += kJoinWarps * C)
            v += *from;
    }
    p[warp][lane] = v;
    __syncthreads();
    if (warp == 0 && c < C) {
        const int n = min(parts, kJoinWarps);
        for (int i = 1; i < n; ++i)
            v += p[i][lane];
        out[c] = v;
    }
}

// ------------------------------------------------------------------ wide
// Up to 16384 columns.  Eight columns (an oct) at a time: thread t of a row's TPR threads owns the octs t, t + TPR,
// ..., NV of them; octs past the row's end hold zeros, and a group's four octs
// lie in four neighbouring lanes.  LPR > 0: LPR lanes of a warp per row, the
// rows of a CTA independent; LPR = 0: the CTA's blockDim.x threads per row.
//
// The grid is persistent, and a shared-memory ring holds the rows that a CTA
// takes next, so that the memory system stays busy through the row sums.
//
// LPR = 0: one thread issues a bulk copy per matrix and row, which costs the
// other threads nothing (per-thread copies took about 60 of a warp's 470
// instructions a row); a stage's mbarrier says when it has arrived, and the
// barrier of the row sums that a row ago's stage may be filled again.
// LPR > 0: each thread copies its own words into its own slots, which needs no
// barrier between the warps' rows.
constexpr int kMaxWide = 16384;
constexpr int kSubThreads = 256;  // CTA size where several rows share a CTA
constexpr int kMaxThreads = 512;  // of a CTA: 128 registers each
constexpr int kMaxStages = 6;
constexpr int kBarBytes = (kMaxStages * 8 + 15) / 16 * 16;

template <typename T>
__device__ __forceinline__ constexpr int chunks() { return sizeof(T) / 2; }  // 16-byte words of an oct

template <int LPR>
struct RowMap {
    int tpr, t;          // threads of a row, this one's place among them
    int64_t first, step; // this thread's first row, rows from one to the next
    int mine, all;       // rows of this thread, iterations of the CTA
    __device__ __forceinline__ explicit RowMap(int64_t rows)
    {
        const int tid = threadIdx.x, per_cta = LPR ? kSubThreads / LPR : 1;
        tpr = LPR ? LPR : blockDim.x;
        t = LPR ? tid % LPR : tid;
        const int64_t cta = static_cast<int64_t>(blockIdx.x) * per_cta;
        step = static_cast<int64_t>(gridDim.x) * per_cta;
        first = cta + (LPR ? tid / LPR : 0);
        all = static_cast<int>((rows - cta + step - 1) / step);
        mine = first < rows ? static_cast<int>((rows - first + step - 1) / step) : 0;
    }
};

// Sums over a row's threads, known to all of them; a CTA's row goes through
// `part` (one entry a warp, zero past the CTA's; two of them used in turn, so
// that one barrier per sum is enough).
template <int LPR>
__device__ __forceinline__ float row_sum(float v, float* part, bool& bad)
{
#pragma unroll
    for (int o = (LPR ? LPR : 32) / 2; o > 0; o >>= 1)
        v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
    if constexpr (LPR == 0) {
        if ((threadIdx.x & 31) == 0)
            part[threadIdx.x >> 5] = v;
        bad = __syncthreads_or(bad);
        const float4 p = *reinterpret_cast<const float4*>(part), q = *reinterpret_cast<const float4*>(part + 4);
        float2 s = __fadd2_rn(__fadd2_rn(make_float2(p.x, p.y), make_float2(p.z, p.w)),
                              __fadd2_rn(make_float2(q.x, q.y), make_float2(q.z, q.w)));
        if (blockDim.x > 256) {
            const float4 t = *reinterpret_cast<const float4*>(part + 8), u = *reinterpret_cast<const float4*>(part + 12);
            s = __fadd2_rn(s, __fadd2_rn(__fadd2_rn(make_float2(t.x, t.y), make_float2(t.z, t.w)),
                                         __fadd2_rn(make_float2(u.x, u.y), make_float2(u.z, u.w))));
        }
        v = s.x + s.y;
    }
    return v;
}
// Two sums.  Where a warp belongs to one row its halves exchange the sums, so
// that each half finishes one of them.
template <int LPR>
__device__ __forceinline__ float2 row_sum2(float2 v, float2* part, bool& bad)
{
    if constexpr (LPR != 0 && LPR < 32) {
#pragma unroll
        for (int o = LPR / 2; o > 0; o >>= 1) {
            v.x += __shfl_xor_sync(0xFFFFFFFFu, v.x, o);
            v.y += __shfl_xor_sync(0xFFFFFFFFu, v.y, o);
        }
        return v;
    } else {
        const bool second = threadIdx.x & 16;
        float s = second ? v.y : v.x;
        s += __shfl_xor_sync(0xFFFFFFFFu, second ? v.x : v.y, 16);
#pragma unroll
        for (int o = 8; o > 0; o >>= 1)
            s += __shfl_xor_sync(0xFFFFFFFFu, s, o);
        if constexpr (LPR == 32)
            return make_float2(__shfl_sync(0xFFFFFFFFu, s, 0), __shfl_sync(0xFFFFFFFFu, s, 16));
        if ((threadIdx.x & 15) == 0)
            reinterpret_cast<float*>(part)[(threadIdx.x >> 5) * 2 + (second ? 1 : 0)] = s;
        bad = __syncthreads_or(bad);
        float2 sum = make_float2(0.0f, 0.0f);
#pragma unroll
        for (int w = 0; w < 8; w += 2) {
            const float4 p = *reinterpret_cast<const float4*>(part + w);
            sum = __fadd2_rn(sum, __fadd2_rn(make_float2(p.x, p.y), make_float2(p.z, p.w)));
        }
        if (blockDim.x > 256)
#pragma unroll
            for (int w = 8; w < 16; w += 2) {
                const float4 p = *reinterpret_cast<const float4*>(part + w);
                sum = __fadd2_rn(sum, __fadd2_rn(make_float2(p.x, p.y), make_float2(p.z, p.w)));
            }
        return sum;
    }
}

// Eight of the weights or biases.  ANY: at any address, those inside the row.
template <bool ANY>
__device__ __forceinline__ void param_oct(const void* p, int dtype, int c, int C, float absent, Oct& o)
{
    if constexpr (ANY) {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            o[i] = c + i < C ? param(p, dtype, c + i, absent) : 0.0f;
    } else {
        mx::param_oct(p, dtype, c, absent, o);
    }
}

// The ring of PARTS matrices.  A matrix may be absent (null).  Its octs take
// 16 (bf16), 32 (fp32) or 8 (codes) bytes.  ANY: rows at any address: a stage
// holds the aligned 16-byte words that a row lies in, one more than its octs
// fill, and an oct is shifted into place when it is read (codes always start on
// a boundary).  The words may hold a neighbouring row's elements; the first and
// the last rows (`edge` of them), whose words would reach past the matrix, are
// not copied but read where they are.
struct RingPart {
    const char* src;    // row 0
    int64_t next_row;   // bytes from one row to the next
    int oct;            // bytes of an oct
    uint32_t at;        // in a stage
};
__host__ __device__ constexpr uint32_t region_bytes(int octs, int oct, bool any)
{
    return (octs * oct + 15) / 16 * 16 + (any && oct != 8 ? 16 : 0);
}
template <int LPR, int NV, int PARTS, bool ANY>
struct RowRing {
    static constexpr int kLanes = LPR ? LPR : 1;
    RingPart part[PARTS];
    uint32_t base, stage_bytes, bars, at_stage = 0;
    int stages, stage = 0, octs, skip = -1;  // skip: test hook, a row that is never copied
    uint32_t phase = 0;
    int64_t rows, row = 0, edge = 1;
    bool direct = false;  // ANY: the current row is read from where it is
    uint32_t here_shift[PARTS], shift_step[PARTS];  // ANY: bytes past a boundary, the current row's and a step's

    __device__ __forceinline__ uint32_t region(int m) const { return region_bytes(octs, part[m].oct, ANY); }
    __device__ __forceinline__ uint32_t shift(int m, int64_t r) const  // bytes past a boundary
    {
        return ANY ? static_cast<uint32_t>(reinterpret_cast<uintptr_t>(part[m].src + r * part[m].next_row)) & 15u : 0u;
    }
    __device__ __forceinline__ bool at_edge(int64_t r) const { return ANY && (r < edge || r >= rows - edge); }

    __device__ __forceinline__ void layout(uint8_t* smem, int stages_, int cols, int64_t rows_)
    {
        stages = stages_;
        octs = (cols + 7) / 8;
        rows = rows_;
        bars = smem_u32(smem);
        base = bars + (LPR == 0 ? kBarBytes : 0);
        uint32_t at = 0;
#pragma unroll
        for (int m = 0; m < PARTS; ++m) {
            part[m].at = at;
            if (part[m].src) {
                at += LPR == 0 ? region(m) : ANY ? kSubThreads / kLanes * region(m) : NV * kSubThreads * part[m].oct;
                if (ANY && part[m].next_row < 16)
                    edge = 16;
            }
        }
        stage_bytes = at;
    }

    // The CTA's row number `it` into stage st: LPR = 0, one thread.
    __device__ __forceinline__ void fill(const RowMap<LPR>& map, int it, int st)
    {
        if (it == skip)
            return;
        const int64_t r = map.first + it * map.step;
        const uint32_t bar = bars + st * 8, to = base + st * stage_bytes;
        if (at_edge(r)) {
            mbar_arrive(bar);
            return;
        }
        uint32_t bytes = 0;
#pragma unroll
        for (int m = 0; m < PARTS; ++m)
            if (part[m].src)
                bytes += copied(m, r);
        mbar_arrive_expect_tx(bar, bytes);
#pragma unroll
        for (int m = 0; m < PARTS; ++m)
            if (part[m].src)
                bulk_load(to + part[m].at, part[m].src + r * part[m].next_row - shift(m, r), copied(m, r), bar);
    }
    // Bytes of the words that row r lies in.
    __device__ __forceinline__ uint32_t copied(int m, int64_t r) const
    {
        if constexpr (!ANY)
            return region(m);
        return part[m].oct == 8 ? region(m) : (shift(m, r) + row_bytes(m) + 15) / 16 * 16;
    }
    int cols_ = 0;
    __device__ __forceinline__ uint32_t row_bytes(int m) const { return static_cast<uint32_t>(cols_) * (part[m].oct / 8); }

    // LPR > 0: this thread's share of its row r into the stage `ahead` rows on.
    __device__ __forceinline__ void copy(int64_t r, bool in, int ahead, int t)
    {
        if (in && !at_edge(r)) {
            const int st = stage + ahead;
            const uint32_t to = base + (st >= stages ? st - stages : st) * stage_bytes;
#pragma unroll
            for (int m = 0; m < PARTS; ++m)
                if (part[m].src) {
                    const char* row_at = part[m].src + r * part[m].next_row;
                    if constexpr (ANY) {  // the row's words over its lanes
                        const uint32_t dst = to + part[m].at + (threadIdx.x / kLanes) * region(m);
                        const uint32_t n = copied(m, r);
                        row_at -= shift(m, r);
                        for (uint32_t w = t * 16; w < n; w += kLanes * 16)
                            copy_async16(dst + w, row_at + w);
                    } else {  // a thread's own octs
                        const int w = min(part[m].oct, 16);
#pragma unroll
                        for (int j = 0; j < NV; ++j)
                            if (t + j * kLanes < octs)
#pragma unroll
                                for (int h = 0; h < part[m].oct / w; ++h) {
                                    const uint32_t dst =
                                        to + part[m].at + ((j * (part[m].oct / w) + h) * kSubThreads + threadIdx.x) * w;
                                    const char* from = row_at + (t + j * kLanes) * part[m].oct + h * 16;
                                    if (w == 16)
                                        copy_async16(dst, from);
                                    else
                                        copy_async8(dst, from);
                                }
                    }
                }
        }
        copy_commit();
    }

    // The first rows.
    __device__ __forceinline__ void start(const RowMap<LPR>& map)
    {
        row = map.first;
        if constexpr (ANY)
#pragma unroll
            for (int m = 0; m < PARTS; ++m) {
                here_shift[m] = shift(m, row);
                shift_step[m] = static_cast<uint32_t>(map.step * part[m].next_row) & 15u;
            }
        if constexpr (LPR == 0) {
            if (threadIdx.x == 0) {
                for (int i = 0; i < stages; ++i)
                    mbar_init(bars + i * 8, 1);
                fence_mbar_init();
                for (int i = 0; i < stages && i < map.all; ++i)
                    fill(map, i, i);
            }
            __syncthreads();
        } else {
            for (int i = 0; i < stages - 1; ++i)
                copy(map.first + i * map.step, i < map.mine, i, map.t);
        }
    }
    // Row `it` has arrived (false: the wait gave up).
    __device__ __forceinline__ bool arrive(const RowMap<LPR>& map, int it, uint64_t limit_ns)
    {
        direct = at_edge(row);
        if constexpr (LPR == 0)
            return mbar_wait_bounded(bars + stage * 8, phase, limit_ns);
        copy(map.first + (it + stages - 1) * map.step, it + stages - 1 < map.mine, stages - 1, map.t);
        copy_wait(stages - 1);
        if (ANY)
            __syncwarp();
        return true;
    }
    // LPR = 0, after a barrier in row `it`: nobody reads row it - 1 any more.
    __device__ __forceinline__ void refill(const RowMap<LPR>& map, int it)
    {
        if (LPR == 0 && threadIdx.x == 0 && stages > 1 && it > 0 && it - 1 + stages < map.all)
            fill(map, it - 1 + stages, stage == 0 ? stages - 1 : stage - 1);
    }
    // The end of row `it`.
    __device__ __forceinline__ void done(const RowMap<LPR>& map, int it)
    {
        if (LPR == 0 && stages == 1) {
            __syncthreads();
            if (threadIdx.x == 0 && it + 1 < map.all)
                fill(map, it + 1, 0);
        }
        if (LPR != 0 && ANY)
            __syncwarp();  // the stage's next words may come from another lane
        row += map.step;
        if constexpr (ANY)
#pragma unroll
            for (int m = 0; m < PARTS; ++m)
                here_shift[m] = (here_shift[m] + shift_step[m]) & 15u;
        at_stage += stage_bytes;
        if (++stage == stages) {
            stage = 0;
            at_stage = 0;
            phase ^= 1;
        }
    }
    // Gave up in row `it`, before its refill: the copies in flight are waited
    // for before the CTA's memory goes back.
    __device__ __forceinline__ void abandon(const RowMap<LPR>& map, int it, uint64_t limit_ns)
    {
        if (LPR == 0 && threadIdx.x == 0)
            for (int i = it; i < map.all && i < (it > 0 && stages > 1 ? it - 1 : it) + stages; ++i) {
                mbar_wait_bounded(bars + stage * 8, phase, limit_ns);
                if (++stage == stages) {
                    stage = 0;
                    phase ^= 1;
                }
            }
    }

    // Address of word h of oct j of matrix m in the current stage.
    __device__ __forceinline__ uint32_t word(int m, int j, int h) const
    {
        const uint32_t at = base + at_stage + part[m].at;
        if constexpr (LPR == 0)
            return at + (threadIdx.x + j * blockDim.x) * part[m].oct + h * 16;
        if constexpr (ANY)
            return at + threadIdx.x / kLanes * region(m) + (threadIdx.x % kLanes + j * kLanes) * part[m].oct + h * 16;
        const int w = min(part[m].oct, 16);
        return at + ((j * (part[m].oct / w) + h) * kSubThreads + threadIdx.x) * w;
    }
    // Oct j, at column c, with n > 0 values inside the row.
    template <typename T>
    __device__ __forceinline__ void read(int m, int j, int c, int n, Oct& o) const
    {
        if constexpr (!ANY) {
            if constexpr (sizeof(T) == 2)
                unpack_oct(lds128(word(m, j, 0)), o);
            else
                words_to_oct(lds128(word(m, j, 0)), lds128(word(m, j, 1)), o);
        } else {
            if (direct) {
                const T* from = reinterpret_cast<const T*>(part[m].src + row * part[m].next_row) + c;
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    o[i] = i < n ? load_f(from + i) : 0.0f;
                return;
            }
            const int s = static_cast<int>(here_shift[m] / sizeof(T));
            if constexpr (sizeof(T) == 2) {
                unpack_oct(shifted(lds128(word(m, j, 0)), lds128(word(m, j, 1)), s), o);
            } else {
                uint4 lo, hi;
                shifted(lds128(word(m, j, 0)), lds128(word(m, j, 1)), lds128(word(m, j, 2)), s, lo, hi);
                words_to_oct(lo, hi, o);
            }
            if (n < 8)
                keep_first(o, n);
        }
    }
    // A checkpoint's codes, as their own values (the pad columns' are zero).
    __device__ __forceinline__ void read_codes(int m, int j, int c, Oct& o) const
    {
        uint2 w;
        if (ANY && direct)
            w = *reinterpret_cast<const uint2*>(part[m].src + row * part[m].next_row + c);
        else
            asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];" : "=r"(w.x), "=r"(w.y) : "r"(word(m, j, 0)) : "memory");
        decode_oct(w, o);
    }
};

// Writes an oct at column c: n of its values, none of them for n <= 0.
template <bool ANY, typename T>
__device__ __forceinline__ void put_oct(T* p, const Oct& o, int n, int c, int C, Top<T>& top)
{
    if constexpr (ANY) {
        const int lane = threadIdx.x & 31;
        store_ragged(p, o, n, lane > 0 && c > 0, lane < 31 && c + 8 < C && n > 0, top);
    } else if (n > 0) {
        store_oct(p, o, top);
    }
}

template <typename T, typename TY, int LPR, int NV, bool ANY>
__global__ void __maxnreg__(ANY || NV > 2 ? 112 : 96) norm_fwd_kernel(NormFwdArgs a, int stages)
{
    extern __shared__ __align__(16) uint8_t ring[];
    __shared__ __align__(16) float part[2][kMaxThreads / 32];
    if (LPR == 0) {
        if (threadIdx.x < kMaxThreads / 32)
            part[0][threadIdx.x] = part[1][threadIdx.x] = 0.0f;
        __syncthreads();
    }
    const RowMap<LPR> map(a.rows);
    const int C = static_cast<int>(a.cols), G = (C + kAct8Group - 1) / kAct8Group;
    const int c0 = 8 * map.t, dc = 8 * map.tpr;  // columns of oct j: c0 + j dc ..
    const float inv_c = 1.0f / static_cast<float>(C);
    const bool layer = a.kind == MX_NORM_LAYER, add = a.residual != nullptr;
    RowRing<LPR, NV, 2, ANY> ring_;
    ring_.part[0] = {static_cast<const char*>(a.x), a.ldx * static_cast<int64_t>(sizeof(T)), 8 * sizeof(T), 0};
    ring_.part[1] = {static_cast<const char*>(a.residual), a.ldr * static_cast<int64_t>(sizeof(T)), 8 * sizeof(T), 0};
    ring_.cols_ = C;
    ring_.layout(ring, stages, C, a.rows);
    auto count = [&](bool in, int j) { return in ? min(C - c0 - j * dc, 8) : 0; };  // an oct's values

    constexpr bool KEEP = NV <= 2;  // weights and biases stay in registers
    Oct wt[KEEP ? NV : 1], bi[KEEP ? NV : 1];
    if constexpr (KEEP)
#pragma unroll
        for (int j = 0; j < NV; ++j)
            if (c0 + j * dc < C) {
                param_oct<ANY>(a.weight, a.w_dtype, c0 + j * dc, C, 1.0f, wt[j]);
                param_oct<ANY>(a.bias, a.w_dtype, c0 + j * dc, C, 0.0f, bi[j]);
            }
    Top<TY> top;
    Top<T> sum_top;
    T* to_sum = static_cast<T*>(a.sum_out) + map.first * a.lds + c0;
    TY* to_y = static_cast<TY*>(a.y) + map.first * a.ldy + c0;
    uint8_t* to_codes = a.save.codes + map.first * (G * kAct8Group) + c0;
    uint8_t* to_sf = a.save.sf + map.first * G + c0 / kAct8Group;
    const int64_t sum_step = map.step * a.lds, y_step = map.step * a.ldy;
    const int64_t codes_step = map.step * (G * kAct8Group), sf_step = map.step * G;
    ring_.skip = a.fail_at;
    ring_.start(map);
    bool bad = false;
    int it = 0;
    for (; it < map.all; ++it) {
        bad = !ring_.arrive(map, it, a.wait_ns);
        const bool in = it < map.mine;
        Oct v[NV];
        float2 sum2 = make_float2(0.0f, 0.0f);
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            const int n = count(in, j);
            v[j].fill(0.0f);
            if (n > 0)
                ring_.template read<T>(0, j, c0 + j * dc, n, v[j]);
            if (add) {
                Oct q;
                q.fill(0.0f);
                if (n > 0)
                    ring_.template read<T>(1, j, c0 + j * dc, n, q);
#pragma unroll
                for (int k = 0; k < 4; ++k)
                    q.p[k] = __fadd2_rn(v[j].p[k], q.p[k]);
                put_oct<ANY>(to_sum + j * dc, q, n, c0 + j * dc, C, sum_top);
                if constexpr (sizeof(T) == 2)
                    unpack_oct(pack_oct(q), v[j]);  // as it was stored
                else
                    v[j] = q;
            }
#pragma unroll
            for (int k = 0; k < 4; ++k)
                sum2 = __fadd2_rn(sum2, v[j].p[k]);
        }
        float mean = 0.0f;
        if (layer) {
            mean = row_sum<LPR>(sum2.x + sum2.y, part[0], bad) * inv_c;
            if (LPR == 0 && bad)
                break;
        }
        float2 sq2 = make_float2(0.0f, 0.0f);
#pragma unroll
        for (int j = 0; j < NV; ++j)
            if (c0 + j * dc < C) {
                Oct d;
#pragma unroll
                for (int k = 0; k < 4; ++k)
                    d.p[k] = __fadd2_rn(v[j].p[k], both(-mean));
                if (ANY && C - c0 - j * dc < 8)
                    keep_first(d, C - c0 - j * dc);
#pragma unroll
                for (int k = 0; k < 4; ++k)
                    sq2 = __ffma2_rn(d.p[k], d.p[k], sq2);
            }
        // RMS norm has one sum per row: its words alternate with the row
        const float rstd = rsqrtf(row_sum<LPR>(sq2.x + sq2.y, part[layer ? 1 : it & 1], bad) * inv_c + a.eps);
        if (LPR == 0 && bad)
            break;
        ring_.refill(map, it);
        if (map.t == 0 && in) {
            const int64_t r = map.first + it * map.step;
            if (a.mean && layer)
                a.mean[r] = mean;
            if (a.rstd)
                a.rstd[r] = rstd;
        }
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            const int n = count(in, j);
            Oct &w = wt[KEEP ? j : 0], &b = bi[KEEP ? j : 0], y;
            if (!KEEP && n > 0) {
                param_oct<ANY>(a.weight, a.w_dtype, c0 + j * dc, C, 1.0f, w);
                param_oct<ANY>(a.bias, a.w_dtype, c0 + j * dc, C, 0.0f, b);
            }
            if (ANY || n > 0) {
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const float2 h = __fmul2_rn(__fadd2_rn(v[j].p[k], both(-mean)), both(rstd));
                    y.p[k] = __ffma2_rn(h, w.p[k], b.p[k]);
                }
                put_oct<ANY>(to_y + j * dc, y, n, c0 + j * dc, C, top);
            }
            if (a.save.codes) {
                uint8_t e;
                const uint2 codes = encode_oct(v[j], e);
                if (in && c0 + j * dc < G * kAct8Group) {
                    *reinterpret_cast<uint2*>(to_codes + j * dc) = codes;
                    if ((threadIdx.x & 3) == 0)
                        to_sf[j * dc / kAct8Group] = e;
                }
            }
        }
        to_sum += sum_step;
        to_y += y_step;
        to_codes += codes_step;
        to_sf += sf_step;
        ring_.done(map, it);
    }
    if (LPR == 0 && bad) {
        if (threadIdx.x == 0)
            atomicExch(a.status, MX_ERR_TIMEOUT);
        ring_.abandon(map, it, a.wait_ns);
        return;
    }
    if (a.amax)
        flush_top(a.amax, top);
}

// dx of each row and the CTA's partial sums of dw and db.  FROM8: the kept input
// is the checkpoint.  The column sums stay in registers over all rows of the
// CTA; dy h and g h come from one reading of the row, dx from what was kept of
// it in registers (up to two octs a thread) or from a second reading of shared
// memory.
template <typename T, typename TY, bool FROM8, int LPR, int NV, bool ANY>
__global__ void __launch_bounds__(LPR ? kSubThreads : kMaxThreads, LPR ? 2 : 1) norm_bwd_kernel(NormBwdArgs a, int stages)
{
    let_next_launch_start();  // the join of the partial sums
    constexpr bool KEEP = NV <= 2;
    extern __shared__ __align__(16) uint8_t ring[];
    __shared__ __align__(16) float2 part[2][kMaxThreads / 32];
    if (LPR == 0) {
        if (threadIdx.x < kMaxThreads / 32)
            part[0][threadIdx.x] = part[1][threadIdx.x] = make_float2(0.0f, 0.0f);
        __syncthreads();
    }
    const RowMap<LPR> map(a.rows);
    const int C = static_cast<int>(a.cols), G = (C + kAct8Group - 1) / kAct8Group;
    const int c0 = 8 * map.t, dc = 8 * map.tpr;
    const float inv_c = 1.0f / static_cast<float>(C);
    const bool layer = a.kind == MX_NORM_LAYER, add = a.dres != nullptr;
    RowRing<LPR, NV, 3, ANY> ring_;
    ring_.part[0] = {static_cast<const char*>(a.dy), a.ldy * static_cast<int64_t>(sizeof(TY)), 8 * sizeof(TY), 0};
    if constexpr (FROM8)
        ring_.part[1] = {reinterpret_cast<const char*>(a.x8.codes), G * int64_t{kAct8Group}, 8, 0};
    else
        ring_.part[1] = {static_cast<const char*>(a.x), a.ldx * static_cast<int64_t>(sizeof(T)), 8 * sizeof(T), 0};
    ring_.part[2] = {static_cast<const char*>(a.dres), a.ldres * static_cast<int64_t>(sizeof(T)), 8 * sizeof(T), 0};
    ring_.cols_ = C;
    ring_.layout(ring, stages, C, a.rows);
    auto count = [&](bool in, int j) { return in ? min(C - c0 - j * dc, 8) : 0; };  // an oct's values

    struct RowWords {  // what a row needs beside its matrices, loaded a row ahead
        float mean, rstd;
        uint32_t e[NV];
    };
    const float* from_mean = a.mean + map.first;
    const float* from_rstd = a.rstd + map.first;
    const uint8_t* from_sf = a.x8.sf + map.first * G + c0 / kAct8Group;
    auto row_words = [&](bool in) {
        RowWords w;
        w.mean = in && layer ? *from_mean : 0.0f;
        w.rstd = in ? *from_rstd : 0.0f;
#pragma unroll
        for (int j = 0; j < NV; ++j)
            w.e[j] = FROM8 && in && c0 + j * dc < C ? from_sf[j * dc / kAct8Group] : 127u;
        from_mean += map.step;
        from_rstd += map.step;
        from_sf += map.step * G;
        return w;
    };

    Oct wt[KEEP ? NV : 1];
    if constexpr (KEEP)
#pragma unroll
        for (int j = 0; j < NV; ++j)
            if (c0 + j * dc < C)
                param_oct<ANY>(a.weight, a.w_dtype, c0 + j * dc, C, 1.0f, wt[j]);
    Oct dw[NV], db[NV];
#pragma unroll
    for (int j = 0; j < NV; ++j) {
        dw[j].fill(0.0f);
        db[j].fill(0.0f);
    }
    Top<T> top;
    T* to_dx = static_cast<T*>(a.dx) + map.first * a.lddx + c0;
    const int64_t dx_step = map.step * a.lddx;
    ring_.skip = a.fail_at;
    ring_.start(map);
    RowWords next = row_words(0 < map.mine);
    bool bad = false;
    int it = 0;
    for (; it < map.all; ++it) {
        const bool in = it < map.mine;
        const RowWords cur = next;
        next = row_words(it + 1 < map.mine);
        bad = !ring_.arrive(map, it, a.wait_ns);
        // dy, and g and h of oct j
        auto load = [&](int j, int n, Oct& dy, Oct& g, Oct& h) {
            ring_.template read<TY>(0, j, c0 + j * dc, n, dy);
            if constexpr (FROM8) {
                ring_.read_codes(1, j, c0 + j * dc, h);
                const float2 scale = both(act8_scale(cur.e[j]));
#pragma unroll
                for (int k = 0; k < 4; ++k)  // the product is exact
                    h.p[k] = __ffma2_rn(h.p[k], scale, both(-cur.mean));
            } else {
                ring_.template read<T>(1, j, c0 + j * dc, n, h);
#pragma unroll
                for (int k = 0; k < 4; ++k)
                    h.p[k] = __fadd2_rn(h.p[k], both(-cur.mean));
            }
            if constexpr (KEEP)
                g = wt[j];
            else
                param_oct<ANY>(a.weight, a.w_dtype, c0 + j * dc, C, 1.0f, g);
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                h.p[k] = __fmul2_rn(h.p[k], both(cur.rstd));
                g.p[k] = __fmul2_rn(g.p[k], dy.p[k]);  // zero past the row's end, as dy
            }
        };
        Oct kg[KEEP ? NV : 1], kh[KEEP ? NV : 1];
        float2 sgh = make_float2(0.0f, 0.0f), sg = sgh;
#pragma unroll
        for (int j = 0; j < NV; ++j)
            if (const int n = count(in, j); n > 0) {
                Oct dy, &g = kg[KEEP ? j : 0], &h = kh[KEEP ? j : 0];
                load(j, n, dy, g, h);
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    sgh = __ffma2_rn(g.p[k], h.p[k], sgh);
                    sg = __fadd2_rn(sg, g.p[k]);
                    dw[j].p[k] = __ffma2_rn(dy.p[k], h.p[k], dw[j].p[k]);
                    db[j].p[k] = __fadd2_rn(db[j].p[k], dy.p[k]);
                }
            }
        const float2 s = row_sum2<LPR>(make_float2(sgh.x + sgh.y, sg.x + sg.y), part[it & 1], bad);
        if (LPR == 0 && bad)
            break;
        ring_.refill(map, it);
        const float2 c1 = both(-s.x * inv_c), c2 = both(layer ? -s.y * inv_c : 0.0f);
#pragma unroll
        for (int j = 0; j < NV; ++j)
            if (const int n = count(in, j); ANY || n > 0) {
                Oct dy, q, &g = kg[KEEP ? j : 0], &h = kh[KEEP ? j : 0];
                q.fill(0.0f);
                if (n > 0) {
                    if constexpr (!KEEP)
                        load(j, n, dy, g, h);
                    if (add)
                        ring_.template read<T>(2, j, c0 + j * dc, n, q);
                }
#pragma unroll
                for (int k = 0; k < 4; ++k)
                    q.p[k] = __ffma2_rn(__fadd2_rn(__ffma2_rn(h.p[k], c1, g.p[k]), c2), both(cur.rstd), q.p[k]);
                put_oct<ANY>(to_dx + j * dc, q, n, c0 + j * dc, C, top);
            }
        to_dx += dx_step;
        ring_.done(map, it);
    }
    if (LPR == 0 && bad) {
        if (threadIdx.x == 0)
            atomicExch(a.status, MX_ERR_TIMEOUT);
        ring_.abandon(map, it, a.wait_ns);
        return;
    }
    if (a.amax)
        flush_top(a.amax, top);
    if (!a.dw && !a.db)
        return;
    float* const out = a.parts + static_cast<int64_t>(blockIdx.x) * C;
    const int64_t to_db = static_cast<int64_t>(gridDim.x) * C;
    if constexpr (LPR == 0) {
#pragma unroll
        for (int j = 0; j < NV; ++j)
            if (ANY) {
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    if (c0 + j * dc + i < C) {
                        out[c0 + j * dc + i] = dw[j][i];
                        out[to_db + c0 + j * dc + i] = db[j][i];
                    }
            } else if (c0 + j * dc < C)
#pragma unroll
                for (int k = 0; k < 4; k += 2) {
                    float* const to = out + c0 + j * dc + 2 * k;
                    *reinterpret_cast<float4*>(to) =
                        make_float4(dw[j].p[k].x, dw[j].p[k].y, dw[j].p[k + 1].x, dw[j].p[k + 1].y);
                    *reinterpret_cast<float4*>(to + to_db) =
                        make_float4(db[j].p[k].x, db[j].p[k].y, db[j].p[k + 1].x, db[j].p[k + 1].y);
                }
    } else {
        // the rows of a warp, then the warps through shared memory, in order
        constexpr int kWarpCols = NV * LPR * 8;
        float* const red = reinterpret_cast<float*>(ring);
#pragma unroll
        for (int j = 0; j < NV; ++j)
#pragma unroll
            for (int i = 0; i < 8; ++i)
#pragma unroll
                for (int o = LPR; o < 32; o <<= 1) {
                    dw[j][i] += __shfl_xor_sync(0xFFFFFFFFu, dw[j][i], o);
                    db[j][i] += __shfl_xor_sync(0xFFFFFFFFu, db[j][i], o);
                }
        copy_wait(0);
#pragma unroll
        for (int which = 0; which < 2; ++which) {
            __syncthreads();
            if ((threadIdx.x & 31) < LPR)
#pragma unroll
                for (int j = 0; j < NV; ++j)
#pragma unroll
                    for (int i = 0; i < 8; ++i)
                        red[(threadIdx.x >> 5) * kWarpCols + (j * 8 + i) * LPR + map.t] = which ? db[j][i] : dw[j][i];
            __syncthreads();
            for (int k = threadIdx.x; k < kWarpCols; k += kSubThreads) {
                float v = 0.0f;
#pragma unroll
                for (int w = 0; w < kSubThreads / 32; ++w)
                    v += red[w * kWarpCols + k];
                const int t = k % LPR, ji = k / LPR, c = 8 * (t + LPR * (ji / 8)) + ji % 8;
                if (c < C)
                    out[which * to_db + c] = v;
            }
        }
    }
}

// How a width is spread over threads: octs of whole groups, so that a group's
// four lanes all exist.  Two octs a thread as long as 512 threads suffice (the
// weights, the column sums and a row's values then fit 128 registers), four
// above 8192 columns.  Up to 512 columns a warp, or a part of one, takes a row
// (`any`: rows at any address: a whole warp).
struct WideShape {
    int lpr, nv, threads;
};
WideShape wide_shape(int64_t cols, bool any)
{
    const int octs = static_cast<int>(act8_groups(cols)) * 4;
    if (octs <= 16 && !any)
        return {octs <= 8 ? 8 : 16, 1, kSubThreads};
    if (octs <= 64)
        return {32, octs <= 32 ? 1 : 2, kSubThreads};
    const int nv = octs <= 2 * kMaxThreads ? 2 : 4;
    return {0, nv, ((octs + nv - 1) / nv + 31) / 32 * 32};
}

constexpr int kRingBytes = 220 * 1024;  // of an SM's shared memory, all its CTAs together
// CTAs of an SM and rows in flight of each, from the bytes of one row's slots:
// as many CTAs as registers allow (with at least two stages each), then the
// stages that fit.
struct RingPlan {
    int per_sm, stages;
};
RingPlan ring_plan(int64_t stage_bytes, int resident, int most)
{
    RingPlan p;
    p.per_sm = resident;
    while (p.per_sm > 1 && p.per_sm * 2 * stage_bytes > kRingBytes)
        --p.per_sm;
    p.stages = static_cast<int>(std::max<int64_t>(1, std::min<int64_t>(most, kRingBytes / (p.per_sm * stage_bytes))));
    return p;
}

bool wide_rows(const void* p, int64_t ld, int bytes)
{
    return (reinterpret_cast<uintptr_t>(p) & 15) == 0 && (ld * bytes) % 16 == 0;
}
bool wide_cols(int64_t cols) { return cols <= kMaxWide; }

// Launches a ring kernel: its grid fills the GPU, or covers the rows, and has
// at most `most` CTAs.  `grid` returns it.
template <auto KERNEL, typename A>
int launch_ring(const A& a, const WideShape& w, int64_t stage_bytes, size_t least_smem, int64_t most, unsigned* grid,
                const Device& d, cudaStream_t s)
{
    const RingPlan p = ring_plan(stage_bytes, resident_ctas<KERNEL>(w.threads),
                                 w.lpr ? 3 : kMaxStages);
    const int64_t per_cta = w.lpr ? w.threads / w.lpr : 1, ctas = (a.rows + per_cta - 1) / per_cta;
    *grid = static_cast<unsigned>(std::min(most, std::min<int64_t>(ctas, int64_t{d.sms} * p.per_sm)));
    const size_t smem = std::max(static_cast<size_t>(stage_bytes) * p.stages + (w.lpr ? 0 : kBarBytes), least_smem);
    if (smem > 40 * 1024 &&  // 48 KiB without asking, the kernels' static words included
        cudaFuncSetAttribute(KERNEL, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(smem)) != cudaSuccess)
        return MX_ERR_CUDA;
    return launch_kernel(KERNEL, *grid, 1, w.threads, smem, a.amax != nullptr, s, a, p.stages);
}

// Bytes of a stage's share of one matrix.
int64_t stage_part(const WideShape& w, int64_t cols, int oct, bool any)
{
    const int64_t region = region_bytes(static_cast<int>((cols + 7) / 8), oct, any);
    return w.lpr == 0 ? region : any ? w.threads / w.lpr * region : static_cast<int64_t>(w.nv) * w.threads * oct;
}

template <typename T, typename TY, bool ANY>
int fwd_wide(const NormFwdArgs& a, const Device& d, cudaStream_t s)
{
    const WideShape w = wide_shape(a.cols, ANY);
    const int64_t bytes = stage_part(w, a.cols, 8 * sizeof(T), ANY) * (a.residual ? 2 : 1);
    const int64_t most = INT32_MAX;
    unsigned grid;
    if constexpr (!ANY) {
        if (w.lpr == 8)
            return launch_ring<norm_fwd_kernel<T, TY, 8, 1, ANY>>(a, w, bytes, 0, most, &grid, d, s);
        if (w.lpr == 16)
            return launch_ring<norm_fwd_kernel<T, TY, 16, 1, ANY>>(a, w, bytes, 0, most, &grid, d, s);
    }
    if (w.lpr == 32 && w.nv == 1)
        return launch_ring<norm_fwd_kernel<T, TY, 32, 1, ANY>>(a, w, bytes, 0, most, &grid, d, s);
    if (w.lpr == 32)
        return launch_ring<norm_fwd_kernel<T, TY, 32, 2, ANY>>(a, w, bytes, 0, most, &grid, d, s);
    return launch_ring<norm_fwd_kernel<T, TY, 0, 4, ANY>>(a, w, bytes, 0, most, &grid, d, s);
}

// Most CTAs of a backward kernel, each with its partial sums: 768 threads an SM
// at most, 152 SMs.  A pure function of the shape: the workspace is sized by it.
constexpr int kPartSms = 152;
int64_t ctas_of(const WideShape& w, int64_t rows)
{
    const int64_t per_cta = w.lpr ? w.threads / w.lpr : 1;
    return std::min<int64_t>((rows + per_cta - 1) / per_cta, kPartSms * std::min(8, std::max(1, 768 / w.threads)));
}

// dw and db from `parts` partial sums of each column, where they are asked for.
int join(const NormBwdArgs& a, int parts, cudaStream_t s)
{
    if (!a.dw && !a.db)
        return MX_OK;
    return launch_kernel(norm_dw_join_kernel, static_cast<unsigned>((a.cols + 31) / 32), 2, kJoinWarps * 32, 0, true, s,
                         a.parts, a.cols, parts, a.dw, a.db);
}

template <typename T, typename TY, bool FROM8, bool ANY>
int bwd_wide(const NormBwdArgs& a, const Device& d, cudaStream_t s)
{
    const WideShape w = wide_shape(a.cols, ANY);
    const int64_t bytes = stage_part(w, a.cols, 8 * sizeof(TY), ANY) +
                          stage_part(w, a.cols, FROM8 ? 8 : 8 * sizeof(T), ANY) +
                          (a.dres ? stage_part(w, a.cols, 8 * sizeof(T), ANY) : 0);
    const int64_t most = ctas_of(w, a.rows);
    // the column sums of a warp-per-row CTA pass through the ring's memory
    const size_t least = w.lpr ? static_cast<size_t>(w.nv) * w.lpr * 8 * sizeof(float) * (w.threads / 32) : 0;
    unsigned grid;
    int rc = MX_ERR_UNSUPPORTED;
    if constexpr (!ANY) {
        if (w.lpr == 8)
            rc = launch_ring<norm_bwd_kernel<T, TY, FROM8, 8, 1, ANY>>(a, w, bytes, least, most, &grid, d, s);
        else if (w.lpr == 16)
            rc = launch_ring<norm_bwd_kernel<T, TY, FROM8, 16, 1, ANY>>(a, w, bytes, least, most, &grid, d, s);
    }
    if (w.lpr == 32 && w.nv == 1)
        rc = launch_ring<norm_bwd_kernel<T, TY, FROM8, 32, 1, ANY>>(a, w, bytes, least, most, &grid, d, s);
    else if (w.lpr == 32)
        rc = launch_ring<norm_bwd_kernel<T, TY, FROM8, 32, 2, ANY>>(a, w, bytes, least, most, &grid, d, s);
    else if (w.lpr == 0 && w.nv == 4)
        rc = launch_ring<norm_bwd_kernel<T, TY, FROM8, 0, 4, ANY>>(a, w, bytes, least, most, &grid, d, s);
    return rc == MX_OK ? join(a, static_cast<int>(grid), s) : rc;
}

int64_t any_parts(int64_t rows) { return std::min<int64_t>((rows + kRowWarps - 1) / kRowWarps, 64); }

template <typename T, typename TY>
int fwd(const NormFwdArgs& a, const Device& d, cudaStream_t s)
{
    const int wb = a.w_dtype == MX_OUT_BF16 ? 2 : 4;
    if (wide_cols(a.cols)) {
        const bool aligned = a.cols % 8 == 0 && wide_rows(a.x, a.ldx, sizeof(T)) && wide_rows(a.residual, a.ldr, sizeof(T)) &&
                             wide_rows(a.sum_out, a.lds, sizeof(T)) && wide_rows(a.y, a.ldy, sizeof(TY)) &&
                             wide_rows(a.weight, 8, wb) && wide_rows(a.bias, 8, wb);
        if (a.cols >= kCtaMinCols && a.cols <= kCtaMaxCols)
            return launch_norm_fwd_cta(a, aligned, d, s);
        return aligned ? fwd_wide<T, TY, false>(a, d, s) : fwd_wide<T, TY, true>(a, d, s);
    }
    const unsigned grid = static_cast<unsigned>(std::min<int64_t>(a.rows, d.sms * 8));
    return launch_kernel(norm_fwd_any_kernel<T, TY>, grid, 1, kRowThreads, 0, a.amax != nullptr, s, a);
}

// Calls of up to 64 rows and 2048 columns: one launch, 3.1 us at
// 32x1024 fp32 where the row kernel and the join take 4.4 us; from 4096 columns
// on, where a row is long for its CTA's scalar accesses, it is the other way
// round (64x4096 bf16 from a checkpoint 9.9 us to 6.2).
bool few_rows(int64_t rows, int64_t cols) { return rows <= 64 && cols <= 2048; }

template <typename T, typename TY>
int bwd_few(const NormBwdArgs& a, cudaStream_t s)
{
    const unsigned rows = static_cast<unsigned>(a.rows);
    const unsigned columns = a.dw || a.db ? static_cast<unsigned>((a.cols + 31) / 32) : 0;
    if (columns == 0 || (a.dx != a.dy && a.dx != a.x))
        return launch_kernel(norm_bwd_few_kernel<T, TY>, rows + columns, 1, kRowThreads, 0, a.amax != nullptr, s, a, 0u);
    const int rc = launch_kernel(norm_bwd_few_kernel<T, TY>, columns, 1, kRowThreads, 0, false, s, a, rows);
    return rc != MX_OK ? rc : launch_kernel(norm_bwd_few_kernel<T, TY>, rows, 1, kRowThreads, 0, false, s, a, 0u);
}

template <typename T, typename TY>
int bwd(const NormBwdArgs& a, const Device& d, cudaStream_t s)
{
    if (few_rows(a.rows, a.cols))
        return bwd_few<T, TY>(a, s);
    const int wb = a.w_dtype == MX_OUT_BF16 ? 2 : 4;
    if (wide_cols(a.cols)) {
        const bool aligned = a.cols % 8 == 0 && wide_rows(a.dy, a.ldy, sizeof(TY)) && wide_rows(a.x, a.ldx, sizeof(T)) &&
                             wide_rows(a.dres, a.ldres, sizeof(T)) && wide_rows(a.dx, a.lddx, sizeof(T)) &&
                             wide_rows(a.weight, 8, wb);
        if (a.cols >= kCtaMinCols && a.cols <= kCtaMaxCols) {
            unsigned grid;
            const int rc = launch_norm_bwd_cta(a, aligned, static_cast<int>(ctas_of(wide_shape(a.cols, false), a.rows)), d, s, &grid);
            return rc == MX_OK ? join(a, static_cast<int>(grid), s) : rc;
        }
        if (a.x8.codes)
            return aligned ? bwd_wide<T, TY, true, false>(a, d, s) : bwd_wide<T, TY, true, true>(a, d, s);
        return aligned ? bwd_wide<T, TY, false, false>(a, d, s) : bwd_wide<T, TY, false, true>(a, d, s);
    }
    if (a.dw || a.db) {  // before dx, which may be dy's memory
        const int parts = static_cast<int>(any_parts(a.rows));
        int rc = launch_kernel(norm_dw_any_kernel<T, TY>, static_cast<unsigned>((a.cols + 31) / 32), parts, kRowThreads, 0,
                               false, s, a);
        if (rc != MX_OK || (rc = join(a, parts, s)) != MX_OK)
            return rc;
    }
    const unsigned grid = static_cast<unsigned>(std::min<int64_t>(a.rows, d.sms * 8));
    return launch_kernel(norm_dx_any_kernel<T, TY>, grid, 1, kRowThreads, 0, false, s, a);
}

}  // namespace

int64_t norm_bwd_parts(int64_t rows, int64_t cols)
{
    if (few_rows(rows, cols))
        return 0;
    if (!wide_cols(cols))
        return any_parts(rows);
    return std::max(ctas_of(wide_shape(cols, false), rows), ctas_of(wide_shape(cols, true), rows));
}

int launch_norm_fwd(const NormFwdArgs& a, const Device& d, cudaStream_t s)
{
    const int rc = launch_zero(a.amax, s);
    if (rc != MX_OK)
        return rc;
    using bf = __nv_bfloat16;
    if (a.x_dtype == MX_OUT_BF16)
        return a.y_dtype == MX_OUT_BF16 ? fwd<bf, bf>(a, d, s) : fwd<bf, float>(a, d, s);
    return a.y_dtype == MX_OUT_BF16 ? fwd<float, bf>(a, d, s) : fwd<float, float>(a, d, s);
}

int launch_norm_bwd(const NormBwdArgs& a, const Device& d, cudaStream_t s)
{
    const int rc = launch_zero(a.amax, s);
    if (rc != MX_OK)
        return rc;
    using bf = __nv_bfloat16;
    if (a.dx_dtype == MX_OUT_BF16)
        return a.dy_dtype == MX_OUT_BF16 ? bwd<bf, bf>(a, d, s) : bwd<bf, float>(a, d, s);
    return a.dy_dtype == MX_OUT_BF16 ? bwd<float, bf>(a, d, s) : bwd<float, float>(a, d, s);
}

}  // namespace mx
