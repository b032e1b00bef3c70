// norm.cu -- layer norm and RMS norm over the rows of a residual stream, forward
// and backward: the choice of the kernel, the kernels for narrow rows (up to 512
// columns), for few short rows and for rows above 16384 columns, and the join of
// the column sums.  The rows between are norm_cta_fwd.cu's and
// norm_cta_bwd.cu's.
#include <algorithm>

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
// One CTA per row, a warp per 32 columns at a time, the row read once per sum:
// right for every width and alignment, and what rows above 16384 columns take.

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
        a.parts[blockIdx.y * part_stride(C) + c] = s.w;
        a.parts[(gridDim.y + blockIdx.y) * part_stride(C) + c] = s.b;
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
        const int64_t stride = part_stride(C);
        const float* from = src + (static_cast<int64_t>(blockIdx.y) * parts + warp) * stride + c;
#pragma unroll 8
        for (int i = warp; i < parts; i += kJoinWarps, from += kJoinWarps * stride)
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

// ------------------------------------------------------------------ narrow
// Rows of up to 512 columns, several to a CTA: LPR lanes of a warp (8, 16 or 32)
// take a row, NV octs (eight columns) each, oct t + j LPR for lane t, so that a
// checkpoint group's four octs lie in four neighbouring lanes.  Rows that start on
// 16-byte boundaries, of a multiple of eight columns, take as few lanes as hold
// them; rows at any address (ANY) a whole warp.
//
// The grid is persistent.  A warp copies the rows that it takes next into a ring
// of shared-memory stages asynchronously, so that the memory system stays busy
// through the row sums; nothing but the warp's own wait synchronises them.
// 262144x128 bf16 measured: forward with residual, checkpoint and maximum 55 us
// (5.5 TB/s), backward from the checkpoint 65 us (3.7 TB/s), 65536x512 57 and 49.
constexpr int kMaxNarrow = 512;
constexpr int kThreads = 256;

template <int LPR>
struct RowMap {
    int t;               // this lane's place among a row's lanes
    int64_t first, step; // its first row, rows from one to the next
    int mine, all;       // rows of this lane, iterations of the CTA
    __device__ __forceinline__ explicit RowMap(int64_t rows)
    {
        constexpr int kRows = kThreads / LPR;
        t = threadIdx.x % LPR;
        const int64_t cta = static_cast<int64_t>(blockIdx.x) * kRows;
        step = static_cast<int64_t>(gridDim.x) * kRows;
        first = cta + threadIdx.x / LPR;
        all = static_cast<int>((rows - cta + step - 1) / step);
        mine = first < rows ? static_cast<int>((rows - first + step - 1) / step) : 0;
    }
};

template <int LPR>
__device__ __forceinline__ float row_sum(float v)
{
#pragma unroll
    for (int o = LPR / 2; o > 0; o >>= 1)
        v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
    return v;
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
// 16 (bf16), 32 (fp32) or 8 (codes) bytes.  ANY: a stage holds the aligned
// 16-byte words that a row lies in, one more than its octs fill, and an oct is
// shifted into place when it is read (codes always start on a boundary).  The
// words may hold a neighbouring row's elements; the first and the last rows
// (`edge` of them), whose words would reach past the matrix, are not copied but
// read where they are.
struct RingPart {
    const char* src;   // row 0
    int64_t next_row;  // bytes from one row to the next
    int oct;           // bytes of an oct
    uint32_t at;       // in a stage
};
__host__ __device__ constexpr uint32_t region_bytes(int octs, int oct, bool any)
{
    return (octs * oct + 15) / 16 * 16 + (any && oct != 8 ? 16 : 0);
}
template <int LPR, int NV, int PARTS, bool ANY>
struct RowRing {
    RingPart part[PARTS];
    uint32_t base, stage_bytes, at_stage = 0;
    int stages, stage = 0, cols, octs;
    int64_t rows, row = 0, edge = 1;
    bool direct = false;  // ANY: the current row is read from where it is
    uint32_t here_shift[PARTS], shift_step[PARTS];  // ANY: bytes past a boundary, the current row's and a step's

    __device__ __forceinline__ uint32_t region(int m) const { return region_bytes(octs, part[m].oct, ANY); }
    __device__ __forceinline__ uint32_t shift(int m, int64_t r) const  // bytes past a boundary
    {
        return ANY ? static_cast<uint32_t>(reinterpret_cast<uintptr_t>(part[m].src + r * part[m].next_row)) & 15u : 0u;
    }
    __device__ __forceinline__ bool at_edge(int64_t r) const { return ANY && (r < edge || r >= rows - edge); }

    __device__ __forceinline__ void layout(uint8_t* smem, int stages_, int cols_, int64_t rows_)
    {
        stages = stages_;
        cols = cols_;
        octs = (cols + 7) / 8;
        rows = rows_;
        base = smem_u32(smem);
        uint32_t at = 0;
#pragma unroll
        for (int m = 0; m < PARTS; ++m) {
            part[m].at = at;
            if (part[m].src) {
                at += ANY ? kThreads / LPR * region(m) : NV * kThreads * part[m].oct;
                if (ANY && part[m].next_row < 16)
                    edge = 16;
            }
        }
        stage_bytes = at;
    }
    // Bytes of the words that row r lies in.
    __device__ __forceinline__ uint32_t copied(int m, int64_t r) const
    {
        return part[m].oct == 8 ? region(m) : (shift(m, r) + static_cast<uint32_t>(cols * (part[m].oct / 8)) + 15) / 16 * 16;
    }
    // This lane's share of its row r into the stage `ahead` rows on.
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
                        const uint32_t dst = to + part[m].at + (threadIdx.x / LPR) * region(m);
                        const uint32_t n = copied(m, r);
                        row_at -= shift(m, r);
                        for (uint32_t w = t * 16; w < n; w += LPR * 16)
                            copy_async16(dst + w, row_at + w);
                    } else {  // a lane's own octs
                        const int w = min(part[m].oct, 16);
#pragma unroll
                        for (int j = 0; j < NV; ++j)
                            if (t + j * LPR < octs)
#pragma unroll
                                for (int h = 0; h < part[m].oct / w; ++h) {
                                    const uint32_t dst =
                                        to + part[m].at + ((j * (part[m].oct / w) + h) * kThreads + threadIdx.x) * w;
                                    const char* from = row_at + (t + j * LPR) * part[m].oct + h * 16;
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
        for (int i = 0; i < stages - 1; ++i)
            copy(map.first + i * map.step, i < map.mine, i, map.t);
    }
    // Row `it` has arrived.
    __device__ __forceinline__ void arrive(const RowMap<LPR>& map, int it)
    {
        direct = at_edge(row);
        copy(map.first + (it + stages - 1) * map.step, it + stages - 1 < map.mine, stages - 1, map.t);
        copy_wait(stages - 1);
        if (ANY)
            __syncwarp();  // words that other lanes copied
    }
    // The end of a row.
    __device__ __forceinline__ void done(const RowMap<LPR>& map)
    {
        if (ANY)
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
        }
    }

    // Address of word h of oct j of matrix m in the current stage.
    __device__ __forceinline__ uint32_t word(int m, int j, int h) const
    {
        const uint32_t at = base + at_stage + part[m].at;
        if constexpr (ANY)
            return at + threadIdx.x / LPR * region(m) + (threadIdx.x % LPR + j * LPR) * part[m].oct + h * 16;
        const int w = min(part[m].oct, 16);
        return at + ((j * (part[m].oct / w) + h) * kThreads + threadIdx.x) * w;
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
        store_ragged(p, o, n, lane > 0, lane < 31 && c + 8 < C && n > 0, top);
    } else if (n > 0) {
        store_oct(p, o, top);
    }
}

template <typename T, typename TY, int LPR, int NV, bool ANY>
__global__ void __launch_bounds__(kThreads, 2) norm_fwd_narrow_kernel(NormFwdArgs a, int stages)
{
    static_assert(!ANY || LPR == 32, "rows at any address take whole warps");
    extern __shared__ __align__(16) uint8_t smem[];
    const RowMap<LPR> map(a.rows);
    const int C = static_cast<int>(a.cols), G = (C + kAct8Group - 1) / kAct8Group;
    const int c0 = 8 * map.t;
    constexpr int dc = 8 * LPR;  // columns of oct j: c0 + j dc ..
    const float inv_c = 1.0f / static_cast<float>(C);
    const bool layer = a.kind == MX_NORM_LAYER, add = a.residual != nullptr;
    RowRing<LPR, NV, 2, ANY> ring;
    ring.part[0] = {static_cast<const char*>(a.x), a.ldx * static_cast<int64_t>(sizeof(T)), 8 * sizeof(T), 0};
    ring.part[1] = {static_cast<const char*>(a.residual), a.ldr * static_cast<int64_t>(sizeof(T)), 8 * sizeof(T), 0};
    ring.layout(smem, stages, C, a.rows);
    auto count = [&](bool in, int j) { return in ? min(C - c0 - j * dc, 8) : 0; };  // an oct's values

    Oct wt[NV], bi[NV];
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
    ring.start(map);
    for (int it = 0; it < map.all; ++it) {
        ring.arrive(map, it);
        const bool in = it < map.mine;
        Oct v[NV];
        float2 sum2 = make_float2(0.0f, 0.0f);
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            const int n = count(in, j);
            v[j].fill(0.0f);
            if (n > 0)
                ring.template read<T>(0, j, c0 + j * dc, n, v[j]);
            if (add) {
                Oct q;
                q.fill(0.0f);
                if (n > 0)
                    ring.template read<T>(1, j, c0 + j * dc, n, q);
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
        const float mean = layer ? row_sum<LPR>(sum2.x + sum2.y) * inv_c : 0.0f;
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
        const float rstd = rsqrtf(row_sum<LPR>(sq2.x + sq2.y) * inv_c + a.eps);
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
            if (ANY || n > 0) {
                Oct y;
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const float2 h = __fmul2_rn(__fadd2_rn(v[j].p[k], both(-mean)), both(rstd));
                    y.p[k] = __ffma2_rn(h, wt[j].p[k], bi[j].p[k]);
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
        ring.done(map);
    }
    if (a.amax)
        flush_top(a.amax, top);
}

// dx of each row and the CTA's partial sums of dw and db.  FROM8: the kept input
// is the checkpoint.  The column sums stay in registers over all of a lane's rows;
// at the end the rows of a warp and the warps join them, in a fixed order.
template <typename T, typename TY, bool FROM8, int LPR, int NV, bool ANY>
__global__ void __launch_bounds__(kThreads, 2) norm_bwd_narrow_kernel(NormBwdArgs a, int stages)
{
    static_assert(!ANY || LPR == 32, "rows at any address take whole warps");
    let_next_launch_start();  // the join of the partial sums
    extern __shared__ __align__(16) uint8_t smem[];
    const RowMap<LPR> map(a.rows);
    const int C = static_cast<int>(a.cols), G = (C + kAct8Group - 1) / kAct8Group;
    const int c0 = 8 * map.t;
    constexpr int dc = 8 * LPR;
    const float inv_c = 1.0f / static_cast<float>(C);
    const bool layer = a.kind == MX_NORM_LAYER, add = a.dres != nullptr;
    RowRing<LPR, NV, 3, ANY> ring;
    ring.part[0] = {static_cast<const char*>(a.dy), a.ldy * static_cast<int64_t>(sizeof(TY)), 8 * sizeof(TY), 0};
    if constexpr (FROM8)
        ring.part[1] = {reinterpret_cast<const char*>(a.x8.codes), G * int64_t{kAct8Group}, 8, 0};
    else
        ring.part[1] = {static_cast<const char*>(a.x), a.ldx * static_cast<int64_t>(sizeof(T)), 8 * sizeof(T), 0};
    ring.part[2] = {static_cast<const char*>(a.dres), a.ldres * static_cast<int64_t>(sizeof(T)), 8 * sizeof(T), 0};
    ring.layout(smem, stages, C, a.rows);
    auto count = [&](bool in, int j) { return in ? min(C - c0 - j * dc, 8) : 0; };

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

    Oct wt[NV], dw[NV], db[NV];
#pragma unroll
    for (int j = 0; j < NV; ++j) {
        if (c0 + j * dc < C)
            param_oct<ANY>(a.weight, a.w_dtype, c0 + j * dc, C, 1.0f, wt[j]);
        dw[j].fill(0.0f);
        db[j].fill(0.0f);
    }
    Top<T> top;
    T* to_dx = static_cast<T*>(a.dx) + map.first * a.lddx + c0;
    const int64_t dx_step = map.step * a.lddx;
    ring.start(map);
    RowWords next = row_words(0 < map.mine);
    for (int it = 0; it < map.all; ++it) {
        const bool in = it < map.mine;
        const RowWords cur = next;
        next = row_words(it + 1 < map.mine);
        ring.arrive(map, it);
        Oct g[NV], h[NV];
        float2 sgh = make_float2(0.0f, 0.0f), sg = sgh;
#pragma unroll
        for (int j = 0; j < NV; ++j)
            if (const int n = count(in, j); n > 0) {
                Oct dy;
                ring.template read<TY>(0, j, c0 + j * dc, n, dy);
                if constexpr (FROM8)
                    ring.read_codes(1, j, c0 + j * dc, h[j]);
                else
                    ring.template read<T>(1, j, c0 + j * dc, n, h[j]);
                const float2 scale = both(act8_scale(cur.e[j]));
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    // the code's product with its scale is exact
                    h[j].p[k] = FROM8 ? __ffma2_rn(h[j].p[k], scale, both(-cur.mean)) : __fadd2_rn(h[j].p[k], both(-cur.mean));
                    h[j].p[k] = __fmul2_rn(h[j].p[k], both(cur.rstd));
                    g[j].p[k] = __fmul2_rn(wt[j].p[k], dy.p[k]);  // zero past the row's end, as dy
                    sgh = __ffma2_rn(g[j].p[k], h[j].p[k], sgh);
                    sg = __fadd2_rn(sg, g[j].p[k]);
                    dw[j].p[k] = __ffma2_rn(dy.p[k], h[j].p[k], dw[j].p[k]);
                    db[j].p[k] = __fadd2_rn(db[j].p[k], dy.p[k]);
                }
            }
        const float c1s = row_sum<LPR>(sgh.x + sgh.y) * inv_c, c2s = row_sum<LPR>(sg.x + sg.y) * inv_c;
        const float2 c1 = both(-c1s), c2 = both(layer ? -c2s : 0.0f);
#pragma unroll
        for (int j = 0; j < NV; ++j)
            if (const int n = count(in, j); ANY || n > 0) {
                Oct q;
                q.fill(0.0f);
                if (add && n > 0)
                    ring.template read<T>(2, j, c0 + j * dc, n, q);
#pragma unroll
                for (int k = 0; k < 4; ++k)
                    q.p[k] = __ffma2_rn(__fadd2_rn(__ffma2_rn(h[j].p[k], c1, g[j].p[k]), c2), both(cur.rstd), q.p[k]);
                put_oct<ANY>(to_dx + j * dc, q, n, c0 + j * dc, C, top);
            }
        to_dx += dx_step;
        ring.done(map);
    }
    if (a.amax)
        flush_top(a.amax, top);
    if (!a.dw && !a.db)
        return;
    float* const out = a.parts + blockIdx.x * part_stride(C);
    const int64_t to_db = gridDim.x * part_stride(C);
    constexpr int kWarpCols = NV * LPR * 8;
    float* const red = reinterpret_cast<float*>(smem);
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
        for (int k = threadIdx.x; k < kWarpCols; k += kThreads) {
            float v = 0.0f;
#pragma unroll
            for (int w = 0; w < kThreads / 32; ++w)
                v += red[w * kWarpCols + k];
            const int t = k % LPR, ji = k / LPR, c = 8 * (t + LPR * (ji / 8)) + ji % 8;
            if (c < C)
                out[which * to_db + c] = v;
        }
    }
}

// Lanes of a narrow row and octs of each: whole checkpoint groups.
struct NarrowShape {
    int lpr, nv;
};
NarrowShape narrow_shape(int64_t cols, bool any)
{
    const int octs = static_cast<int>(act8_groups(cols)) * 4;
    if (octs <= 16 && !any)
        return {octs <= 8 ? 8 : 16, 1};
    return {32, octs <= 32 ? 1 : 2};
}
// Bytes of a stage's share of one matrix.
int64_t stage_part(const NarrowShape& w, int64_t cols, int oct, bool any)
{
    return any ? int64_t{kThreads / w.lpr} * region_bytes(static_cast<int>((cols + 7) / 8), oct, true)
               : int64_t{w.nv} * kThreads * oct;
}
bool wide_rows(const void* p, int64_t ld, int bytes)
{
    return (reinterpret_cast<uintptr_t>(p) & 15) == 0 && (ld * bytes) % 16 == 0;
}

// Launches a ring kernel: up to three rows in flight for each of the CTAs that
// an SM holds, a grid that fills the GPU or covers the rows, with at most `most`
// CTAs.  *grid returns it.
template <auto KERNEL, typename A>
int launch_narrow(const A& a, const NarrowShape& w, int64_t stage_bytes, size_t least_smem, int64_t most, unsigned* grid,
                  const Device& d, cudaStream_t s)
{
    int per_sm = resident_ctas<KERNEL>(kThreads);
    while (per_sm > 1 && per_sm * 2 * stage_bytes > kRingBytes)
        --per_sm;
    const int stages = static_cast<int>(std::max<int64_t>(1, std::min<int64_t>(3, kRingBytes / (per_sm * stage_bytes))));
    const int64_t per_cta = kThreads / w.lpr, ctas = (a.rows + per_cta - 1) / per_cta;
    *grid = static_cast<unsigned>(std::min(most, std::min<int64_t>(ctas, int64_t{d.sms} * per_sm)));
    const size_t smem = std::max(static_cast<size_t>(stage_bytes) * stages, least_smem);
    if (const int rc = allow_ring<KERNEL>(smem, d); rc != MX_OK)
        return rc;
    return launch_kernel(KERNEL, *grid, 1, kThreads, smem, a.amax != nullptr, s, a, stages);
}

template <typename T, typename TY, bool ANY>
int fwd_narrow(const NormFwdArgs& a, const Device& d, cudaStream_t s)
{
    const NarrowShape w = narrow_shape(a.cols, ANY);
    const int64_t bytes = stage_part(w, a.cols, 8 * sizeof(T), ANY) * (a.residual ? 2 : 1);
    const int64_t most = INT32_MAX;
    unsigned grid;
    if constexpr (!ANY) {
        if (w.lpr == 8)
            return launch_narrow<norm_fwd_narrow_kernel<T, TY, 8, 1, ANY>>(a, w, bytes, 0, most, &grid, d, s);
        if (w.lpr == 16)
            return launch_narrow<norm_fwd_narrow_kernel<T, TY, 16, 1, ANY>>(a, w, bytes, 0, most, &grid, d, s);
    }
    if (w.nv == 1)
        return launch_narrow<norm_fwd_narrow_kernel<T, TY, 32, 1, ANY>>(a, w, bytes, 0, most, &grid, d, s);
    return launch_narrow<norm_fwd_narrow_kernel<T, TY, 32, 2, ANY>>(a, w, bytes, 0, most, &grid, d, s);
}

// Most CTAs of a backward kernel, each with its partial sums: 768 threads an SM
// at most, 152 SMs.  A pure function of the shape: the workspace is sized by it.
constexpr int kPartSms = 152;
int64_t cta_parts(int64_t rows, int64_t cols)
{
    return std::min<int64_t>(rows, kPartSms * std::min(8, std::max(1, 768 / cta_threads(cols))));
}
int64_t narrow_parts(int64_t rows, int64_t cols, bool any)
{
    const int64_t per_cta = kThreads / narrow_shape(cols, any).lpr;
    return std::min<int64_t>((rows + per_cta - 1) / per_cta, kPartSms * (768 / kThreads));
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
int bwd_narrow(const NormBwdArgs& a, const Device& d, cudaStream_t s)
{
    const NarrowShape w = narrow_shape(a.cols, ANY);
    const int64_t bytes = stage_part(w, a.cols, 8 * sizeof(TY), ANY) +
                          stage_part(w, a.cols, FROM8 ? 8 : 8 * sizeof(T), ANY) +
                          (a.dres ? stage_part(w, a.cols, 8 * sizeof(T), ANY) : 0);
    const int64_t most = narrow_parts(a.rows, a.cols, ANY);
    // the warps' column sums pass through the ring's memory
    const size_t least = static_cast<size_t>(w.nv) * w.lpr * 8 * sizeof(float) * (kThreads / 32);
    unsigned grid;
    int rc = MX_ERR_UNSUPPORTED;
    if constexpr (!ANY) {
        if (w.lpr == 8)
            rc = launch_narrow<norm_bwd_narrow_kernel<T, TY, FROM8, 8, 1, ANY>>(a, w, bytes, least, most, &grid, d, s);
        else if (w.lpr == 16)
            rc = launch_narrow<norm_bwd_narrow_kernel<T, TY, FROM8, 16, 1, ANY>>(a, w, bytes, least, most, &grid, d, s);
    }
    if (w.lpr == 32 && w.nv == 1)
        rc = launch_narrow<norm_bwd_narrow_kernel<T, TY, FROM8, 32, 1, ANY>>(a, w, bytes, least, most, &grid, d, s);
    else if (w.lpr == 32)
        rc = launch_narrow<norm_bwd_narrow_kernel<T, TY, FROM8, 32, 2, ANY>>(a, w, bytes, least, most, &grid, d, s);
    return rc == MX_OK ? join(a, static_cast<int>(grid), s) : rc;
}

int64_t any_parts(int64_t rows) { return std::min<int64_t>((rows + kRowWarps - 1) / kRowWarps, 64); }

template <typename T, typename TY>
int fwd(const NormFwdArgs& a, const Device& d, cudaStream_t s)
{
    const int wb = a.w_dtype == MX_OUT_BF16 ? 2 : 4;
    const bool aligned = a.cols % 8 == 0 && wide_rows(a.x, a.ldx, sizeof(T)) && wide_rows(a.residual, a.ldr, sizeof(T)) &&
                         wide_rows(a.sum_out, a.lds, sizeof(T)) && wide_rows(a.y, a.ldy, sizeof(TY)) &&
                         wide_rows(a.weight, 8, wb) && wide_rows(a.bias, 8, wb);
    if (a.cols <= kMaxNarrow)
        return aligned ? fwd_narrow<T, TY, false>(a, d, s) : fwd_narrow<T, TY, true>(a, d, s);
    if (a.cols <= kCtaMaxCols)
        return launch_norm_fwd_cta(a, aligned, d, s);
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
    const bool aligned = a.cols % 8 == 0 && wide_rows(a.dy, a.ldy, sizeof(TY)) && wide_rows(a.x, a.ldx, sizeof(T)) &&
                         wide_rows(a.dres, a.ldres, sizeof(T)) && wide_rows(a.dx, a.lddx, sizeof(T)) &&
                         wide_rows(a.weight, 8, wb);
    if (a.cols <= kMaxNarrow) {
        if (a.x8.codes)
            return aligned ? bwd_narrow<T, TY, true, false>(a, d, s) : bwd_narrow<T, TY, true, true>(a, d, s);
        return aligned ? bwd_narrow<T, TY, false, false>(a, d, s) : bwd_narrow<T, TY, false, true>(a, d, s);
    }
    if (a.cols <= kCtaMaxCols) {
        unsigned grid;
        const int rc = launch_norm_bwd_cta(a, aligned, static_cast<int>(cta_parts(a.rows, a.cols)), d, s, &grid);
        return rc == MX_OK ? join(a, static_cast<int>(grid), s) : rc;
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
    if (cols <= kMaxNarrow)
        return std::max(narrow_parts(rows, cols, false), narrow_parts(rows, cols, true));
    return cols <= kCtaMaxCols ? cta_parts(rows, cols) : any_parts(rows);
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
