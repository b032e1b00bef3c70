// norm_cta.cu -- the norm's kernels for rows of 513 to 16384 columns.
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
// with residual, checkpoint and maximum 55 us (303 MB, 5.5 TB/s; 65536 rows 6.0),
// backward from the checkpoint with the residual's gradient 45.5 us (236 MB, 5.2
// TB/s; 65536 rows 6.8), of which the partial sums and their join take 5; layer
// norm alone at 32768 rows 90 us (537 MB, 5.9 TB/s).  At odd addresses the
// shifts double the instructions: 8192x4099 fp32 in, bf16 out 88 us, where
// 8192x4096 takes 34.
#include <algorithm>

#include "mx_act8.cuh"
#include "mx_internal.cuh"
#include "mx_norm.cuh"
#include "mx_ptx.cuh"

namespace mx {
namespace {

constexpr int kMaxThreads = 512;  // 128 registers each
constexpr int kMaxStages = 6;
constexpr int kBarBytes = 64;
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
    if constexpr (ANY) {
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

// ADD: the residual is added; SAVE: the checkpoint is kept; R rows at a time;
// FULL: every thread's octs lie inside the row (cols a multiple of 512), which
// saves a tenth of the instructions.
template <typename T, typename TY, bool ADD, bool SAVE, int R, int NV, bool FULL, bool ANY>
__global__ void __launch_bounds__(kMaxThreads) norm_fwd_cta_kernel(NormFwdArgs a, int stages)
{
    extern __shared__ __align__(128) uint8_t smem[];
    __shared__ __align__(16) float2 part[2][kWarps];
    if (threadIdx.x < kWarps)
        part[0][threadIdx.x] = part[1][threadIdx.x] = make_float2(0.0f, 0.0f);
    const int C = static_cast<int>(a.cols), G = (C + kAct8Group - 1) / kAct8Group;
    const int c0 = 8 * threadIdx.x, dc = 8 * blockDim.x;
    constexpr bool KEEP = NV <= 2;
    int own[NV];  // values of each oct, <= 0: none
#pragma unroll
    for (int j = 0; j < NV; ++j)
        own[j] = FULL ? 8 : min(C - c0 - j * dc, 8);
    const float inv_c = 1.0f / static_cast<float>(C);
    const bool layer = a.kind == MX_NORM_LAYER;
    const int64_t tiles_of_all = (a.rows + R - 1) / R;
    const int tiles = static_cast<int>((tiles_of_all - blockIdx.x + gridDim.x - 1) / gridDim.x);

    Pipe<ADD ? 2 : 1, R, ANY> pipe;
    pipe.matrix(0, a.x, a.ldx * static_cast<int64_t>(sizeof(T)), C * sizeof(T), false);
    if constexpr (ADD)
        pipe.matrix(1, a.residual, a.ldr * static_cast<int64_t>(sizeof(T)), C * sizeof(T), false);
    pipe.layout(smem, stages, a.fail_at, a.rows);
    pipe.start(a.rows, tiles);

    Oct wt[KEEP ? NV : 1], bi[KEEP ? NV : 1];
#pragma unroll
    for (int j = 0; j < (KEEP ? NV : 0); ++j) {
        params<ANY>(a.weight, a.w_dtype, c0 + j * dc, own[j], 1.0f, wt[j]);
        params<ANY>(a.bias, a.w_dtype, c0 + j * dc, own[j], 0.0f, bi[j]);
    }
    int64_t r = static_cast<int64_t>(blockIdx.x) * R;
    const int64_t step = static_cast<int64_t>(gridDim.x) * R;
    TY* to_y = static_cast<TY*>(a.y) + r * a.ldy + c0;
    T* to_sum = ADD ? static_cast<T*>(a.sum_out) + r * a.lds + c0 : nullptr;
    uint8_t* to_codes = SAVE ? a.save.codes + r * (G * kAct8Group) + c0 : nullptr;
    const int64_t y_step = step * a.ldy, sum_step = step * a.lds, codes_step = step * (G * kAct8Group);

    Top<TY> top;
    Top<T> unused;
    bool bad = false;
    int it = 0;
    for (; it < tiles; ++it) {
        bad = !pipe.wait(a.wait_ns);
        const bool two = R == 2 && r + 1 < a.rows;  // the last tile may have one row
        Oct v[R][NV];
        float sum[2] = {0.0f, 0.0f};
#pragma unroll
        for (int q = 0; q < R; ++q) {
            float2 s2 = make_float2(0.0f, 0.0f);
#pragma unroll
            for (int j = 0; j < NV; ++j) {
                v[q][j].fill(0.0f);
                if (own[j] > 0)
                    pipe.template oct<T>(0, q, j, r + q, own[j], v[q][j]);
                if constexpr (ADD) {
                    Oct o;
                    o.fill(0.0f);
                    if (own[j] > 0)
                        pipe.template oct<T>(1, q, j, r + q, own[j], o);
#pragma unroll
                    for (int k = 0; k < 4; ++k)
                        o.p[k] = __fadd2_rn(v[q][j].p[k], o.p[k]);
                    if (q == 0 || two)
                        put<ANY>(to_sum + q * a.lds + j * dc, o, own[j], c0 + j * dc, C, unused);
                    if constexpr (sizeof(T) == 2)
                        unpack_oct(pack_oct(o), v[q][j]);  // as it was stored
                    else
                        v[q][j] = o;
                }
#pragma unroll
                for (int k = 0; k < 4; ++k)
                    s2 = __fadd2_rn(s2, v[q][j].p[k]);
            }
            sum[q] = s2.x + s2.y;
        }
        float2 mean = make_float2(0.0f, 0.0f);
        if (layer) {
            mean = cta_sum2(sum[0], sum[1], part[0], bad);
            if (bad)
                break;
            mean.x *= inv_c;
            mean.y *= inv_c;
        }
        if constexpr (SAVE) {
#pragma unroll
            for (int q = 0; q < R; ++q)
#pragma unroll
                for (int j = 0; j < NV; ++j) {
                    uint8_t e;
                    const uint2 codes = encode_oct(v[q][j], e);
                    if ((FULL || c0 + j * dc < G * kAct8Group) && (q == 0 || two)) {
                        *reinterpret_cast<uint2*>(to_codes + q * (G * kAct8Group) + j * dc) = codes;
                        if ((threadIdx.x & 3) == 0)
                            a.save.sf[(r + q) * G + (c0 + j * dc) / kAct8Group] = e;
                    }
                }
        }
        float sq[2] = {0.0f, 0.0f};
#pragma unroll
        for (int q = 0; q < R; ++q) {
            const float2 m = both(q == 0 ? -mean.x : -mean.y);
            float2 s2 = make_float2(0.0f, 0.0f);
#pragma unroll
            for (int j = 0; j < NV; ++j)
                if (own[j] > 0) {
#pragma unroll
                    for (int k = 0; k < 4; ++k)
                        v[q][j].p[k] = __fadd2_rn(v[q][j].p[k], m);
                    if (ANY && own[j] < 8)
                        keep_first(v[q][j], own[j]);
#pragma unroll
                    for (int k = 0; k < 4; ++k)
                        s2 = __ffma2_rn(v[q][j].p[k], v[q][j].p[k], s2);
                }
            sq[q] = s2.x + s2.y;
        }
        // RMS norm has one barrier per tile: its words alternate
        const float2 var = cta_sum2(sq[0], sq[1], part[layer ? 1 : it & 1], bad);
        if (bad)
            break;
        pipe.refill(it, a.rows, tiles, pipe.stage);  // the tile's rows are in registers
        const float2 rstd = make_float2(rsqrtf(var.x * inv_c + a.eps), rsqrtf(var.y * inv_c + a.eps));
        if (threadIdx.x < R && (threadIdx.x == 0 || two)) {
            const bool first = threadIdx.x == 0;
            if (a.mean && layer)
                a.mean[r + threadIdx.x] = first ? mean.x : mean.y;
            if (a.rstd)
                a.rstd[r + threadIdx.x] = first ? rstd.x : rstd.y;
        }
#pragma unroll
        for (int q = 0; q < R; ++q)
            if (q == 0 || two) {
                const float2 s = both(q == 0 ? rstd.x : rstd.y);
#pragma unroll
                for (int j = 0; j < NV; ++j) {
                    Oct y, &w = wt[KEEP ? j : 0], &b = bi[KEEP ? j : 0];
                    if constexpr (!KEEP) {
                        params<ANY>(a.weight, a.w_dtype, c0 + j * dc, own[j], 1.0f, w);
                        params<ANY>(a.bias, a.w_dtype, c0 + j * dc, own[j], 0.0f, b);
                    }
#pragma unroll
                    for (int k = 0; k < 4; ++k)
                        y.p[k] = __ffma2_rn(__fmul2_rn(v[q][j].p[k], s), w.p[k], b.p[k]);
                    put<ANY>(to_y + q * a.ldy + j * dc, y, own[j], c0 + j * dc, C, top);
                }
            }
        r += step;
        to_y += y_step;
        if constexpr (ADD)
            to_sum += sum_step;
        if constexpr (SAVE)
            to_codes += codes_step;
        pipe.next(r, a.rows);
    }
    if (bad) {
        pipe.abandon(it, min(tiles, it + stages), a.wait_ns, a.status);
        return;
    }
    if (a.amax)
        flush_top(a.amax, top);
}

// dx of each row and the CTA's partial sums of dw and db.  FROM8: the kept input
// is the checkpoint.  ADD: the residual path's gradient joins dx.
template <typename T, typename TY, bool FROM8, bool ADD, int NV, bool FULL, bool ANY>
__global__ void __launch_bounds__(kMaxThreads) norm_bwd_cta_kernel(NormBwdArgs a, int stages)
{
    extern __shared__ __align__(128) uint8_t smem[];
    __shared__ __align__(16) float2 part[2][kWarps];
    let_next_launch_start();  // the join of the partial sums
    if (threadIdx.x < kWarps)
        part[0][threadIdx.x] = part[1][threadIdx.x] = make_float2(0.0f, 0.0f);
    const int C = static_cast<int>(a.cols), G = (C + kAct8Group - 1) / kAct8Group;
    const int c0 = 8 * threadIdx.x, dc = 8 * blockDim.x;
    constexpr bool KEEP = NV <= 2;
    int own[NV];  // values of each oct, <= 0: none
#pragma unroll
    for (int j = 0; j < NV; ++j)
        own[j] = FULL ? 8 : min(C - c0 - j * dc, 8);
    const float inv_c = 1.0f / static_cast<float>(C);
    const bool layer = a.kind == MX_NORM_LAYER;
    const int tiles = static_cast<int>((a.rows - blockIdx.x + gridDim.x - 1) / gridDim.x);

    Pipe<ADD ? 3 : 2, 1, ANY> pipe;
    pipe.matrix(0, a.dy, a.ldy * static_cast<int64_t>(sizeof(TY)), C * sizeof(TY), false);
    if constexpr (FROM8)
        pipe.matrix(1, a.x8.codes, G * int64_t{kAct8Group}, G * kAct8Group, true);
    else
        pipe.matrix(1, a.x, a.ldx * static_cast<int64_t>(sizeof(T)), C * sizeof(T), false);
    if constexpr (ADD)
        pipe.matrix(2, a.dres, a.ldres * static_cast<int64_t>(sizeof(T)), C * sizeof(T), false);
    pipe.layout(smem, stages, a.fail_at, a.rows);
    pipe.start(a.rows, tiles);

    Oct wt[KEEP ? NV : 1], dw[NV], db[NV];
#pragma unroll
    for (int j = 0; j < NV; ++j) {
        if constexpr (KEEP)
            params<ANY>(a.weight, a.w_dtype, c0 + j * dc, own[j], 1.0f, wt[j]);
        dw[j].fill(0.0f);
        db[j].fill(0.0f);
    }
    int64_t r = blockIdx.x;
    const int64_t step = gridDim.x;
    T* to_dx = static_cast<T*>(a.dx) + r * a.lddx + c0;
    const int64_t dx_step = step * a.lddx;
    // what a row needs beside its matrices, loaded a row ahead
    float mean = 0.0f, rstd = 0.0f;
    uint32_t e[NV];
    auto row_words = [&] {
        rstd = a.rstd[r];
        if (layer)
            mean = a.mean[r];
        if constexpr (FROM8)
#pragma unroll
            for (int j = 0; j < NV; ++j)
                e[j] = a.x8.sf[r * G + min((c0 + j * dc) / kAct8Group, G - 1)];
    };
    row_words();

    Top<T> top;
    bool bad = false;
    int it = 0;
    for (; it < tiles; ++it) {
        const float2 m = both(-mean), s = both(rstd);
        float2 scale[NV];
#pragma unroll
        for (int j = 0; j < (FROM8 ? NV : 0); ++j)
            scale[j] = both(act8_scale(e[j]));
        const int64_t row = r;
        r += step;
        if (it + 1 < tiles)
            row_words();
        bad = !pipe.wait(a.wait_ns);
        // g and h of oct j
        auto load = [&](int j, Oct& dy, Oct& g, Oct& h) {
            pipe.template oct<TY>(0, 0, j, row, own[j], dy);
            if constexpr (FROM8)
                pipe.codes(1, j, row, h);
            else
                pipe.template oct<T>(1, 0, j, row, own[j], h);
            Oct& w = wt[KEEP ? j : 0];
            if constexpr (!KEEP)
                params<ANY>(a.weight, a.w_dtype, c0 + j * dc, own[j], 1.0f, w);
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                // the code's product with its scale is exact
                h.p[k] = FROM8 ? __ffma2_rn(h.p[k], scale[j], m) : __fadd2_rn(h.p[k], m);
                h.p[k] = __fmul2_rn(h.p[k], s);
                g.p[k] = __fmul2_rn(dy.p[k], w.p[k]);
            }
        };
        Oct keep_g[KEEP ? NV : 1], keep_h[KEEP ? NV : 1];
        float2 sgh = make_float2(0.0f, 0.0f), sg = sgh;
#pragma unroll
        for (int j = 0; j < NV; ++j)
            if (own[j] > 0) {
                Oct dy, &g = keep_g[KEEP ? j : 0], &h = keep_h[KEEP ? j : 0];
                load(j, dy, g, h);
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    sgh = __ffma2_rn(g.p[k], h.p[k], sgh);
                    sg = __fadd2_rn(sg, g.p[k]);
                    dw[j].p[k] = __ffma2_rn(dy.p[k], h.p[k], dw[j].p[k]);
                    db[j].p[k] = __fadd2_rn(db[j].p[k], dy.p[k]);
                }
            }
        const float2 sums = cta_sum2(sgh.x + sgh.y, sg.x + sg.y, part[it & 1], bad);
        if (bad)
            break;
        if (stages > 1)
            pipe.refill(it - 1, a.rows, tiles, pipe.before());  // nobody reads the row before any more
        const float2 c1 = both(-sums.x * inv_c), c2 = both(layer ? -sums.y * inv_c : 0.0f);
#pragma unroll
        for (int j = 0; j < NV; ++j)
            if (ANY || own[j] > 0) {
                Oct dy, q, &g = keep_g[KEEP ? j : 0], &h = keep_h[KEEP ? j : 0];
                if (!KEEP && own[j] > 0)
                    load(j, dy, g, h);
                q.fill(0.0f);
                if (ADD && own[j] > 0)
                    pipe.template oct<T>(2, 0, j, row, own[j], q);
#pragma unroll
                for (int k = 0; k < 4; ++k)
                    q.p[k] = __ffma2_rn(__fadd2_rn(__ffma2_rn(h.p[k], c1, g.p[k]), c2), s, q.p[k]);
                put<ANY>(to_dx + j * dc, q, own[j], c0 + j * dc, C, top);
            }
        to_dx += dx_step;
        if (stages == 1) {
            __syncthreads();
            pipe.refill(it, a.rows, tiles, 0);
        }
        pipe.next(r, a.rows);
    }
    if (bad) {
        pipe.abandon(it, min(tiles, stages > 1 ? max(it - 1, 0) + stages : it + 1), a.wait_ns, a.status);
        return;
    }
    if (a.amax)
        flush_top(a.amax, top);
    if (!a.dw && !a.db)
        return;
    float* const out = a.parts + static_cast<int64_t>(blockIdx.x) * C + c0;
    const int64_t to_db = static_cast<int64_t>(gridDim.x) * C;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
        float* const to = out + j * dc;
        if constexpr (ANY) {
#pragma unroll
            for (int i = 0; i < 8; ++i)
                if (i < own[j]) {
                    to[i] = dw[j][i];
                    to[to_db + i] = db[j][i];
                }
        } else if (own[j] > 0) {
#pragma unroll
            for (int k = 0; k < 4; k += 2) {
                *reinterpret_cast<float4*>(to + 2 * k) =
                    make_float4(dw[j].p[k].x, dw[j].p[k].y, dw[j].p[k + 1].x, dw[j].p[k + 1].y);
                *reinterpret_cast<float4*>(to + to_db + 2 * k) =
                    make_float4(db[j].p[k].x, db[j].p[k].y, db[j].p[k + 1].x, db[j].p[k + 1].y);
            }
        }
    }
}

constexpr int64_t kRingBytes = 220 * 1024;  // of an SM's shared memory, all its CTAs together

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
int launch(const A& a, int threads, int64_t stage_bytes, int per_sm, unsigned grid, cudaStream_t s)
{
    const int stages =
        static_cast<int>(std::max<int64_t>(1, std::min<int64_t>(kMaxStages, kRingBytes / (per_sm * stage_bytes))));
    const size_t smem = static_cast<size_t>(stage_bytes) * stages + kBarBytes;
    if (smem > 40 * 1024 &&  // 48 KiB without asking, the kernels' static words included
        cudaFuncSetAttribute(KERNEL, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(smem)) != cudaSuccess)
        return MX_ERR_CUDA;
    return launch_kernel(KERNEL, grid, 1, threads, smem, a.amax != nullptr, s, a, stages);
}

// How the rows of a call lie: every thread's octs inside the row, some past it,
// or rows at any address.
enum Rows { kFull, kPart, kAny };

template <typename T, typename TY, bool ADD, bool SAVE, Rows ROWS, int NV>
int fwd(const NormFwdArgs& a, const Device& d, cudaStream_t s)
{
    constexpr bool FULL = ROWS == kFull, ANY = ROWS == kAny;
    const int threads = cta_threads(a.cols);
    const int64_t row = int64_t{Pipe<1, 1, ANY>::room(static_cast<uint32_t>(a.cols * sizeof(T)), ANY)} * (ADD ? 2 : 1);
    // Two rows at a time for the norm without a residual, whose few bytes a row
    // leave it bound by instructions (32768x4096 bf16: 125 -> 90 us), where every
    // CTA still has several tiles and a ring of three stages fits.  With the
    // addition one row is faster (8192x4096: 42.6 us, 45.9 for two).
    if constexpr (!ADD && !ANY && NV == 2) {
        constexpr auto two = norm_fwd_cta_kernel<T, TY, ADD, SAVE, 2, NV, FULL, false>;
        const int n2 = ctas_per_sm<two>(threads, 2 * row);
        if (a.rows >= 4ll * n2 * d.sms && n2 * 3 * 2 * row <= kRingBytes)
            return launch<two>(a, threads, 2 * row, n2, static_cast<unsigned>(n2 * d.sms), s);
    }
    constexpr auto one = norm_fwd_cta_kernel<T, TY, ADD, SAVE, 1, NV, FULL, ANY>;
    const int n1 = ctas_per_sm<one>(threads, row);
    return launch<one>(a, threads, row, n1, static_cast<unsigned>(std::min<int64_t>(a.rows, int64_t{n1} * d.sms)), s);
}
template <typename T, typename TY, Rows ROWS, int NV>
int fwd_options(const NormFwdArgs& a, const Device& d, cudaStream_t s)
{
    if (a.residual)
        return a.save.codes ? fwd<T, TY, true, true, ROWS, NV>(a, d, s) : fwd<T, TY, true, false, ROWS, NV>(a, d, s);
    return a.save.codes ? fwd<T, TY, false, true, ROWS, NV>(a, d, s) : fwd<T, TY, false, false, ROWS, NV>(a, d, s);
}

// Above 8192 columns the rows may always end before a thread's octs do (as
// kPart), which halves the kernels there.
bool full_rows(int64_t cols) { return cols == 16 * cta_threads(cols); }

template <typename T, typename TY>
int fwd_rows(const NormFwdArgs& a, bool aligned, const Device& d, cudaStream_t s)
{
    if (a.cols > kCtaTwoOcts)
        return aligned ? fwd_options<T, TY, kPart, 4>(a, d, s) : fwd_options<T, TY, kAny, 4>(a, d, s);
    if (!aligned)
        return fwd_options<T, TY, kAny, 2>(a, d, s);
    return full_rows(a.cols) ? fwd_options<T, TY, kFull, 2>(a, d, s) : fwd_options<T, TY, kPart, 2>(a, d, s);
}

template <typename T, typename TY, bool FROM8, bool ADD, Rows ROWS, int NV>
int bwd(const NormBwdArgs& a, int most, const Device& d, cudaStream_t s, unsigned* grid)
{
    constexpr bool ANY = ROWS == kAny;
    const int threads = cta_threads(a.cols);
    auto room = [&](size_t bytes) { return int64_t{Pipe<2, 1, ANY>::room(static_cast<uint32_t>(a.cols * bytes), ANY)}; };
    const int64_t row =
        room(sizeof(TY)) + (FROM8 ? act8_groups(a.cols) * kAct8Group : room(sizeof(T))) + (ADD ? room(sizeof(T)) : 0);
    constexpr auto kernel = norm_bwd_cta_kernel<T, TY, FROM8, ADD, NV, ROWS == kFull, ANY>;
    const int n = ctas_per_sm<kernel>(threads, row);
    *grid = static_cast<unsigned>(std::min<int64_t>(std::min<int64_t>(a.rows, most), int64_t{n} * d.sms));
    return launch<kernel>(a, threads, row, n, *grid, s);
}
template <typename T, typename TY, Rows ROWS, int NV>
int bwd_options(const NormBwdArgs& a, int most, const Device& d, cudaStream_t s, unsigned* grid)
{
    if (a.x8.codes)
        return a.dres ? bwd<T, TY, true, true, ROWS, NV>(a, most, d, s, grid) : bwd<T, TY, true, false, ROWS, NV>(a, most, d, s, grid);
    return a.dres ? bwd<T, TY, false, true, ROWS, NV>(a, most, d, s, grid) : bwd<T, TY, false, false, ROWS, NV>(a, most, d, s, grid);
}
template <typename T, typename TY>
int bwd_rows(const NormBwdArgs& a, bool aligned, int most, const Device& d, cudaStream_t s, unsigned* grid)
{
    if (a.cols > kCtaTwoOcts)
        return aligned ? bwd_options<T, TY, kPart, 4>(a, most, d, s, grid) : bwd_options<T, TY, kAny, 4>(a, most, d, s, grid);
    if (!aligned)
        return bwd_options<T, TY, kAny, 2>(a, most, d, s, grid);
    return full_rows(a.cols) ? bwd_options<T, TY, kFull, 2>(a, most, d, s, grid)
                             : bwd_options<T, TY, kPart, 2>(a, most, d, s, grid);
}

}  // namespace

int launch_norm_fwd_cta(const NormFwdArgs& a, bool aligned, const Device& d, cudaStream_t s)
{
    using bf = __nv_bfloat16;
    if (a.x_dtype == MX_OUT_BF16)
        return a.y_dtype == MX_OUT_BF16 ? fwd_rows<bf, bf>(a, aligned, d, s) : fwd_rows<bf, float>(a, aligned, d, s);
    return a.y_dtype == MX_OUT_BF16 ? fwd_rows<float, bf>(a, aligned, d, s) : fwd_rows<float, float>(a, aligned, d, s);
}

int launch_norm_bwd_cta(const NormBwdArgs& a, bool aligned, int most, const Device& d, cudaStream_t s, unsigned* grid)
{
    using bf = __nv_bfloat16;
    if (a.dx_dtype == MX_OUT_BF16)
        return a.dy_dtype == MX_OUT_BF16 ? bwd_rows<bf, bf>(a, aligned, most, d, s, grid)
                                         : bwd_rows<bf, float>(a, aligned, most, d, s, grid);
    return a.dy_dtype == MX_OUT_BF16 ? bwd_rows<float, bf>(a, aligned, most, d, s, grid)
                                     : bwd_rows<float, float>(a, aligned, most, d, s, grid);
}

}  // namespace mx
