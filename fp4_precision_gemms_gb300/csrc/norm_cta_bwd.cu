// norm_cta_bwd.cu -- the norm's backward kernels for rows of 513 to 16384 columns.
#include "mx_norm_cta.cuh"

namespace mx {
namespace {

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
    float* const out = a.parts + blockIdx.x * part_stride(C) + c0;
    const int64_t to_db = gridDim.x * part_stride(C);
#pragma unroll
    for (int j = 0; j < NV; ++j)
        if (own[j] > 0) {  // zeros past the row's end, up to the stride
            float* const to = out + j * dc;
#pragma unroll
            for (int k = 0; k < 4; k += 2) {
                *reinterpret_cast<float4*>(to + 2 * k) =
                    make_float4(dw[j].p[k].x, dw[j].p[k].y, dw[j].p[k + 1].x, dw[j].p[k + 1].y);
                *reinterpret_cast<float4*>(to + to_db + 2 * k) =
                    make_float4(db[j].p[k].x, db[j].p[k].y, db[j].p[k + 1].x, db[j].p[k + 1].y);
            }
        }
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
    return launch<kernel>(a, threads, row, n, *grid, d, s);
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
