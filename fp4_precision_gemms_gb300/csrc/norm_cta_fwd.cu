// norm_cta_fwd.cu -- the norm's forward kernels for rows of 513 to 16384 columns.
#include "mx_norm_cta.cuh"

namespace mx {
namespace {

// ADD: the residual is added; SAVE: the checkpoint is kept; R rows at a time;
// FULL: every thread's octs lie inside the row (cols a multiple of 512), which
// saves a tenth of the instructions.  The mean is summed first and the variance
// around it, from the values in registers: a second barrier, but no cancellation.
// Figures stand in mx_norm_cta.cuh.
// BOUND: the threads that the compiler limits registers for, 512: 128 a thread, 544
// to 640: 96.
template <typename T, typename TY, bool ADD, bool SAVE, int R, int NV, bool FULL, bool ANY, int BOUND>
__global__ void __launch_bounds__(BOUND) norm_fwd_cta_kernel(NormFwdArgs a, int stages)
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

template <auto KERNEL>
int fwd_one(const NormFwdArgs& a, int threads, int64_t row, int n, const Device& d, cudaStream_t s)
{
    return launch<KERNEL>(a, threads, row, n, static_cast<unsigned>(std::min<int64_t>(a.rows, int64_t{n} * d.sms)), d, s);
}

// Registers.  Where 96 a thread leave an SM two CTAs, up to 341 threads, a sum that
// is also saved takes 96 and above 128; the sum alone takes 128 up to there and 96
// above.  The CTAs' number is not all: the compiler's schedule is another one, as it
// is between bounds of 576 and 640, which allow the same 96 (saved sum 8192x4096 50.2
// and 51.7 us, but 65536x4096 396 and 365; sum alone 4096x8192 43.5 and 45).  Measured over 2^25 bf16 values,
// columns: us at 128 | 96 registers:
//   saved sum     768: 92 | 70   4096: 54.9 | 51.7   5120: 58 | 52   8192: 50.9 | 56.6
//   sum alone     768: 47 | 51   4096: 43.3 | 46.9   5120: 46 | 48   8192: 47 | 43.5
// Rows at any address take 96 (2^24 values fp32, 2049 columns 34 | 31, 4099 48 | 34,
// 8191 33.7 | 34.2; bf16 8193 columns 96 | 71), one row at a time without a residual
// too, for the second CTA; two rows take 128 (8192x4096 34, at 96 42).
template <typename T, typename TY, bool ADD, bool SAVE, Rows ROWS, int NV>
int fwd(const NormFwdArgs& a, const Device& d, cudaStream_t s)
{
    constexpr bool FULL = ROWS == kFull, ANY = ROWS == kAny;
    constexpr int tight = ANY || (ADD && !SAVE && NV == 2) ? 576 : NV == 2 ? 640 : kMaxThreads;
    const int threads = cta_threads(a.cols);
    const int64_t row = int64_t{Pipe<1, 1, ANY>::room(static_cast<uint32_t>(a.cols * sizeof(T)), ANY)} * (ADD ? 2 : 1);
    if constexpr (ADD && !ANY && NV == 2) {
        if (SAVE != (threads <= 65536 / (2 * 96))) {
            constexpr auto loose = norm_fwd_cta_kernel<T, TY, ADD, SAVE, 1, NV, FULL, false, kMaxThreads>;
            return fwd_one<loose>(a, threads, row, ctas_per_sm<loose>(threads, row), d, s);
        }
    }
    constexpr auto one = norm_fwd_cta_kernel<T, TY, ADD, SAVE, 1, NV, FULL, ANY, tight>;
    const int n1 = ctas_per_sm<one>(threads, row);
    // Two rows at a time for the norm without a residual, whose few bytes a row
    // leave it bound by instructions (32768x4096 bf16: 125 -> 90 us), where every
    // CTA still has several tiles and a ring of three stages fits, unless that
    // leaves an SM one CTA where one row leaves it two (257 to 341 threads; 8192x5120
    // 38.0 us and 35.8, with the checkpoint 53.3 and 46.8).  With the addition one
    // row is faster (8192x4096: 42.6 us, 45.9 for two).
    if constexpr (!ADD && !ANY && NV == 2) {
        constexpr auto two = norm_fwd_cta_kernel<T, TY, ADD, SAVE, 2, NV, FULL, false, kMaxThreads>;
        const int n2 = ctas_per_sm<two>(threads, 2 * row);
        if ((n2 > 1 || n1 == 1) && a.rows >= 4ll * n2 * d.sms && n2 * 3 * 2 * row <= kRingBytes)
            return launch<two>(a, threads, 2 * row, n2, static_cast<unsigned>(n2 * d.sms), d, s);
    }
    return fwd_one<one>(a, threads, row, n1, d, s);
}
template <typename T, typename TY, Rows ROWS, int NV>
int fwd_options(const NormFwdArgs& a, const Device& d, cudaStream_t s)
{
    if (a.residual)
        return a.save.codes ? fwd<T, TY, true, true, ROWS, NV>(a, d, s) : fwd<T, TY, true, false, ROWS, NV>(a, d, s);
    return a.save.codes ? fwd<T, TY, false, true, ROWS, NV>(a, d, s) : fwd<T, TY, false, false, ROWS, NV>(a, d, s);
}

template <typename T, typename TY>
int fwd_rows(const NormFwdArgs& a, bool aligned, const Device& d, cudaStream_t s)
{
    if (a.cols > kCtaTwoOcts)
        return aligned ? fwd_options<T, TY, kPart, 4>(a, d, s) : fwd_options<T, TY, kAny, 4>(a, d, s);
    if (!aligned)
        return fwd_options<T, TY, kAny, 2>(a, d, s);
    return full_rows(a.cols) ? fwd_options<T, TY, kFull, 2>(a, d, s) : fwd_options<T, TY, kPart, 2>(a, d, s);
}

}  // namespace

int launch_norm_fwd_cta(const NormFwdArgs& a, bool aligned, const Device& d, cudaStream_t s)
{
    using bf = __nv_bfloat16;
    if (a.x_dtype == MX_OUT_BF16)
        return a.y_dtype == MX_OUT_BF16 ? fwd_rows<bf, bf>(a, aligned, d, s) : fwd_rows<bf, float>(a, aligned, d, s);
    return a.y_dtype == MX_OUT_BF16 ? fwd_rows<float, bf>(a, aligned, d, s) : fwd_rows<float, float>(a, aligned, d, s);
}

}  // namespace mx
