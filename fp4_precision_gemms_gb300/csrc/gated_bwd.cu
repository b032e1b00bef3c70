// gated_bwd.cu -- the gated block's backward activation and the quantization of its
// result in one pass: from dH and the checkpoints of g and u straight to the MXFP8 /
// MXFP4 operands of both gradient products.
//
//   D[T, 2F] = [dH u act'(g), dH act(g)], rounded to bf16 as mx_act_bwd writes it, then
//   encoded along its rows (the data gradient's operand) and along its columns (the
//   weight gradient's, transposed), to nearest with the FLOOR rule
//
// A CTA takes 128 tokens x 128 features, the extent of one 512-byte scale chunk in both
// directions.  First each thread computes eights of a row, encodes them (four lanes share
// a block's maximum) and leaves the bf16 values in shared memory; then each thread
// encodes two columns of 32 tokens.  Chunks of scale bytes are gathered in shared memory
// and written whole.  Where F is an odd multiple of 64 (MXFP8 only), up's columns of D start
// in the middle of a chunk: tiles of 64 features then, whose scale bytes go out one by one.
// Bytes: 2 + 2.06 a value of dH read, 4.12 written (FP8); the two passes that this replaces
// move D's 4 bytes out and in again as well (149 + 166 us).
// Bound by issue and latency together: 48 instructions a value of dH, 55 % of the issue
// slots (66 % at 2048 tokens), two CTAs an SM whose loading and encoding phases overlap only
// with each other's.
#include <cuda_bf16.h>

#include "mx_act8.cuh"
#include "mx_activate.cuh"
#include "mx_codec.cuh"
#include "mx_internal.cuh"

namespace mx {
namespace {

constexpr int kTokens = 128;  // of a tile
template <int FEATURES>
struct Shape {
    static constexpr int threads = 4 * FEATURES, ctas = 1024 / threads;
    static constexpr int pitch = FEATURES * 2 + 16;    // bytes of a staged row
    static constexpr int stage = kTokens * pitch;      // of one operand
    static constexpr int smem = 2 * stage + 4 * 512;
    static constexpr int octs = FEATURES / 8;          // of a row
    static constexpr int rows = threads / octs;        // that the threads take at once
};
// Eights of a thread whose loads are in flight together: all four of a tile.  8192 x 14336
// SiLU: 230 us (960 MB, 4.2 TB/s); two at a time 248, three CTAs of 256 threads 246.
constexpr int kFlight = 4;

struct BwdQuantParams {
    const __nv_bfloat16* dh;
    int64_t ldh;
    Act8View g8, u8;
    int64_t T, F;
    uint8_t* row_codes;  // [T, 2F]
    uint8_t* row_sf;
    uint8_t* col_codes;  // [2F, T]
    uint8_t* col_sf;
};

// max(|a|, |b|) by halves; the signs of the result are not cleared.
__device__ __forceinline__ uint32_t top_bf16x2(uint32_t a, uint32_t b)
{
    uint32_t r;
    asm("max.xorsign.abs.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}
__device__ __forceinline__ float2 scaled(uint32_t w, float2 s) { return __fmul2_rn(unpack_bf16x2(w), s); }

// Offset of (row r of 128, block kb of 4) in a chunk of scale bytes.
__device__ __forceinline__ int chunk_at(int r, int kb) { return (r & 31) * 16 + (r >> 5) * 4 + kb; }

// Eight values of a row whose block four lanes hold: their codes and the block's byte.
template <int ELEM>
__device__ __forceinline__ uint32_t encode_row(uint4 w, uint2& codes)
{
    uint32_t m = top_bf16x2(top_bf16x2(w.x, w.y), top_bf16x2(w.z, w.w));
    m = top_bf16x2(m, __shfl_xor_sync(0xFFFFFFFFu, m, 1));
    m = top_bf16x2(m, __shfl_xor_sync(0xFFFFFFFFu, m, 2)) & 0x7FFF7FFFu;
    // as floats: where one half of every word is NaN, which no maximum counts, the other half's values have a scale
    const int e = pow2_exponent<ELEM>(fmaxf(__uint_as_float(m << 16), __uint_as_float(m & 0xFFFF0000u)), MX_SCALE_FLOOR);
    const float2 s = both(exp2_neg(e));
    const float2 a = scaled(w.x, s), b = scaled(w.y, s), c = scaled(w.z, s), d = scaled(w.w, s);
    if constexpr (ELEM == kElemE4M3) {
        codes = make_uint2(cvt_e4m3x2(a.x, a.y) | cvt_e4m3x2(b.x, b.y) << 16, cvt_e4m3x2(c.x, c.y) | cvt_e4m3x2(d.x, d.y) << 16);
    } else {
        const float q[8] = {a.x, a.y, b.x, b.y, c.x, c.y, d.x, d.y};
        codes.x = cvt_e2m1x8(q);
    }
    return static_cast<uint32_t>(e + 127);
}

// 32 tokens of two neighbouring columns.
template <int ELEM>
__device__ __forceinline__ void encode_columns(const uint32_t (&w)[32], uint8_t* to_a, uint8_t* to_b, uint8_t& byte_a,
                                               uint8_t& byte_b)
{
    uint32_t m[8];
#pragma unroll
    for (int i = 0; i < 8; ++i)
        m[i] = top_bf16x2(top_bf16x2(w[i], w[i + 8]), top_bf16x2(w[i + 16], w[i + 24]));
#pragma unroll
    for (int h = 4; h > 0; h >>= 1)
#pragma unroll
        for (int i = 0; i < h; ++i)
            m[i] = top_bf16x2(m[i], m[i + h]);
    m[0] &= 0x7FFF7FFFu;
    const int ea = pow2_exponent<ELEM>(__uint_as_float(m[0] << 16), MX_SCALE_FLOOR);
    const int eb = pow2_exponent<ELEM>(__uint_as_float(m[0] & 0xFFFF0000u), MX_SCALE_FLOOR);
    const float2 s = make_float2(exp2_neg(ea), exp2_neg(eb));
    byte_a = static_cast<uint8_t>(ea + 127);
    byte_b = static_cast<uint8_t>(eb + 127);
    if constexpr (ELEM == kElemE4M3) {
        uint32_t a[8], b[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const float2 p = scaled(w[4 * i], s), q = scaled(w[4 * i + 1], s), r = scaled(w[4 * i + 2], s), t = scaled(w[4 * i + 3], s);
            a[i] = cvt_e4m3x2(p.x, q.x) | cvt_e4m3x2(r.x, t.x) << 16;
            b[i] = cvt_e4m3x2(p.y, q.y) | cvt_e4m3x2(r.y, t.y) << 16;
        }
        store_sector(to_a, a);  // in two halves each: 20 us more at 8192 x 14336 in an earlier form
        store_sector(to_b, b);
    } else {
        uint32_t a[4], b[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            float qa[8], qb[8];
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                const float2 p = scaled(w[8 * i + k], s);
                qa[k] = p.x;
                qb[k] = p.y;
            }
            a[i] = cvt_e2m1x8(qa);
            b[i] = cvt_e2m1x8(qb);
        }
        *reinterpret_cast<uint4*>(to_a) = make_uint4(a[0], a[1], a[2], a[3]);
        *reinterpret_cast<uint4*>(to_b) = make_uint4(b[0], b[1], b[2], b[3]);
    }
}

template <int ACT, int ELEM, int FEATURES>
__global__ void __launch_bounds__(Shape<FEATURES>::threads, Shape<FEATURES>::ctas) gated_bwd_quantize_kernel(const BwdQuantParams p)
{
    using S = Shape<FEATURES>;
    constexpr int EPB = ELEM == kElemE4M3 ? 1 : 2;  // values a byte
    constexpr bool CHUNKS = FEATURES == 128;        // a tile's scale bytes are whole chunks
    constexpr int kStage = S::stage, kPitch = S::pitch;
    extern __shared__ __align__(16) uint8_t smem[];
    uint8_t* chunks = smem + 2 * kStage;  // rowwise gate, up; columnwise gate, up
    const int f_tiles = static_cast<int>(p.F / FEATURES);
    const int tt = blockIdx.x / f_tiles, ft = blockIdx.x - tt * f_tiles;
    const int64_t t0 = static_cast<int64_t>(tt) * kTokens, f0 = static_cast<int64_t>(ft) * FEATURES;
    const int64_t row_kgroups = p.F / 64, col_kgroups = p.T / 128;  // 2F / 32 / 4, T / 32 / 4
    const int64_t groups = p.F / kAct8Group;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

    // rows: a warp takes two or four at a time
    const int oct = threadIdx.x % S::octs, row = threadIdx.x / S::octs;
#pragma unroll 1
    for (int it = 0; it < kTokens / S::rows; it += kFlight) {
        RawOct<__nv_bfloat16> dh[kFlight];
        uint2 cg[kFlight], cu[kFlight];
        uint32_t bg[kFlight], bu[kFlight];
#pragma unroll
        for (int k = 0; k < kFlight; ++k) {
            const int64_t t = t0 + (it + k) * S::rows + row;
            dh[k].load(p.dh + t * p.ldh + f0 + oct * 8);
            const int64_t at = t * p.F + f0 + oct * 8;  // F is a multiple of 32: the checkpoints' rows have no pads
            cg[k] = __ldcs(reinterpret_cast<const uint2*>(p.g8.codes + at));
            cu[k] = __ldcs(reinterpret_cast<const uint2*>(p.u8.codes + at));
            const int64_t group = t * groups + (f0 >> 5) + (oct >> 2);
            bg[k] = p.g8.sf[group];
            bu[k] = p.u8.sf[group];
        }
#pragma unroll
        for (int k = 0; k < kFlight; ++k) {
            const int r = (it + k) * S::rows + row;
            Oct d, g, u, dg, du;
            dh[k].get(d);
            decode_oct(cg[k], g);
            decode_oct(cu[k], u);
            const float2 sg = both(act8_scale(bg[k])), su = both(act8_scale(bu[k]));
#pragma unroll
            for (int j = 0; j < 4; ++j) {  // the order of mx_act_bwd's products
                const ValueSlope f = activate<ACT, true>(__fmul2_rn(g.p[j], sg));
                const float2 up = __fmul2_rn(u.p[j], su);
                dg.p[j].x = d.p[j].x * f.slope.x, dg.p[j].y = d.p[j].y * f.slope.y;
                dg.p[j].x *= up.x, dg.p[j].y *= up.y;
                du.p[j].x = d.p[j].x * f.value.x, du.p[j].y = d.p[j].y * f.value.y;
            }
            const uint4 wg = pack_oct(dg), wu = pack_oct(du);
            *reinterpret_cast<uint4*>(smem + r * kPitch + oct * 16) = wg;
            *reinterpret_cast<uint4*>(smem + kStage + r * kPitch + oct * 16) = wu;
            uint2 g_codes, u_codes;
            const uint32_t g_byte = encode_row<ELEM>(wg, g_codes), u_byte = encode_row<ELEM>(wu, u_codes);
            uint8_t* to = p.row_codes + ((t0 + r) * 2 * p.F + f0 + oct * 8) / EPB;
            if constexpr (ELEM == kElemE4M3) {
                *reinterpret_cast<uint2*>(to) = g_codes;
                *reinterpret_cast<uint2*>(to + p.F) = u_codes;
            } else {
                *reinterpret_cast<uint32_t*>(to) = g_codes.x;
                *reinterpret_cast<uint32_t*>(to + p.F / 2) = u_codes.x;
            }
            if ((lane & 3) == 0) {
                if constexpr (CHUNKS) {
                    chunks[chunk_at(r, oct >> 2)] = static_cast<uint8_t>(g_byte);
                    chunks[512 + chunk_at(r, oct >> 2)] = static_cast<uint8_t>(u_byte);
                } else {
                    const int64_t kb = (f0 >> 5) + (oct >> 2);
                    p.row_sf[sf_offset(t0 + r, kb, row_kgroups)] = static_cast<uint8_t>(g_byte);
                    p.row_sf[sf_offset(t0 + r, kb + (p.F >> 5), row_kgroups)] = static_cast<uint8_t>(u_byte);
                }
            }
        }
    }
    __syncthreads();
    // columns: a thread takes two neighbouring features of an operand and 32 tokens, a warp 64
    // features
    constexpr int kWarpsOfOperand = S::threads / 64;
    const int operand = warp / kWarpsOfOperand, pair = (warp % (FEATURES / 64)) * 32 + lane;
    const int block = (warp % kWarpsOfOperand) / (FEATURES / 64);
    uint32_t w[32];
#pragma unroll
    for (int i = 0; i < 32; ++i)
        w[i] = *reinterpret_cast<const uint32_t*>(smem + operand * kStage + (block * 32 + i) * kPitch + pair * 4);
    const int64_t f = operand * p.F + f0 + 2 * pair;
    uint8_t* to = p.col_codes + (f * p.T + t0 + block * 32) / EPB;
    uint8_t byte_a, byte_b;
    encode_columns<ELEM>(w, to, to + p.T / EPB, byte_a, byte_b);
    if constexpr (!CHUNKS) {
        p.col_sf[sf_offset(f, (t0 >> 5) + block, col_kgroups)] = byte_a;
        p.col_sf[sf_offset(f + 1, (t0 >> 5) + block, col_kgroups)] = byte_b;
    } else {
        uint8_t* bytes = chunks + (2 + operand) * 512;
        bytes[chunk_at(2 * pair, block)] = byte_a;
        bytes[chunk_at(2 * pair + 1, block)] = byte_b;
        __syncthreads();
        if (threadIdx.x < 128) {  // four chunks of 32 x 16 bytes
            const int c = threadIdx.x >> 5;
            const int64_t f_chunks = p.F / 128;
            uint8_t* out = c < 2 ? p.row_sf + (tt * row_kgroups + c * f_chunks + ft) * 512
                                 : p.col_sf + (((c - 2) * f_chunks + ft) * col_kgroups + tt) * 512;
            reinterpret_cast<uint4*>(out)[lane] = reinterpret_cast<const uint4*>(chunks + c * 512)[lane];
        }
    }
}

template <int ACT, int ELEM, int FEATURES>
int launch(const BwdQuantParams& p, const Device& d, cudaStream_t s)
{
    using S = Shape<FEATURES>;
    constexpr auto kernel = gated_bwd_quantize_kernel<ACT, ELEM, FEATURES>;
    static int configured_device = -1;
    if (configured_device != d.id) {
        if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, S::smem) != cudaSuccess)
            return MX_ERR_CUDA;
        configured_device = d.id;
    }
    return launch_kernel(kernel, static_cast<unsigned>((p.T / kTokens) * (p.F / FEATURES)), 1, S::threads, S::smem, false, s, p);
}
template <int ACT, int ELEM>
int launch(const BwdQuantParams& p, const Device& d, cudaStream_t s)
{
    if constexpr (ELEM == kElemE4M3)
        if (p.F % 128 != 0)
            return launch<ACT, ELEM, 64>(p, d, s);
    return launch<ACT, ELEM, 128>(p, d, s);
}
template <int ELEM>
int launch(int act, const BwdQuantParams& p, const Device& d, cudaStream_t s)
{
    switch (act) {
    case MX_ACT_SILU: return launch<MX_ACT_SILU, ELEM>(p, d, s);
    case MX_ACT_GELU: return launch<MX_ACT_GELU, ELEM>(p, d, s);
    default: return launch<MX_ACT_GELU_TANH, ELEM>(p, d, s);
    }
}

}  // namespace

bool gated_bwd_quantize_takes(const ActArgs& a, int fmt)
{
    // FP4's data gradient multiplies along 2 F in steps of 256: whole tiles of 128 features
    const int64_t multiple = fmt == MX_FMT_MXFP8_E4M3 ? 64 : fmt == MX_FMT_MXFP4_E2M1 ? 128 : 0;
    return multiple != 0 && a.rows % kTokens == 0 && a.cols % multiple == 0 && a.ldh % 8 == 0 &&
           reinterpret_cast<uintptr_t>(a.h) % 16 == 0 && (a.rows / kTokens) * (a.cols / 64) <= INT32_MAX;
}

int launch_gated_bwd_quantize(const ActArgs& a, const mx_tensor& rows, const mx_tensor& cols, int fmt, const Device& d,
                              cudaStream_t s)
{
    BwdQuantParams p;
    p.dh = static_cast<const __nv_bfloat16*>(a.h);
    p.ldh = a.ldh;
    p.g8 = a.gate8;
    p.u8 = a.up8;
    p.T = a.rows;
    p.F = a.cols;
    p.row_codes = static_cast<uint8_t*>(rows.codes);
    p.row_sf = rows.sf;
    p.col_codes = static_cast<uint8_t*>(cols.codes);
    p.col_sf = cols.sf;
    return fmt == MX_FMT_MXFP8_E4M3 ? launch<kElemE4M3>(a.act, p, d, s) : launch<kElemE2M1>(a.act, p, d, s);
}

}  // namespace mx
