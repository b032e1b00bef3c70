// gated.cu -- the gated feed-forward block's first half in one kernel: both
// projections, the activation and the product, with the checkpoints that the
// backward pass reads.
//
//   h = act(g) * u,   g = A gate^T, u = A up^T
//
// The kernel is the linear layer's warp-specialised CTA pair (mx_gemm_ws.cuh): of
// its 256 x 256 tile the first 128 columns are gate features and the last 128 the
// same up features, each CTA of the pair loading one operand's 128 rows, so that an
// epilogue thread holds both factors of 64 values of h.  Nothing of g and u leaves
// the chip but their 8-bit checkpoints.
#include "mx_act8.cuh"
#include "mx_activate.cuh"
#include "mx_gemm_ws.cuh"

namespace mx {
namespace {

struct GatedParams {
    const float* tsa;
    const float* tsg;
    const float* tsu;
    __nv_bfloat16* h;
    int64_t ldh;
    int M, N, K;  // N: features
    int act;
    int ts_region;
    Act8View gate8, up8;
    int64_t groups;   // checkpoint groups of a row
    int pair_bytes;   // a thread's two exponent bytes are an aligned pair
    int64_t kgroups;
    int m_tiles, n_tiles, group_m;  // 256 x 128 tiles
    unsigned* amax_out;
    int* status;
    uint64_t wait_ns;
};

// 32 values of a row in pairs.
struct Chunk {
    float2 v[16];
};

// A checkpoint group with values that are not finite: these count for nothing but their
// own codes.
__device__ __noinline__ uint32_t encode_not_finite(Chunk& x)
{
    float m = 0.0f;
#pragma unroll
    for (int i = 0; i < 16; ++i) {
        x.v[i] = make_float2(finite_or_nan(x.v[i].x), finite_or_nan(x.v[i].y));
        m = fmaxf(m, fmaxf(fabsf(x.v[i].x), fabsf(x.v[i].y)));
    }
    return act8_byte(m);
}

// The checkpoint of 32 columns that one thread holds; returns their exponent byte.
__device__ __forceinline__ uint32_t save_codes(uint8_t* codes, Chunk x)
{
    float m[2] = {0.0f, 0.0f};
#pragma unroll
    for (int i = 0; i < 16; ++i)
        m[i & 1] = max_abs(m[i & 1], x.v[i]);
    m[0] = max_nan(m[0], m[1]);
    const uint32_t e = non_finite(m[0]) ? encode_not_finite(x) : act8_byte(m[0]);
    const float2 s = both(act8_inverse(e));
    uint32_t w[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const float2 a = __fmul2_rn(x.v[2 * i], s), b = __fmul2_rn(x.v[2 * i + 1], s);
        w[i] = cvt_e4m3x2(a.x, a.y) | cvt_e4m3x2(b.x, b.y) << 16;
    }
    uint4* dst = reinterpret_cast<uint4*>(codes);
    dst[0] = make_uint4(w[0], w[1], w[2], w[3]);
    dst[1] = make_uint4(w[4], w[5], w[6], w[7]);
    return e;
}

template <int ACT>
__device__ __forceinline__ void gated32(const Chunk& g, const Chunk& u, uint32_t (&pk)[16])
{
#pragma unroll
    for (int i = 0; i < 16; ++i)
        pk[i] = pack_bf16x2(__fmul2_rn(activate<ACT, true>(g.v[i]).value, u.v[i]));
}

// Accumulators times their factor, zeros past the first n (most chunks are whole).
__device__ __forceinline__ void scaled(Chunk& x, const uint32_t (&r)[32], float alpha, int n)
{
#pragma unroll
    for (int i = 0; i < 16; ++i)
        x.v[i] = __fmul2_rn(make_float2(__uint_as_float(r[2 * i]), __uint_as_float(r[2 * i + 1])), both(alpha));
    if (n < 32)
#pragma unroll
        for (int i = 0; i < 16; ++i)
            x.v[i] = make_float2(2 * i < n ? x.v[i].x : 0.0f, 2 * i + 1 < n ? x.v[i].y : 0.0f);
}

struct GatedEpilogue {
    using Params = GatedParams;
    static constexpr int kHalves = 2;
    float ag, au;
    Top<__nv_bfloat16> top;

    __device__ __forceinline__ explicit GatedEpilogue(const GatedParams& p)
    {
        const float ta = p.tsa ? *p.tsa : 1.0f;
        ag = __fmul_rn(ta, p.tsg ? *p.tsg : 1.0f);
        au = __fmul_rn(ta, p.tsu ? *p.tsu : 1.0f);
    }
    // chunks 0, 1: gate columns, 2, 3: the same up columns
    static __device__ __forceinline__ int column(int half, int j) { return (j >> 1) * 128 + half * 64 + (j & 1) * 32; }

    __device__ __forceinline__ void tile(const GatedParams& p, int mt, int nt, int rank, int q, int half, int lane,
                                         uint32_t (&r)[4][32], uint8_t* stg)
    {
        const int row0 = mt * 256 + rank * 128 + q * 32;
        const int row = row0 + lane;
        if (row0 >= p.M)
            return;
        const int64_t group0 = static_cast<int64_t>(row) * p.groups + nt * 4 + half * 2;
        uint32_t byte_g = 0, byte_u = 0;
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            const int col0 = nt * 128 + half * 64 + j * 32;
            const int n = p.N - col0;
            if (n <= 0)
                break;
            if (p.ts_region && row < p.M) {
                ag = region_alpha(p.tsa, p.tsg, 1.0f, row, col0);
                au = region_alpha(p.tsa, p.tsu, 1.0f, row, col0);
            }
            Chunk g, u;
            scaled(g, r[j], ag, n);
            scaled(u, r[2 + j], au, n);
            if (p.gate8.codes && row < p.M) {
                byte_g |= save_codes(p.gate8.codes + (group0 + j) * kAct8Group, g) << (8 * j);
                byte_u |= save_codes(p.up8.codes + (group0 + j) * kAct8Group, u) << (8 * j);
            }
            uint32_t pk[16];
            if (p.act == MX_ACT_SILU)
                gated32<MX_ACT_SILU>(g, u, pk);
            else if (p.act == MX_ACT_GELU)
                gated32<MX_ACT_GELU>(g, u, pk);
            else
                gated32<MX_ACT_GELU_TANH>(g, u, pk);
            if (p.amax_out && row < p.M)  // what lies past the columns is 0: act(0) * 0
#pragma unroll
                for (int i = 0; i < 16; ++i)
                    top.word(pk[i]);
            // 64 bytes of a row through the staging box: lane l writes row l, then reads and
            // stores 16 bytes of row 8 i + l / 4
#pragma unroll
            for (int w = 0; w < 4; ++w)
                *reinterpret_cast<uint4*>(stg + lane * kStgPitch + w * 16) =
                    make_uint4(pk[4 * w], pk[4 * w + 1], pk[4 * w + 2], pk[4 * w + 3]);
            __syncwarp();
            const int piece = lane & 3, c = col0 + piece * 8;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int rr = 8 * i + (lane >> 2);
                const uint4 v = *reinterpret_cast<const uint4*>(stg + rr * kStgPitch + piece * 16);
                if (row0 + rr < p.M && c < p.N) {
                    __nv_bfloat16* dst = p.h + static_cast<int64_t>(row0 + rr) * p.ldh + c;
                    if (c + 8 <= p.N) {
                        st_global_v4(dst, v);
                    } else {
                        const uint32_t w4[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
                        for (int e = 0; e < 8; ++e)
                            if (c + e < p.N)
                                reinterpret_cast<uint16_t*>(dst)[e] = static_cast<uint16_t>(w4[e >> 1] >> (16 * (e & 1)));
                    }
                }
            }
            __syncwarp();
        }
        if (p.gate8.codes && row < p.M) {  // the thread's two exponent bytes, at once where they are an aligned pair
            if (p.pair_bytes) {
                if (nt * 128 + half * 64 < p.N) {
                    *reinterpret_cast<uint16_t*>(p.gate8.sf + group0) = static_cast<uint16_t>(byte_g);
                    *reinterpret_cast<uint16_t*>(p.up8.sf + group0) = static_cast<uint16_t>(byte_u);
                }
            } else {
#pragma unroll
                for (int j = 0; j < 2; ++j)
                    if (nt * 128 + half * 64 + j * 32 < p.N) {
                        p.gate8.sf[group0 + j] = static_cast<uint8_t>(byte_g >> (8 * j));
                        p.up8.sf[group0 + j] = static_cast<uint8_t>(byte_u >> (8 * j));
                    }
            }
        }
    }
    __device__ __forceinline__ void finish(const GatedParams& p)
    {
        if (p.amax_out)
            flush_top(p.amax_out, top);
    }
};

template <int KIND, int STAGES, int BKB, int SFS>
int launch_gated_ws(const GatedArgs& a, const Device& d, cudaStream_t s)
{
    using G = CfgWs<KIND, STAGES, BKB, SFS>;
    int clusters = 0;
    const int rc = ws_max_clusters<G, GatedEpilogue>(d, &clusters);
    if (rc != MX_OK)
        return rc;
    const int64_t M = a.x->rows, N = a.gate->rows, K = a.x->k, kbytes = K / G::EPB;
    const int64_t sfa = sf_layout_bytes(M, K / G::BLOCK), sfb = sf_layout_bytes(N, K / G::BLOCK);
    WsMaps<2> maps;
    if (!make_code_map(&maps.a, a.x->codes, M, kbytes, 128) || !make_sf_map(&maps.sfa, a.x->sf, sfa, G::NCHUNK) ||
        !make_code_map(&maps.b[0], a.gate->codes, N, kbytes, 128) || !make_sf_map(&maps.sfb[0], a.gate->sf, sfb, G::NCHUNK) ||
        !make_code_map(&maps.b[1], a.up->codes, N, kbytes, 128) || !make_sf_map(&maps.sfb[1], a.up->sf, sfb, G::NCHUNK))
        return MX_ERR_CUDA;
    GatedParams p;
    const bool ts = fmt_has_tensor_scale(a.x->fmt);
    p.tsa = ts ? a.x->tensor_scale : nullptr;
    p.tsg = ts ? a.gate->tensor_scale : nullptr;
    p.tsu = ts ? a.up->tensor_scale : nullptr;
    p.h = static_cast<__nv_bfloat16*>(a.h);
    p.ldh = a.ldh;
    p.M = static_cast<int>(M);
    p.N = static_cast<int>(N);
    p.K = static_cast<int>(K);
    p.act = a.act;
    p.ts_region = fmt_is_local(a.x->fmt) ? 1 : 0;
    p.gate8 = a.gate8;
    p.up8 = a.up8;
    p.groups = act8_groups(N);
    p.pair_bytes = N % 64 == 0 && reinterpret_cast<uintptr_t>(a.gate8.sf) % 2 == 0 && reinterpret_cast<uintptr_t>(a.up8.sf) % 2 == 0;
    p.kgroups = sf_kgroups(K / G::BLOCK);
    p.m_tiles = static_cast<int>((M + 255) / 256);
    p.n_tiles = static_cast<int>((N + 127) / 128);
    p.group_m = raster_group_m(M, 2 * N, kbytes, 256, 256, p.m_tiles, p.n_tiles, clusters);
    p.amax_out = a.amax;
    p.status = d.status;
    p.wait_ns = kWaitLimitNs;
    return ws_launch<G, GatedEpilogue>(maps, p, clusters, s);
}

}  // namespace

int launch_gated(const GatedArgs& a, const Device& d, cudaStream_t s)
{
    const int64_t K = a.x->k;
    if (a.x->rows <= kGatedFewTokens && !a.gate8.codes)
        return launch_gated_few(a, a.early, d, s);
    switch (a.x->fmt) {  // stages as the plain GEMM has them
    case MX_FMT_MXFP8_E4M3:
    case MX_FMT_MOSS_FP8:
        return K % 256 == 0 ? launch_gated_ws<0, 3, 256, 4>(a, d, s) : launch_gated_ws<0, 5, 128, 6>(a, d, s);
    case MX_FMT_MXFP4_E2M1:
        return K % 512 == 0 ? launch_gated_ws<1, 3, 256, 2>(a, d, s) : launch_gated_ws<1, 5, 128, 6>(a, d, s);
    default: return launch_gated_ws<2, 5, 128, 5>(a, d, s);
    }
}

}  // namespace mx
