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
//
// Bound by the tensor pipe without checkpoints: 8192 tokens, 4096 x 14336, MXFP8 526 us
// (3.66 PFLOP/s; the plain GEMM of both projections, which writes twice as much, 547),
// NVFP4 311 us (plain 336).  With checkpoints 610 and 414 us: a tile's epilogue is then
// longer than its products, by the codes' scattered sectors (NVFP4: 60 us of the 414 in an
// earlier form), the exponent bytes (40) and the encoding (50).  Through the staging box, or
// as tensor stores of 64-byte rows, the codes took longer still.
#include "mx_act8.cuh"
#include "mx_activate.cuh"
#include "mx_gemm_ws.cuh"

namespace mx {
namespace {

struct GatedParams {
    CUtensorMap map_h;  // h's columns up to a multiple of eight, in boxes of 32 rows x 32 columns
    __nv_bfloat16* h;
    int64_t ldh;
    const float* tsa;
    const float* tsg;
    const float* tsu;
    int M, N, K;  // N: features
    int act;
    int ts_region;
    Act8View gate8, up8;
    int64_t groups;   // checkpoint groups of a row
    int pair_bytes;   // a thread's two exponent bytes are an aligned pair
    int sectors;      // the checkpoints' codes start on 32-byte boundaries
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

// 32 bytes to a multiple of 32 (sectors) or of 16.
__device__ __forceinline__ void store32(uint8_t* to, bool sectors, const uint32_t (&w)[8])
{
    if (sectors) {
        store_sector(to, w);
    } else {
        reinterpret_cast<uint4*>(to)[0] = make_uint4(w[0], w[1], w[2], w[3]);
        reinterpret_cast<uint4*>(to)[1] = make_uint4(w[4], w[5], w[6], w[7]);
    }
}

// The checkpoint codes of 32 columns that one thread holds; returns their exponent byte.
__device__ __forceinline__ uint32_t encode_group(Chunk x, uint32_t (&w)[8])
{
    float m[2] = {0.0f, 0.0f};
#pragma unroll
    for (int i = 0; i < 16; ++i)
        m[i & 1] = max_abs(m[i & 1], x.v[i]);
    m[0] = max_nan(m[0], m[1]);
    const uint32_t e = non_finite(m[0]) ? encode_not_finite(x) : act8_byte(m[0]);
    const float2 s = both(act8_inverse(e));
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const float2 a = __fmul2_rn(x.v[2 * i], s), b = __fmul2_rn(x.v[2 * i + 1], s);
        w[i] = cvt_e4m3x2(a.x, a.y) | cvt_e4m3x2(b.x, b.y) << 16;
    }
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
    bool busy = false;  // the warp's staging box may still be read by a store
    Top<__nv_bfloat16> top;

    __device__ __forceinline__ explicit GatedEpilogue(const GatedParams& p)
    {
        const float ta = p.tsa ? *p.tsa : 1.0f;
        ag = __fmul_rn(ta, p.tsg ? *p.tsg : 1.0f);
        au = __fmul_rn(ta, p.tsu ? *p.tsu : 1.0f);
    }
    // 64 bytes of each of the warp's 32 rows to column x on, by a tensor store that clips
    // what lies outside the map.  The box is swizzled (16-byte pieces of a 64-byte row
    // exchanged by the row's pair number), which keeps the lanes' writes apart in the banks.
    // The stores that leave the chip then cost the load/store unit nothing, on which the
    // warps that feed the scales depend.
    // A store writes its last 16 bytes whole, so the map ends at a multiple of eight columns;
    // those after it the lanes take from the box one by one.
    __device__ __forceinline__ void send(const GatedParams& p, const uint32_t (&w)[16], int x, int row0, int lane, uint8_t* stg)
    {
        if (busy) {  // the previous store has read the box
            if (lane == 0)
                bulk_wait_read_all();
            __syncwarp();
        }
#pragma unroll
        for (int i = 0; i < 4; ++i)
            *reinterpret_cast<uint4*>(stg + lane * 64 + ((i ^ (lane >> 1)) & 3) * 16) =
                make_uint4(w[4 * i], w[4 * i + 1], w[4 * i + 2], w[4 * i + 3]);
        const int edge = p.N & ~7;
        busy = x < edge;
        if (busy) {
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) {
                tma_store_2d(&p.map_h, smem_u32(stg), x, row0);
                bulk_commit();
            }
        }
        if (x + 32 > edge && edge < p.N && row0 + lane < p.M) {
            const uint8_t* from = stg + lane * 64 + (((edge - x) >> 3 ^ (lane >> 1)) & 3) * 16;
            __nv_bfloat16* to = p.h + (row0 + lane) * p.ldh + edge;
#pragma unroll 1
            for (int i = 0; i < p.N - edge; ++i)
                to[i] = reinterpret_cast<const __nv_bfloat16*>(from)[i];
        }
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
        const int col = nt * 128 + half * 64;
        if (col >= p.N)
            return;
        const int64_t group0 = static_cast<int64_t>(row) * p.groups + col / kAct8Group;
        const bool save = p.gate8.codes && row < p.M;
        uint32_t byte_g = 0, byte_u = 0;
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            const int col0 = col + j * 32;
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
            if (save) {
                uint32_t w[8];
                byte_g |= encode_group(g, w) << (8 * j);
                store32(p.gate8.codes + (group0 + j) * kAct8Group, p.sectors, w);
                byte_u |= encode_group(u, w) << (8 * j);
                store32(p.up8.codes + (group0 + j) * kAct8Group, p.sectors, w);
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
            send(p, pk, col0, row0, lane, stg);
        }
        if (!save)
            return;
        if (p.pair_bytes) {  // the thread's two exponent bytes at once
            *reinterpret_cast<uint16_t*>(p.gate8.sf + group0) = static_cast<uint16_t>(byte_g);
            *reinterpret_cast<uint16_t*>(p.up8.sf + group0) = static_cast<uint16_t>(byte_u);
            return;
        }
#pragma unroll
        for (int j = 0; j < 2; ++j)
            if (col + j * 32 < p.N) {
                p.gate8.sf[group0 + j] = static_cast<uint8_t>(byte_g >> (8 * j));
                p.up8.sf[group0 + j] = static_cast<uint8_t>(byte_u >> (8 * j));
            }
    }
    __device__ __forceinline__ void finish(const GatedParams& p)
    {
        if ((threadIdx.x & 31) == 0)
            bulk_wait_all();  // the box's next use may have waited for a store's reads only
        __syncwarp();
        if (p.amax_out)
            flush_top(p.amax_out, top);
    }
};

// 2-D map over h (row stride ld) for stores of 32 x 32 boxes with the 64-byte swizzle.  With
// fewer than eight columns no store is made through it.
bool make_h_map(CUtensorMap* m, void* base, int64_t rows, int64_t cols, int64_t ld)
{
    EncodeTiledFn enc = encode_fn();
    if (!enc)
        return false;
    const cuuint64_t dims[2] = {static_cast<cuuint64_t>(std::max<int64_t>(cols & ~int64_t{7}, 8)), static_cast<cuuint64_t>(rows)};
    const cuuint64_t strides[1] = {static_cast<cuuint64_t>(ld) * 2};
    const cuuint32_t box[2] = {32u, 32u};
    const cuuint32_t estr[2] = {1u, 1u};
    return enc(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, base, dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
               CU_TENSOR_MAP_SWIZZLE_64B, CU_TENSOR_MAP_L2_PROMOTION_NONE, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

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
    if (!make_h_map(&p.map_h, a.h, M, N, a.ldh))
        return MX_ERR_CUDA;
    p.h = static_cast<__nv_bfloat16*>(a.h);
    p.ldh = a.ldh;
    const bool ts = fmt_has_tensor_scale(a.x->fmt);
    p.tsa = ts ? a.x->tensor_scale : nullptr;
    p.tsg = ts ? a.gate->tensor_scale : nullptr;
    p.tsu = ts ? a.up->tensor_scale : nullptr;
    p.M = static_cast<int>(M);
    p.N = static_cast<int>(N);
    p.K = static_cast<int>(K);
    p.act = a.act;
    p.ts_region = fmt_is_local(a.x->fmt) ? 1 : 0;
    p.gate8 = a.gate8;
    p.up8 = a.up8;
    p.groups = act8_groups(N);
    p.pair_bytes = N % 64 == 0 && reinterpret_cast<uintptr_t>(a.gate8.sf) % 2 == 0 && reinterpret_cast<uintptr_t>(a.up8.sf) % 2 == 0;
    p.sectors = reinterpret_cast<uintptr_t>(a.gate8.codes) % 32 == 0 && reinterpret_cast<uintptr_t>(a.up8.codes) % 32 == 0;
    p.kgroups = sf_kgroups(K / G::BLOCK);
    p.m_tiles = static_cast<int>((M + 255) / 256);
    p.n_tiles = static_cast<int>((N + 127) / 128);
    p.group_m = raster_group_m(M, 2 * N, kbytes, 256, 256, p.m_tiles, p.n_tiles, clusters);
    p.amax_out = a.amax;
    p.status = d.status;
    p.wait_ns = kWaitLimitNs;
    return ws_launch<G, GatedEpilogue>(maps, p, clusters, s);
}

__global__ void __launch_bounds__(256) move_scales_kernel(const uint8_t* __restrict__ sf, int64_t from, int64_t rows,
                                                         int64_t kgroups, uint8_t* __restrict__ to)
{
    const int64_t words = (rows + 127) / 128 * 128 * kgroups, stride = static_cast<int64_t>(gridDim.x) * 256;
    for (int64_t i = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x; i < words; i += stride) {
        // 128 words of a chunk at a time: word i % 128 of its chunk in the order of the layout
        const int64_t chunk = i >> 7, tile = chunk / kgroups, kg = chunk - tile * kgroups;
        const int64_t r = tile * 128 + (i & 3) * 32 + ((i & 127) >> 2);
        if (r < rows)
            *reinterpret_cast<uint32_t*>(to + sf_offset(r, kg * 4, kgroups)) =
                *reinterpret_cast<const uint32_t*>(sf + sf_offset(from + r, kg * 4, kgroups));
    }
}

}  // namespace

int launch_move_scales(const uint8_t* sf, int64_t from, int64_t rows, int64_t kgroups, uint8_t* to, cudaStream_t s)
{
    const int64_t padded = (rows + 127) / 128 * 128;  // whole chunks
    const unsigned ctas = static_cast<unsigned>(std::min<int64_t>((padded * kgroups + 255) / 256, 152 * 8));
    return launch_kernel(move_scales_kernel, ctas, 1, 256, 0, false, s, sf, from, rows, kgroups, to);
}

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
