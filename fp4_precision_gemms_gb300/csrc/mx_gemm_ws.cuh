// mx_gemm_ws.cuh -- the warp-specialised CTA-pair GEMM kernel on sm_103a tensor
// cores, with the output's arithmetic left to its user, and the host-side pieces
// that the block-scaled GEMM kernels share.
#pragma once
#include <algorithm>
#include <cmath>

#include <cuda.h>
#include <cuda_bf16.h>

#include "mx_internal.cuh"
#include "mx_ptx.cuh"

namespace mx {
namespace {

// ------------------------------------------------------------- host side
using EncodeTiledFn = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                                   const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                                   CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeTiledFn encode_fn()
{
    static EncodeTiledFn fn = [] {
        void* p = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &q) != cudaSuccess ||
            q != cudaDriverEntryPointSuccess)
            p = nullptr;
        return reinterpret_cast<EncodeTiledFn>(p);
    }();
    return fn;
}

// 2-D map over a row-major byte matrix [rows, row_bytes] with 128-byte swizzled
// boxes of box_rows x 128 bytes.
bool make_code_map(CUtensorMap* m, const void* base, int64_t rows, int64_t row_bytes, int box_rows)
{
    EncodeTiledFn enc = encode_fn();
    if (!enc)
        return false;
    const cuuint64_t dims[2] = {static_cast<cuuint64_t>(row_bytes), static_cast<cuuint64_t>(rows)};
    const cuuint64_t strides[1] = {static_cast<cuuint64_t>(row_bytes)};
    const cuuint32_t box[2] = {128u, static_cast<cuuint32_t>(box_rows)};
    const cuuint32_t estr[2] = {1u, 1u};
    return enc(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<void*>(base), dims, strides, box, estr,
               CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
               CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Tile raster: the group size in M-tiles of the grouped order (tiles walk M
// within a group, then N).  `wave` tiles run at once, and what a wave reads
// should stay in L2 (129 MB, of which 96 MB is budgeted for operand tiles).
// When all of one operand plus the other operand's tiles one wave touches fit
// the budget, that operand stays resident and the other streams once: B with
// N-fastest order (groups of one M-tile), A with one group of all M-tiles
// (the smaller resident set when both fit).  Otherwise a wave of groups of g
// M-tiles touches g A tiles and wave / g B tiles, and g near
// sqrt(wave * b_tile / a_tile) makes that set smallest.
int raster_group_m(int64_t M, int64_t N, int64_t kbytes, int bm, int bn, int m_tiles, int n_tiles, int wave)
{
    constexpr int64_t kBudget = int64_t(96) << 20;
    const int64_t a_tile = static_cast<int64_t>(bm) * kbytes, b_tile = static_cast<int64_t>(bn) * kbytes;
    const int64_t b_resident = N * kbytes + (wave + n_tiles - 1) / n_tiles * a_tile;
    const int64_t a_resident = M * kbytes + (wave + m_tiles - 1) / m_tiles * b_tile;
    const bool b_fits = b_resident <= kBudget, a_fits = a_resident <= kBudget;
    if (b_fits && (!a_fits || N <= M))
        return 1;
    if (a_fits)
        return m_tiles;
    const double g = std::sqrt(static_cast<double>(wave) * static_cast<double>(b_tile) / static_cast<double>(a_tile));
    return std::max(1, std::min(m_tiles, static_cast<int>(g + 0.5)));
}

// 2-D map over a scale-factor buffer viewed as rows of 128 bytes; one box is
// `chunks` consecutive 512-byte chunks.  Boxes past the end read zeros.
bool make_sf_map(CUtensorMap* m, const void* base, int64_t bytes, int chunks)
{
    EncodeTiledFn enc = encode_fn();
    if (!enc)
        return false;
    const cuuint64_t dims[2] = {128u, static_cast<cuuint64_t>(bytes / 128)};
    const cuuint64_t strides[1] = {128u};
    const cuuint32_t box[2] = {128u, static_cast<cuuint32_t>(4 * chunks)};
    const cuuint32_t estr[2] = {1u, 1u};
    return enc(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<void*>(base), dims, strides, box, estr,
               CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_NONE, CU_TENSOR_MAP_L2_PROMOTION_L2_128B,
               CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// ----------------------------------------------------------- device side
// One 32-bit TMEM column per lane of the calling warp's lane quarter.
__device__ __forceinline__ void tmem_st1(uint32_t taddr, uint32_t v)
{
    asm volatile("tcgen05.st.sync.aligned.32x32b.x1.b32 [%0], {%1};" ::"r"(taddr), "r"(v) : "memory");
}

__device__ __forceinline__ uint32_t lds32(uint32_t saddr)
{
    uint32_t v;
    asm volatile("ld.shared.u32 %0, [%1];" : "=r"(v) : "r"(saddr) : "memory");
    return v;
}

__device__ __forceinline__ void grouped_tile(int tile, int m_tiles, int n_tiles, int group_m, int& mt, int& nt)
{
    const int per_group = group_m * n_tiles;
    const int g = tile / per_group;
    const int first_m = g * group_m;
    const int gm = min(group_m, m_tiles - first_m);
    const int r = tile - g * per_group;
    mt = first_m + r % gm;
    nt = r / gm;
}

// The epilogue factor of output (row, col) when the tensor scales are per
// region of 128 operand rows (NVFP4_LOCAL): fl32(fl32(sA * sB) * extra), the
// same product order as the global alpha; constant over a 32-column chunk.
__device__ __forceinline__ float region_alpha(const float* tsa, const float* tsb, float extra, int row, int col0)
{
    return __fmul_rn(__fmul_rn(tsa[row >> 7], tsb[col0 >> 7]), extra);
}

__device__ __forceinline__ float max_nan(float a, float b)
{
    float d;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(d) : "f"(a), "f"(b));
    return d;
}

// ---------------------------------------------------------------------------
// Warp-specialised CTA-pair kernel.  Same tiles, operand rings, scale-factor
// layout and MMA loop as bs_gemm_pair_kernel, with the two jobs of that
// kernel's epilogue warps given to separate warps, so that neither waits for
// the other:
//   warp 0        code-tile TMA producer (both CTAs).
//   warp 1        TMEM allocation (both CTAs); in rank 0 the MMA loop.
//   warp 2        scale-factor TMA producer (both CTAs).
//   warp 3        idle.
//   warps 4-7     scale-factor stores: warp 4 + q copies every stage's scale
//                 chunks from the shared ring into lane quarter q of the
//                 stage's TMEM slot with wide tcgen05.st, as soon as the MMAs
//                 that last read that slot have completed.
//   warps 8-15    epilogue: pull this CTA's 128 x 256 accumulator rows into
//                 registers, release the accumulator, scale by alpha and write
//                 the output.  bf16 / fp32 chunks are transposed through a
//                 padded 32-row staging box per warp, so that each store
//                 instruction writes eight rows of 64 contiguous bytes.
// A stage's barrier counts the code bytes of both CTAs and one arrival from
// each of the eight scale-store warps.  Warpgroups 0 and 1 hand registers to
// the epilogue warpgroups (setmaxnreg), whose threads hold 128 accumulator
// values each.  What they make of a tile is Epi's: its chunks' columns and the
// output's arithmetic; with Epi::kHalves 2 the B tile is 128 rows of each of two
// operands, so that a tile holds the same 128 columns of both products.
constexpr int kStgPitch = 80;  // 64 data bytes per staged row + 16 of padding (no bank conflicts)

template <int HALVES>
struct WsMaps {
    CUtensorMap a, sfa, b[HALVES], sfb[HALVES];
};

template <int KIND_, int STAGES_, int BKB_ = 128, int SFS_ = 5>
struct CfgWs {
    static constexpr int KIND = KIND_;
    static constexpr int BM = 128, BN = 256;
    static constexpr int STAGES = STAGES_;
    static constexpr int BKB = BKB_;
    static constexpr int SUB = BKB / 128;
    static constexpr int EPB = KIND == 0 ? 1 : 2;
    static constexpr int BK = BKB * EPB;
    static constexpr int BLOCK = KIND == 2 ? 16 : 32;
    static constexpr int MMA_K_BYTES = 32;
    static constexpr int MMAS = BKB / MMA_K_BYTES;
    static constexpr int BPM = MMA_K_BYTES * EPB / BLOCK;
    static constexpr int NCHUNK = MMAS * BPM / 4;  // 512-byte scale chunks per 128 rows per stage
    static constexpr int A_BYTES = BM * BKB;
    static constexpr int B_BYTES = (BN / 2) * BKB;
    static constexpr int SFS = SFS_;
    static constexpr int SFA_BYTES = NCHUNK * 512;
    static constexpr int SFB_BYTES = 2 * NCHUNK * 512;
    static constexpr int STG_BOX = 32 * kStgPitch;
    static constexpr int EPI_WARPS = 8;
    static constexpr int OFF_A = 0;
    static constexpr int OFF_B = OFF_A + STAGES * A_BYTES;
    static constexpr int OFF_SFA = OFF_B + STAGES * B_BYTES;
    static constexpr int OFF_SFB = OFF_SFA + SFS * SFA_BYTES;
    static constexpr int OFF_STG = OFF_SFB + SFS * SFB_BYTES;
    static constexpr int OFF_BAR = OFF_STG + EPI_WARPS * STG_BOX;
    static constexpr int NBAR = 2 * STAGES + 3 + 2 * SFS;
    static constexpr int SMEM_BYTES = OFF_BAR + NBAR * 8 + 16;
    static constexpr int SMEM_ALLOC = SMEM_BYTES + 1024;
    static constexpr int SFA_COLS = 4 * NCHUNK;
    static constexpr int SFB_COLS = 8 * NCHUNK;
    static constexpr int TM_SFA = BN;
    static constexpr int TM_SFB = TM_SFA + STAGES * SFA_COLS;
    static constexpr int TM_USED = TM_SFB + STAGES * SFB_COLS;
    static constexpr int TM_ALLOC = 512;
    static constexpr int THREADS = 512;
    static constexpr int REGS_LOW = 64;    // warpgroups 0 and 1
    static constexpr int REGS_HIGH = 192;  // epilogue warpgroups 2 and 3
    static constexpr uint32_t AB_TYPE = KIND == 0 ? 0u : 1u;
    static constexpr uint32_t SF_E8M0 = KIND == 2 ? 0u : 1u;
    static constexpr uint32_t TX = A_BYTES + B_BYTES;
    static constexpr uint32_t SF_TX = SFA_BYTES + SFB_BYTES;
    static_assert(TM_USED <= TM_ALLOC, "TMEM budget");
    static_assert(SMEM_ALLOC <= 232448, "shared memory budget");
    static_assert(NCHUNK == 1 || NCHUNK == 2 || NCHUNK == 4, "scale chunks per stage");
    // the register pool the block launches with (128 per thread) covers the split
    static_assert(128 * (REGS_LOW + REGS_LOW) + 256 * REGS_HIGH <= THREADS * 128, "register split");
};

template <class G, class Epi>
__global__ void __launch_bounds__(512, 1)
    bs_gemm_ws_kernel(const __grid_constant__ WsMaps<Epi::kHalves> maps, const __grid_constant__ typename Epi::Params p)
{
    constexpr int KIND = G::KIND, STAGES = G::STAGES;
    constexpr int kHalves = Epi::kHalves;  // 2: the tile's two halves of 128 columns come from two operands
    const CUtensorMap &tmA = maps.a, &tmSFA = maps.sfa;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    const uint32_t s0 = smem_u32(smem);
    const uint32_t bar0 = s0 + G::OFF_BAR;
    auto full = [&](int s) { return bar0 + 8u * s; };
    auto empty = [&](int s) { return bar0 + 8u * (STAGES + s); };
    const uint32_t accf = bar0 + 8u * (2 * STAGES);
    const uint32_t acce = accf + 8u;
    const uint32_t tdone = acce + 8u;
    auto sffull = [&](int q) { return bar0 + 8u * (2 * STAGES + 3 + q); };
    auto sfempty = [&](int q) { return bar0 + 8u * (2 * STAGES + 3 + G::SFS + q); };
    volatile uint32_t* tmem_slot = reinterpret_cast<volatile uint32_t*>(smem + G::OFF_BAR + 8 * G::NBAR);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);

    const uint32_t rank = cluster_ctarank();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int cluster_id = blockIdx.x >> 1, nclusters = gridDim.x >> 1;
    const int tiles = p.m_tiles * p.n_tiles;
    const int num_kt = p.K / G::BK;
    const int my_tiles = cluster_id < tiles ? (tiles - cluster_id + nclusters - 1) / nclusters : 0;
    const int total_it = my_tiles * num_kt;

    if (threadIdx.x == 0) {
        for (int s = 0; s < STAGES; ++s) {
            mbar_init(full(s), 2 + 8);  // both code producers + four scale-store warps per CTA
            mbar_init(empty(s), 1);     // rank 0's multicast commit
        }
        mbar_init(accf, 1);
        mbar_init(acce, 2);
        mbar_init(tdone, G::EPI_WARPS);
        for (int q = 0; q < G::SFS; ++q) {
            mbar_init(sffull(q), 1);   // this CTA's scale producer
            mbar_init(sfempty(q), 4);  // this CTA's four scale-store warps
        }
        *abort_flag = 0;
        fence_mbar_init();
        prefetch_tmap(&tmA);
        prefetch_tmap(&tmSFA);
        for (int i = 0; i < kHalves; ++i) {
            prefetch_tmap(&maps.b[i]);
            prefetch_tmap(&maps.sfb[i]);
        }
    }
    if (warp == 1) {
        tmem_alloc_pair(smem_u32(const_cast<uint32_t*>(tmem_slot)), G::TM_ALLOC);
        tmem_relinquish_pair();
    }
    tc_fence_before();
    cluster_sync();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    auto fail = [&]() {
        atomicExch(p.status, MX_ERR_TIMEOUT);
        *abort_flag = 1;
    };

    // Each warpgroup changes its register allotment at one point, before its
    // warps take their roles.
    if (warp < 8) {
    regs_dec<G::REGS_LOW>();
    if (warp == 0) {
        if (lane == 0) {
            const uint32_t full0_r0 = mapa_shared(full(0), 0);
            int it = 0;
            bool stop = false;
            for (int tile = cluster_id; tile < tiles && !stop; tile += nclusters) {
                int mt, nt;
                grouped_tile(tile, p.m_tiles, p.n_tiles, p.group_m, mt, nt);
                const int arow = mt * 256 + static_cast<int>(rank) * 128;
                const CUtensorMap& tmB = maps.b[kHalves == 2 ? rank : 0];
                const int brow = kHalves == 2 ? nt * 128 : nt * 256 + static_cast<int>(rank) * 128;
                for (int kt = 0; kt < num_kt; ++kt, ++it) {
                    const int s = it % STAGES;
                    const uint32_t round = static_cast<uint32_t>(it / STAGES);
                    if (it >= STAGES && !mbar_wait_bounded(empty(s), (round - 1) & 1u, p.wait_ns))
                        fail();
                    if (*abort_flag) {
                        stop = true;
                        break;
                    }
                    const uint32_t fb = full0_r0 + 8u * s;
                    mbar_arrive_expect_tx_cluster(fb, G::TX);
#pragma unroll
                    for (int sub = 0; sub < G::SUB; ++sub) {
                        tma_load_2d_pair(s0 + G::OFF_A + s * G::A_BYTES + sub * (G::BM * 128), &tmA, fb,
                                         kt * G::BKB + sub * 128, arow);
                        tma_load_2d_pair(s0 + G::OFF_B + s * G::B_BYTES + sub * ((G::BN / 2) * 128), &tmB, fb,
                                         kt * G::BKB + sub * 128, brow);
                    }
                }
            }
            if (stop) {  // give copies already issued time to land before the CTA can exit
                const uint64_t t0 = globaltimer_ns();
                while (globaltimer_ns() - t0 < 2000000ull) {
                }
            }
        }
    } else if (warp == 1) {
        if (rank == 0) {
            const bool leader = elect_one();
            int it = 0, titer = 0;
            bool stop = false;
            for (int tile = cluster_id; tile < tiles && !stop; tile += nclusters, ++titer) {
                if (titer > 0 &&
                    !__all_sync(0xffffffffu, mbar_wait_bounded(acce, static_cast<uint32_t>(titer - 1) & 1u, p.wait_ns))) {
                    if (leader)
                        fail();
                    break;
                }
                tc_fence_after();
                for (int kt = 0; kt < num_kt; ++kt, ++it) {
                    const int s = it % STAGES;
                    const uint32_t round = static_cast<uint32_t>(it / STAGES);
                    if (!__all_sync(0xffffffffu, mbar_wait_bounded(full(s), round & 1u, p.wait_ns))) {
                        if (leader)
                            fail();
                        stop = true;
                        break;
                    }
                    tc_fence_after();
                    const uint32_t sfa_t = tmem + G::TM_SFA + s * G::SFA_COLS;
                    const uint32_t sfb_t = tmem + G::TM_SFB + s * G::SFB_COLS;
                    if (leader) {
#pragma unroll
                        for (int i = 0; i < G::MMAS; ++i) {
                            constexpr int PER_SUB = 128 / G::MMA_K_BYTES;
                            const int sub = i / PER_SUB;
                            const uint64_t adesc =
                                sdesc_kmajor_sw128(s0 + G::OFF_A + s * G::A_BYTES + sub * (G::BM * 128));
                            const uint64_t bdesc =
                                sdesc_kmajor_sw128(s0 + G::OFF_B + s * G::B_BYTES + sub * ((G::BN / 2) * 128));
                            const int fb = i * G::BPM;
                            const int chunk = fb / 4;
                            const uint32_t sf_id = static_cast<uint32_t>(fb % 4);
                            const uint32_t idesc = idesc_block_scaled(G::AB_TYPE, G::SF_E8M0, 256, G::BN, sf_id, sf_id);
                            const uint64_t koff = static_cast<uint64_t>(((i % PER_SUB) * G::MMA_K_BYTES) >> 4);
                            mma_bs_pair<KIND>(tmem, adesc + koff, bdesc + koff, idesc, sfa_t + 4 * chunk,
                                              sfb_t + 8 * chunk, (kt > 0 || i > 0) ? 1u : 0u);
                        }
                        tc_commit_pair(empty(s), 0x3);
                    }
                    __syncwarp();
                }
                if (leader)
                    tc_commit_pair(accf, 0x3);
                __syncwarp();
            }
        }
        __syncwarp();
    } else if (warp == 2) {
        if (lane == 0) {
            int it = 0;
            bool stop = false;
            for (int tile = cluster_id; tile < tiles && !stop; tile += nclusters) {
                int mt, nt;
                grouped_tile(tile, p.m_tiles, p.n_tiles, p.group_m, mt, nt);
                for (int kt = 0; kt < num_kt; ++kt, ++it) {
                    const int q = it % G::SFS;
                    const uint32_t round = static_cast<uint32_t>(it / G::SFS);
                    if (it >= G::SFS && !mbar_wait_bounded(sfempty(q), (round - 1) & 1u, p.wait_ns))
                        fail();
                    if (*abort_flag) {
                        stop = true;
                        break;
                    }
                    const int cha = static_cast<int>((mt * 2 + static_cast<int>(rank)) * p.kgroups + kt * G::NCHUNK);
                    const uint32_t fl = sffull(q);
                    mbar_arrive_expect_tx(fl, G::SF_TX);
                    tma_load_2d(s0 + G::OFF_SFA + q * G::SFA_BYTES, &tmSFA, fl, 0, cha * 4);
#pragma unroll
                    for (int r = 0; r < 2; ++r) {
                        const int chb = static_cast<int>((kHalves == 2 ? nt : nt * 2 + r) * p.kgroups + kt * G::NCHUNK);
                        tma_load_2d(s0 + G::OFF_SFB + q * G::SFB_BYTES + r * (G::SFB_BYTES / 2),
                                    &maps.sfb[kHalves == 2 ? r : 0], fl, 0, chb * 4);
                    }
                }
            }
            if (stop) {
                const uint64_t t0 = globaltimer_ns();
                while (globaltimer_ns() - t0 < 2000000ull) {
                }
            }
        }
        __syncwarp();
    } else if (warp >= 4 && warp < 8) {
        // Scale-factor stores into lane quarter q.  Lane l of the quarter gets
        // line l of every 512-byte chunk (the scales of rows l, l + 32, l + 64,
        // l + 96); A's chunks fill the slot's SFA columns in order, B's chunk c
        // of row tile r fills columns 8c + 4r .. 8c + 4r + 3 of its SFB columns.
        // Lane quarter q computes output rows 32q .. 32q + 31, so of A's chunk
        // it reads only word q (the scales of its own rows, column 4c + q):
        // NVFP4, with four A chunks per stage, stores just that word (measured:
        // the same results, 0.4-1.4 % faster; for MXFP8 no difference).  B's
        // chunks are read by every quarter (each computes all N columns) and
        // must be complete in all four (measured: storing word q alone gives
        // wrong products).
        const int q = warp & 3;
        const uint32_t lanes = static_cast<uint32_t>(q * 32) << 16;
        const uint32_t full0_r0 = mapa_shared(full(0), 0);
        for (int it = 0; it < total_it; ++it) {
            const int s = it % STAGES;
            const int qs = it % G::SFS;
            bool ok = mbar_wait_bounded(sffull(qs), static_cast<uint32_t>(it / G::SFS) & 1u, p.wait_ns) &&
                      (it < STAGES ||
                       mbar_wait_bounded(empty(s), static_cast<uint32_t>(it / STAGES - 1) & 1u, p.wait_ns));
            ok = __all_sync(0xffffffffu, ok);
            if (!ok || *abort_flag) {
                if (lane == 0 && !ok)
                    fail();
                break;
            }
            tc_fence_after();
            const uint32_t sfa_s = s0 + G::OFF_SFA + qs * G::SFA_BYTES + lane * 16;
            const uint32_t sfb_s = s0 + G::OFF_SFB + qs * G::SFB_BYTES + lane * 16;
            constexpr bool A_WORD = KIND == 2;  // A's scales: only the word this quarter reads
            uint4 va[A_WORD ? 1 : G::NCHUNK];
            if constexpr (!A_WORD) {
#pragma unroll
                for (int c = 0; c < G::NCHUNK; ++c)
                    va[c] = lds128(sfa_s + c * 512);
            }
            uint4 vb[2 * G::NCHUNK];
#pragma unroll
            for (int c = 0; c < G::NCHUNK; ++c)
#pragma unroll
                for (int r = 0; r < 2; ++r)
                    vb[2 * c + r] = lds128(sfb_s + (r * G::NCHUNK + c) * 512);
            if constexpr (A_WORD) {
#pragma unroll
                for (int c = 0; c < G::NCHUNK; ++c)
                    tmem_st1(tmem + lanes + G::TM_SFA + s * G::SFA_COLS + 4 * c + q, lds32(sfa_s + c * 512 + 4 * q));
            } else {
                tmem_st_wide<G::NCHUNK>(tmem + lanes + G::TM_SFA + s * G::SFA_COLS, va);
            }
            tmem_st_wide<2 * G::NCHUNK>(tmem + lanes + G::TM_SFB + s * G::SFB_COLS, vb);
            tmem_st_wait();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) {
                mbar_arrive(sfempty(qs));
                mbar_arrive_cluster(full0_r0 + 8u * s);
            }
        }
        __syncwarp();
    }
    } else {
        regs_inc<G::REGS_HIGH>();
        const int ew = warp - 8;   // 0 .. 7
        const int q = warp & 3;    // TMEM lane quarter this warp may access
        const int half = ew >> 2;  // accumulator columns half*128 .. +127
        const uint32_t acce_r0 = mapa_shared(acce, 0);
        Epi epi(p);
        uint8_t* stg = smem + G::OFF_STG + ew * G::STG_BOX;
        int titer = 0;
        for (int tile = cluster_id; tile < tiles; tile += nclusters, ++titer) {
            int mt, nt;
            grouped_tile(tile, p.m_tiles, p.n_tiles, p.group_m, mt, nt);
            const bool acc_ok =
                __all_sync(0xffffffffu, mbar_wait_bounded(accf, static_cast<uint32_t>(titer) & 1u, p.wait_ns));
            if (!acc_ok || *abort_flag) {
                if (lane == 0 && !acc_ok)
                    fail();
                break;
            }
            tc_fence_after();
            uint32_t r[4][32];
#pragma unroll
            for (int j = 0; j < 4; ++j)
                tmem_ld32(tmem + (static_cast<uint32_t>(q * 32) << 16) + Epi::column(half, j), r[j]);
            tmem_ld_wait();
            tc_fence_before();
            __syncwarp();
            if (lane == 0)
                mbar_arrive(tdone);
            if (ew == 0 && lane == 0) {
                if (mbar_wait_bounded(tdone, static_cast<uint32_t>(titer) & 1u, p.wait_ns))
                    mbar_arrive_cluster(acce_r0);
                else
                    fail();
            }
            epi.tile(p, mt, nt, static_cast<int>(rank), q, half, lane, r, stg);
        }
        __syncwarp();
        epi.finish(p);
    }
    tc_fence_before();
    __syncthreads();
    cluster_sync();  // remote arrivals and the peer's TMEM reads are finished
    if (warp == 1) {
        if (*abort_flag && lane == 0 && rank == 0)
            (void)mbar_wait_bounded(accf, 0, kWaitLimitNs);
        __syncwarp();
        tc_fence_after();
        tmem_dealloc_pair(tmem, G::TM_ALLOC);
    }
}

// Sets the kernel up for the device on its first launch there, then launches as many
// CTA pairs as there are tiles, or as fit.
template <class G, class Epi>
int ws_max_clusters(const Device& d, int* clusters)
{
    auto kernel = bs_gemm_ws_kernel<G, Epi>;
    // a thread's own: another's could see the device before the number of clusters
    static thread_local int configured_device = -1;
    static thread_local int max_clusters = 0;
    if (configured_device != d.id) {
        // The register split (setmaxnreg) assumes the kernel launches with 128
        // registers per thread: with fewer, the epilogue's increase could not be
        // met, so such a build is refused instead of launched.
        cudaFuncAttributes fa;
        if (cudaFuncGetAttributes(&fa, kernel) != cudaSuccess || fa.numRegs != 128)
            return MX_ERR_UNSUPPORTED;
        if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, G::SMEM_ALLOC) != cudaSuccess)
            return MX_ERR_CUDA;
        cudaLaunchConfig_t cfg = {};
        cudaLaunchAttribute attr[1];
        attr[0].id = cudaLaunchAttributeClusterDimension;
        attr[0].val.clusterDim = {2, 1, 1};
        cfg.blockDim = dim3(G::THREADS);
        cfg.dynamicSmemBytes = G::SMEM_ALLOC;
        cfg.attrs = attr;
        cfg.numAttrs = 1;
        cfg.gridDim = dim3(2 * (d.sms / 2));
        int n = 0;
        if (cudaOccupancyMaxActiveClusters(&n, kernel, &cfg) != cudaSuccess || n < 1)
            return MX_ERR_CUDA;
        max_clusters = n;
        configured_device = d.id;
    }
    *clusters = max_clusters;
    return MX_OK;
}

template <class G, class Epi>
int ws_launch(const WsMaps<Epi::kHalves>& maps, const typename Epi::Params& p, int clusters, cudaStream_t s)
{
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim = {2, 1, 1};
    cfg.gridDim = dim3(2 * std::min(p.m_tiles * p.n_tiles, clusters));
    cfg.blockDim = dim3(G::THREADS);
    cfg.dynamicSmemBytes = G::SMEM_ALLOC;
    cfg.stream = s;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    if (cudaLaunchKernelEx(&cfg, bs_gemm_ws_kernel<G, Epi>, maps, p) != cudaSuccess)
        return MX_ERR_CUDA;
    count_launch();
    return MX_OK;
}

}  // namespace
}  // namespace mx
