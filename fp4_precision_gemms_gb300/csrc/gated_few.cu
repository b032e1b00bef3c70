// gated_few.cu -- the gated feed-forward block's first half for few tokens: the
// weights' bytes are all that counts, so the weights are the M side of the tensor
// core's tile and the tokens, padded to a multiple of 16, its N side.
//
// A tile is 128 features: two accumulators of 128 x N in TMEM, gate and up, from the
// same token tile.  Warp 0 (one thread) streams both weight tiles through a ring of
// stages, warp 2 (one thread) the token tile and all scales; warps 4-7 store a stage's
// scales to TMEM, each the quarter of the lanes that it may; warp 1 (one thread) issues the
// MMAs; warps 8-15 hold one feature a lane and write h, sixteen tokens at a time.  With the
// scales copied by tcgen05.cp, which takes the tensor pipe 30 ns each, a step of 32 KB of
// weights took 514 ns (MXFP8) and 790 (NVFP4, twelve copies).  Launched with programmatic dependent launch behind
// the tokens' quantization, the kernel fills its ring with weights before that has finished.
//
// Where the tiles are too few, or a little more than the SMs, their steps along K, one tile
// after another, are cut into equal ranges, one an SM (gated_few_cut).  A tile
// that lies in several ranges leaves partial sums in a workspace; the CTA that counts
// itself last for the tile, after its own partial sums are visible, adds them up in the
// ranges' order.  No CTA waits for another.
//
// 14336 x 4096 with the tokens' quantization: MXFP8, 1 token 24 us (121 MB, 5.1 TB/s),
// NVFP4, 48 tokens 17.2 us (66 MB; 15 with the weights partly in L2).  Bound by DRAM and by
// what does not stream: launch, first and last tile, 5 us.  The tokens end where TMEM does
// (two accumulators twice, beside the scales); the kernel for many takes 35.6 and 31.2 us for
// 65 tokens, where this one takes 25.3 and 17.3 for 64.
//
// Every wait is bounded, as in gemm.cu.
#include <algorithm>

#include "mx_act8.cuh"
#include "mx_activate.cuh"
#include "mx_gemm_ws.cuh"

namespace mx {
namespace {

template <int KIND>
struct CfgFew {
    static constexpr int BM = 128, BN = kGatedFewTokens;
    static constexpr int BKB = 128;
    static constexpr int EPB = KIND == 0 ? 1 : 2;
    static constexpr int BK = BKB * EPB;
    static constexpr int BLOCK = KIND == 2 ? 16 : 32;
    static constexpr int MMA_K_BYTES = 32;
    static constexpr int MMAS = BKB / MMA_K_BYTES;
    static constexpr int BPM = MMA_K_BYTES * EPB / BLOCK;
    static constexpr int NCHUNK = MMAS * BPM / 4;
    static constexpr int STAGES = KIND == 2 ? 4 : 5;
    static constexpr int W_BYTES = BM * BKB;  // of each weight tile
    static constexpr int X_BYTES = BN * BKB;
    static constexpr int SF_BYTES = NCHUNK * 512;  // of each of the three
    static constexpr int OFF_W = 0;
    static constexpr int OFF_X = OFF_W + STAGES * 2 * W_BYTES;
    static constexpr int OFF_SF = OFF_X + STAGES * X_BYTES;
    static constexpr int OFF_BAR = OFF_SF + STAGES * 3 * SF_BYTES;
    static constexpr int SMEM_BYTES = OFF_BAR + (3 * STAGES + 4) * 8 + 16;
    static constexpr int SMEM_ALLOC = SMEM_BYTES + 1024;
    // TMEM: two accumulators twice (a tile's sums are read while the next one's are
    // formed), then three scale regions a stage
    static constexpr int SF_COLS = 4 * NCHUNK;
    static constexpr int TM_SF = 4 * BN;
    static constexpr int TM_USED = TM_SF + STAGES * 3 * SF_COLS;
    static constexpr int TM_ALLOC = 512;
    static constexpr uint32_t AB_TYPE = KIND == 0 ? 0u : 1u;
    static constexpr uint32_t SF_E8M0 = KIND == 2 ? 0u : 1u;
    static_assert(TM_USED <= 512, "TMEM budget");
    static_assert(SMEM_ALLOC <= 232448, "shared memory budget");
};

struct FewParams {
    const uint8_t* sfx;
    const uint8_t* sfg;
    const uint8_t* sfu;
    const float* tsa;
    const float* tsg;
    const float* tsu;
    __nv_bfloat16* h;
    int64_t ldh;
    int M, N, K;  // tokens, features
    int n_pad;    // the MMA's N: tokens up to a multiple of 16
    int act, ts_region;
    int early;    // weights may be read before the launch before this one has finished
    int64_t kgroups;
    unsigned* amax_out;
    float4* parts;      // two slots of partial sums a CTA; null: every range is whole tiles
    unsigned* counters; // one a tile, zero before the kernel
    int* status;
    uint64_t wait_ns;
};

// CTA c has the steps from first_step(c) to first_step(c + 1) of tiles x num_kt.
struct Ranges {
    int64_t steps;
    int ctas, num_kt;
    __device__ __forceinline__ int64_t first_step(int c) const { return steps * c / ctas; }
    __device__ __forceinline__ int cta_of(int64_t step) const  // the last c with first_step(c) <= step
    {
        return static_cast<int>(((step + 1) * ctas - 1) / steps);
    }
};
constexpr int kJoin = 2;  // fours of tokens whose partial sums are read together

// Each thread of the warp reads 16 consecutive fp32 columns of its TMEM lane.
__device__ __forceinline__ void tmem_ld16(uint32_t taddr, float (&r)[16])
{
    uint32_t v[16];
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
        : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]), "=r"(v[7]), "=r"(v[8]), "=r"(v[9]),
          "=r"(v[10]), "=r"(v[11]), "=r"(v[12]), "=r"(v[13]), "=r"(v[14]), "=r"(v[15])
        : "r"(taddr)
        : "memory");
    tmem_ld_wait();
#pragma unroll
    for (int i = 0; i < 16; ++i)
        r[i] = __uint_as_float(v[i]);
}

// h of N tokens' sums of one feature, of which the first n are written.  All are
// computed, so that the exponentials overlap.  The maximum goes by the fp32 form of what
// is written.
template <int ACT, int N>
__device__ __forceinline__ void write_h(const float (&g)[N], const float (&u)[N], float ag, float au, int n,
                                        __nv_bfloat16* dst, int64_t ldh, Top<float>& top)
{
    float v[N];
#pragma unroll
    for (int i = 0; i < N; i += 2) {
        const float2 a = activate<ACT, true>(make_float2(__fmul_rn(g[i], ag), __fmul_rn(g[i + 1], ag))).value;
        v[i] = a.x * __fmul_rn(u[i], au);
        v[i + 1] = a.y * __fmul_rn(u[i + 1], au);
    }
#pragma unroll
    for (int i = 0; i < N; ++i)
        if (i < n) {
            const __nv_bfloat16 r = __float2bfloat16_rn(v[i]);
            dst[i * ldh] = r;
            top.value(__bfloat162float(r));
        }
}
template <int N>
__device__ __forceinline__ void write_h(int act, const float (&g)[N], const float (&u)[N], float ag, float au, int n,
                                        __nv_bfloat16* dst, int64_t ldh, Top<float>& top)
{
    if (act == MX_ACT_SILU)
        write_h<MX_ACT_SILU>(g, u, ag, au, n, dst, ldh, top);
    else if (act == MX_ACT_GELU)
        write_h<MX_ACT_GELU>(g, u, ag, au, n, dst, ldh, top);
    else
        write_h<MX_ACT_GELU_TANH>(g, u, ag, au, n, dst, ldh, top);
}

template <int KIND>
__global__ void __launch_bounds__(512, 1)
    gated_few_kernel(const __grid_constant__ CUtensorMap tmX, const __grid_constant__ CUtensorMap tmG,
                     const __grid_constant__ CUtensorMap tmU, const FewParams p)
{
    using G = CfgFew<KIND>;
    constexpr int STAGES = G::STAGES;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    const uint32_t s0 = smem_u32(smem);
    const uint32_t bar0 = s0 + G::OFF_BAR;
    auto full = [&](int s) { return bar0 + 8u * s; };
    auto empty = [&](int s) { return bar0 + 8u * (STAGES + s); };
    auto scales = [&](int s) { return bar0 + 8u * (2 * STAGES + s); };
    auto accf = [&](int b) { return bar0 + 8u * (3 * STAGES + b); };
    auto acce = [&](int b) { return bar0 + 8u * (3 * STAGES + 2 + b); };
    volatile uint32_t* tmem_slot = reinterpret_cast<volatile uint32_t*>(smem + G::OFF_BAR + 8 * (3 * STAGES + 4));
    volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
    volatile uint32_t* arrived = tmem_slot + 2;

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int num_kt = p.K / G::BK;
    const Ranges ranges = {static_cast<int64_t>((p.N + 127) / 128) * num_kt, static_cast<int>(gridDim.x), num_kt};
    const int64_t begin = ranges.first_step(blockIdx.x), last = ranges.first_step(blockIdx.x + 1);
    const int my_steps = static_cast<int>(last - begin);
    const int tile0 = static_cast<int>(begin / num_kt), kt0 = static_cast<int>(begin - static_cast<int64_t>(tile0) * num_kt);

    if (threadIdx.x == 0) {
        for (int s = 0; s < STAGES; ++s) {
            mbar_init(full(s), 2 + 4);  // both producers and the warps that store the scales
            mbar_init(empty(s), 1);
            mbar_init(scales(s), 1);
        }
        for (int b = 0; b < 2; ++b) {
            mbar_init(accf(b), 1);
            mbar_init(acce(b), 8);  // the epilogue warps
        }
        *abort_flag = 0;
        fence_mbar_init();
        prefetch_tmap(&tmX);
        prefetch_tmap(&tmG);
        prefetch_tmap(&tmU);
    }
    if (warp == 1) {
        tmem_alloc(smem_u32(const_cast<uint32_t*>(tmem_slot)), G::TM_ALLOC);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    auto fail = [&]() {
        atomicExch(p.status, MX_ERR_TIMEOUT);
        *abort_flag = 1;
    };
    // Runs load(stage, tile, kt) for every step whose stage is free; false when a wait ran out.
    auto produce = [&](auto load, int& it) -> bool {
        int tile = tile0, kt = kt0;
        for (; it < my_steps; ++it) {
            const int s = it % STAGES;
            if (it >= STAGES && !mbar_wait_bounded(empty(s), static_cast<uint32_t>(it / STAGES - 1) & 1u, p.wait_ns))
                fail();
            if (*abort_flag)
                return false;
            load(s, tile, kt);
            if (++kt == num_kt) {
                kt = 0;
                ++tile;
            }
        }
        return true;
    };
    // Lets the copies already issued land before the CTA can exit (the other producer's of
    // a stage may be missing: the waits are bounded).
    auto drain = [&](int it) {
        for (int k = max(0, it - STAGES); k < it; ++k)
            (void)mbar_wait_bounded(full(k % STAGES), static_cast<uint32_t>(k / STAGES) & 1u, 2000000ull);
    };

    if (warp == 0) {
        if (lane == 0) {
            auto load = [&](int s, int tile, int kt) {
                mbar_arrive_expect_tx(full(s), 2 * G::W_BYTES);
                tma_load_2d(s0 + G::OFF_W + (2 * s) * G::W_BYTES, &tmG, full(s), kt * G::BKB, tile * 128);
                tma_load_2d(s0 + G::OFF_W + (2 * s + 1) * G::W_BYTES, &tmU, full(s), kt * G::BKB, tile * 128);
            };
            if (!p.early)
                wait_for_launch_before();
            int it = 0;
            if (!produce(load, it))
                drain(it);
            wait_for_launch_before();  // this CTA ends after the launch before it in any case
        }
        __syncwarp();
    } else if (warp == 2) {
        if (lane == 0) {
            auto load = [&](int s, int tile, int kt) {
                const int64_t chunk = static_cast<int64_t>(tile) * p.kgroups + static_cast<int64_t>(kt) * G::NCHUNK;
                mbar_arrive_expect_tx(scales(s), 3 * G::SF_BYTES);
                bulk_load(s0 + G::OFF_SF + (3 * s) * G::SF_BYTES, p.sfg + chunk * 512, G::SF_BYTES, scales(s));
                bulk_load(s0 + G::OFF_SF + (3 * s + 1) * G::SF_BYTES, p.sfu + chunk * 512, G::SF_BYTES, scales(s));
                bulk_load(s0 + G::OFF_SF + (3 * s + 2) * G::SF_BYTES, p.sfx + static_cast<int64_t>(kt) * G::NCHUNK * 512,
                          G::SF_BYTES, scales(s));
                mbar_arrive_expect_tx(full(s), p.n_pad * G::BKB);
                tma_load_2d(s0 + G::OFF_X + s * G::X_BYTES, &tmX, full(s), kt * G::BKB, 0);
            };
            wait_for_launch_before();
            int it = 0;
            if (!produce(load, it)) {
                drain(it);
                for (int k = max(0, it - STAGES); k < it; ++k)
                    (void)mbar_wait_bounded(scales(k % STAGES), static_cast<uint32_t>(k / STAGES) & 1u, 2000000ull);
            }
        }
        __syncwarp();
    } else if (warp >= 4 && warp < 8) {
        // Lane l of lane quarter q gets line l of every 512-byte chunk.  The quarter computes
        // weight rows 32 q .. 32 q + 31 of either operand, whose scales are word q of the
        // lines; of the tokens' it needs all words.  A stage's slot is free once its bytes
        // have been loaded again.
        const int q = warp & 3;
        const uint32_t lanes = static_cast<uint32_t>(q * 32) << 16;
        for (int it = 0; it < my_steps; ++it) {
            const int s = it % STAGES;
            const bool ok =
                __all_sync(0xffffffffu, mbar_wait_bounded(scales(s), static_cast<uint32_t>(it / STAGES) & 1u, p.wait_ns));
            if (!ok || *abort_flag) {
                if (lane == 0 && !ok)
                    fail();
                break;
            }
            tc_fence_after();
            const uint32_t from = s0 + G::OFF_SF + 3 * s * G::SF_BYTES + lane * 16;
            const uint32_t to = tmem + lanes + G::TM_SF + s * 3 * G::SF_COLS;
            uint4 x[G::NCHUNK];
            uint32_t w[2][G::NCHUNK];
#pragma unroll
            for (int c = 0; c < G::NCHUNK; ++c) {
                w[0][c] = lds32(from + c * 512 + 4 * q);
                w[1][c] = lds32(from + G::SF_BYTES + c * 512 + 4 * q);
                x[c] = lds128(from + 2 * G::SF_BYTES + c * 512);
            }
#pragma unroll
            for (int o = 0; o < 2; ++o)
#pragma unroll
                for (int c = 0; c < G::NCHUNK; ++c)
                    tmem_st1(to + o * G::SF_COLS + 4 * c + q, w[o][c]);
            tmem_st_wide<G::NCHUNK>(to + 2 * G::SF_COLS, x);
            tmem_st_wait();
            tc_fence_before();
            __syncwarp();
            if (lane == 0)
                mbar_arrive(full(s));
        }
        __syncwarp();
    } else if (warp == 1) {
        if (lane == 0) {
            int it = 0, n = 0, kt = kt0;
            bool stop = false;
            for (int left = my_steps; left > 0 && !stop; ++n) {
                const int end = min(num_kt, kt + left);
                const uint32_t acc = tmem + (n & 1) * 2 * G::BN;
                if (n >= 2 && !mbar_wait_bounded(acce(n & 1), static_cast<uint32_t>((n >> 1) - 1) & 1u, p.wait_ns)) {
                    fail();
                    break;
                }
                tc_fence_after();
                left -= end - kt;
                for (int k = kt; k < end; ++k, ++it) {
                    const int s = it % STAGES;
                    if (!mbar_wait_bounded(full(s), static_cast<uint32_t>(it / STAGES) & 1u, p.wait_ns)) {
                        fail();
                        stop = true;
                        break;
                    }
                    tc_fence_after();
                    const uint32_t sf_t = tmem + G::TM_SF + s * 3 * G::SF_COLS;
                    const uint64_t xdesc = sdesc_kmajor_sw128(s0 + G::OFF_X + s * G::X_BYTES);
#pragma unroll
                    for (int o = 0; o < 2; ++o) {
                        const uint64_t wdesc = sdesc_kmajor_sw128(s0 + G::OFF_W + (2 * s + o) * G::W_BYTES);
#pragma unroll
                        for (int i = 0; i < G::MMAS; ++i) {
                            const int fb = i * G::BPM, chunk = fb / 4;
                            const uint32_t sf_id = static_cast<uint32_t>(fb % 4);
                            const uint32_t idesc = idesc_block_scaled(G::AB_TYPE, G::SF_E8M0, 128, 0, sf_id, sf_id) |
                                                   static_cast<uint32_t>(p.n_pad >> 3) << 17;
                            const uint64_t koff = static_cast<uint64_t>((i * G::MMA_K_BYTES) >> 4);
                            mma_bs<KIND>(acc + o * G::BN, wdesc + koff, xdesc + koff, idesc, sf_t + o * G::SF_COLS + 4 * chunk,
                                         sf_t + 2 * G::SF_COLS + 4 * chunk, (k > kt || i > 0) ? 1u : 0u);
                        }
                    }
                    tc_commit(empty(s));
                }
                tc_commit(accf(n & 1));
                kt = 0;
            }
        }
        __syncwarp();
    } else if (warp >= 8) {
        const int q = warp & 3;            // TMEM lane quarter
        const int half = (warp - 8) >> 2;  // of the sixteens of tokens, every other one
        const int tokens4 = (p.M + 3) / 4;
        const int64_t slot_size = static_cast<int64_t>(2) * tokens4 * 128;  // float4 of a slot: [gate, up][token / 4][feature]
        Top<float> top;
        wait_for_launch_before();  // the tensor scale of the tokens, the counters
        const float ta = p.tsa ? *p.tsa : 1.0f;
        int n = 0, kt = kt0, tile = tile0;
        for (int left = my_steps; left > 0; ++n, ++tile) {
            const int end = min(num_kt, kt + left);
            const bool whole = kt == 0 && end == num_kt;
            left -= end - kt;
            kt = 0;
            const int f = tile * 128 + q * 32 + lane;
            const int region = p.ts_region ? tile : 0;  // of 128 weight rows
            const float ag = __fmul_rn(ta, p.tsg ? p.tsg[region] : 1.0f), au = __fmul_rn(ta, p.tsu ? p.tsu[region] : 1.0f);
            // after a wait that ran out the warp waits no more, but keeps meeting the others
            const bool ok = !*abort_flag && mbar_wait_bounded(accf(n & 1), static_cast<uint32_t>(n >> 1) & 1u, p.wait_ns);
            if (!__all_sync(0xffffffffu, ok)) {
                if (lane == 0)
                    fail();
                if (!whole)
                    for (int k = 0; k < 3; ++k)
                        named_barrier_sync(1, 256);
                continue;
            }
            tc_fence_after();
            const uint32_t acc = tmem + (n & 1) * 2 * G::BN + (static_cast<uint32_t>(q * 32) << 16);
            const int live = f < p.N ? p.M : 0;  // tokens whose h this lane writes
#pragma unroll 1
            for (int t0 = half * 16; t0 < p.M; t0 += 32) {
                float g[16], u[16];
                tmem_ld16(acc + t0, g);
                tmem_ld16(acc + G::BN + t0, u);
                if (whole) {
                    write_h(p.act, g, u, ag, au, live - t0, p.h + static_cast<int64_t>(t0) * p.ldh + f, p.ldh, top);
                } else {
                    float4* slot = p.parts + (2 * blockIdx.x + (n > 0 ? 1 : 0)) * slot_size + q * 32 + lane;
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        if (t0 + 4 * i < p.M) {
                            float4* at = slot + (t0 / 4 + i) * 128;
                            __stcg(at, make_float4(g[4 * i], g[4 * i + 1], g[4 * i + 2], g[4 * i + 3]));
                            __stcg(at + tokens4 * 128, make_float4(u[4 * i], u[4 * i + 1], u[4 * i + 2], u[4 * i + 3]));
                        }
                }
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0)
                mbar_arrive(acce(n & 1));
            if (whole)
                continue;
            const int64_t at = static_cast<int64_t>(tile) * num_kt;
            const int c0 = ranges.cta_of(at), c1 = ranges.cta_of(at + num_kt - 1);
            __threadfence();
            named_barrier_sync(1, 256);
            if (threadIdx.x == 256 && !*abort_flag)  // a piece that some warp did not write is not counted
                *arrived = atomicAdd(p.counters + tile, 1u);
            named_barrier_sync(1, 256);
            const bool join = __all_sync(0xffffffffu, !*abort_flag && *arrived == static_cast<uint32_t>(c1 - c0));
            named_barrier_sync(1, 256);  // the word is read before the next piece's arrival
            if (!join)
                continue;
            __threadfence();
#pragma unroll 1
            for (int t4 = half * kJoin; t4 < tokens4; t4 += 2 * kJoin) {
                float g[4 * kJoin] = {}, u[4 * kJoin] = {};
#pragma unroll 4
                for (int c = c0; c <= c1; ++c) {
                    const bool second = c == c0 && ranges.first_step(c) < at;  // the tile is not its range's first
                    const float4* from = p.parts + (2 * c + (second ? 1 : 0)) * slot_size + q * 32 + lane;
#pragma unroll
                    for (int i = 0; i < kJoin; ++i) {
                        const int at4 = min(t4 + i, tokens4 - 1) * 128;
                        const float4 a = __ldcg(from + at4), b = __ldcg(from + tokens4 * 128 + at4);
                        g[4 * i] += a.x, g[4 * i + 1] += a.y, g[4 * i + 2] += a.z, g[4 * i + 3] += a.w;
                        u[4 * i] += b.x, u[4 * i + 1] += b.y, u[4 * i + 2] += b.z, u[4 * i + 3] += b.w;
                    }
                }
                write_h(p.act, g, u, ag, au, live - 4 * t4, p.h + static_cast<int64_t>(4 * t4) * p.ldh + f, p.ldh, top);
            }
        }
        __syncwarp();
        if (p.amax_out)
            flush_top(p.amax_out, top);
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 1) {
        if (*abort_flag && lane == 0) {  // no MMA may still write TMEM
            (void)mbar_wait_bounded(accf(0), 0, kWaitLimitNs);
            (void)mbar_wait_bounded(accf(1), 0, kWaitLimitNs);
        }
        __syncwarp();
        tc_fence_after();
        tmem_dealloc(tmem, G::TM_ALLOC);
    }
}

template <int KIND>
int launch_few(const GatedArgs& a, bool early, const Device& d, cudaStream_t s)
{
    using G = CfgFew<KIND>;
    static int configured_device = -1;
    if (configured_device != d.id) {
        if (cudaFuncSetAttribute(gated_few_kernel<KIND>, cudaFuncAttributeMaxDynamicSharedMemorySize, G::SMEM_ALLOC) !=
            cudaSuccess)
            return MX_ERR_CUDA;
        configured_device = d.id;
    }
    const int64_t M = a.x->rows, N = a.gate->rows, K = a.x->k, kbytes = K / G::EPB;
    FewParams p;
    p.n_pad = static_cast<int>((M + 15) / 16 * 16);
    CUtensorMap mx, mg, mu;
    if (!make_code_map(&mx, a.x->codes, M, kbytes, p.n_pad) || !make_code_map(&mg, a.gate->codes, N, kbytes, 128) ||
        !make_code_map(&mu, a.up->codes, N, kbytes, 128))
        return MX_ERR_CUDA;
    const bool ts = fmt_has_tensor_scale(a.x->fmt);
    p.sfx = a.x->sf;
    p.sfg = a.gate->sf;
    p.sfu = a.up->sf;
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
    p.early = early ? 1 : 0;
    p.kgroups = sf_kgroups(K / G::BLOCK);
    p.amax_out = a.amax;
    p.status = d.status;
    p.wait_ns = kWaitLimitNs;
    const int64_t tiles = (N + 127) / 128;
    const int64_t ctas = a.parts ? gated_few_cut(N, K, a.x->fmt).ranges : tiles;
    p.parts = static_cast<float4*>(a.parts);
    p.counters = a.counters;
    return launch_kernel(gated_few_kernel<KIND>, static_cast<unsigned>(ctas), 1, 512, G::SMEM_ALLOC, early, s, mx, mg, mu, p);
}

}  // namespace

// Cut where that takes less time: a tile a CTA, in as many waves as it takes, against equal
// ranges of at least four steps and the join of the tiles that lie in several.  Times by
// rates that 456 pairs of measurements gave (MXFP8 and NVFP4, K 1024 to 8192, 8 to 320
// tiles, 1 to 64 tokens, weights not in L2): the memory 7500 bytes a ns, an SM 80, a wave
// after the first 5 us, a join 2 us, 0.05 a token, and 0.2 and 0.015 a token for each of a
// tile's pieces.  What is chosen is 0.2 % slower than the better of the two on average, 6 %
// at most; on 900 other pairs (all kinds of format, K 768 to 5120, 4 to 460 tiles) 0.5 and
// 13 %.  K = 4096, whole / cut in us: 32 tiles MXFP8 1 token 18.9 / 14.2, 64 tokens 19.9 /
// 26.3; 80 tiles NVFP4 48 tokens 15.8 / 19.7; 112 tiles MXFP8 1 token 23.6 / 26.5; 160
// tiles, of which 8 would be a wave of their own, 43.3 / 33.4; 304 tiles, as ranges of two
// whole ones, 54.5 / 51.5.
FewCut gated_few_cut(int64_t features, int64_t k, int fmt)
{
    const int64_t num_kt = k / gemm_k_multiple(fmt), tiles = (features + 127) / 128, steps = tiles * num_kt;
    if (steps == 0)
        return {0, 0};
    const int64_t ranges = std::max<int64_t>(1, std::min<int64_t>(kGatedFewCtas, steps / 4));
    const double step_us = 256.0 * static_cast<double>(codes_row_bytes(fmt, k) + k / fmt_block(fmt)) / static_cast<double>(num_kt) / 80e3;
    const double memory_us = static_cast<double>(steps) * step_us * (80.0 / 7500.0);
    const int64_t waves = (tiles + kGatedFewCtas - 1) / kGatedFewCtas;
    const double whole_us = std::max(memory_us, static_cast<double>(waves * num_kt) * step_us) + 5.0 * static_cast<double>(waves - 1);
    const double spare_us = whole_us - std::max(memory_us, static_cast<double>((steps + ranges - 1) / ranges) * step_us);
    if (steps % ranges == 0 && steps / ranges % num_kt == 0)  // ranges of whole tiles: nothing to join
        return {ranges, spare_us > 0.0 ? kGatedFewTokens : 0};
    const double pieces = static_cast<double>((num_kt * ranges + steps - 1) / steps);
    const double most = (spare_us - 2.0 - 0.2 * pieces) / (0.05 + 0.015 * pieces);
    return {ranges, std::max<int64_t>(0, static_cast<int64_t>(std::min<double>(most, kGatedFewTokens)))};
}

int launch_gated_few(const GatedArgs& a, bool early, const Device& d, cudaStream_t s)
{
    switch (a.x->fmt) {
    case MX_FMT_MXFP8_E4M3:
    case MX_FMT_MOSS_FP8: return launch_few<0>(a, early, d, s);
    case MX_FMT_MXFP4_E2M1: return launch_few<1>(a, early, d, s);
    default: return launch_few<2>(a, early, d, s);
    }
}

}  // namespace mx
