// gated_few.cu -- the gated feed-forward block's first half for few tokens: the
// weights' bytes are all that counts, so the weights are the M side of the tensor
// core's tile and the tokens, padded to a multiple of 16, its N side.
//
// One CTA computes 128 features: two accumulators of 128 x N in TMEM, gate and up,
// from the same token tile.  Warp 0 (one thread) streams both weight tiles, the token
// tile and their scales through a ring of stages; warp 1 (one thread) copies the
// stage's scales into TMEM and issues the MMAs; warps 2-5 hold one feature a lane and
// write h.  Launched with programmatic dependent launch behind the tokens'
// quantization, it fills its ring with weights before that has finished.
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
    static constexpr int SMEM_BYTES = OFF_BAR + (2 * STAGES + 1) * 8 + 16;
    static constexpr int SMEM_ALLOC = SMEM_BYTES + 1024;
    // TMEM: two accumulators, then three scale regions a stage
    static constexpr int SF_COLS = 4 * NCHUNK;
    static constexpr int TM_SF = 2 * BN;
    static constexpr int TM_USED = TM_SF + STAGES * 3 * SF_COLS;
    static constexpr int TM_ALLOC = TM_USED <= 256 ? 256 : 512;
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
    int* status;
    uint64_t wait_ns;
};

template <int ACT>
__device__ __forceinline__ float gate_value(float z)
{
    return activate<ACT, true>(make_float2(z, 0.0f)).value.x;
}

template <int KIND>
__global__ void __launch_bounds__(192, 1)
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
    const uint32_t accf = bar0 + 8u * (2 * STAGES);
    volatile uint32_t* tmem_slot = reinterpret_cast<volatile uint32_t*>(smem + G::OFF_BAR + 8 * (2 * STAGES + 1));
    volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int tile = blockIdx.x;
    const int num_kt = p.K / G::BK;

    if (threadIdx.x == 0) {
        for (int s = 0; s < STAGES; ++s) {
            mbar_init(full(s), 1);
            mbar_init(empty(s), 1);
        }
        mbar_init(accf, 1);
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

    if (warp == 0) {
        if (lane == 0) {
            const uint32_t tx = 2 * G::W_BYTES + p.n_pad * G::BKB + 3 * G::SF_BYTES;
            auto load_weights = [&](int kt) {
                const int s = kt % STAGES;
                const int64_t chunk = static_cast<int64_t>(tile) * p.kgroups + static_cast<int64_t>(kt) * G::NCHUNK;
                mbar_arrive_expect_tx(full(s), tx);
                tma_load_2d(s0 + G::OFF_W + (2 * s) * G::W_BYTES, &tmG, full(s), kt * G::BKB, tile * 128);
                tma_load_2d(s0 + G::OFF_W + (2 * s + 1) * G::W_BYTES, &tmU, full(s), kt * G::BKB, tile * 128);
                bulk_load(s0 + G::OFF_SF + (3 * s) * G::SF_BYTES, p.sfg + chunk * 512, G::SF_BYTES, full(s));
                bulk_load(s0 + G::OFF_SF + (3 * s + 1) * G::SF_BYTES, p.sfu + chunk * 512, G::SF_BYTES, full(s));
            };
            auto load_tokens = [&](int kt) {
                const int s = kt % STAGES;
                tma_load_2d(s0 + G::OFF_X + s * G::X_BYTES, &tmX, full(s), kt * G::BKB, 0);
                bulk_load(s0 + G::OFF_SF + (3 * s + 2) * G::SF_BYTES, p.sfx + static_cast<int64_t>(kt) * G::NCHUNK * 512,
                          G::SF_BYTES, full(s));
            };
            const int ahead = min(STAGES, num_kt);
            if (!p.early)
                wait_for_launch_before();
            for (int kt = 0; kt < ahead; ++kt)
                load_weights(kt);
            if (p.early)
                wait_for_launch_before();
            for (int kt = 0; kt < ahead; ++kt)
                load_tokens(kt);
            int kt = ahead;
            for (; kt < num_kt; ++kt) {
                if (!mbar_wait_bounded(empty(kt % STAGES), static_cast<uint32_t>(kt / STAGES - 1) & 1u, p.wait_ns))
                    fail();
                if (*abort_flag)
                    break;
                load_weights(kt);
                load_tokens(kt);
            }
            if (*abort_flag)  // let the copies already issued land before the CTA can exit
                for (int k = max(0, kt - STAGES); k < kt; ++k)
                    (void)mbar_wait_bounded(full(k % STAGES), static_cast<uint32_t>(k / STAGES) & 1u, kWaitLimitNs);
        }
        __syncwarp();
    } else if (warp == 1) {
        if (lane == 0) {
            for (int kt = 0; kt < num_kt; ++kt) {
                const int s = kt % STAGES;
                if (!mbar_wait_bounded(full(s), static_cast<uint32_t>(kt / STAGES) & 1u, p.wait_ns)) {
                    fail();
                    break;
                }
                tc_fence_after();
                const uint32_t sf_t = tmem + G::TM_SF + s * 3 * G::SF_COLS;
#pragma unroll
                for (int o = 0; o < 3; ++o)
#pragma unroll
                    for (int c = 0; c < G::NCHUNK; ++c)
                        tc_cp_sf(sf_t + o * G::SF_COLS + 4 * c, sdesc_sf(s0 + G::OFF_SF + (3 * s + o) * G::SF_BYTES + c * 512));
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
                        mma_bs<KIND>(tmem + o * G::BN, wdesc + koff, xdesc + koff, idesc, sf_t + o * G::SF_COLS + 4 * chunk,
                                     sf_t + 2 * G::SF_COLS + 4 * chunk, (kt > 0 || i > 0) ? 1u : 0u);
                    }
                }
                tc_commit(empty(s));
            }
            tc_commit(accf);
        }
        __syncwarp();
    } else {
        const int q = warp & 3;  // TMEM lane quarter
        const int f = tile * 128 + q * 32 + lane;
        Top<float> top;
        wait_for_launch_before();  // the tensor scale of the tokens
        const float ta = p.tsa ? *p.tsa : 1.0f;
        const int region = p.ts_region ? tile : 0;  // of 128 weight rows
        const float ag = __fmul_rn(ta, p.tsg ? p.tsg[region] : 1.0f), au = __fmul_rn(ta, p.tsu ? p.tsu[region] : 1.0f);
        const bool ok = __all_sync(0xffffffffu, mbar_wait_bounded(accf, 0, p.wait_ns));
        if (!ok) {
            if (lane == 0)
                fail();
        } else {
            tc_fence_after();
#pragma unroll 1
            for (int t0 = 0; t0 < p.M; t0 += 32) {
                uint32_t g[32], u[32];
                tmem_ld32(tmem + (static_cast<uint32_t>(q * 32) << 16) + t0, g);
                tmem_ld32(tmem + (static_cast<uint32_t>(q * 32) << 16) + G::BN + t0, u);
                tmem_ld_wait();
                __nv_bfloat16* dst = p.h + static_cast<int64_t>(t0) * p.ldh + f;
#pragma unroll
                for (int i = 0; i < 32; ++i) {
                    if (t0 + i >= p.M)
                        break;
                    const float z = __fmul_rn(__uint_as_float(g[i]), ag);
                    const float a = p.act == MX_ACT_SILU   ? gate_value<MX_ACT_SILU>(z)
                                    : p.act == MX_ACT_GELU ? gate_value<MX_ACT_GELU>(z)
                                                           : gate_value<MX_ACT_GELU_TANH>(z);
                    const __nv_bfloat16 v = __float2bfloat16_rn(a * __fmul_rn(__uint_as_float(u[i]), au));
                    if (f < p.N) {
                        dst[i * p.ldh] = v;
                        top.value(__bfloat162float(v));
                    }
                }
            }
        }
        __syncwarp();
        if (p.amax_out)
            flush_top(p.amax_out, top);
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 1) {
        if (*abort_flag && lane == 0)
            (void)mbar_wait_bounded(accf, 0, kWaitLimitNs);  // no MMA may still write TMEM
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
    return launch_kernel(gated_few_kernel<KIND>, static_cast<unsigned>((N + 127) / 128), 1, 192, G::SMEM_ALLOC, early, s, mx,
                         mg, mu, p);
}

}  // namespace

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
