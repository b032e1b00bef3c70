// optim.cu -- the optimizer's step and the gradients' norm over many tensors in
// one launch each.
#include <algorithm>
#include <cmath>
#include <type_traits>

#include "mx_act8.cuh"
#include "mx_internal.cuh"
#include "mx_units.cuh"

namespace mx {
namespace {

constexpr int kThreads = 256;
// Octs (eight consecutive values) that a thread takes of a tile.  8-bit moments: four, 32
// apart, so that a warp has 32 whole groups and reads and writes their exponent bytes as
// one sector each (a quarter of a sector at a time cost a layer 57 us more in an earlier form).
__host__ __device__ constexpr int octs_of(int bits) { return bits == 8 ? 4 : 1; }

// Eight fp32 values at a multiple of 32 bytes in one access.  (In two of 16 bytes each, a
// warp's access touches every sector of its kilobyte twice.)
__device__ __forceinline__ void load_sector(const float* p, RawOct<float>& w)
{
    asm volatile("ld.global.L1::no_allocate.v8.f32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                 : "=f"(w.a.x), "=f"(w.a.y), "=f"(w.a.z), "=f"(w.a.w), "=f"(w.b.x), "=f"(w.b.y), "=f"(w.b.z), "=f"(w.b.w)
                 : "l"(p)
                 : "memory");
}
__device__ __forceinline__ void store_sector(float* p, const Oct& o)
{
    asm volatile("st.global.v8.f32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "f"(o.p[0].x), "f"(o.p[0].y), "f"(o.p[1].x),
                 "f"(o.p[1].y), "f"(o.p[2].x), "f"(o.p[2].y), "f"(o.p[3].x), "f"(o.p[3].y)
                 : "memory");
}

// Eight values of a flat tensor.  Not ANY: the tensor starts on a boundary of eight values
// and holds a multiple of eight.  ANY: it need not; which of its arrays do is looked at
// for each, since most start where an allocation does and only their sizes are odd.
template <typename T, bool ANY>
struct Values {
    Unit<T, true> u;

    static __device__ __forceinline__ bool on_boundary(const void* base)
    {
        return (reinterpret_cast<uintptr_t>(base) & (8 * sizeof(T) - 1)) == 0;
    }
    __device__ __forceinline__ void load(const void* base, const Place& at, int64_t n)
    {
        const T* src = static_cast<const T*>(base) + static_cast<int64_t>(at.unit) * 8;
        if (ANY && !on_boundary(base)) {
            u.load(base, 0, at, 1, n);
            return;
        }
        u.s = 0;
        u.w.clear();
        if (at.cols == 8) {
            if constexpr (sizeof(T) == 4)
                load_sector(src, u.w);
            else
                u.w.load(src);
        } else if (ANY && at.cols > 0) {
            T v[8];
#pragma unroll
            for (int c = 0; c < 8; ++c)
                v[c] = c < at.cols ? src[c] : T(0.0f);
            memcpy(&u.w, v, sizeof v);
        }
    }
    __device__ __forceinline__ void get(Oct& o, int n) const
    {
        if (ANY && u.s != 0)
            u.get(o, n);
        else
            u.w.get(o);
    }
    // Executed by whole warps.
    static __device__ __forceinline__ void store(void* base, const Place& at, const Oct& o, int64_t n)
    {
        if (ANY && !on_boundary(base)) {
            Top<T> unused;
            store_unit<T, true>(base, 0, at, o, n, unused);
            return;
        }
        T* dst = static_cast<T*>(base) + static_cast<int64_t>(at.unit) * 8;
        if (at.cols == 8) {
            if constexpr (sizeof(T) == 4)
                store_sector(dst, o);
            else
                *reinterpret_cast<uint4*>(dst) = pack_oct(o);
        } else if (ANY) {
#pragma unroll
            for (int c = 0; c < 8; ++c)
                if (c < at.cols)
                    store_f(dst + c, o[c]);
        }
    }
};
__device__ __forceinline__ void fold(Top<float>& top, const Oct& o)
{
    top.pair(o.p[0]), top.pair(o.p[1]), top.pair(o.p[2]), top.pair(o.p[3]);
}
__device__ __forceinline__ void fold(Top<__nv_bfloat16>& top, const Oct& o)
{
    const uint4 w = pack_oct(o);
    top.word(w.x), top.word(w.y), top.word(w.z), top.word(w.w);
}
bool whole(const void* p, int64_t n, unsigned bytes)  // bytes of a value: 2 or 4
{
    return ((n & 7) | static_cast<int64_t>(reinterpret_cast<uintptr_t>(p) & (8 * bytes - 1))) == 0;
}

// ---------------------------------------------------------------- AdamW
// The tensors of one launch, in its parameters: no table to copy to the device
// before it and nothing that a captured graph would have to keep alive.
constexpr int kAdamwEntries = 128;
struct AdamwEntry {
    void* p;
    const void* g;  // null: the tensor has no gradient and stays as it is
    void* m;
    void* v;
    uint8_t* m_sf;
    uint8_t* v_sf;
    __nv_bfloat16* copy;
    int64_t n;
    uint32_t first;  // the launch's tile at which the tensor starts
    uint32_t index;  // in the call
    float wd, decay;
};
struct AdamwTable {
    AdamwEntry e[kAdamwEntries];
    int count;
    uint32_t tiles;
    float b1, c1, b2, c2;    // beta, 1 - beta
    float eps, lr;
    float step, root;        // lr / (1 - beta1^t), 1 / sqrt(1 - beta2^t)
    float log_b1, log_b2;
    const float* lr_at;      // these two replace lr, t and what follows from them
    const int64_t* t_at;
    const float* scale;
    unsigned* amax;
    uint32_t t;
    uint32_t keys[20];  // Philox's two, round by round: operands from the constant bank
};

// The entry that holds tile i.
__device__ __forceinline__ int entry_of(const AdamwTable& t, uint32_t i)
{
    int lo = 0, hi = t.count;
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (t.e[mid].first <= i)
            lo = mid;
        else
            hi = mid;
    }
    return lo;
}

// 1 / x for x >= 0; below 2^-126 that number's.
__device__ __forceinline__ float rcp_approx(float x)
{
    float r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(max_nan(x, 1.17549435e-38f)));
    return r;
}
__device__ __forceinline__ float sqrt_approx(float x)
{
    float r;
    asm("sqrt.approx.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}

// Philox4x32-10 (Salmon et al., SC'11) for values 8 unit .. 8 unit + 7: u[k] holds
// the number of value 2 k in its low half and that of value 2 k + 1 in its high one.
__device__ __forceinline__ void random8(const AdamwTable& a, uint32_t t, uint32_t unit, uint32_t word, uint32_t (&u)[4])
{
    uint32_t c0 = unit, c1 = 0, c2 = t, c3 = word;
#pragma unroll
    for (int round = 0; round < 10; ++round) {
        const uint64_t x = uint64_t{0xD2511F53u} * c0, y = uint64_t{0xCD9E8D57u} * c2;
        c0 = static_cast<uint32_t>(y >> 32) ^ c1 ^ a.keys[2 * round];
        c2 = static_cast<uint32_t>(x >> 32) ^ c3 ^ a.keys[2 * round + 1];
        c1 = static_cast<uint32_t>(y);
        c3 = static_cast<uint32_t>(x);
    }
    u[0] = c0, u[1] = c1, u[2] = c2, u[3] = c3;
}

// The E4M3 codes of four values |y| <= 448, each up iff u16 < p 2^16; u as random8 gives
// it.  From 2^-6 on a float's upper bits are the code (less 960), and the 20 that go are
// p 2^20: adding 2^20 - 1 - 16 u16 carries into the code where they are above 16 u16.
// Below 2^-6, adding 2^-6 brings the value to the same spacing of 2^-9, eight codes up;
// rounding that sum up keeps the comparison, whose other side is whole, what it is on the
// exact p.
template <bool SIGNED>
__device__ __forceinline__ uint32_t e4m3_sr4(const float (&y)[4], uint32_t u01, uint32_t u23)
{
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float a = SIGNED ? fabsf(y[i]) : y[i];
        const uint32_t u = i < 2 ? u01 : u23;
        const uint32_t r = ((i & 1 ? u >> 12 : u << 4) & 0xFFFF0u) ^ 0xFFFFFu;
        const uint32_t b = a < 0.015625f ? __float_as_uint(__fadd_ru(a, 0.015625f)) - (8u << 20) : __float_as_uint(a);
        w[i] = (b + r) << 4;  // the code + 0xC0 in the top byte
    }
    const uint32_t four = __byte_perm(__byte_perm(w[0], w[1], 0x0073), __byte_perm(w[2], w[3], 0x0073), 0x5410);
    // less 0xC0 again: a byte's upper bits are 11 for codes below 0x40 and 00 (carried) above
    uint32_t codes = (four & 0x3F3F3F3Fu) | (~four & 0x40404040u);
    if constexpr (SIGNED) {
        const uint32_t s = __byte_perm(__byte_perm(__float_as_uint(y[0]), __float_as_uint(y[1]), 0x0073),
                                       __byte_perm(__float_as_uint(y[2]), __float_as_uint(y[3]), 0x0073), 0x5410);
        codes |= s & 0x80808080u;
    }
    return codes;
}

// A moment in the 8-bit checkpoint's format: like encode_oct, but rounded
// stochastically where SR, and with ROOT a value that is not zero keeps at least
// the smallest code: a root that vanished would divide its first moment by eps.
template <bool ROOT, bool SR>
__device__ __forceinline__ uint2 encode_moment(Oct z, uint8_t& byte, const uint32_t (&u)[4])
{
    if constexpr (!ROOT && !SR)
        return encode_oct(z, byte);
    float m = max_abs(max_abs(max_abs(max_abs(0.0f, z.p[0]), z.p[1]), z.p[2]), z.p[3]);
    m = max_nan(m, __shfl_xor_sync(0xFFFFFFFFu, m, 1));
    m = max_nan(m, __shfl_xor_sync(0xFFFFFFFFu, m, 2));
    const bool odd = __any_sync(0xFFFFFFFFu, non_finite(m));
    if (odd) {
        m = 0.0f;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            z[i] = finite_or_nan(z[i]);
            m = fmaxf(m, fabsf(z[i]));
        }
        m = fmaxf(m, __shfl_xor_sync(0xFFFFFFFFu, m, 1));
        m = fmaxf(m, __shfl_xor_sync(0xFFFFFFFFu, m, 2));
    }
    const uint32_t e = act8_byte(m);
    byte = static_cast<uint8_t>(e);
    const float s = act8_inverse(e);
    float y[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        y[i] = __fmul_rn(z[i], s);
        if constexpr (ROOT)
            y[i] = z[i] == 0.0f ? 0.0f : max_nan(y[i], 0.001953125f);
    }
    uint32_t w[2];
    if constexpr (SR) {
        w[0] = e4m3_sr4<!ROOT>({y[0], y[1], y[2], y[3]}, u[0], u[1]);
        w[1] = e4m3_sr4<!ROOT>({y[4], y[5], y[6], y[7]}, u[2], u[3]);
        if (odd)
#pragma unroll
            for (int i = 0; i < 8; ++i)
                if (y[i] != y[i])
                    w[i >> 2] |= 0x7Fu << (8 * (i & 3));
    } else {
        w[0] = cvt_e4m3x2(y[0], y[1]) | cvt_e4m3x2(y[2], y[3]) << 16;
        w[1] = cvt_e4m3x2(y[4], y[5]) | cvt_e4m3x2(y[6], y[7]) << 16;
    }
    return make_uint2(w[0], w[1]);
}

// bf16 values by 16-bit numbers: up where the number is below the 16 bits that go, which is
// where these and 2^16 - 1 - u16 carry.  A NaN becomes the one whose bits that go are 0.
__device__ __forceinline__ void round_bf16_sr(Oct& p, const uint32_t (&u)[4])
{
    float m = max_abs(max_abs(max_abs(max_abs(0.0f, p.p[0]), p.p[1]), p.p[2]), p.p[3]);
    if (m != m)
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (p[i] != p[i])
                p[i] = __uint_as_float(0x7FC00000u);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const uint32_t r = i & 1 ? ~u[i >> 1] >> 16 : ~u[i >> 1] & 0xFFFFu;
        p[i] = __uint_as_float((__float_as_uint(p[i]) + r) & 0xFFFF0000u);
    }
}

// Each operation of the moments is rounded on its own, so that the codes of 8-bit ones
// are a function of the formula alone.  The scalar intrinsics: the compiler fuses the
// two-wide product and sum.
__device__ __forceinline__ float first_moment(const AdamwTable& a, float m, float g)
{
    return __fadd_rn(__fmul_rn(m, a.b1), __fmul_rn(g, a.c1));
}
__device__ __forceinline__ float second_moment(const AdamwTable& a, float v, float g)
{
    return __fadd_rn(__fmul_rn(v, a.b2), __fmul_rn(__fmul_rn(g, g), a.c2));
}

// Eight codes of an 8-bit moment.
struct Codes {
    uint2 w;
    __device__ __forceinline__ void load(const void* codes, const Place& at)
    {
        w = make_uint2(0u, 0u);
        if (at.cols > 0)
            asm volatile("ld.global.L1::no_allocate.v2.u32 {%0, %1}, [%2];"
                         : "=r"(w.x), "=r"(w.y)
                         : "l"(static_cast<const uint8_t*>(codes) + static_cast<int64_t>(at.unit) * 8)
                         : "memory");
    }
    __device__ __forceinline__ void get(Oct& o, uint32_t byte) const
    {
        decode_oct(w, o);
        const float2 s = both(act8_scale(byte));
#pragma unroll
        for (int k = 0; k < 4; ++k)
            o.p[k] = __fmul2_rn(o.p[k], s);
    }
};
// A tensor's values as one thread takes them from memory.
template <typename P, typename G, int BITS, bool ANY>
struct Loaded {
    Place at;
    Values<P, ANY> p;
    Values<G, ANY> g;
    std::conditional_t<BITS == 8, Codes, Values<float, ANY>> m, v;
};

// CTAs an SM that the registers are held to, 0: the compiler's choice.  Odd sizes, 100 tensors
// of 300001 values, choice / three / four: fp32 180 / 178 / 195 us, bf16 stochastic 140 / 125 /
// 133, 8-bit moments 121 / 120 / 129, stochastic 158 / 149 / 139.
constexpr int least_ctas(int bits, bool sr, bool any) { return !any ? 0 : bits == 8 && sr ? 4 : 3; }

// m' = b1 m + (1 - b1) g, v' = b2 v + (1 - b2) g^2, and the weight's step, which divides
// by approximation (2^-21 of the step; a divisor below 2^-126 counts as that).
// Of 8-bit moments the second one's root is kept: it spans half the octaves, and
// E4M3's 18 then hold 36 of the moment's.
//
// Bound by DRAM: a layer of 218e6 values, fp32 with bf16 copies and maxima, 990 us (6.54
// GB, 6.6 TB/s; 1408 with fp32 accesses of 16 bytes), 8-bit moments and bf16 gradients
// 564 us (3.52 GB, 6.2 TB/s).  Stochastic rounding of 8-bit moments is bound by
// instructions, 125 a value at odd addresses against 60 to nearest: about 19 are the random
// numbers (three sets for eight values), the others the two roundings to E4M3, bf16's and the
// shifts.  7.7e6 bf16 values at odd addresses 37 us; 218e6 aligned ones with bf16 gradients and
// no copies, stochastic / to nearest: fp32 813 / 516 us, bf16 833 / 470.
template <typename P, typename G, int BITS, bool SR, bool ANY>
__global__ void __launch_bounds__(kThreads, least_ctas(BITS, SR, ANY)) adamw_kernel(const __grid_constant__ AdamwTable a)
{
    constexpr int kOcts = octs_of(BITS);
    // octs whose loads are in flight together (a layer with 8-bit moments: one 573 us, two
    // 562, four 589), and how often the loop over them is unrolled: at any address its body
    // is long, and unrolled it takes the registers of a CTA an SM
    constexpr int kBatch = ANY || kOcts == 1 ? 1 : 2;
    constexpr int kUnroll = ANY ? 1 : kOcts / kBatch;
    const int lane = threadIdx.x & 31;
    const float scale = a.scale ? *a.scale : 1.0f;
    float step = a.step, root = a.root, lr = a.lr;
    uint32_t t = a.t;
    if (a.lr_at || a.t_at) {
        if (a.lr_at)
            lr = *a.lr_at;
        float n = static_cast<float>(a.t);
        if (a.t_at) {
            t = static_cast<uint32_t>(*a.t_at);
            n = static_cast<float>(*a.t_at);
        }
        step = lr / -expm1f(n * a.log_b1);
        root = 1.0f / sqrtf(-expm1f(n * a.log_b2));
    }
    const bool skip = scale != scale;
    Top<P> top;
    Top<__nv_bfloat16> top16;
    int cur = -1;
    auto flush = [&](int i) {
        if (!a.amax)
            return;
        if (sizeof(P) == 4 && a.e[i].copy)
            flush_top(a.amax + a.e[i].index, top16);
        else
            flush_top(a.amax + a.e[i].index, top);
        top = Top<P>();
        top16 = Top<__nv_bfloat16>();
    };
    for (uint32_t tile = blockIdx.x; tile < a.tiles; tile += gridDim.x) {
        const int i = entry_of(a, tile);
        const AdamwEntry& e = a.e[i];
        if (cur >= 0 && i != cur)
            flush(cur);
        cur = i;
        const bool still = skip || !e.g;
        const float decay = a.lr_at ? 1.0f - lr * e.wd : e.decay;
        // this lane's first oct of the warp's 32 kOcts
        const uint32_t first = (tile - e.first) * (kThreads * kOcts) + (threadIdx.x - lane) * kOcts + lane;
        uint32_t bytes_m = 127, bytes_v = 127;  // 8-bit moments: of the warp's group `lane`
        uint8_t new_m = 0, new_v = 0;
        const int64_t group = static_cast<int64_t>(first - lane) / 4 + lane;
        const bool has_group = BITS == 8 && group * kAct8Group < e.n;
        if (has_group && !still) {
            bytes_m = e.m_sf[group];
            bytes_v = e.v_sf[group];
        }
#pragma unroll kUnroll
        for (int batch = 0; batch < kOcts; batch += kBatch) {
            Loaded<P, G, BITS, ANY> w[kBatch];
#pragma unroll
            for (int o = 0; o < kBatch; ++o) {
                const uint32_t unit = first + (batch + o) * 32;
                w[o].at = {0, unit, static_cast<int32_t>(max(min(e.n - static_cast<int64_t>(unit) * 8, int64_t{8}), int64_t{0}))};
                w[o].p.load(e.p, w[o].at, e.n);
                if (still)
                    continue;
                w[o].g.load(e.g, w[o].at, e.n);
                if constexpr (BITS == 8) {
                    w[o].m.load(e.m, w[o].at);
                    w[o].v.load(e.v, w[o].at);
                } else {
                    w[o].m.load(e.m, w[o].at, e.n);
                    w[o].v.load(e.v, w[o].at, e.n);
                }
            }
#pragma unroll
            for (int o = 0; o < kBatch; ++o) {
                const Place at = w[o].at;
                const uint32_t unit = at.unit;
                Oct p;
                w[o].p.get(p, at.cols);
                if (!still) {
                    Oct g, m, v, r;
                    w[o].g.get(g, at.cols);
                    if constexpr (BITS == 8) {
                        const int from = (batch + o) * 8 + (lane >> 2);
                        w[o].m.get(m, __shfl_sync(0xFFFFFFFFu, bytes_m, from));
                        w[o].v.get(v, __shfl_sync(0xFFFFFFFFu, bytes_v, from));
#pragma unroll
                        for (int k = 0; k < 4; ++k)
                            v.p[k] = __fmul2_rn(v.p[k], v.p[k]);
                    } else {
                        w[o].m.get(m, at.cols);
                        w[o].v.get(v, at.cols);
                    }
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        const float x = __fmul_rn(g.p[k].x, scale), y = __fmul_rn(g.p[k].y, scale);
                        m.p[k] = make_float2(first_moment(a, m.p[k].x, x), first_moment(a, m.p[k].y, y));
                        v.p[k] = make_float2(second_moment(a, v.p[k].x, x), second_moment(a, v.p[k].y, y));
                        if constexpr (BITS == 8)
                            r.p[k] = make_float2(__fsqrt_rn(v.p[k].x), __fsqrt_rn(v.p[k].y));
                        else
                            r.p[k] = make_float2(sqrt_approx(v.p[k].x), sqrt_approx(v.p[k].y));
                        const float2 d = __ffma2_rn(r.p[k], both(root), both(a.eps));
                        const float2 q = __fmul2_rn(m.p[k], make_float2(rcp_approx(d.x), rcp_approx(d.y)));
                        p.p[k] = __ffma2_rn(q, both(-step), __fmul2_rn(p.p[k], both(decay)));
                    }
                    uint32_t u[4] = {};
                    if constexpr (BITS == 8) {
                        if (at.cols < 8) {
                            keep_first(m, at.cols);
                            keep_first(r, at.cols);
                        }
                        uint8_t bm, bv;
                        if constexpr (SR)
                            random8(a, t, unit, 4 * e.index, u);
                        const uint2 cm = encode_moment<false, SR>(m, bm, u);
                        if constexpr (SR)
                            random8(a, t, unit, 4 * e.index + 1, u);
                        const uint2 cv = encode_moment<true, SR>(r, bv, u);
                        const uint32_t from = (lane & 7) * 4;
                        const uint32_t both_bytes = __shfl_sync(0xFFFFFFFFu, uint32_t{bm} | uint32_t{bv} << 8, from);
                        if ((lane >> 3) == batch + o) {
                            new_m = static_cast<uint8_t>(both_bytes);
                            new_v = static_cast<uint8_t>(both_bytes >> 8);
                        }
                        // whole groups: a tensor's last one is padded with zeros
                        if (static_cast<int64_t>(unit) * 8 < (e.n + 31) / 32 * 32) {
                            *reinterpret_cast<uint2*>(static_cast<uint8_t*>(e.m) + static_cast<int64_t>(unit) * 8) = cm;
                            *reinterpret_cast<uint2*>(static_cast<uint8_t*>(e.v) + static_cast<int64_t>(unit) * 8) = cv;
                        }
                    } else {
                        Values<float, ANY>::store(e.m, at, m, e.n);
                        Values<float, ANY>::store(e.v, at, v, e.n);
                    }
                    if constexpr (SR && sizeof(P) == 2) {
                        random8(a, t, unit, 4 * e.index + 2, u);
                        round_bf16_sr(p, u);
                    }
                    Values<P, ANY>::store(e.p, at, p, e.n);
                }
                if (at.cols < 8)
                    keep_first(p, at.cols);
                if (sizeof(P) == 4 && e.copy) {
                    Values<__nv_bfloat16, ANY>::store(e.copy, at, p, e.n);
                    if (a.amax)
                        fold(top16, p);
                } else if (a.amax) {
                    fold(top, p);
                }
            }
        }
        if (has_group && !still) {
            e.m_sf[group] = new_m;
            e.v_sf[group] = new_v;
        }
    }
    if (cur >= 0)
        flush(cur);
}

template <typename P, typename G, int BITS, bool SR, bool ANY>
int launch_adamw(const AdamwTable& t, const Device& d, cudaStream_t s)
{
    constexpr auto kernel = adamw_kernel<P, G, BITS, SR, ANY>;
    const unsigned most = static_cast<unsigned>(d.sms * resident_ctas<kernel>(kThreads));
    return launch_kernel(kernel, std::min(t.tiles, most), 1, kThreads, 0, false, s, t);
}
template <typename P, typename G, int BITS, bool SR>
int launch_adamw(const AdamwTable& t, bool any, const Device& d, cudaStream_t s)
{
    return any ? launch_adamw<P, G, BITS, SR, true>(t, d, s) : launch_adamw<P, G, BITS, SR, false>(t, d, s);
}
template <typename P, typename G>
int launch_adamw(const AdamwTable& t, int bits, bool sr, bool any, const Device& d, cudaStream_t s)
{
    if (bits == 8)
        return sr ? launch_adamw<P, G, 8, true>(t, any, d, s) : launch_adamw<P, G, 8, false>(t, any, d, s);
    if constexpr (sizeof(P) == 2)
        if (sr)
            return launch_adamw<P, G, 32, true>(t, any, d, s);
    return launch_adamw<P, G, 32, false>(t, any, d, s);
}

uint32_t tiles_of(int64_t n, int bits)
{
    const int64_t tile = 8 * kThreads * octs_of(bits);
    return static_cast<uint32_t>((n + tile - 1) / tile);
}

}  // namespace

int launch_adamw(const mx_adamw_tensor* tensors, int64_t count, const mx_adamw_opts& o, const float* scale, float* amax,
                 const Device& d, cudaStream_t s)
{
    AdamwTable t;
    t.b1 = static_cast<float>(o.beta1);
    t.c1 = static_cast<float>(1.0 - o.beta1);
    t.b2 = static_cast<float>(o.beta2);
    t.c2 = static_cast<float>(1.0 - o.beta2);
    t.eps = static_cast<float>(o.eps);
    t.lr = static_cast<float>(o.lr);
    t.step = static_cast<float>(o.lr / -std::expm1(static_cast<double>(o.t) * std::log(o.beta1)));
    t.root = static_cast<float>(1.0 / std::sqrt(-std::expm1(static_cast<double>(o.t) * std::log(o.beta2))));
    t.log_b1 = static_cast<float>(std::log(o.beta1));
    t.log_b2 = static_cast<float>(std::log(o.beta2));
    t.lr_at = o.lr_at;
    t.t_at = o.t_at;
    t.scale = scale;
    t.amax = reinterpret_cast<unsigned*>(amax);
    t.t = static_cast<uint32_t>(o.t);
    for (uint32_t i = 0; i < 10; ++i) {
        t.keys[2 * i] = static_cast<uint32_t>(o.seed) + i * 0x9E3779B9u;
        t.keys[2 * i + 1] = static_cast<uint32_t>(o.seed >> 32) + i * 0xBB67AE85u;
    }
    // one launch for each kind of tensor (types, 8-bit moments, alignment) and 128 of them
    auto kind_of = [](const mx_adamw_tensor& x) {
        const bool p16 = x.p_dtype == MX_OUT_BF16, g16 = x.g_dtype == MX_OUT_BF16, eight = x.bits == 8;
        const bool wide = whole(x.param, x.n, p16 ? 2 : 4) && whole(x.grad, x.n, g16 ? 2 : 4) && whole(x.copy, x.n, 2) &&
                          (eight || (whole(x.m, x.n, 4) && whole(x.v, x.n, 4)));
        return (p16 ? 1 : 0) | (g16 ? 2 : 0) | (eight ? 4 : 0) | (wide ? 0 : 8);
    };
    unsigned kinds = 0;
    for (int64_t i = 0; i < count; ++i)
        if (tensors[i].n > 0)
            kinds |= 1u << kind_of(tensors[i]);
    for (int kind = 0; kind < 16; ++kind) {
        if (!(kinds >> kind & 1))
            continue;
        const bool p16 = kind & 1, g16 = kind & 2, any = kind & 8;
        const int bits = kind & 4 ? 8 : 32;
        const bool sr = o.rounding == MX_ROUND_SR;
        t.count = 0;
        t.tiles = 0;
        auto flush = [&]() -> int {
            const int rc = p16 ? (g16 ? launch_adamw<__nv_bfloat16, __nv_bfloat16>(t, bits, sr, any, d, s)
                                      : launch_adamw<__nv_bfloat16, float>(t, bits, sr, any, d, s))
                               : (g16 ? launch_adamw<float, __nv_bfloat16>(t, bits, sr, any, d, s)
                                      : launch_adamw<float, float>(t, bits, sr, any, d, s));
            t.count = 0;
            t.tiles = 0;
            return rc;
        };
        for (int64_t i = 0; i < count; ++i) {
            const mx_adamw_tensor& x = tensors[i];
            if (x.n == 0 || kind_of(x) != kind)
                continue;
            if (t.count == kAdamwEntries) {
                const int rc = flush();
                if (rc != MX_OK)
                    return rc;
            }
            AdamwEntry& e = t.e[t.count++];
            e.p = x.param;
            e.g = x.grad;
            e.m = x.m;
            e.v = x.v;
            e.m_sf = x.m_sf;
            e.v_sf = x.v_sf;
            e.copy = static_cast<__nv_bfloat16*>(x.copy);
            e.n = x.n;
            e.first = t.tiles;
            e.index = static_cast<uint32_t>(i);
            e.wd = static_cast<float>(x.weight_decay);
            e.decay = static_cast<float>(1.0 - o.lr * x.weight_decay);
            t.tiles += tiles_of(x.n, x.bits);  // at most 2^23 each
        }
        const int rc = flush();
        if (rc != MX_OK)
            return rc;
    }
    return MX_OK;
}

// ---------------------------------------------------------------- gradient norm
namespace {

constexpr int kNormEntries = 512;
constexpr int kNormUnits = 4;  // octs a thread in flight
struct NormEntry {
    const void* g;
    int64_t n;
    uint32_t first, bf16;
};
struct NormTable {
    NormEntry e[kNormEntries];
    int count;
    uint32_t tiles;
    double* parts;
};

__device__ __forceinline__ double block_sum(double v)
{
    __shared__ double of_warp[kThreads / 32];
#pragma unroll
    for (int k = 16; k > 0; k >>= 1)
        v += __shfl_xor_sync(0xFFFFFFFFu, v, k);
    __syncthreads();
    if ((threadIdx.x & 31) == 0)
        of_warp[threadIdx.x >> 5] = v;
    __syncthreads();
    v = 0.0;
    for (int k = 0; k < kThreads / 32; ++k)
        v += of_warp[k];
    return v;
}

template <typename G, bool ANY>
__device__ __forceinline__ float squares(const NormEntry& e, uint32_t tile)
{
    constexpr int kFlight = ANY && sizeof(G) == 4 ? 1 : kNormUnits;  // loads in flight, by registers
    const int64_t first = static_cast<int64_t>(tile - e.first) * (kThreads * kNormUnits) + threadIdx.x;
    float2 sum = both(0.0f);
#pragma unroll 1
    for (int batch = 0; batch < kNormUnits; batch += kFlight) {
        Values<G, ANY> w[kFlight];
        Place at[kFlight];
#pragma unroll
        for (int k = 0; k < kFlight; ++k) {
            const int64_t unit = first + (batch + k) * kThreads;
            at[k] = {0, static_cast<uint32_t>(unit), static_cast<int32_t>(max(min(e.n - unit * 8, int64_t{8}), int64_t{0}))};
            w[k].load(e.g, at[k], e.n);
        }
#pragma unroll
        for (int k = 0; k < kFlight; ++k) {
            Oct o;
            w[k].get(o, at[k].cols);
#pragma unroll
            for (int j = 0; j < 4; ++j)
                sum = __ffma2_rn(o.p[j], o.p[j], sum);
        }
    }
    return sum.x + sum.y;
}

// Bound by DRAM: 218e6 fp32 values 126 us (6.9 TB/s, some of them still in L2).
//
// Squares and the sums of a thread's 32 values in fp32, everything above in fp64:
// no chain of fp32 additions grows with the tensors.  Partial sums by tile order and
// CTA, which the shapes alone fix.
__global__ void __launch_bounds__(kThreads) square_sum_kernel(const __grid_constant__ NormTable a)
{
    let_next_launch_start();
    double sum = 0.0;
    for (uint32_t tile = blockIdx.x; tile < a.tiles; tile += gridDim.x) {
        int lo = 0, hi = a.count;
        while (hi - lo > 1) {
            const int mid = (lo + hi) >> 1;
            if (a.e[mid].first <= tile)
                lo = mid;
            else
                hi = mid;
        }
        const NormEntry& e = a.e[lo];
        const bool any = e.n % 8 != 0 || reinterpret_cast<uintptr_t>(e.g) % (e.bf16 ? 16 : 32) != 0;
        sum += any ? (e.bf16 ? squares<__nv_bfloat16, true>(e, tile) : squares<float, true>(e, tile))
                   : (e.bf16 ? squares<__nv_bfloat16, false>(e, tile) : squares<float, false>(e, tile));
    }
    sum = block_sum(sum);
    if (threadIdx.x == 0)
        a.parts[blockIdx.x] = sum;
}

// out[0] = the norm, out[1] = min(1, max_norm / (norm + 1e-6)), NaN for a norm that is
// not finite.
__global__ void __launch_bounds__(kThreads) norm_join_kernel(const double* parts, int count, double max_norm, float* out)
{
    wait_for_launch_before();
    double sum = 0.0;
    for (int i = threadIdx.x; i < count; i += kThreads)
        sum += parts[i];
    sum = block_sum(sum);
    if (threadIdx.x == 0) {
        const double norm = sqrt(sum);
        out[0] = static_cast<float>(norm);
        const double f = max_norm / (norm + 1e-6);
        out[1] = isfinite(norm) ? static_cast<float>(f < 1.0 ? f : 1.0) : __int_as_float(0x7FC00000);
    }
}

}  // namespace

int64_t grad_norm_parts(int64_t count) { return (count / kNormEntries + 1) * kGradNormCtas; }

int launch_grad_norm(const mx_grad* grads, int64_t count, double max_norm, float* out, double* parts, const Device& d,
                     cudaStream_t s)
{
    NormTable t;
    t.count = 0;
    t.tiles = 0;
    int used = 0;
    auto flush = [&]() -> int {
        const unsigned most =
            std::min<unsigned>(kGradNormCtas, d.sms * resident_ctas<square_sum_kernel>(kThreads));
        const unsigned ctas = std::min(t.tiles, most);
        t.parts = parts + used;
        used += static_cast<int>(ctas);
        const int rc = ctas ? launch_kernel(square_sum_kernel, ctas, 1, kThreads, 0, false, s, t) : MX_OK;
        t.count = 0;
        t.tiles = 0;
        return rc;
    };
    for (int64_t i = 0; i < count; ++i) {
        if (grads[i].n == 0)
            continue;
        if (t.count == kNormEntries) {
            const int rc = flush();
            if (rc != MX_OK)
                return rc;
        }
        NormEntry& e = t.e[t.count++];
        e.g = grads[i].data;
        e.n = grads[i].n;
        e.first = t.tiles;
        e.bf16 = grads[i].dtype == MX_OUT_BF16;
        t.tiles += static_cast<uint32_t>((e.n + 8 * kThreads * kNormUnits - 1) / (8 * kThreads * kNormUnits));
    }
    int rc = flush();
    if (rc == MX_OK)
        rc = launch_kernel(norm_join_kernel, 1, 1, kThreads, 0, used > 0, s, static_cast<const double*>(parts), used, max_norm,
                           out);
    return rc;
}

}  // namespace mx
