// mx_units.cuh -- eight consecutive elements a thread: loads and stores of a
// matrix's units at any address, and their checkpoints.
#pragma once
#include <cstring>

#include "mx_act8.cuh"

namespace mx {

// ANY: rows of any address and length; else they start on 16-byte boundaries and
// their length is a multiple of eight.
struct Place {
    int64_t row;
    uint32_t unit;  // in the row
    int32_t cols;   // columns of the unit inside the row: 8, fewer at its end, <= 0 past it
};
// A unit's words.  ANY: the aligned words that it lies in; they may hold a
// neighbouring row's elements, but nothing before the matrix's first element or
// after its last one is touched.
template <typename T, bool ANY>
struct Unit {
    RawOct<T> w;
    uint4 more;
    int s;

    __device__ __forceinline__ void load(const void* base, int64_t ld, const Place& p, int64_t rows, int64_t cols)
    {
        const T* src = static_cast<const T*>(base) + p.row * ld + static_cast<int64_t>(p.unit) * 8;
        if constexpr (!ANY) {
            if (p.cols > 0)
                w.load(src);
            else
                w.clear();
        } else {
            s = misaligned(src, sizeof(T));
            const int64_t at = p.row * ld + static_cast<int64_t>(p.unit) * 8, end = (rows - 1) * ld + cols;
            w.clear();
            more = make_uint4(0, 0, 0, 0);
            if (p.cols <= 0)
                return;
            if (at < 8 || at + 16 > end) {  // the aligned words may reach past the matrix
                T v[8];
#pragma unroll
                for (int c = 0; c < 8; ++c)
                    v[c] = c < p.cols ? src[c] : T(0.0f);
                memcpy(&w, v, sizeof v);
                s = 0;
                return;
            }
            w.load(src - s);
            if (s + p.cols > 8) {
                RawOct<__nv_bfloat16> m;
                m.load(reinterpret_cast<const __nv_bfloat16*>(src - s + 8));
                more = m.w;
            }
        }
    }
    __device__ __forceinline__ void get(Oct& o, int n) const
    {
        if constexpr (!ANY) {
            w.get(o);
        } else {
            if constexpr (sizeof(T) == 2) {
                unpack_oct(shifted(w.w, more, s), o);
            } else {
                uint4 a, b, lo, hi;
                memcpy(&a, &w.a, 16);
                memcpy(&b, &w.b, 16);
                shifted(a, b, more, s, lo, hi);
                words_to_oct(lo, hi, o);
            }
            if (n < 8)
                keep_first(o, n);
        }
    }
};

template <typename T, bool ANY>
__device__ __forceinline__ void store_unit(void* base, int64_t ld, const Place& p, const Oct& o, int64_t cols, Top<T>& top)
{
    T* dst = static_cast<T*>(base) + p.row * ld + static_cast<int64_t>(p.unit) * 8;
    if constexpr (!ANY) {
        if (p.cols > 0)
            store_oct(dst, o, top);
    } else {
        const int lane = threadIdx.x & 31;
        store_ragged(dst, o, p.cols, lane > 0 && p.unit > 0, lane < 31 && static_cast<int64_t>(p.unit) * 8 + 8 < cols, top);
    }
}

__device__ __forceinline__ void save_unit(const Act8View& out, int64_t unit, bool in, const Oct& o)
{
    uint8_t e;
    const uint2 codes = encode_oct(o, e);
    if (in) {
        *reinterpret_cast<uint2*>(out.codes + unit * 8) = codes;
        if ((threadIdx.x & 3) == 0)
            out.sf[unit >> 2] = e;
    }
}

}  // namespace mx
