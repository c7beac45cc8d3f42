// mx_rows.h -- kernels that go over the rows of a matrix once: the grid, and loads and stores
// of a lane's 16 bytes of a row from any address aligned to the element.
#pragma once

#include <algorithm>

#include "mx.h"

namespace bitopt {

// Lanes along a row: 2^lanes_log2 of a workgroup's 256, the rest of the workgroup takes
// further rows; `steps` row groups per workgroup.
struct RowGrid {
    int32_t lanes_log2, chunks, steps;
};

constexpr int kRowSteps = 4;

inline RowGrid row_grid(int64_t rows, int64_t items, dim3& grid) {
    RowGrid g{};
    g.lanes_log2 = 4;
    while (g.lanes_log2 < 8 && (int64_t{1} << g.lanes_log2) < items) ++g.lanes_log2;
    g.chunks = (int32_t)((items + (int64_t{1} << g.lanes_log2) - 1) >> g.lanes_log2);
    const int64_t per = kThreads >> g.lanes_log2;
    const int64_t groups = (rows + per - 1) / per;
    g.steps = groups * g.chunks >= 4096 ? kRowSteps : 1;
    grid = dim3((unsigned)g.chunks, (unsigned)std::min<int64_t>((groups + g.steps - 1) / g.steps, 65535));
    return g;
}

#ifdef __HIPCC__

// Elements per lane.
template <int DT> constexpr int kPer = DT == kF32 ? 4 : 8;

// One item of a row as fp32, from any address aligned to the element; zeros from element n on.
// before: elements of the row ahead of it.
template <int DT, bool NT> __device__ __forceinline__ void ld_item(const void* base, int64_t e, int n, int64_t before,
                                                                         float v[kPer<DT>]) {
    if constexpr (DT == kF32) {
        const float* p = reinterpret_cast<const float*>(base) + e;
        if (n >= 4) {
            const f32x4 a = ld16_a4<NT>(p);
#pragma unroll
            for (int j = 0; j < 4; ++j) v[j] = a[j];
        } else {
#pragma unroll
            for (int j = 0; j < 4; ++j) v[j] = j < n ? gbl(p)[j] : 0.0f;
        }
    } else {
        const u32x4 r = ld_half8<NT>(reinterpret_cast<const uint16_t*>(base) + e, n, before);
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] = widen<DT>(r[j / 2] >> (16 * (j & 1)));
    }
}

template <int DT, bool NT = true> __device__ __forceinline__ void st_item(void* base, int64_t e, int n, const float v[kPer<DT>]) {
    if constexpr (DT == kF32) {
        float* p = reinterpret_cast<float*>(base) + e;
        if (n >= 4) {
            st16_a4<NT>(p, f32x4{v[0], v[1], v[2], v[3]});
        } else {
#pragma unroll
            for (int j = 0; j < 4; ++j)
                if (j < n) gbl(p)[j] = v[j];
        }
    } else {
        uint16_t* p = reinterpret_cast<uint16_t*>(base) + e;
        const u32x4 r = {narrow2<DT>(v[0], v[1]), narrow2<DT>(v[2], v[3]), narrow2<DT>(v[4], v[5]),
                         narrow2<DT>(v[6], v[7])};
        if (n >= 8) {
            st16_a2<NT>(p, r);
        } else {
#pragma unroll
            for (int j = 0; j < 8; ++j)
                if (j < n) gbl(p)[j] = (uint16_t)(r[j / 2] >> (16 * (j & 1)));
        }
    }
}

// PER elements of a row whatever the type: eight (fp32 in two loads or stores), or four (fp32, and
// 16-bit loads of half the width).  A matrix of fp32 is best written in fours: lanes that write eight leave
// every other 16 bytes to the next store, and such streamed stores reach 2 TB/s instead of 6.
template <int DT, int PER>
__device__ __forceinline__ void ld_row(const void* base, int64_t e, int n, int64_t before, float v[PER]) {
    if constexpr (PER == kPer<DT>) {
        ld_item<DT, false>(base, e, n, before, v);
    } else if constexpr (DT == kF32) {
        ld_item<DT, false>(base, e, n, before, v);
        ld_item<DT, false>(base, e + 4, n - 4, before + 4, v + 4);
    } else {
        const uint16_t* p = reinterpret_cast<const uint16_t*>(base) + e;
        if (n >= 4) {
            const u32x2a2 r = *(const BITOPT_GLOBAL u32x2a2*)p;
#pragma unroll
            for (int j = 0; j < 4; ++j) v[j] = widen<DT>(r[j / 2] >> (16 * (j & 1)));
        } else {
#pragma unroll
            for (int j = 0; j < 4; ++j) v[j] = j < n ? widen<DT>(gbl(p)[j]) : 0.0f;
        }
    }
}
template <int DT, int PER, bool NT = true> __device__ __forceinline__ void st_row(void* base, int64_t e, int n, const float v[PER]) {
    static_assert(DT == kF32 || PER == kPer<DT>, "16-bit elements are written in eights");
    st_item<DT, NT>(base, e, n, v);
    if constexpr (PER > kPer<DT>) st_item<DT, NT>(base, e + 4, n - 4, v + 4);
}

// Eight elements of a row of at least eight as they lie, from column c or, near its end, the row's
// last eight: loads without a branch, so those of several rows are under way together.  values()
// brings them to their places, with zeros from the row's end on.
template <int DT> struct Eight {
    u32x4 r[DT == kF32 ? 2 : 1];
    template <bool NT> __device__ __forceinline__ void load(const void* base, int64_t row, int64_t c, int64_t cols) {
        const int64_t e = row + min(c, cols - 8);
        if constexpr (DT == kF32) {
            const float* p = reinterpret_cast<const float*>(base) + e;
            r[0] = __builtin_bit_cast(u32x4, ld16_a4<NT>(p));
            r[1] = __builtin_bit_cast(u32x4, ld16_a4<NT>(p + 4));
        } else {
            r[0] = ld16_a2<NT>(reinterpret_cast<const uint16_t*>(base) + e);
        }
    }
    // over = c + 8 - cols, how many of the eight lie beyond the row
    __device__ __forceinline__ void values(int64_t over, float v[8]) const {
        if constexpr (DT == kF32) {
            u32x4 lo = r[0], hi = r[1];
            if (over > 0) {
                if (over & 4) lo = hi, hi = u32x4{0u, 0u, 0u, 0u};
                if (over & 2) lo = u32x4{lo.z, lo.w, hi.x, hi.y}, hi = u32x4{hi.z, hi.w, 0u, 0u};
                if (over & 1) lo = u32x4{lo.y, lo.z, lo.w, hi.x}, hi = u32x4{hi.y, hi.z, hi.w, 0u};
                if (over >= 8) lo = hi = u32x4{0u, 0u, 0u, 0u};
            }
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                v[j] = __uint_as_float(lo[j]);
                v[4 + j] = __uint_as_float(hi[j]);
            }
        } else {
            u32x4 w = r[0];
            if (over > 0) w = over >= 8 ? u32x4{0u, 0u, 0u, 0u} : half_shift(w, (int)over);
#pragma unroll
            for (int j = 0; j < 8; ++j) v[j] = widen<DT>(w[j / 2] >> (16 * (j & 1)));
        }
    }
};

// Runs f(row, item) for every item of the rows.  Where a row has a multiple of 16 items, the
// lanes of an aligned group of 16 are in or out together.
template <class F> __device__ __forceinline__ void for_items(const RowGrid& g, int64_t rows, int32_t items, F f) {
    const int lanes = 1 << g.lanes_log2;
    const int32_t item = (int32_t)blockIdx.x * lanes + ((int)threadIdx.x & (lanes - 1));
    const int64_t per = kThreads >> g.lanes_log2;
    if (item >= items) return;
    const int64_t stride = per * gridDim.y;
    int64_t row = per * blockIdx.y + (threadIdx.x >> g.lanes_log2);
    for (; row + (kRowSteps - 1) * stride < rows; row += kRowSteps * stride) {
#pragma unroll
        for (int s = 0; s < kRowSteps; ++s) f(row + s * stride, item);
    }
    for (; row < rows; row += stride) f(row, item);
}

template <int DT> __device__ __forceinline__ int item_elems(int64_t cols, int32_t item) {
    return (int)max((int64_t)0, min((int64_t)kPer<DT>, cols - kPer<DT> * (int64_t)item));
}

#endif  // __HIPCC__

}  // namespace bitopt
