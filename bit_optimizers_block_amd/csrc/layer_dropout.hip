// Dropout whose mask is never stored: the backward pass draws the same random bits again.
//
// The bits come from a counter-based generator, Philox4x32 with ten rounds (Salmon, Moraes,
// Dror, Shaw, "Parallel random numbers: as easy as 1, 2, 3", 2011), keyed by the seed.  Its
// counter is (column / 8, row, call, call >> 32), so an element's bits depend on its place in
// the matrix alone, not on strides, tiles or the launch.  128 bits serve eight elements, 16 for
// each: the probability is a multiple of 2^-16, and the generator costs an eighth of its rounds
// per element, which keeps the pass bound by HBM: 32768 x 2048 bf16 with a residual 63 us (6.4 TB/s),
// without 43.7 (6.1 TB/s).
#include "launch.h"
#include "layer.h"
#include "mx_rows.h"

namespace bitopt {

__device__ __forceinline__ u32x4 philox(u32x4 c, uint32_t k0, uint32_t k1) {
#pragma unroll
    for (int i = 0; i < 10; ++i) {
        const uint64_t p = (uint64_t)0xD2511F53u * c.x, q = (uint64_t)0xCD9E8D57u * c.z;
        c = u32x4{(uint32_t)(q >> 32) ^ c.y ^ k0, (uint32_t)q, (uint32_t)(p >> 32) ^ c.w ^ k1, (uint32_t)p};
        k0 += 0x9E3779B9u;
        k1 += 0xBB67AE85u;
    }
    return c;
}

// y may lie over x or the residual: a lane reads its elements before it writes them, and what the
// last item's load takes from the item before is shifted out.  A dropped element is zero whatever x
// holds there.  In fp32 a lane takes four elements, and two lanes draw the same eight.
template <int DT, bool RESIDUAL> __global__ __launch_bounds__(kThreads) void k_dropout(DropoutArgs a, RowGrid g) {
    constexpr int PER = kPer<DT>;
    const uint64_t call = a.call + (a.counter ? *a.counter : 0);
    for_items(g, a.rows, (int32_t)((a.cols + PER - 1) / PER), [&](int64_t row, int32_t item) {
        const int64_t e = PER * (int64_t)item;
        const int n = (int)min((int64_t)PER, a.cols - e);
        float x[PER], r[PER];
        ld_item<DT, true>(a.x, row * a.ldx + e, n, e, x);
        if constexpr (RESIDUAL) ld_item<DT, true>(a.residual, row * a.ldr + e, n, e, r);
        const u32x4 bits = philox(u32x4{(uint32_t)(e / 8), (uint32_t)row, (uint32_t)call, (uint32_t)(call >> 32)},
                                  (uint32_t)a.seed, (uint32_t)(a.seed >> 32));
#pragma unroll
        for (int j = 0; j < PER; ++j) {
            const uint32_t w = PER == 8 ? bits[j / 2] : item & 1 ? bits[2 + j / 2] : bits[j / 2];
            const uint32_t u = j & 1 ? w >> 16 : w & 0xffffu;
            x[j] = u >= a.threshold ? x[j] * a.grow : 0.0f;
            if constexpr (RESIDUAL) x[j] += r[j];
        }
        st_item<DT>(a.y, row * a.ldy + e, n, x);
    });
}

template <int DT> static hipError_t dropout(const DropoutArgs& a, hipStream_t s) {
    dim3 grid;
    const RowGrid g = row_grid(a.rows, (a.cols + kPer<DT> - 1) / kPer<DT>, grid);
    if (a.residual) hipLaunchKernelGGL((k_dropout<DT, true>), grid, dim3(kThreads), 0, s, a, g);
    else hipLaunchKernelGGL((k_dropout<DT, false>), grid, dim3(kThreads), 0, s, a, g);
    return hipGetLastError();
}

hipError_t launch_dropout(const DropoutArgs& a, int dtype, hipStream_t s) {
    return dtype == kF32 ? dropout<kF32>(a, s) : dtype == kF16 ? dropout<kF16>(a, s) : dropout<kBF16>(a, s);
}

}  // namespace bitopt
