// Products of few rows (decoding steps, small batches) with an MX matrix.
//
// out[m][n] = sum_k A[m][k] B[n][k] with M <= 64: bound by reading B's codes once, so
// nothing goes through LDS on the way in.  A workgroup owns 16 rows of B; its waves take
// the 128-element chunks of the contraction in turn and their partial sums meet in LDS,
// in a fixed order.  In a chunk, lane l holds the whole block l / 16 of row l % 16 (one
// scale, 16 or 32 bytes of codes, one or two wide loads); the contraction may be summed
// in any order, so matrix instruction j simply takes elements 8 j .. 8 j + 7 of every
// lane's block, and A's fragment is the same slice of its row.
#include "launch.h"
#include "mx.h"

namespace bitopt {

enum { kX16, kXE2M1, kXE4M3 };

// The 32 elements of one block of a row as four 16-bit fragments.
template <int DT, int FMT>
__device__ __forceinline__ void ld_block16(const uint8_t* row, const uint8_t* scales, int64_t block, u32x4 f[4]) {
    const float s = mx_scale_f32(gbl(scales)[block]);
    if constexpr (FMT == kMxE2M1) {
        const u32x4 c = gbl(reinterpret_cast<const u32x4*>(row))[block];
#pragma unroll
        for (int j = 0; j < 4; ++j) f[j] = mx_half8_e2m1<DT>(c[j], s);
    } else {
        const u32x4 c0 = gbl(reinterpret_cast<const u32x4*>(row))[2 * block];
        const u32x4 c1 = gbl(reinterpret_cast<const u32x4*>(row))[2 * block + 1];
        f[0] = mx_half8_e4m3<DT>(c0.x, c0.y, s);
        f[1] = mx_half8_e4m3<DT>(c0.z, c0.w, s);
        f[2] = mx_half8_e4m3<DT>(c1.x, c1.y, s);
        f[3] = mx_half8_e4m3<DT>(c1.z, c1.w, s);
    }
}

// MT: tiles of 16 rows of A.
template <int DT, int XSRC, int FMT, int MT, int WAVES>
__global__ __launch_bounds__(WAVES * 64) void k_mx_skinny(MxGemmArgs g) {
    __shared__ f32x4 part[WAVES > 1 ? (WAVES - 1) * MT * 64 : 1];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, i = lane & 15, q = lane >> 4;
    const int n0 = blockIdx.x * 16;
    const int chunks = (int)(mx_padded(g.K) / kMxPad);
    const int64_t brow = min(n0 + i, g.N - 1);
    const uint8_t* bc = g.b + brow * g.b_row_bytes;
    const uint8_t* bs = g.b_scales + brow * g.b_row_scales;

    f32x4 acc[MT];
#pragma unroll
    for (int t = 0; t < MT; ++t) acc[t] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};

    constexpr bool scaled = XSRC == kXE2M1 && FMT == kMxE2M1;
#pragma unroll 2
    for (int c = wave; c < chunks; c += WAVES) {
        const int64_t block = 4 * (int64_t)c + q;
        if constexpr (scaled) {
            const u32x4 fb = gbl(reinterpret_cast<const u32x4*>(bc))[block];
            const uint32_t sb = gbl(bs)[block];
#pragma unroll
            for (int t = 0; t < MT; ++t) {
                const int64_t m = min(16 * t + i, g.M - 1);
                const u32x4 fa = gbl(reinterpret_cast<const u32x4*>(reinterpret_cast<const uint8_t*>(g.a) + m * g.a_row_bytes))[block];
                acc[t] = mfma_e2m1(fb, fa, acc[t], sb, gbl(g.a_scales)[m * g.a_row_scales + block]);
            }
        } else {
            u32x4 fb[4];
            ld_block16<DT, FMT>(bc, bs, block, fb);
#pragma unroll
            for (int t = 0; t < MT; ++t) {
                const int64_t m = min(16 * t + i, g.M - 1);
                u32x4 fa[4];
                if constexpr (XSRC == kX16) {
                    const uint16_t* p = reinterpret_cast<const uint16_t*>(g.a) + m * g.lda + block * kMxBlock;
                    const int left = g.K - (int)block * kMxBlock;
#pragma unroll
                    for (int j = 0; j < 4; ++j) fa[j] = ld_half8(p + 8 * j, left - 8 * j);
                } else {
                    ld_block16<DT, XSRC == kXE2M1 ? kMxE2M1 : kMxE4M3>(
                        reinterpret_cast<const uint8_t*>(g.a) + m * g.a_row_bytes, g.a_scales + m * g.a_row_scales, block,
                        fa);
                }
#pragma unroll
                for (int j = 0; j < 4; ++j) acc[t] = mfma16<DT>(fb[j], fa[j], acc[t]);
            }
        }
    }
    if constexpr (WAVES > 1) {
        if (wave > 0) {
#pragma unroll
            for (int t = 0; t < MT; ++t) part[((wave - 1) * MT + t) * 64 + lane] = acc[t];
        }
        __syncthreads();
        if (wave > 0) return;
#pragma unroll
        for (int w = 0; w < WAVES - 1; ++w)
#pragma unroll
            for (int t = 0; t < MT; ++t) acc[t] += part[(w * MT + t) * 64 + lane];
    }
    const int n = n0 + 4 * q;
#pragma unroll
    for (int t = 0; t < MT; ++t) {
        const int m = 16 * t + i;
        if (m < g.M && n < g.N) mx_store4(g, m, n, acc[t]);
    }
}

template <int DT, int XSRC, int FMT> static hipError_t skinny(const MxGemmArgs& g, hipStream_t s) {
    const dim3 grid((unsigned)((g.N + 15) / 16));
    if (g.M <= 16) hipLaunchKernelGGL((k_mx_skinny<DT, XSRC, FMT, 1, 8>), grid, dim3(512), 0, s, g);
    else if (g.M <= 32) hipLaunchKernelGGL((k_mx_skinny<DT, XSRC, FMT, 2, 8>), grid, dim3(512), 0, s, g);
    else hipLaunchKernelGGL((k_mx_skinny<DT, XSRC, FMT, 4, 8>), grid, dim3(512), 0, s, g);
    return hipGetLastError();
}

hipError_t launch_mx_linear_skinny(const MxGemmArgs& g, int dtype, int fmt, hipStream_t s) {
    const bool four = fmt == kMxE2M1;
    if (dtype == kBF16) return four ? skinny<kBF16, kX16, kMxE2M1>(g, s) : skinny<kBF16, kX16, kMxE4M3>(g, s);
    return four ? skinny<kF16, kX16, kMxE2M1>(g, s) : skinny<kF16, kX16, kMxE4M3>(g, s);
}

hipError_t launch_mx_matmul_skinny(const MxGemmArgs& g, int a_fmt, int b_fmt, hipStream_t s) {
    if (a_fmt == kMxE2M1)
        return b_fmt == kMxE2M1 ? skinny<kBF16, kXE2M1, kMxE2M1>(g, s) : skinny<kBF16, kXE2M1, kMxE4M3>(g, s);
    return b_fmt == kMxE2M1 ? skinny<kBF16, kXE4M3, kMxE2M1>(g, s) : skinny<kBF16, kXE4M3, kMxE4M3>(g, s);
}

}  // namespace bitopt
