// F8 products with up to 32 rows of A (single tokens, small decoding batches).
//
// Bound by reading B once.  A workgroup takes 16 rows of B, and its waves take blocks of 128
// contraction elements in turn: a wave's load covers 16 whole lines.  Codes are decoded to
// bf16 (exact) for the 16-bit matrix instructions, which keep pace with memory here, so one
// form serves 16-bit and fp32 results (one row x 50257 x 2048, B by tiles: 17.6 us, 5.9 TB/s).  The waves'
// sums meet in LDS, in the order of the waves.
#include <type_traits>

#include "f8.h"

namespace bitopt {

template <int AF, int BF, bool BTILES, int MT, int WAVES>
__global__ __launch_bounds__(WAVES * 64) void k_f8_few(F8GemmArgs g) {
    constexpr int U = MT * WAVES == 4 ? 4 : 2;  // blocks of a wave in flight
    __shared__ f32x4 part[WAVES * MT * 64];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), i = lane & 15, q = lane >> 4;
    const int n0 = (int)blockIdx.x * 16, blocks = (int)f8_blocks(g.K);
    // rows beyond the matrix repeat its last one
    const uint8_t* b = g.b + min((int64_t)n0 + i, (int64_t)g.N - 1) * g.row_bytes + 32 * q;
    const float* tile = g.b_scales + (int64_t)(n0 / kF8Block) * blocks;
    const uint8_t* a[MT];
    int am[MT];
#pragma unroll
    for (int t = 0; t < MT; ++t) {
        am[t] = min(16 * t + i, g.M - 1);
        a[t] = g.a + am[t] * g.row_bytes + 32 * q;
    }
    f32x4 acc[MT];
    // every `waves`-th of the waves' blocks, with scales as they are or taken apart
    auto run = [&](int first, int waves, auto apart) __attribute__((always_inline)) {
        constexpr bool APART = decltype(apart)::value;
#pragma unroll
        for (int t = 0; t < MT; ++t) acc[t] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};

        for (int c0 = U * first; c0 < blocks; c0 += U * waves) {
            u32x4 bx[U][2], ax[U][MT][2];
            float sa[U][MT];
            f32x4 sb[U];
#pragma unroll
            for (int u = 0; u < U; ++u) {
                // past the last block: codes and scales of zero
                const int c = c0 + u;
                const bool in = c < blocks;
                const int at = in ? c : blocks - 1;
                bx[u][0] = *gbl(reinterpret_cast<const u32x4*>(b + (int64_t)at * kF8Block));
                bx[u][1] = *gbl(reinterpret_cast<const u32x4*>(b + (int64_t)at * kF8Block + 16));
                if (!in) bx[u][0] = bx[u][1] = u32x4{0u, 0u, 0u, 0u};
                if constexpr (BTILES) {
                    const float s = in ? gbl(tile)[at] : 0.0f;
                    sb[u] = f32x4{s, s, s, s};
                } else {
#pragma unroll
                    for (int r = 0; r < 4; ++r)
                        sb[u][r] = in ? gbl(g.b_scales)[(int64_t)at * g.N + min((int64_t)n0 + 4 * q + r, (int64_t)g.N - 1)] : 0.0f;
                }
#pragma unroll
                for (int t = 0; t < MT; ++t) {
                    ax[u][t][0] = *gbl(reinterpret_cast<const u32x4*>(a[t] + (int64_t)at * kF8Block));
                    ax[u][t][1] = *gbl(reinterpret_cast<const u32x4*>(a[t] + (int64_t)at * kF8Block + 16));
                    if (!in) ax[u][t][0] = ax[u][t][1] = u32x4{0u, 0u, 0u, 0u};
                    sa[u][t] = in ? gbl(g.a_scales)[(int64_t)at * g.M + am[t]] : 0.0f;
                }
            }
#pragma unroll
            for (int u = 0; u < U; ++u) {
                u32x4 bh[4];
                float fb = 1.0f;
                if constexpr (APART) {
                    const int64_t row = min((int64_t)n0 + i, (int64_t)g.N - 1), at = min(c0 + u, blocks - 1);
                    fb = f8_fold(BTILES ? sb[u].x : gbl(g.b_scales)[at * g.N + row]).f;
#pragma unroll
                    for (int r = 0; r < 4; ++r) sb[u][r] = f8_fold(sb[u][r]).s;
                }
#pragma unroll
                for (int h = 0; h < 4; ++h) bh[h] = f8_half8<BF>(bx[u][h / 2][2 * (h & 1)], bx[u][h / 2][2 * (h & 1) + 1], fb);
#pragma unroll
                for (int t = 0; t < MT; ++t) {
                    f32x4 p = {0.0f, 0.0f, 0.0f, 0.0f};
                    float fa = 1.0f;
                    if constexpr (APART) {
                        const F8Fold v = f8_fold(sa[u][t]);
                        fa = v.f;
                        sa[u][t] = v.s;
                    }
#pragma unroll
                    for (int h = 0; h < 4; ++h)
                        p = mfma16<kBF16>(bh[h], f8_half8<AF>(ax[u][t][h / 2][2 * (h & 1)], ax[u][t][h / 2][2 * (h & 1) + 1], fa), p);
#pragma unroll
                    for (int r = 0; r < 4; ++r) acc[t][r] = __builtin_fmaf(p[r], sa[u][t] * sb[u][r], acc[t][r]);
                }
            }
        }
    };
    run(wave, WAVES, std::false_type{});
#pragma unroll
    for (int t = 0; t < MT; ++t) part[(wave * MT + t) * 64 + lane] = acc[t];
    __syncthreads();
    for (int t = wave; t < MT; t += WAVES) {
        f32x4 v[1][1] = {{part[t * 64 + lane]}};
#pragma unroll
        for (int w = 1; w < WAVES; ++w) v[0][0] += part[(w * MT + t) * 64 + lane];
        f8_store(g.accumulate, blocks > 0,
                 [&] __attribute__((always_inline)) {
                     if (16 * t + i < g.M && n0 + 4 * q < g.N) mx_store4(g, 16 * t + i, n0 + 4 * q, v[0][0]);
                 },
                 [&] __attribute__((always_inline)) { return f8_again(g, v, 16 * t, n0, f8_least<AF, BF>(blocks)); },
                 [&] __attribute__((always_inline)) {
                     // this wave alone, in the same order
                     for (int w = 0; w < WAVES; ++w) {
                         run(w, WAVES, std::true_type{});
                         const f32x4 p = MT > 1 && t > 0 ? acc[MT - 1] : acc[0];
                         v[0][0] = w > 0 ? v[0][0] + p : p;
                     }
                 });
    }
}

// ------------------------------------------------------------------------- launches

// us a launch among others with four and with eight waves, B by tiles: 1 x 50257 x 2048 18.1, 18.6; 1 x 2048 x 8192
// 8.0, 7.0; 16 x 8192 x 8192 18.3, 17.1; 32 x 8192 x 8192 25.3, 25.0; by rows: 19.5, 23.5; 9.5, 7.6; 19.9, 18.6; 26.6,
// 26.3.  Beyond 32 rows the tiled forms are faster; us with this form and with those: 64 x 8192 x 2048
// 13.1 and 8.1, 64 x 50257 x 2048 65 and 39 (17 x 4093 x 1999 5.6 and 7.2).
template <int AF, int BF, bool BTILES> static hipError_t few(const F8GemmArgs& g, hipStream_t s) {
    const dim3 grid((unsigned)(((int64_t)g.N + 15) / 16));
    const bool deep = f8_blocks(g.K) >= 32;
    if (g.M <= 16 && deep) hipLaunchKernelGGL((k_f8_few<AF, BF, BTILES, 1, 8>), grid, dim3(512), 0, s, g);
    else if (g.M <= 16) hipLaunchKernelGGL((k_f8_few<AF, BF, BTILES, 1, 4>), grid, dim3(256), 0, s, g);
    else if (deep) hipLaunchKernelGGL((k_f8_few<AF, BF, BTILES, 2, 8>), grid, dim3(512), 0, s, g);
    else hipLaunchKernelGGL((k_f8_few<AF, BF, BTILES, 2, 4>), grid, dim3(256), 0, s, g);
    return hipGetLastError();
}

hipError_t launch_f8_few(const F8GemmArgs& g, int a_fmt, int b_fmt, int b_blocks, hipStream_t s) {
    const bool a4 = a_fmt == kF8E4M3, b4 = b_fmt == kF8E4M3, t = b_blocks == kF8Tiles;
    if (a4 && b4) return t ? few<0, 0, true>(g, s) : few<0, 0, false>(g, s);
    if (b4) return t ? few<1, 0, true>(g, s) : few<1, 0, false>(g, s);
    if (a4) return t ? few<0, 1, true>(g, s) : few<0, 1, false>(g, s);
    return t ? few<1, 1, true>(g, s) : few<1, 1, false>(g, s);
}

}  // namespace bitopt
