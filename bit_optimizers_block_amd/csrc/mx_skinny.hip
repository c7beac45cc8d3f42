// Products of few rows (decoding steps, small batches) with an MX matrix.
//
// out[m][n] = sum_k A[m][k] B[n][k] with M <= 64: bound by reading B's codes once, so
// nothing goes through LDS on the way in.  A workgroup owns 16 R rows of B; its waves take
// units of U 128-element chunks of the contraction in turn and their partial sums meet in
// LDS, in a fixed order.
//
// Two E2M1 operands: lane (row i, group q) of a chunk loads block q of its row, 16 bytes of
// codes, which is what the scaled matrix instruction takes.
//
// Decoded operands: the four 16-bit matrix instructions of a chunk need elements 32 j + 8 q
// .. + 7 in lane group q, and those of a 16-bit A are four 16-byte loads of which a row's
// four lanes read 64 consecutive bytes.  Codes are loaded 16 bytes a lane as well and
// brought into that order by exchanges between lane groups (E2M1: a 4 x 4 transpose of
// dwords, four exchanges for 128 elements; E4M3: half a transpose, four exchanges, which
// leaves groups 1 and 2 with each other's elements, so the other operand follows).
//
// Measured, bf16 A, E2M1 B: one row against 50257 x 2048 (55 MB of codes and scales) 16.3 us,
// two E2M1 operands 12.9 us, of which a launch is 2.6 (E4M3 B 24.2 us); 64 rows against
// 8192 x 8192 38 us (E4M3 B 42.5), 17 rows against 4093 x 1999 8.5.  Those wait for one unit's loads
// after the other with two waves a SIMD; A in E4M3, half the bytes, takes 32 and 5.7, so its
// rows, which every workgroup reads from the caches, are not all of it.
#include <algorithm>
#include <type_traits>

#include "launch.h"
#include "mx.h"

namespace bitopt {

enum { kX16, kXE2M1, kXE4M3 };

__device__ __forceinline__ void swap32(uint32_t& a, uint32_t& b) {
    const auto r = __builtin_amdgcn_permlane32_swap(a, b, false, false);
    a = r[0];
    b = r[1];
}
__device__ __forceinline__ void swap16(uint32_t& a, uint32_t& b) {
    const auto r = __builtin_amdgcn_permlane16_swap(a, b, false, false);
    a = r[0];
    b = r[1];
}

// The codes of one 128-element chunk of a row, and their order for the 16-bit products.
template <int FMT> struct ChunkCodes {
    static constexpr int N = FMT == kMxE2M1 ? 1 : 2;
    u32x4 c[N];

    // Lane group q: 16-byte piece q of each 64 bytes of the chunk.
    __device__ __forceinline__ void load(const uint8_t* row, int chunk, int q, bool in) {
        const u32x4* p = reinterpret_cast<const u32x4*>(row) + (4 * N) * (int64_t)chunk + q;
#pragma unroll
        for (int h = 0; h < N; ++h) c[h] = in ? *gbl(p + 4 * h) : u32x4{0u, 0u, 0u, 0u};
    }

    // Fragment j in 16 bits: lane group q gets elements 32 j + 8 q .. + 7, or with CROSSED
    // those of group {0, 2, 1, 3}[q].  s: the chunk's four scale bytes.
    template <int DT, bool CROSSED> __device__ __forceinline__ void half(uint32_t s, u32x4 f[4]) const {
        if constexpr (FMT == kMxE2M1) {
            uint32_t d0 = c[0][0], d1 = CROSSED ? c[0][2] : c[0][1], d2 = CROSSED ? c[0][1] : c[0][2], d3 = c[0][3];
            swap32(d0, d2);
            swap32(d1, d3);
            swap16(d0, d1);
            swap16(d2, d3);
            const uint32_t d[4] = {d0, d1, d2, d3};
#pragma unroll
            for (int j = 0; j < 4; ++j) f[j] = mx_half8_e2m1<DT>(d[j], mx_scale_f32((s >> (8 * j)) & 255u));
        } else {
            static_assert(CROSSED, "E4M3 chunks come out crossed");
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                uint32_t a0 = c[h][0], a1 = c[h][1], b0 = c[h][2], b1 = c[h][3];
                swap32(a0, b0);
                swap32(a1, b1);
                f[2 * h] = mx_half8_e4m3<DT>(a0, a1, mx_scale_f32((s >> (16 * h)) & 255u));
                f[2 * h + 1] = mx_half8_e4m3<DT>(b0, b1, mx_scale_f32((s >> (16 * h + 8)) & 255u));
            }
        }
    }
};

// The four scale bytes of each of U chunks from c0.
template <int U> __device__ __forceinline__ void ld_scales(const uint8_t* row, int c0, int chunks, uint32_t s[U]) {
    const uint32_t* p = reinterpret_cast<const uint32_t*>(row) + c0;
    if (c0 + U <= chunks) {
#pragma unroll
        for (int u = 0; u < U; ++u) s[u] = gbl(p)[u];
    } else {
#pragma unroll
        for (int u = 0; u < U; ++u) s[u] = c0 + u < chunks ? gbl(p)[u] : 0u;
    }
}

// A chunk's four fragments of a 16-bit row from element k on: zeros where the lane has no
// row or the chunk does not exist, element by element only where the row ends in it.
__device__ __forceinline__ void ld_chunk16(const uint16_t* row, int chunk, int octet, int K, bool in, u32x4 f[4]) {
    const int k = chunk * kMxPad + 8 * octet;
#pragma unroll
    for (int j = 0; j < 4; ++j) f[j] = u32x4{0u, 0u, 0u, 0u};
    if (in) {
        if (K - chunk * kMxPad >= kMxPad) {
#pragma unroll
            for (int j = 0; j < 4; ++j) f[j] = ld16_a2(row + k + 32 * j);
        } else {
#pragma unroll
            for (int j = 0; j < 4; ++j) f[j] = ld_half8(row + k + 32 * j, K - k - 32 * j, k + 32 * j);
        }
    }
}

// MT: tiles of 16 rows of A; R: tiles of 16 rows of B; U: chunks per unit.
template <int DT, int XSRC, int FMT, int MT, int R, int U, int WAVES>
__global__ __launch_bounds__(WAVES * 64) void k_mx_skinny(MxGemmArgs g) {
    constexpr int T = R * MT;
    constexpr bool scaled = XSRC == kXE2M1 && FMT == kMxE2M1;
    constexpr int XFMT = XSRC == kXE4M3 ? kMxE4M3 : kMxE2M1;
    constexpr bool crossed = FMT == kMxE4M3 || XSRC == kXE4M3;
    static_assert(!scaled || U == 4, "scales of two E2M1 operands are transposed four chunks at a time");
    __shared__ f32x4 part[WAVES * T * 64];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), i = lane & 15, q = lane >> 4;
    const int n0 = blockIdx.x * (16 * R);
    const int chunks = (int)(mx_padded(g.K) / kMxPad);

    const uint8_t *bc[R], *bs[R];
#pragma unroll
    for (int r = 0; r < R; ++r) {
        const int64_t row = min(n0 + 16 * r + i, g.N - 1);
        bc[r] = g.b + row * g.b_row_bytes;
        bs[r] = g.b_scales + row * g.b_row_scales;
    }
    const uint8_t *ax[MT], *as[MT];
    bool live[MT];
#pragma unroll
    for (int t = 0; t < MT; ++t) {
        live[t] = 16 * t + i < g.M;
        const int64_t row = min(16 * t + i, g.M - 1);
        ax[t] = reinterpret_cast<const uint8_t*>(g.a) + (XSRC == kX16 ? 2 * row * g.lda : row * g.a_row_bytes);
        as[t] = XSRC == kX16 ? nullptr : g.a_scales + row * g.a_row_scales;
    }
    const int octet = crossed ? ((q & 1) << 1 | q >> 1) : q;

    f32x4 acc[R][MT];
#pragma unroll
    for (int r = 0; r < R; ++r)
#pragma unroll
        for (int t = 0; t < MT; ++t) acc[r][t] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};

    struct Unit {
        ChunkCodes<FMT> b[U][R];
        uint32_t sb[R][scaled ? 1 : U];
        ChunkCodes<XFMT> xc[XSRC == kX16 ? 1 : U][MT];
        uint32_t sx[MT][scaled ? 1 : U];
        u32x4 xh[XSRC == kX16 ? U : 1][MT][4];
    };
    auto load = [&](Unit& d, int c0) {
#pragma unroll
        for (int r = 0; r < R; ++r)
#pragma unroll
            for (int u = 0; u < U; ++u) d.b[u][r].load(bc[r], c0 + u, q, c0 + u < chunks);
#pragma unroll
        for (int r = 0; r < R; ++r) {
            if constexpr (scaled) d.sb[r][0] = gbl(reinterpret_cast<const uint32_t*>(bs[r]))[min(c0 + q, chunks - 1)];
            else ld_scales<U>(bs[r], c0, chunks, d.sb[r]);
        }
#pragma unroll
        for (int t = 0; t < MT; ++t) {
            if constexpr (scaled) d.sx[t][0] = gbl(reinterpret_cast<const uint32_t*>(as[t]))[min(c0 + q, chunks - 1)];
            else if constexpr (XSRC != kX16) ld_scales<U>(as[t], c0, chunks, d.sx[t]);
#pragma unroll
            for (int u = 0; u < U; ++u) {
                // lanes without a row of A load nothing: their sums are not stored
                const bool in = c0 + u < chunks && live[t];
                if constexpr (XSRC == kX16) {
                    ld_chunk16(reinterpret_cast<const uint16_t*>(ax[t]), c0 + u, octet, g.K, in, d.xh[u][t]);
                } else {
                    d.xc[u][t].load(ax[t], c0 + u, q, in);
                }
            }
        }
    };
    auto multiply = [&](const Unit& d) {
        if constexpr (scaled) {
            uint32_t sb[R], sx[MT];
#pragma unroll
            for (int r = 0; r < R; ++r) sb[r] = transpose_bytes(d.sb[r][0], lane);
#pragma unroll
            for (int t = 0; t < MT; ++t) sx[t] = transpose_bytes(d.sx[t][0], lane);
            auto chunk = [&](auto at) {
                constexpr int u = decltype(at)::value;
#pragma unroll
                for (int r = 0; r < R; ++r)
#pragma unroll
                    for (int t = 0; t < MT; ++t)
                        acc[r][t] = mfma_e2m1_at<u>(d.b[u][r].c[0], d.xc[u][t].c[0], acc[r][t], sb[r], sx[t]);
            };
            chunk(std::integral_constant<int, 0>{});
            chunk(std::integral_constant<int, 1>{});
            chunk(std::integral_constant<int, 2>{});
            chunk(std::integral_constant<int, 3>{});
        } else {
#pragma unroll
            for (int u = 0; u < U; ++u) {
                u32x4 f[R][4];
#pragma unroll
                for (int r = 0; r < R; ++r) d.b[u][r].template half<DT, crossed>(d.sb[r][u], f[r]);
#pragma unroll
                for (int t = 0; t < MT; ++t) {
                    u32x4 x[4];
                    if constexpr (XSRC == kX16) {
#pragma unroll
                        for (int j = 0; j < 4; ++j) x[j] = d.xh[u][t][j];
                    } else {
                        d.xc[u][t].template half<DT, crossed>(d.sx[t][u], x);
                    }
#pragma unroll
                    for (int j = 0; j < 4; ++j)
#pragma unroll
                        for (int r = 0; r < R; ++r) acc[r][t] = mfma16<DT>(f[r][j], x[j], acc[r][t]);
                }
            }
        }
    };

    for (int c0 = U * wave; c0 < chunks; c0 += U * WAVES) {
        Unit d;
        load(d, c0);
        multiply(d);
    }
    // tile (r, t) is summed over the waves, in their order, by wave (r MT + t) % WAVES
#pragma unroll
    for (int r = 0; r < R; ++r)
#pragma unroll
        for (int t = 0; t < MT; ++t) part[(wave * T + r * MT + t) * 64 + lane] = acc[r][t];
    __syncthreads();
    for (int tile = wave; tile < T; tile += WAVES) {
        f32x4 v = part[tile * 64 + lane];
#pragma unroll
        for (int w = 1; w < WAVES; ++w) v += part[(w * T + tile) * 64 + lane];
        const int m = 16 * (tile % MT) + i, n = n0 + 16 * (tile / MT) + 4 * q;
        if (m < g.M && n < g.N) mx_store4(g, m, n, v);
    }
}

// Up to 16 rows of A and a contraction that the waves hold at four chunks each: A's
// fragments are loaded once and stay in registers, and a workgroup goes through tiles of 16
// rows of B, the next tile's codes on their way while one is multiplied (one row against
// 50257 x 2048: 16.3 us, against 20.8 with A's rows loaded for every tile;
// registers for a fourth wave a SIMD spill: 24).
template <int DT, int XSRC, int FMT, int WAVES>
__global__ __launch_bounds__(WAVES * 64) void k_mx_tokens(MxGemmArgs g) {
    constexpr bool scaled = XSRC == kXE2M1 && FMT == kMxE2M1;
    constexpr int XFMT = XSRC == kXE4M3 ? kMxE4M3 : kMxE2M1;
    constexpr bool crossed = FMT == kMxE4M3 || XSRC == kXE4M3;
    constexpr int U = 4;
    __shared__ f32x4 part[2][WAVES * 64];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), i = lane & 15, q = lane >> 4;
    const int chunks = (int)(mx_padded(g.K) / kMxPad), c0 = U * wave;
    const int tiles = (g.N + 15) / 16;

    struct Unit {
        ChunkCodes<FMT> b[U];
        uint32_t s[scaled ? 1 : U];
    };
    auto load = [&](Unit& d, int tile) {
        const int64_t row = min(16 * tile + i, g.N - 1);
        const uint8_t* codes = g.b + row * g.b_row_bytes;
        const uint8_t* scales = g.b_scales + row * g.b_row_scales;
#pragma unroll
        for (int u = 0; u < U; ++u) d.b[u].load(codes, c0 + u, q, c0 + u < chunks);
        if constexpr (scaled) d.s[0] = gbl(reinterpret_cast<const uint32_t*>(scales))[min(c0 + q, chunks - 1)];
        else ld_scales<U>(scales, c0, chunks, d.s);
    };
    int tile = blockIdx.x;
    Unit a, b;
    if (c0 < chunks) load(a, tile);

    const bool live = i < g.M;
    const int64_t m = min(i, g.M - 1);
    u32x4 x[U][scaled ? 1 : 4];
    uint32_t sx = 0;
#pragma unroll
    for (int u = 0; u < U; ++u) {
        const bool in = c0 + u < chunks && live;
        if constexpr (XSRC == kX16) {
            const int octet = crossed ? ((q & 1) << 1 | q >> 1) : q;
            ld_chunk16(reinterpret_cast<const uint16_t*>(g.a) + m * g.lda, c0 + u, octet, g.K, in, x[u]);
        } else {
            ChunkCodes<XFMT> c;
            const uint8_t* scales = g.a_scales + m * g.a_row_scales;
            c.load(reinterpret_cast<const uint8_t*>(g.a) + m * g.a_row_bytes, c0 + u, q, in);
            if constexpr (scaled) {
                x[u][0] = c.c[0];
            } else {
                const uint32_t s = c0 + u < chunks ? gbl(reinterpret_cast<const uint32_t*>(scales))[c0 + u] : 0u;
                c.template half<DT, crossed>(s, x[u]);
            }
        }
    }
    if constexpr (scaled) {
        const uint8_t* scales = g.a_scales + m * g.a_row_scales;
        if (c0 < chunks)
            sx = transpose_bytes(gbl(reinterpret_cast<const uint32_t*>(scales))[min(c0 + q, chunks - 1)], lane);
    }

    int turn = 0;
    auto step = [&](const Unit& cur, Unit& next) {
        if (c0 < chunks && tile + (int)gridDim.x < tiles) load(next, tile + (int)gridDim.x);
        f32x4 acc = {0.0f, 0.0f, 0.0f, 0.0f};
        if (c0 < chunks) {
            if constexpr (scaled) {
                const uint32_t s = transpose_bytes(cur.s[0], lane);
                acc = mfma_e2m1_at<0>(cur.b[0].c[0], x[0][0], acc, s, sx);
                acc = mfma_e2m1_at<1>(cur.b[1].c[0], x[1][0], acc, s, sx);
                acc = mfma_e2m1_at<2>(cur.b[2].c[0], x[2][0], acc, s, sx);
                acc = mfma_e2m1_at<3>(cur.b[3].c[0], x[3][0], acc, s, sx);
            } else {
#pragma unroll
                for (int u = 0; u < U; ++u) {
                    u32x4 f[4];
                    cur.b[u].template half<DT, crossed>(cur.s[u], f);
#pragma unroll
                    for (int j = 0; j < 4; ++j) acc = mfma16<DT>(f[j], x[u][j], acc);
                }
            }
        }
        // the sums of two tiles back in this half were read before the last barrier
        part[turn & 1][wave * 64 + lane] = acc;
        asm volatile("" ::: "memory");
        __builtin_amdgcn_s_waitcnt(0xC07F);        // LDS only: the next tile's loads stay in flight
        __builtin_amdgcn_s_barrier();
        asm volatile("" ::: "memory");
        if (wave == turn % WAVES) {
            f32x4 v = part[turn & 1][lane];
#pragma unroll
            for (int w = 1; w < WAVES; ++w) v += part[turn & 1][w * 64 + lane];
            const int n = 16 * tile + 4 * q;
            if (live && n < g.N) mx_store4(g, i, n, v);
        }
        ++turn;
        tile += gridDim.x;
    };
    while (true) {
        step(a, b);
        if (tile >= tiles) break;
        step(b, a);
        if (tile >= tiles) break;
    }
}

template <int DT, int XSRC, int FMT, int MT, int R, int WAVES>
static hipError_t skinny_launch(const MxGemmArgs& g, hipStream_t s) {
    // several chunks in flight where A's fragments leave the registers for them
    constexpr int U = (XSRC == kXE2M1 && FMT == kMxE2M1) || (MT == 1 && R == 1) ? 4 : 1;
    hipLaunchKernelGGL((k_mx_skinny<DT, XSRC, FMT, MT, R, U, WAVES>), dim3((unsigned)((g.N + 16 * R - 1) / (16 * R))),
                       dim3(WAVES * 64), 0, s, g);
    return hipGetLastError();
}

// A's rows are read once per workgroup, so more rows of B a workgroup save cache traffic as
// long as N still occupies the CUs.  bf16 A, E2M1 B, us with 1, 2 and 4 tiles of 16 rows:
// 64 x 8192 x 8192 (M x N x K) 67, 39, 48; 64 x 50257 x 2048 125, 79, 49; 17 x 4093 x 1999
// 9.6, 10.2, 11.9; 16 x 8192 x 8192 24.4, 18.0, 26.2.
template <int DT, int XSRC, int FMT, int MT> static hipError_t skinny_rows(const MxGemmArgs& g, hipStream_t s) {
    if (g.N >= 64 * 512) return skinny_launch<DT, XSRC, FMT, MT, 4, 4>(g, s);
    if (g.N >= 32 * 192) return skinny_launch<DT, XSRC, FMT, MT, 2, 8>(g, s);
    return skinny_launch<DT, XSRC, FMT, MT, 1, 8>(g, s);
}

template <int DT, int XSRC, int FMT, int WAVES> static hipError_t tokens_launch(const MxGemmArgs& g, hipStream_t s) {
    static const int per_cu = [] {
        int n = 0;
        if (hipOccupancyMaxActiveBlocksPerMultiprocessor(
                &n, reinterpret_cast<const void*>(&k_mx_tokens<DT, XSRC, FMT, WAVES>), WAVES * 64, 0) != hipSuccess || n < 1) {
            (void)hipGetLastError();
            return 1;
        }
        return n;
    }();
    const int64_t tiles = (g.N + 15) / 16;
    const unsigned grid = (unsigned)std::min<int64_t>(tiles, group_cap(per_cu));
    hipLaunchKernelGGL((k_mx_tokens<DT, XSRC, FMT, WAVES>), dim3(grid), dim3(WAVES * 64), 0, s, g);
    return hipGetLastError();
}

template <int DT, int XSRC, int FMT> static hipError_t skinny(const MxGemmArgs& g, hipStream_t s) {
    if (g.M <= 16 && g.K > 0) {
        if (g.K <= 4 * 512) return tokens_launch<DT, XSRC, FMT, 4>(g, s);
        if (g.K <= 8 * 512) return tokens_launch<DT, XSRC, FMT, 8>(g, s);
        if constexpr (XSRC == kXE2M1 && FMT == kMxE2M1)
            if (g.K <= 16 * 512) return tokens_launch<DT, XSRC, FMT, 16>(g, s);
    }
    if (g.M <= 16) return skinny_rows<DT, XSRC, FMT, 1>(g, s);
    if (g.M <= 32) return skinny_rows<DT, XSRC, FMT, 2>(g, s);
    return skinny_rows<DT, XSRC, FMT, 4>(g, s);
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
