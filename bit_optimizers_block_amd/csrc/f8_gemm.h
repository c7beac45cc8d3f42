// f8_gemm.h -- tiled products of F8 matrices, out = A B^T, both contracted along their rows.
//
// Each block of 128 contraction elements is a product of its own, multiplied by its rows' and
// columns' scales and added to the fp32 sums.  Two ways to that product:
//   fast   the 8-bit matrix instruction, one for 128 elements.  It aligns the products of a
//          step to the largest one and drops what lies some 17 bits below: far below half a
//          step of a 16-bit result, and visible in an fp32 one.
//   exact  the codes decoded to bf16 in registers (every element is exact there) and four
//          16-bit matrix instructions, which keep fp32: for fp32 results, at half the rate.
#pragma once

#include <algorithm>

#include "f8.h"

namespace bitopt {

template <int AF, int BF> __device__ __forceinline__ f32x4 mfma_f8(i32x8 a, i32x8 b, f32x4 c) {
    // scale operands of zero select the instruction without scales
    return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(a, b, c, AF, BF, 0, 0, 0, 0);
}

// Waits for the wave's loads and LDS accesses, then for the workgroup.  The empty statements
// keep memory accesses on their side.
__device__ __forceinline__ void f8_barrier() {
    asm volatile("" ::: "memory");
    __builtin_amdgcn_s_waitcnt(0x70);
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
}

// Workgroup tile BM x BN, wave tile WM x WN, two LDS buffers of one block of 128 contraction
// elements: rows of 128 bytes, filled by direct loads while the other buffer is multiplied, one
// barrier a block.  A wave's load fills 1024 consecutive bytes of LDS, so the swizzle that spreads
// a fragment's rows over the banks -- 16-byte chunk c of row r lies at chunk c ^ (r % 8) -- is
// applied to the source address.  A lane holds row l % 16 and chunks q and q + 4, q = l / 16, of
// either operand: which elements those are does not matter to the sum, as long as both agree.
template <int AF, int BF, bool BTILES, bool EXACT, int BM, int BN, int WM, int WN>
__global__ __launch_bounds__((BM / WM) * (BN / WN) * 64) void k_f8_gemm(F8GemmArgs g) {
    constexpr int NT = (BM / WM) * (BN / WN) * 64, FM = WM / 16, FN = WN / 16;
    constexpr int STAGE = (BM + BN) * 128, PASS_ROWS = NT / 8, LOADS = (BM + BN) / PASS_ROWS;
    constexpr int SCALES = (BM + (BTILES ? 0 : BN)) * 4;
    static_assert(BM % PASS_ROWS == 0 && BN % PASS_ROWS == 0 && PASS_ROWS % 8 == 0, "whole passes per operand");
    static_assert(BM + BN <= NT && kF8Block % WN == 0, "a scale for each thread at most; a wave's columns in one tile");
    __shared__ __attribute__((aligned(16))) char lds[2 * STAGE + 2 * SCALES];

    int tm, tn;
    mx_tile((g.M + BM - 1) / BM, (g.N + BN - 1) / BN, tm, tn);
    const int m0 = tm * BM, n0 = tn * BN;
    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int wm = wave % (BM / WM) * WM, wn = wave / (BM / WM) * WN;
    const int q = lane >> 4, li = lane & 15;
    const int steps = (int)f8_blocks(g.K);

    // this lane's part of pass i, from the tile's first byte of a block: rows beyond the matrix
    // repeat its last row
    const int pr = tid >> 3, chunk = (tid & 7) ^ (pr & 7);
    const uint8_t* a_next = g.a + (int64_t)m0 * g.row_bytes;
    const uint8_t* b_next = g.b + (int64_t)n0 * g.row_bytes;
    uint32_t off[LOADS];
#pragma unroll
    for (int i = 0; i < LOADS; ++i) {
        const int r = i * PASS_ROWS + pr;
        off[i] = (uint32_t)(i * PASS_ROWS < BM ? min(r, g.M - 1 - m0) : min(r - BM, g.N - 1 - n0)) * (uint32_t)g.row_bytes +
                 chunk * 16;
    }
    const float* s_next = tid < BM ? g.a_scales + min(m0 + tid, g.M - 1) : g.b_scales + min(n0 + tid - BM, g.N - 1);
    const int64_t s_step = tid < BM ? g.M : g.N;
    auto issue = [&](int buffer) {
#pragma unroll
        for (int i = 0; i < LOADS; ++i)
            __builtin_amdgcn_global_load_lds(
                (const BITOPT_GLOBAL void*)((i * PASS_ROWS < BM ? a_next : b_next) + off[i]),
                (__attribute__((address_space(3))) void*)(lds + buffer * STAGE + i * NT * 16 + wave * 1024), 16, 0, 0);
        if (wave * 256 < SCALES)
            __builtin_amdgcn_global_load_lds(
                (const BITOPT_GLOBAL void*)s_next,
                (__attribute__((address_space(3))) void*)(lds + 2 * STAGE + buffer * SCALES + wave * 256), 4, 0, 0);
        a_next += kF8Block;
        b_next += kF8Block;
        s_next += s_step;
    };
    // the wave's columns lie in one tile of 128; beyond the last, one whose results are not stored
    const float* b_tile = g.b_scales + (int64_t)min((n0 + wn) / kF8Block, (g.N - 1) / kF8Block) * steps;

    f32x4 acc[FM][FN];
#pragma unroll
    for (int i = 0; i < FM; ++i)
#pragma unroll
        for (int j = 0; j < FN; ++j) acc[i][j] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};

    if (steps > 0) {
        issue(0);
        f8_barrier();
    }
    for (int t = 0; t < steps; ++t) {
        const int buffer = t & 1;
        if (t + 1 < steps) issue(buffer ^ 1);
        const char* cur = lds + buffer * STAGE + li * 128;
        const float* sc = reinterpret_cast<const float*>(lds + 2 * STAGE + buffer * SCALES);
        const int lo = (q ^ (li & 7)) << 4, hi = ((q + 4) ^ (li & 7)) << 4;
        auto read = [&](int row, u32x4& x, u32x4& y) {
            x = *reinterpret_cast<const u32x4*>(cur + row * 128 + lo);
            y = *reinterpret_cast<const u32x4*>(cur + row * 128 + hi);
        };
        float tile = 0.0f;
        f32x4 sb[BTILES ? 1 : FN];
        if constexpr (BTILES) {
            tile = b_tile[t];
        } else {
#pragma unroll
            for (int j = 0; j < FN; ++j) sb[j] = *reinterpret_cast<const f32x4*>(sc + BM + wn + 16 * j + 4 * q);
        }
        u32x4 bx[FN], by[FN];
#pragma unroll
        for (int j = 0; j < FN; ++j) read(BM + wn + 16 * j, bx[j], by[j]);
        u32x4 bh[EXACT ? FN : 1][4];
        if constexpr (EXACT) {
#pragma unroll
            for (int j = 0; j < FN; ++j) {
                bh[j][0] = f8_half8<BF>(bx[j].x, bx[j].y); bh[j][1] = f8_half8<BF>(bx[j].z, bx[j].w);
                bh[j][2] = f8_half8<BF>(by[j].x, by[j].y); bh[j][3] = f8_half8<BF>(by[j].z, by[j].w);
            }
        }
#pragma unroll
        for (int i = 0; i < FM; ++i) {
            u32x4 ax, ay;
            read(wm + 16 * i, ax, ay);
            float sa = sc[wm + 16 * i + li];
            if constexpr (BTILES) sa *= tile;
            u32x4 ah[4];
            if constexpr (EXACT) {
                ah[0] = f8_half8<AF>(ax.x, ax.y); ah[1] = f8_half8<AF>(ax.z, ax.w);
                ah[2] = f8_half8<AF>(ay.x, ay.y); ah[3] = f8_half8<AF>(ay.z, ay.w);
            }
            // B first: a lane then holds four consecutive columns of one output row
#pragma unroll
            for (int j = 0; j < FN; ++j) {
                f32x4 p = {0.0f, 0.0f, 0.0f, 0.0f};
                if constexpr (EXACT) {
#pragma unroll
                    for (int h = 0; h < 4; ++h) p = mfma16<kBF16>(bh[j][h], ah[h], p);
                } else {
                    const i32x8 x = {(int)bx[j].x, (int)bx[j].y, (int)bx[j].z, (int)bx[j].w,
                                     (int)by[j].x, (int)by[j].y, (int)by[j].z, (int)by[j].w};
                    const i32x8 y = {(int)ax.x, (int)ax.y, (int)ax.z, (int)ax.w, (int)ay.x, (int)ay.y, (int)ay.z, (int)ay.w};
                    p = mfma_f8<BF, AF>(x, y, p);
                }
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    if constexpr (BTILES) acc[i][j][r] = __builtin_fmaf(p[r], sa, acc[i][j][r]);
                    else acc[i][j][r] = __builtin_fmaf(p[r], sa * sb[j][r], acc[i][j][r]);
                }
            }
        }
        // the next block has to be there, and every wave to have read this one
        f8_barrier();
    }
#pragma unroll
    for (int i = 0; i < FM; ++i) {
        const int m = m0 + wm + 16 * i + li;
#pragma unroll
        for (int j = 0; j < FN; j += 2) mx_store_pair(g, m, n0 + wn + 16 * j, q, acc[i][j], acc[i][j + 1]);
    }
}

// ------------------------------------------------------------------------ tile choice

template <int AF, int BF, bool BTILES, bool EXACT> hipError_t f8_tiled(const F8GemmArgs& g, hipStream_t s) {
    auto tiles = [&](int t) { return ((int64_t)g.M + t - 1) / t * (((int64_t)g.N + t - 1) / t); };
    if (tiles(256) >= 192)
        hipLaunchKernelGGL((k_f8_gemm<AF, BF, BTILES, EXACT, 256, 256, 128, 64>), dim3((unsigned)tiles(256)), dim3(512), 0, s, g);
    else if (tiles(128) >= 160)
        hipLaunchKernelGGL((k_f8_gemm<AF, BF, BTILES, EXACT, 128, 128, 64, 32>), dim3((unsigned)tiles(128)), dim3(512), 0, s, g);
    else
        hipLaunchKernelGGL((k_f8_gemm<AF, BF, BTILES, EXACT, 64, 64, 32, 32>), dim3((unsigned)tiles(64)), dim3(256), 0, s, g);
    return hipGetLastError();
}

template <bool EXACT> hipError_t f8_product(const F8GemmArgs& g, int a_fmt, int b_fmt, int b_blocks, hipStream_t s) {
    const bool a4 = a_fmt == kF8E4M3, b4 = b_fmt == kF8E4M3, t = b_blocks == kF8Tiles;
    if (a4 && b4) return t ? f8_tiled<0, 0, true, EXACT>(g, s) : f8_tiled<0, 0, false, EXACT>(g, s);
    if (b4) return t ? f8_tiled<1, 0, true, EXACT>(g, s) : f8_tiled<1, 0, false, EXACT>(g, s);
    if (a4) return t ? f8_tiled<0, 1, true, EXACT>(g, s) : f8_tiled<0, 1, false, EXACT>(g, s);
    return t ? f8_tiled<1, 1, true, EXACT>(g, s) : f8_tiled<1, 1, false, EXACT>(g, s);
}

}  // namespace bitopt
