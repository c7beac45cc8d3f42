// mx_gemm.h -- tiled products with MX operands on the matrix cores.
//
// k_mx_gemm16: out = A B^T with 16-bit matrix instructions.  A is a 16-bit matrix or an
// MX matrix, B an MX matrix; codes are decoded to 16 bits on their way into LDS, once per
// workgroup, so the inner loop is that of an ordinary 16-bit product.
// k_mx_gemm4: both operands E2M1, fed to the scaled matrix instruction as codes.
//
// An operand lies "along" when the contraction index runs along its rows in memory (a
// lane's eight contraction elements are one 16-byte LDS read) and "across" when its rows
// are the contraction index (the LDS transpose read gathers a lane's four elements of a
// column from four rows).  The three products of a linear layer y = x W^T:
//   forward       y[t][n]  = sum_k x[t][k] W[n][k]     A along,  B along
//   input grad    dx[t][k] = sum_n dy[t][n] W[n][k]    A along,  B across
//   weight grad   dw[n][k] = sum_t dy[t][n] x[t][k]    A across, B across
#pragma once

#include <type_traits>

#include "mx.h"

namespace bitopt {

enum MxSource { kAlong16, kAcross16, kAlongE2M1, kAlongE4M3, kAcrossE2M1, kAcrossE4M3 };

constexpr bool mx_is_along(int s) { return s == kAlong16 || s == kAlongE2M1 || s == kAlongE4M3; }
constexpr bool mx_is_codes(int s) { return s >= kAlongE2M1; }
constexpr bool mx_is_4bit(int s) { return s == kAlongE2M1 || s == kAcrossE2M1; }

constexpr int kGemmK = 64;      // contraction elements per LDS stage of the 16-bit product

// One operand's way from global memory to LDS: R rows (columns, if across) by kGemmK
// contraction elements of 16 bits.
//
// LDS image, along: R rows of 128 bytes; 16-byte chunk c of row r is stored at chunk
// c ^ (r & 7), so the 16 rows of a fragment read fall on different banks.  Across: kGemmK
// rows of 2R bytes; 32-byte segment s of row k is stored at segment s ^ f(k), f of the four
// rows and two row groups that one transpose read touches, for the same reason.
template <int DT, int SRC, int R, int NT> struct MxStage {
    static constexpr bool along = mx_is_along(SRC), codes = mx_is_codes(SRC), four = mx_is_4bit(SRC);
    // elements per thread item: one 16-byte load
    static constexpr int EL = !codes ? 8 : (four ? 32 : 16);
    static constexpr int PER_ROW = (along ? kGemmK : R) / EL;
    static constexpr int ITEMS = PER_ROW * (along ? R : kGemmK);
    static constexpr int N = (ITEMS + NT - 1) / NT;
    static constexpr int BYTES = R * kGemmK * 2;
    static_assert(PER_ROW >= 1, "tile narrower than an item");

    u32x4 raw[N];
    float scale[codes ? N : 1];

    static __device__ __forceinline__ int swizzle(int k) { return (k & 3) | (R >= 128 ? ((k >> 3) & 1) << 2 : 0); }

    // r0: first row (column) of the tile, k0: first contraction element.
    __device__ __forceinline__ void load(const void* base, int64_t ld, const uint8_t* sc, int64_t ld_sc, int rows, int K,
                                         int r0, int k0, int tid) {
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const int idx = i * NT + tid;
            const int a = idx / PER_ROW, b = idx % PER_ROW * EL;
            raw[i] = u32x4{0u, 0u, 0u, 0u};
            if constexpr (codes) scale[i] = 0.0f;
            if (ITEMS % NT != 0 && idx >= ITEMS) continue;
            // memory row and first element of the item
            const int64_t row = along ? min(r0 + a, rows - 1) : k0 + a;
            const int col = (along ? k0 : r0) + b;
            if constexpr (!codes) {
                // elements left in the row: beyond it, and on rows past the contraction, zero
                const int left = along ? K - col : (row < K ? rows - col : 0);
                if (left > 0)
                    raw[i] = ld_half8(reinterpret_cast<const uint16_t*>(base) + row * ld + col, left);
            } else {
                // rows of codes are padded with zeros to 128 elements
                const int width = (int)mx_padded(along ? K : rows);
                if (col < width && (along || row < K)) {
                    raw[i] = *gbl(reinterpret_cast<const u32x4*>(reinterpret_cast<const uint8_t*>(base) + row * ld +
                                                                (four ? col / 2 : col)));
                    scale[i] = mx_scale_f32(gbl(sc)[row * ld_sc + col / kMxBlock]);
                }
            }
        }
    }

    __device__ __forceinline__ void store(char* lds, int tid) const {
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const int idx = i * NT + tid;
            const int a = idx / PER_ROW, b = idx % PER_ROW * EL;
            if (ITEMS % NT != 0 && idx >= ITEMS) continue;
#pragma unroll
            for (int h = 0; h < EL / 8; ++h) {
                u32x4 v;
                if constexpr (!codes) v = raw[i];
                else if constexpr (four) v = mx_half8_e2m1<DT>(raw[i][h], scale[i]);
                else v = mx_half8_e4m3<DT>(raw[i][2 * h], raw[i][2 * h + 1], scale[i]);
                const int c = b / 8 + h;            // 16-byte chunk of the row
                const int at = along ? a * (kGemmK * 2) + ((c ^ (a & 7)) << 4)
                                     : a * (R * 2) + (((c >> 1) ^ swizzle(a)) << 5) + ((c & 1) << 4);
                *reinterpret_cast<u32x4*>(lds + at) = v;
            }
        }
    }

    // Fragment of rows r .. r+15 and contraction elements 32 ks .. 32 ks + 31: lane l holds
    // row l % 16, elements 8 (l / 16) .. + 7.
    static __device__ __forceinline__ u32x4 fragment(const char* lds, int r, int ks, int lane) {
        const int i = lane & 15, q = lane >> 4;
        if constexpr (along) {
            const int row = r + i;
            return *reinterpret_cast<const u32x4*>(lds + row * (kGemmK * 2) + (((ks * 4 + q) ^ (row & 7)) << 4));
        } else {
            typedef short s16x4 __attribute__((ext_vector_type(4)));
            typedef __attribute__((address_space(3))) s16x4* lds_ptr;
            const int k = ks * 32 + q * 8 + (i >> 2);
            const char* p = lds + k * (R * 2) + (((r >> 4) ^ swizzle(k)) << 5) + ((i & 3) << 3);
            const s16x4 lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_ptr)p);
            const s16x4 hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_ptr)(p + 4 * (R * 2)));
            const u32x2 a = __builtin_bit_cast(u32x2, lo), b = __builtin_bit_cast(u32x2, hi);
            return u32x4{a.x, a.y, b.x, b.y};
        }
    }
};

// Workgroup tile BM x BN, wave tile WM x WN.
template <int DT, int ASRC, int BSRC, int BM, int BN, int WM, int WN>
__global__ __launch_bounds__((BM / WM) * (BN / WN) * 64) void k_mx_gemm16(MxGemmArgs g) {
    constexpr int NT = (BM / WM) * (BN / WN) * 64, FM = WM / 16, FN = WN / 16;
    using SA = MxStage<DT, ASRC, BM, NT>;
    using SB = MxStage<DT, BSRC, BN, NT>;
    constexpr int STAGE = SA::BYTES + SB::BYTES;
    __shared__ __attribute__((aligned(16))) char lds[2 * STAGE];

    int tm, tn;
    mx_tile((g.M + BM - 1) / BM, (g.N + BN - 1) / BN, tm, tn);
    const int m0 = tm * BM, n0 = tn * BN;
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const int wm = wave % (BM / WM) * WM, wn = wave / (BM / WM) * WN;
    const int64_t lda = SA::codes ? g.a_row_bytes : g.lda;

    SA sa;
    SB sb;
    f32x4 acc[FM][FN];
#pragma unroll
    for (int i = 0; i < FM; ++i)
#pragma unroll
        for (int j = 0; j < FN; ++j) acc[i][j] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};

    const int steps = (g.K + kGemmK - 1) / kGemmK;
    sa.load(g.a, lda, g.a_scales, g.a_row_scales, g.M, g.K, m0, 0, tid);
    sb.load(g.b, g.b_row_bytes, g.b_scales, g.b_row_scales, g.N, g.K, n0, 0, tid);
    sa.store(lds, tid);
    sb.store(lds + SA::BYTES, tid);
    __syncthreads();
    for (int t = 0; t < steps; ++t) {
        const char* cur = lds + (t & 1) * STAGE;
        if (t + 1 < steps) {
            sa.load(g.a, lda, g.a_scales, g.a_row_scales, g.M, g.K, m0, (t + 1) * kGemmK, tid);
            sb.load(g.b, g.b_row_bytes, g.b_scales, g.b_row_scales, g.N, g.K, n0, (t + 1) * kGemmK, tid);
        }
#pragma unroll
        for (int ks = 0; ks < kGemmK / 32; ++ks) {
            u32x4 fa[FM], fb[FN];
#pragma unroll
            for (int i = 0; i < FM; ++i) fa[i] = SA::fragment(cur, wm + 16 * i, ks, lane);
#pragma unroll
            for (int j = 0; j < FN; ++j) fb[j] = SB::fragment(cur + SA::BYTES, wn + 16 * j, ks, lane);
            // B first: a lane then holds four consecutive columns of one output row
#pragma unroll
            for (int i = 0; i < FM; ++i)
#pragma unroll
                for (int j = 0; j < FN; ++j) acc[i][j] = mfma16<DT>(fb[j], fa[i], acc[i][j]);
        }
        if (t + 1 < steps) {
            // the other buffer was last read before the barrier that ended step t - 1
            char* next = lds + ((t + 1) & 1) * STAGE;
            sa.store(next, tid);
            sb.store(next + SA::BYTES, tid);
            __syncthreads();
        }
    }
#pragma unroll
    for (int i = 0; i < FM; ++i) {
        const int m = m0 + wm + 16 * i + (lane & 15);
#pragma unroll
        for (int j = 0; j < FN; j += 2) mx_store_pair(g, m, n0 + wn + 16 * j, lane >> 4, acc[i][j], acc[i][j + 1]);
    }
}

// ------------------------------------------------------------------ both operands E2M1

// Codes go from global memory straight to LDS in two stages of 256 contraction elements in
// turn: 128 bytes of codes a row, a whole cache line (stages of 64 bytes a row fetched
// lines twice).  A stage is multiplied in two steps of 128.  While the fragments of one step
// are multiplied, those of the next are read from LDS; when the second step of a stage
// begins, all of the stage is in registers and the stage after the next is asked for into
// its buffer, two steps before it is needed.  That is one barrier per stage.  A wave's load
// fills 1024 consecutive bytes of LDS, so the swizzle that spreads a fragment's rows over
// the banks -- 16-byte chunk c of row r lies at chunk c ^ (r % 8) -- is applied to the source
// address.
//
// Scales never touch LDS.  Lane (row i, group q) loads the four scale bytes of its row in
// step q of a group of four steps; a byte transpose across the four lane groups leaves it
// with the bytes of its own block in all four steps, and the matrix instruction selects
// byte t itself.

constexpr int kGemm4K = 128;

// Waits until at most N of the wave's global loads are outstanding and its LDS reads are
// done, then for the workgroup.  The empty statements keep memory accesses on their side.
template <int N> __device__ __forceinline__ void stage_barrier() {
    asm volatile("" ::: "memory");
    __builtin_amdgcn_s_waitcnt((N & 15) | 0x70 | ((N >> 4) << 14));
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
}

template <int BM, int BN, int WM, int WN>
__global__ __launch_bounds__((BM / WM) * (BN / WN) * 64) void k_mx_gemm4(MxGemmArgs g) {
    constexpr int NT = (BM / WM) * (BN / WN) * 64, FM = WM / 16, FN = WN / 16;
    constexpr int STAGE = (BM + BN) * 128, PASS_ROWS = NT / 8, LOADS = (BM + BN) / PASS_ROWS;
    static_assert(BM % PASS_ROWS == 0 && BN % PASS_ROWS == 0 && PASS_ROWS % 8 == 0, "whole passes per operand");
    __shared__ __attribute__((aligned(16))) char lds[2 * STAGE];

    int tm, tn;
    mx_tile((g.M + BM - 1) / BM, (g.N + BN - 1) / BN, tm, tn);
    const int m0 = tm * BM, n0 = tn * BN;
    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int wm = wave % (BM / WM) * WM, wn = wave / (BM / WM) * WN;
    const int q = lane >> 4, li = lane & 15;
    const int steps = (int)(mx_padded(g.K) / kGemm4K);

    // this lane's source of pass i in stage 0: rows beyond the matrix repeat its last row
    const int pr = tid >> 3, chunk = (tid & 7) ^ (pr & 7);
    const uint8_t* src[LOADS];
#pragma unroll
    for (int i = 0; i < LOADS; ++i) {
        const int r = i * PASS_ROWS + pr;
        src[i] = i * PASS_ROWS < BM
                     ? reinterpret_cast<const uint8_t*>(g.a) + (int64_t)min(m0 + r, g.M - 1) * g.a_row_bytes + chunk * 16
                     : g.b + (int64_t)min(n0 + r - BM, g.N - 1) * g.b_row_bytes + chunk * 16;
    }
    // t: the stage's first step
    auto issue = [&](int t, int buffer) {
        // a last stage of one step: its second half repeats the first and is not multiplied
        const int back = t + 1 < steps || chunk < 4 ? 0 : 64;
#pragma unroll
        for (int i = 0; i < LOADS; ++i)
            __builtin_amdgcn_global_load_lds((const BITOPT_GLOBAL void*)(src[i] + ((int64_t)t * 64 - back)),
                                             (__attribute__((address_space(3))) void*)(lds + buffer * STAGE +
                                                                                       i * NT * 16 + wave * 1024),
                                             16, 0, 0);
    };

    // scale bytes of the fragments' rows, four steps at a time (rows of them hold a multiple of 4)
    const uint8_t* sa0 = g.a_scales + (int64_t)m0 * g.a_row_scales;
    const uint8_t* sb0 = g.b_scales + (int64_t)n0 * g.b_row_scales;
    auto scales = [&](int step, uint32_t xa[FM], uint32_t xb[FN]) {
        const int t = min(step + q, steps - 1);     // bytes of steps that are not taken are not looked at
#pragma unroll
        for (int i = 0; i < FM; ++i) {
            const uint32_t r = (uint32_t)min(wm + 16 * i + li, g.M - 1 - m0);
            xa[i] = *gbl(reinterpret_cast<const uint32_t*>(sa0 + (r * (uint32_t)g.a_row_scales + 4 * t)));
        }
#pragma unroll
        for (int j = 0; j < FN; ++j) {
            const uint32_t r = (uint32_t)min(wn + 16 * j + li, g.N - 1 - n0);
            xb[j] = *gbl(reinterpret_cast<const uint32_t*>(sb0 + (r * (uint32_t)g.b_row_scales + 4 * t)));
        }
    };

    f32x4 acc[FM][FN];
#pragma unroll
    for (int i = 0; i < FM; ++i)
#pragma unroll
        for (int j = 0; j < FN; ++j) acc[i][j] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};

    struct Fragments {
        u32x4 a[FM], b[FN];
    };
    auto read = [&](int buffer, int half, Fragments& f) {
        const char* cur = lds + buffer * STAGE + li * 128 + (((half * 4 + q) ^ (li & 7)) << 4);
#pragma unroll
        for (int j = 0; j < FN; ++j) f.b[j] = *reinterpret_cast<const u32x4*>(cur + (BM + wn + 16 * j) * 128);
#pragma unroll
        for (int i = 0; i < FM; ++i) f.a[i] = *reinterpret_cast<const u32x4*>(cur + (wm + 16 * i) * 128);
    };

    if (steps > 0) issue(0, 0);
    if (steps > 2) issue(2, 1);
    uint32_t xa[FM], xb[FN], ya[FM], yb[FN];
    Fragments even, odd;
    if (steps > 0) {
        scales(0, xa, xb);
        stage_barrier<0>();
        read(0, 0, even);
    }
    for (int t0 = 0; t0 < steps; t0 += 4) {
#pragma unroll
        for (int i = 0; i < FM; ++i) ya[i] = transpose_bytes(xa[i], lane);
#pragma unroll
        for (int j = 0; j < FN; ++j) yb[j] = transpose_bytes(xb[j], lane);
        auto step = [&](auto byte, const Fragments& cur, Fragments& next) {
            constexpr int B = decltype(byte)::value;
            const int t = t0 + B;
            if (t >= steps) return;
            if constexpr (B & 1) {
                // the next stage has to be there, and every wave to have read this one
                stage_barrier<0>();
                if (t + 3 < steps) issue(t + 3, B >> 1);
                if constexpr (B == 1) scales(t0 + 4, xa, xb);
            }
            read((B + 1) / 2 % 2, (B + 1) % 2, next);      // after the last step: not looked at
#pragma unroll
            for (int i = 0; i < FM; ++i)
#pragma unroll
                for (int j = 0; j < FN; ++j) acc[i][j] = mfma_e2m1_at<B>(cur.b[j], cur.a[i], acc[i][j], yb[j], ya[i]);
#pragma unroll
            for (int r = 0; r < FM + FN; ++r) {
                __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);                     // one LDS read
                __builtin_amdgcn_sched_group_barrier(0x008, FM * FN / (FM + FN), 0);   // its share of products
            }
        };
        step(std::integral_constant<int, 0>{}, even, odd);
        step(std::integral_constant<int, 1>{}, odd, even);
        step(std::integral_constant<int, 2>{}, even, odd);
        step(std::integral_constant<int, 3>{}, odd, even);
    }
#pragma unroll
    for (int i = 0; i < FM; ++i) {
        const int m = m0 + wm + 16 * i + li;
#pragma unroll
        for (int j = 0; j < FN; j += 2) mx_store_pair(g, m, n0 + wn + 16 * j, q, acc[i][j], acc[i][j + 1]);
    }
}

// ------------------------------------------------------------------------ tile choice

// Launches `big` (256 x 256 tiles), `mid` (128 x 128) or `small` (64 x 64): the largest
// tile whose grid still gives the 256 CUs about one workgroup each.
template <class Big, class Mid, class Small>
hipError_t mx_by_tile(const MxGemmArgs& g, Big big, Mid mid, Small small) {
    auto tiles = [&](int t) { return ((int64_t)g.M + t - 1) / t * (((int64_t)g.N + t - 1) / t); };
    if (tiles(256) >= 192) return big(dim3((unsigned)tiles(256)));
    if (tiles(128) >= 160) return mid(dim3((unsigned)tiles(128)));
    return small(dim3((unsigned)tiles(64)));
}

template <int DT, int ASRC, int BSRC> hipError_t mx_gemm16(const MxGemmArgs& g, hipStream_t s) {
    return mx_by_tile(
        g,
        [&](dim3 grid) {
            hipLaunchKernelGGL((k_mx_gemm16<DT, ASRC, BSRC, 256, 256, 128, 64>), grid, dim3(512), 0, s, g);
            return hipGetLastError();
        },
        [&](dim3 grid) {
            hipLaunchKernelGGL((k_mx_gemm16<DT, ASRC, BSRC, 128, 128, 64, 64>), grid, dim3(256), 0, s, g);
            return hipGetLastError();
        },
        [&](dim3 grid) {
            hipLaunchKernelGGL((k_mx_gemm16<DT, ASRC, BSRC, 64, 64, 32, 32>), grid, dim3(256), 0, s, g);
            return hipGetLastError();
        });
}

}  // namespace bitopt
