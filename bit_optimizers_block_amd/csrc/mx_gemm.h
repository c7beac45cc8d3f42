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

// One operand's way from global memory through registers to LDS: R rows (columns, if
// across) by kGemmK contraction elements of 16 bits.
//
// LDS image, along: R rows of 128 bytes; 16-byte chunk c of row r is stored at chunk
// c ^ (r & 7), so the 16 rows of a fragment read fall on different banks.  Across: kGemmK
// rows of 2R bytes and 32 of padding, so the four rows of a transpose read do (a swizzle of
// the segments does the same, but costs a register of addresses for every fragment).
template <int DT, int SRC, int R, int NT, bool WHOLE> struct MxStage {
    static constexpr bool along = mx_is_along(SRC), codes = mx_is_codes(SRC), four = mx_is_4bit(SRC);
    // elements per thread item: one 16-byte load, or one of 8 where a small tile's 4-bit codes
    // would leave half of the workgroup without
    static constexpr bool HALF = four && R * kGemmK / 32 < NT;
    static constexpr int EL = !codes ? 8 : (four && !HALF ? 32 : 16);
    static constexpr int PER_ROW = (along ? kGemmK : R) / EL;
    static constexpr int ITEMS = PER_ROW * (along ? R : kGemmK);
    static constexpr int N = (ITEMS + NT - 1) / NT;
    static constexpr int PIECES = N * EL / 8;           // 16-byte LDS writes of a thread
    static constexpr int PITCH = along ? kGemmK * 2 : R * 2 + 32;
    static constexpr int BYTES = PITCH * (along ? R : kGemmK);
    static_assert(PER_ROW >= 1, "tile narrower than an item");

    // Offsets of this thread's items from the tile's first byte of a stage, where they fit 32
    // bits; otherwise, and where a stage reaches over an edge, load_any() is taken.  Across,
    // item i lies a uniform distance behind item 0; along, rows beyond the last repeat it.
    static constexpr int OFFS = along ? N : 1;
    static constexpr int ROWS = NT / PER_ROW;           // memory rows from an item to the next
    static_assert(along || N == 1 || NT % PER_ROW == 0, "items of a thread in one column");
    // Across, an item's scale byte is loaded with it.  Along, scale bytes go to LDS by direct
    // loads, eight stages (16 bytes a row) at a time: loaded with the items, a byte each, every
    // two or four lanes are an access to another row, which cost as much as the codes
    // themselves.
    static constexpr bool own_scales = codes && !along;
    static constexpr int SCALES = codes && along ? R * 16 : 0;
    // WHOLE: every stage of every tile lies inside the operand and its offsets fit, so nothing is
    // looked at on the way.  Otherwise a stage over an edge takes load_any().  Along, that is the
    // last stage only, and its items are shifted as they are loaded.  Across, a ragged tile has
    // one in every stage: an item is one load of the row's last eight elements at most, and
    // store() shifts it and zeroes what lies beyond, so the load stays in flight.
    static constexpr bool SHIFTS = !codes && !along && !WHOLE;
    int span;               // elements of a memory row from the tile's first (across)
    uint32_t off[OFFS], soff;
    u32x4 raw[N];
    uint32_t scale[own_scales ? N : 1];

    static __device__ __forceinline__ u32x4 ld_codes(const uint8_t* p) {
        if constexpr (HALF) {
            const u32x2 v = *gbl(reinterpret_cast<const u32x2*>(p));
            return u32x4{v.x, v.y, 0u, 0u};
        } else {
            return *gbl(reinterpret_cast<const u32x4*>(p));
        }
    }
    // rows: the operand's rows (columns, if across); r0: the tile's first
    __device__ __forceinline__ void init(int64_t ld, int64_t ld_sc, int rows, int r0, int tid) {
        span = rows - r0;
#pragma unroll
        for (int i = 0; i < OFFS; ++i) {
            const int idx = min(i * NT + tid, ITEMS - 1);
            const int a = idx / PER_ROW;
            int b = idx % PER_ROW * EL;
            if constexpr (SHIFTS) b = max(0, min(b, rows - r0 - 8));
            const uint32_t row = along ? (uint32_t)min(a, rows - 1 - r0) : (uint32_t)a;
            off[i] = row * (uint32_t)(codes ? ld : 2 * ld) + (codes ? (four ? b / 2 : b) : 2 * b);
            if constexpr (own_scales) soff = row * (uint32_t)ld_sc + b / kMxBlock;
        }
    }
    // Whether every stage of every tile is inside().
    static bool whole(int64_t ld, int64_t rows, int64_t K) {
        if (ld >= (1 << 22)) return false;
        if (along) return codes || K % kGemmK == 0;
        return K % kGemmK == 0 && (rows + R - 1) / R * R <= (codes ? mx_padded(rows) : rows);
    }
    // Whether the stage from k0 lies inside the operand and its offsets fit (wave-uniform).
    static __device__ __forceinline__ bool inside(int64_t ld, int rows, int K, int r0, int k0) {
        if (ld >= (1 << 22)) return false;
        if (along) return codes || k0 + kGemmK <= K;
        return k0 + kGemmK <= K && (codes ? r0 + R <= (int)mx_padded(rows) : rows - r0 >= 8);
    }
    __device__ __forceinline__ void load_inside(const void* base, int64_t ld, const uint8_t* sc, int64_t ld_sc, int r0,
                                                int k0) {
        const int64_t row = along ? r0 : k0, col = along ? k0 : r0;
        const uint8_t* p = reinterpret_cast<const uint8_t*>(base) + row * (codes ? ld : 2 * ld) +
                           (codes ? (four ? col / 2 : col) : 2 * col);
        const int64_t next = along ? 0 : ROWS * (codes ? ld : 2 * ld);
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const uint8_t* q = p + i * next + off[along ? i : 0];
            if constexpr (codes) raw[i] = ld_codes(q);
            else raw[i] = ld16_a2(q);
        }
        if constexpr (own_scales) {
            const uint8_t* s = sc + row * ld_sc + col / kMxBlock;
#pragma unroll
            for (int i = 0; i < N; ++i) scale[i] = gbl(s + i * ROWS * ld_sc)[soff];
        }
    }
    __device__ __forceinline__ void load_any(const void* base, int64_t ld, const uint8_t* sc, int64_t ld_sc, int rows,
                                             int K, int r0, int k0, int tid) {
#pragma unroll
        for (int i = 0; i < N; ++i) {
            // computed here each time: ahead of the loop, the addresses of all items would take
            // registers in every stage
            int idx = i * NT + tid;
            asm volatile("" : "+v"(idx));
            const int a = idx / PER_ROW, b = idx % PER_ROW * EL;
            raw[i] = u32x4{0u, 0u, 0u, 0u};
            if constexpr (own_scales) scale[i] = 0u;
            if (ITEMS % NT != 0 && idx >= ITEMS) continue;
            // memory row and first element of the item
            const int64_t row = along ? min(r0 + a, rows - 1) : k0 + a;
            const int col = (along ? k0 : r0) + b;
            if constexpr (!codes) {
                const uint16_t* p = reinterpret_cast<const uint16_t*>(base) + row * ld;
                if constexpr (along) {
                    raw[i] = ld_half8(p + col, K - col, col);
                } else if (row < K) {           // rows past the contraction are zero
                    if (span >= 8) raw[i] = ld16_a2(p + min(col, rows - 8));
                    else raw[i] = ld_half8(p + col, rows - col, 0);
                }
            } else {
                // rows of codes are padded with zeros to 128 elements
                const int width = (int)mx_padded(along ? K : rows);
                if (col < width && (along || row < K)) {
                    raw[i] = ld_codes(reinterpret_cast<const uint8_t*>(base) + row * ld + (four ? col / 2 : col));
                    if constexpr (own_scales) scale[i] = gbl(sc)[row * ld_sc + col / kMxBlock];
                }
            }
        }
    }
    __device__ __forceinline__ void load(const void* base, int64_t ld, const uint8_t* sc, int64_t ld_sc, int rows, int K,
                                         int r0, int k0, int tid) {
        if (WHOLE || inside(ld, rows, K, r0, k0)) load_inside(base, ld, sc, ld_sc, r0, k0);
        else load_any(base, ld, sc, ld_sc, rows, K, r0, k0, tid);
    }

    // Scale bytes of the eight stages of group n: rows beyond the last repeat it, bytes beyond
    // a row's are not looked at.
    static __device__ __forceinline__ void issue_scales(char* lds, const uint8_t* sc, int64_t ld_sc, int rows, int r0,
                                                        int n, int tid, int wave) {
#pragma unroll
        for (int i = 0; i < R * 4 / NT; ++i) {
            const int d = i * NT + tid;
            const uint8_t* p = sc + (int64_t)min(r0 + (d >> 2), rows - 1) * ld_sc +
                               min((int64_t)n * 16 + (d & 3) * 4, ld_sc - 4);
            __builtin_amdgcn_global_load_lds((const BITOPT_GLOBAL void*)p,
                                             (__attribute__((address_space(3))) void*)(lds + i * NT * 4 + wave * 256), 4,
                                             0, 0);
        }
    }

    // Write p of this thread for stage s: eight elements, decoded on the way.
    __device__ __forceinline__ void store(char* lds, const char* scales, int tid, int s, int p) const {
        const int i = p / (EL / 8), h = p % (EL / 8);
        const int idx = i * NT + tid;
        const int a = idx / PER_ROW, c = idx % PER_ROW * (EL / 8) + h;      // row, 16-byte chunk of it
        if (ITEMS % NT != 0 && idx >= ITEMS) return;
        u32x4 v;
        if constexpr (!codes) {
            v = raw[i];
            if constexpr (SHIFTS) {
                if (span >= 8 && span < R) {
                    const int left = span - c * 8;
                    v = left >= 8 ? v : left > 0 ? half_shift(v, 8 - left) : u32x4{0u, 0u, 0u, 0u};
                }
            }
        } else {
            uint32_t b;
            if constexpr (own_scales) b = scale[i];
            else b = *reinterpret_cast<const uint8_t*>(scales + a * 16 + (s & 7) * 2 + c * 8 / kMxBlock);
            if constexpr (four) v = mx_half8_e2m1<DT>(raw[i][h], mx_scale_f32(b));
            else v = mx_half8_e4m3<DT>(raw[i][2 * h], raw[i][2 * h + 1], mx_scale_f32(b));
        }
        const int at = a * PITCH + ((along ? c ^ (a & 7) : c) << 4);
        *reinterpret_cast<u32x4*>(lds + at) = v;
    }

    // Fragment of rows r .. r+15 and contraction elements 32 ks .. 32 ks + 31: lane l holds
    // row l % 16, elements 8 (l / 16) .. + 7.
    static __device__ __forceinline__ u32x4 fragment(const char* lds, int r, int ks, int lane) {
        const int i = lane & 15, q = lane >> 4;
        if constexpr (along) {
            const int row = r + i;
            return *reinterpret_cast<const u32x4*>(lds + row * PITCH + (((ks * 4 + q) ^ (i & 7)) << 4));
        } else {
            typedef short s16x4 __attribute__((ext_vector_type(4)));
            typedef __attribute__((address_space(3))) s16x4* lds_ptr;
            const int k = ks * 32 + q * 8 + (i >> 2);
            const char* p = lds + k * PITCH + 2 * r + ((i & 3) << 3);
            const s16x4 lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_ptr)p);
            const s16x4 hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_ptr)(p + 4 * PITCH));
            const u32x2 a = __builtin_bit_cast(u32x2, lo), b = __builtin_bit_cast(u32x2, hi);
            return u32x4{a.x, a.y, b.x, b.y};
        }
    }
};

// Waits until at most N of the wave's global loads are outstanding and its LDS reads are
// done, then for the workgroup.  The empty statements keep memory accesses on their side.
template <int N> __device__ __forceinline__ void stage_barrier() {
    asm volatile("" ::: "memory");
    __builtin_amdgcn_s_waitcnt((N & 15) | 0x70 | ((N >> 4) << 14));
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
}

// Waits for the wave's LDS accesses, then for the workgroup; global loads stay in flight.
// The empty statements keep memory accesses on their side.
__device__ __forceinline__ void lds_barrier() {
    asm volatile("" ::: "memory");
    __builtin_amdgcn_s_waitcnt(0xC07F);
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
}

// Workgroup tile BM x BN, wave tile WM x WN.  Two LDS buffers of one stage of 64 contraction
// elements.  While a stage is multiplied, the next one, whose loads were sent a stage before,
// is decoded and written to the other buffer between the products, and the loads of the one
// after that are sent; the barrier that ends a stage leaves them in flight.
//
// Bound: no unit alone.  A 256 x 256 tile on eight waves of 128 x 64 moves 96 KB of fragments and
// 32 KB of writes through LDS per 32 contraction elements, against 1024 cycles of products;
// counters show the matrix pipes busy 51% of the cycles and LDS 34% (57% in the gradients, whose
// transpose reads conflict on banks), the rest is waits that two waves a SIMD do not fill.
// Measured at 8192 x 8192 x 2048, bf16 and E2M1: input grad 203 us (1350 TFLOP/s), weight grad
// 215 us, forward 212 us; E4M3: 209, 208 and 221.  Earlier forms: the next stage written after the
// products 304, 316, 314; four waves of 128 x 128, whose LDS traffic is a quarter less, which leave
// one wave a SIMD and too few registers, 360, 499, 322.
template <int DT, int ASRC, int BSRC, int BM, int BN, int WM, int WN, bool WHOLE>
__global__ __launch_bounds__((BM / WM) * (BN / WN) * 64) void k_mx_gemm16(MxGemmArgs g) {
    constexpr int NT = (BM / WM) * (BN / WN) * 64, FM = WM / 16, FN = WN / 16;
    using SA = MxStage<DT, ASRC, BM, NT, WHOLE>;
    using SB = MxStage<DT, BSRC, BN, NT, WHOLE>;
    constexpr int STAGE = SA::BYTES + SB::BYTES, SCALES = SA::SCALES + SB::SCALES;
    __shared__ __attribute__((aligned(16))) char lds[2 * STAGE + 2 * SCALES];

    int tm, tn;
    mx_tile((g.M + BM - 1) / BM, (g.N + BN - 1) / BN, tm, tn);
    const int m0 = tm * BM, n0 = tn * BN;
    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int wm = wave % (BM / WM) * WM, wn = wave / (BM / WM) * WN;
    const int64_t lda = SA::codes ? g.a_row_bytes : g.lda;
    const int stages = (g.K + kGemmK - 1) / kGemmK;

    SA sa;
    SB sb;
    sa.init(lda, g.a_row_scales, g.M, m0, tid);
    sb.init(g.b_row_bytes, g.b_row_scales, g.N, n0, tid);
    f32x4 acc[FM][FN];
#pragma unroll
    for (int i = 0; i < FM; ++i)
#pragma unroll
        for (int j = 0; j < FN; ++j) acc[i][j] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};

    auto load = [&](int s) {
        if (s >= stages) return;
        sa.load(g.a, lda, g.a_scales, g.a_row_scales, g.M, g.K, m0, s * kGemmK, tid);
        sb.load(g.b, g.b_row_bytes, g.b_scales, g.b_row_scales, g.N, g.K, n0, s * kGemmK, tid);
    };
    constexpr int P = SA::PIECES + SB::PIECES;
    // scale bytes of stage s lie in the half of group s / 8
    auto scales_of = [&](int n) { return lds + 2 * STAGE + (n & 1) * SCALES; };
    auto issue_scales = [&](int n) {
        if constexpr (SA::SCALES > 0) SA::issue_scales(scales_of(n), g.a_scales, g.a_row_scales, g.M, m0, n, tid, wave);
        if constexpr (SB::SCALES > 0)
            SB::issue_scales(scales_of(n) + SA::SCALES, g.b_scales, g.b_row_scales, g.N, n0, n, tid, wave);
    };
    auto store = [&](int buffer, int s, int p) {
        if (p < SA::PIECES) sa.store(lds + buffer * STAGE, scales_of(s >> 3), tid, s, p);
        else sb.store(lds + buffer * STAGE + SA::BYTES, scales_of(s >> 3) + SA::SCALES, tid, s, p - SA::PIECES);
    };
    struct Fragments {
        u32x4 a[FM], b[FN];
    };
    // fragment r of a step: B's, then A's
    constexpr int G = FM + FN;
    auto read = [&](int buffer, int ks, Fragments& f, int r) {
        if (r < FN) f.b[r] = SB::fragment(lds + buffer * STAGE + SA::BYTES, wn + 16 * r, ks, lane);
        else f.a[r - FN] = SA::fragment(lds + buffer * STAGE, wm + 16 * (r - FN), ks, lane);
    };
    // B first: a lane then holds four consecutive columns of one output row
    auto multiply = [&](const Fragments& f) {
#pragma unroll
        for (int i = 0; i < FM; ++i)
#pragma unroll
            for (int j = 0; j < FN; ++j) acc[i][j] = mfma16<DT>(f.b[j], f.a[i], acc[i][j]);
    };

    if (stages > 0) {
        issue_scales(0);
        load(0);
        stage_barrier<0>();
#pragma unroll
        for (int p = 0; p < P; ++p) store(0, 0, p);
        load(1);
        lds_barrier();
    }
    for (int s0 = 0; s0 < stages; s0 += 2) {
        auto stage = [&](auto buffer) {
            constexpr int B = decltype(buffer)::value;
            const int s = s0 + B;
            if (s >= stages) return;
            if constexpr (B == 0 && SCALES > 0) {
                // The other half was last read for stage s - 1.  Loads complete in order: a wave
                // that has the items it asks for below has written its part, and the barriers
                // of the stages until the group begins tell the others.
                if ((s & 7) == 0 && s + 8 < stages) {
                    issue_scales((s >> 3) + 1);
                    asm volatile("" ::: "memory");
                }
            }
            Fragments f;
#pragma unroll
            for (int r = 0; r < G; ++r) read(B, 0, f, r);
            multiply(f);
            Fragments h;
#pragma unroll
            for (int r = 0; r < G; ++r) {
                read(B, 1, h, r);
#pragma unroll
                for (int p = r * P / G; p < (r + 1) * P / G; ++p) store(B ^ 1, s + 1, p);
            }
            multiply(h);
            load(s + 2);
            lds_barrier();
        };
        stage(std::integral_constant<int, 0>{});
        stage(std::integral_constant<int, 1>{});
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
// turn: 128 bytes of codes a row, a whole cache line.  A stage is multiplied in two steps of
// 128.  Once the second step's fragments are in registers, and the barrier has said so for
// every wave and that the next stage is there, the stage after it is asked for into the
// buffer, under the products.  That is one barrier per stage.  A wave's load fills 1024
// consecutive bytes of LDS, so the swizzle that spreads a fragment's rows over the banks --
// 16-byte chunk c of row r lies at chunk c ^ (r % 8) -- is applied to the source address.
//
// Scales come by the same direct loads, eight steps (32 bytes a row) at a time.  Lane (row
// i, group q) reads the four scale bytes of its row in step q of four; a byte transpose
// across the four lane groups leaves it with the bytes of its own block in all four steps,
// and the matrix instruction selects byte t itself.  (Loaded from global memory in that
// pattern, 64 separate dwords an instruction, scales were two thirds of the cache's
// accesses: 8192 x 8192 x 8192 took 347 us.)
//
// Measured: 8192 x 8192 x 8192 262 us (4200 TFLOP/s), 8192 x 8192 x 2048 87 to 98 us, of which the
// results' stores are 16 and the steps 55: with one workgroup a CU, each of the four rounds of
// tiles begins with empty buffers and ends in 128 KB of results that nothing overlaps.  The
// matrix instructions alone reach 9500 TFLOP/s on zeros and 7000 on random codes, where the
// card's power sets the clock; here their pipes are busy 44 to 47% of the cycles, LDS 25 to 27%, and the larger
// size takes 230 us on zeros and 233 with the loads left out.  Four waves of 128 x 128 that
// read a step's fragments under the one before took 266 and 110 us; eight such waves spill.
// Reads and products of a SIMD's two waves in alternate phases, with a barrier after each: 265
// and 100 (1024 x 4096 x 4096 16 -> 18).  One resident grid with the next tile's loads ahead of
// the last one's stores took 154 us at the second size, non-temporal stores 138, against 116 at
// the time: both on earlier forms, of which the first spilled.  This one holds 208 registers of
// 256, and neither has been tried on it.

constexpr int kGemm4K = 128;

template <int BM, int BN, int WM, int WN>
__global__ __launch_bounds__((BM / WM) * (BN / WN) * 64) void k_mx_gemm4(MxGemmArgs g) {
    constexpr int NT = (BM / WM) * (BN / WN) * 64, FM = WM / 16, FN = WN / 16;
    constexpr int STAGE = (BM + BN) * 128, PASS_ROWS = NT / 8, LOADS = (BM + BN) / PASS_ROWS;
    constexpr int SCALES = (BM + BN) * 32, SCALE_LOADS = SCALES / (NT * 4);
    static_assert(BM % PASS_ROWS == 0 && BN % PASS_ROWS == 0 && PASS_ROWS % 8 == 0, "whole passes per operand");
    static_assert(SCALES % (NT * 4) == 0 && BM * 8 % NT == 0, "whole passes per operand");
    __shared__ __attribute__((aligned(16))) char lds[2 * STAGE + 2 * SCALES];

    int tm, tn;
    mx_tile((g.M + BM - 1) / BM, (g.N + BN - 1) / BN, tm, tn);
    const int m0 = tm * BM, n0 = tn * BN;
    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int wm = wave % (BM / WM) * WM, wn = wave / (BM / WM) * WN;
    const int q = lane >> 4, li = lane & 15;
    const int steps = (int)(mx_padded(g.K) / kGemm4K);

    // this lane's part of pass i, from the tile's first byte of a stage: rows beyond the
    // matrix repeat its last row
    const int pr = tid >> 3, chunk = (tid & 7) ^ (pr & 7);
    const uint8_t* a_stage = reinterpret_cast<const uint8_t*>(g.a) + (int64_t)m0 * g.a_row_bytes;
    const uint8_t* b_stage = g.b + (int64_t)n0 * g.b_row_bytes;
    uint32_t off[LOADS];
#pragma unroll
    for (int i = 0; i < LOADS; ++i) {
        const int r = i * PASS_ROWS + pr;
        off[i] = (i * PASS_ROWS < BM ? (uint32_t)min(r, g.M - 1 - m0) * (uint32_t)g.a_row_bytes
                                     : (uint32_t)min(r - BM, g.N - 1 - n0) * (uint32_t)g.b_row_bytes) + chunk * 16;
    }
    auto issue = [&](int i, int buffer, uint32_t back) {
        __builtin_amdgcn_global_load_lds(
            (const BITOPT_GLOBAL void*)((i * PASS_ROWS < BM ? a_stage : b_stage) + (off[i] - back)),
            (__attribute__((address_space(3))) void*)(lds + buffer * STAGE + i * NT * 16 + wave * 1024), 16, 0, 0);
    };
    // The source moves on while there are stages; after the last, loads repeat it into buffers
    // that are not read.  Of a last stage of one step the second half repeats the first.
    const int last = (steps - 1) & ~1;
    auto back = [&](int t) { return (steps & 1) && t >= last && chunk >= 4 ? 64u : 0u; };
    auto advance = [&](int t) {
        a_stage += t < last ? 128 : 0;
        b_stage += t < last ? 128 : 0;
    };

    // scale bytes of eight steps: lane l of a pass takes step l % 8 of row l / 8
    const uint8_t* sa0 = g.a_scales + (int64_t)m0 * g.a_row_scales;
    const uint8_t* sb0 = g.b_scales + (int64_t)n0 * g.b_row_scales;
    uint32_t soff[SCALE_LOADS];
#pragma unroll
    for (int i = 0; i < SCALE_LOADS; ++i) {
        const int r = i * PASS_ROWS + pr;
        soff[i] = i * PASS_ROWS < BM ? (uint32_t)min(r, g.M - 1 - m0) * (uint32_t)g.a_row_scales
                                     : (uint32_t)min(r - BM, g.N - 1 - n0) * (uint32_t)g.b_row_scales;
    }
    auto issue_scales = [&](int t, int buffer) {
        const uint32_t o = 4u * (uint32_t)min(t + (tid & 7), steps - 1);    // beyond the last step: not looked at
#pragma unroll
        for (int i = 0; i < SCALE_LOADS; ++i)
            __builtin_amdgcn_global_load_lds(
                (const BITOPT_GLOBAL void*)((i * PASS_ROWS < BM ? sa0 : sb0) + (soff[i] + o)),
                (__attribute__((address_space(3))) void*)(lds + 2 * STAGE + buffer * SCALES + i * NT * 4 + wave * 256), 4, 0,
                0);
    };
    // four steps from t
    auto scales = [&](int t, uint32_t ya[FM], uint32_t yb[FN]) {
        const char* cur = lds + 2 * STAGE + (t >> 3 & 1) * SCALES + li * 32 + (t & 4) * 4 + q * 4;
#pragma unroll
        for (int i = 0; i < FM; ++i)
            ya[i] = transpose_bytes(*reinterpret_cast<const uint32_t*>(cur + (wm + 16 * i) * 32), lane);
#pragma unroll
        for (int j = 0; j < FN; ++j)
            yb[j] = transpose_bytes(*reinterpret_cast<const uint32_t*>(cur + (BM + wn + 16 * j) * 32), lane);
    };

    f32x4 acc[FM][FN];
#pragma unroll
    for (int i = 0; i < FM; ++i)
#pragma unroll
        for (int j = 0; j < FN; ++j) acc[i][j] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};

    struct Fragments {
        u32x4 a[FM], b[FN];
    };
    // fragment r of the step: B's, then A's
    auto read = [&](int buffer, int half, Fragments& f, int r) {
        const char* cur = lds + buffer * STAGE + li * 128 + (((half * 4 + q) ^ (li & 7)) << 4);
        if (r < FN) f.b[r] = *reinterpret_cast<const u32x4*>(cur + (BM + wn + 16 * r) * 128);
        else f.a[r - FN] = *reinterpret_cast<const u32x4*>(cur + (wm + 16 * (r - FN)) * 128);
    };

    if (steps > 0) {
        issue_scales(0, 0);
#pragma unroll
        for (int s = 0; s < 2; ++s) {
#pragma unroll
            for (int i = 0; i < LOADS; ++i) issue(i, s, back(2 * s));
            advance(2 * s);
            asm volatile("" ::: "memory");      // in this order: the wait below counts on it
        }
        stage_barrier<LOADS>();         // all but the second stage
    }
    for (int t0 = 0; t0 < steps; t0 += 4) {
        uint32_t ya[FM], yb[FN];
        scales(t0, ya, yb);
        if ((t0 & 4) == 0 && t0 + 8 < steps) issue_scales(t0 + 8, (t0 >> 3 & 1) ^ 1);
        auto step = [&](auto byte) {
            constexpr int B = decltype(byte)::value;
            const int t = t0 + B;
            if (t >= steps) return;
            Fragments f;
#pragma unroll
            for (int r = 0; r < FM + FN; ++r) read(B / 2, B % 2, f, r);
            if constexpr (B & 1) {
                // the next stage has to be there, and every wave to have read this one
                stage_barrier<0>();
                const uint32_t less = back(t + 3);
#pragma unroll
                for (int i = 0; i < LOADS; ++i) issue(i, B >> 1, less);
                advance(t + 3);
            }
#pragma unroll
            for (int i = 0; i < FM; ++i)
#pragma unroll
                for (int j = 0; j < FN; ++j) acc[i][j] = mfma_e2m1_at<B>(f.b[j], f.a[i], acc[i][j], yb[j], ya[i]);
        };
        step(std::integral_constant<int, 0>{});
        step(std::integral_constant<int, 1>{});
        step(std::integral_constant<int, 2>{});
        step(std::integral_constant<int, 3>{});
    }
    stage_barrier<0>();             // no load to LDS outlives its workgroup
#pragma unroll
    for (int i = 0; i < FM; ++i) {
        const int m = m0 + wm + 16 * i + li;
#pragma unroll
        for (int j = 0; j < FN; j += 2) mx_store_pair(g, m, n0 + wn + 16 * j, q, acc[i][j], acc[i][j + 1]);
    }
}

// ------------------------------------------------------------------------ tile choice

// Launches `big` (256 x 256 tiles), `mid` (128 x 128) or `small` (64 x 64): the largest tile of
// which there are enough for most of the 256 CUs; without enough of any, the smallest.  us with
// big, mid and small tiles (E2M1; weight gradient E4M3):
//   M x N (big tiles, mid tiles)   forward, K          input grad     weight grad    E2M1 x E2M1
//   3584 x 3584 (196, 784)         55, 69, 84  2048                                  25, 26, 29
//   3328 x 4096 (208, 832)         54, 67, 82  2048    57, 69, 96     60, 83, 105    23, 25, 29
//   4096 x 2816 (176, 704)         99, 99, 141  4096   60, 55, 77     61, 65, 86     37, 35, 44
//   4096 x 2048 (128, 512)         179, 135, 215  8192 60, 39, 56     61, 46, 64     65, 44, 64
//   1792 x 1792 (49, 196)          50, 22, 30  2048    55, 23, 31     58, 28, 37     20, 9.6, 10
//   2048 x 1280 (40, 160)          91, 39, 44  4096    55, 23, 25     58, 27, 30     32, 14.4, 13.5
//   2048 x 1152 (40, 144)          91, 39, 44  4096    65, 22, 25     76, 27, 30     32, 14.0, 13.0
//   2048 x 1024 (32, 128)          49, 21, 19  2048    55, 22, 19     57, 26, 22     19, 8.9, 7.1
// (the gradients over 2048).  It does not look at how full the last round of tiles is: 4096 x 4608
// (288, 1152), whose second round holds 32 big tiles, takes 107, 86 and 121 over 2048; and at 144
// mid tiles small ones are taken, 12% slower but for two E2M1 operands.
template <class Big, class Mid, class Small>
hipError_t mx_by_tile(const MxGemmArgs& g, Big big, Mid mid, Small small) {
    auto tiles = [&](int t) { return ((int64_t)g.M + t - 1) / t * (((int64_t)g.N + t - 1) / t); };
    if (tiles(256) >= 192) return big(dim3((unsigned)tiles(256)));
    if (tiles(128) >= 160) return mid(dim3((unsigned)tiles(128)));
    return small(dim3((unsigned)tiles(64)));
}

// Sizes whose every stage lies inside both operands take the form that looks for no edge: us
// general and whole, bf16, 8192 x 8192 x 2048: forward E2M1 220, 212, E4M3 251, 221; weight grad
// 233, 215 and 227, 208; 512 x 2048 x 2048 forward 14.3, 12.7.  Input grad is alike in both.
template <int DT, int ASRC, int BSRC, int T, int WM, int WN>
hipError_t mx_gemm16_tile(const MxGemmArgs& g, dim3 grid, hipStream_t s) {
    constexpr int threads = (T / WM) * (T / WN) * 64;
    using SA = MxStage<DT, ASRC, T, threads, true>;
    using SB = MxStage<DT, BSRC, T, threads, true>;
    if (SA::whole(SA::codes ? g.a_row_bytes : g.lda, g.M, g.K) && SB::whole(g.b_row_bytes, g.N, g.K))
        hipLaunchKernelGGL((k_mx_gemm16<DT, ASRC, BSRC, T, T, WM, WN, true>), grid, dim3(threads), 0, s, g);
    else
        hipLaunchKernelGGL((k_mx_gemm16<DT, ASRC, BSRC, T, T, WM, WN, false>), grid, dim3(threads), 0, s, g);
    return hipGetLastError();
}

template <int DT, int ASRC, int BSRC> hipError_t mx_gemm16(const MxGemmArgs& g, hipStream_t s) {
    return mx_by_tile(
        g, [&](dim3 grid) { return mx_gemm16_tile<DT, ASRC, BSRC, 256, 128, 64>(g, grid, s); },
        [&](dim3 grid) { return mx_gemm16_tile<DT, ASRC, BSRC, 128, 64, 32>(g, grid, s); },
        [&](dim3 grid) { return mx_gemm16_tile<DT, ASRC, BSRC, 64, 32, 32>(g, grid, s); });
}

}  // namespace bitopt
