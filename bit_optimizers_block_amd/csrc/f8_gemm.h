// f8_gemm.h -- tiled products of F8 matrices, out = A B^T, both contracted along their rows.
//
// Each block of 128 contraction elements is a product of its own, multiplied by its rows' and
// columns' scales and added to the fp32 sums.  Two ways to that product:
//   fast   the 8-bit matrix instruction, one for 128 elements.  It aligns the products of a
//          step to the largest one and drops what lies some 17 bits below.
//   exact  the codes decoded to bf16 in registers (every element is exact there) and four
//          16-bit matrix instructions, which keep fp32: at half the rate.
// Error of the sums, in norm, as a share of the results' norm (1024 x 1024 x K, K from 128 to 8192, normal
// values): fast 1.4e-5 (E4M3) and 1.1e-5 (E5M2 x E4M3) at any K, without a bias, at most 2e-5 of the sum
// of magnitudes at K = 128 and 1.2e-6 at 8192; exact 5e-8 to 1e-7.  Rounding to bf16 is 1.657e-3 with either: one
// result in a hundred rounds to the other side.  Rounding to fp16 is 2.074e-4 and became 2.079e-4, six in a hundred.
// So bf16 results are fast, fp16 and fp32 ones exact.
#pragma once

#include <algorithm>
#include <type_traits>

#include "f8.h"

namespace bitopt {

template <int AF, int BF> __device__ __forceinline__ f32x4 mfma_f8(i32x8 a, i32x8 b, f32x4 c) {
    // scale operands of zero select the instruction without scales
    return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(a, b, c, AF, BF, 0, 0, 0, 0);
}
// The same times 2^(ea - 127) for a lane's row of A and 2^(eb - 127) for its row of B.
template <int AF, int BF> __device__ __forceinline__ f32x4 mfma_f8(i32x8 a, i32x8 b, f32x4 c, int ea, int eb) {
    return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(a, b, c, AF, BF, 0, ea, 0, eb);
}

// A scale taken apart: what goes into the products of a lane's row, and the rest of it.
template <bool EXACT> using F8Factor = std::conditional_t<EXACT, float, int>;
template <bool EXACT> __device__ __forceinline__ F8Factor<EXACT> f8_take(float scale, float& rest) {
    if constexpr (EXACT) {
        const F8Fold v = f8_fold(scale);
        rest = v.s;
        return v.f;
    } else {
        const F8Parts v = f8_parts(scale);
        rest = v.s;
        return v.e;
    }
}
template <bool EXACT> __device__ __forceinline__ f32x4 f8_rest(f32x4 scale) {
    float r[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) f8_take<EXACT>(scale[i], r[i]);
    return f32x4{r[0], r[1], r[2], r[3]};
}

// Waits until at most N of the wave's global loads are outstanding and its LDS reads are done, then
// for the workgroup.  The empty statements keep memory accesses on their side.
template <int N> __device__ __forceinline__ void f8_barrier() {
    asm volatile("" ::: "memory");
    __builtin_amdgcn_s_waitcnt((N & 15) | 0x70 | ((N >> 4) << 14));
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
}

// SIZE bytes for each lane from a uniform base and the lane's offset to LDS, the wave's one behind the
// other.  A buffer load: its address takes one register, and the compiler counts it apart from the
// LDS reads, where after a global load to LDS it waits for all of them at each.
template <int SIZE> __device__ __forceinline__ void load_to_lds(const void* base, uint32_t offset, char* to) {
#ifdef __HIP_DEVICE_COMPILE__
    const auto from = __builtin_amdgcn_make_buffer_rsrc((void*)base, 0, -1, 0x00027000);
    const auto at = (__attribute__((address_space(3))) void*)to;
    if constexpr (SIZE == 16) __builtin_amdgcn_raw_ptr_buffer_load_lds(from, at, 16, offset, 0, 0, 0);
    else __builtin_amdgcn_raw_ptr_buffer_load_lds(from, at, 4, offset, 0, 0, 0);
#endif
}

// Workgroup tile BM x BN, wave tile WM x WN, NS LDS buffers of one block of 128 contraction elements:
// rows of 128 bytes, filled by direct loads NS - 1 blocks ahead.  A wave's load fills 1024
// consecutive bytes of LDS, so the swizzle that spreads a fragment's rows over the banks -- 16-byte
// chunk c of row r lies at chunk c ^ (r % 8) -- is applied to the source address.  A lane holds row
// l % 16 and chunks q and q + 4, q = l / 16, of either operand: which elements those are does not
// matter to the sum, as long as both agree.
//
// A block goes in groups of one A fragment by all of B's; under a group's products run the reads of
// a later A fragment and the additions of the group before.  Where every fragment left is in
// registers the barrier that ends the block stands, and its buffer is filled anew.  Fast: that is
// ahead of the last two groups, which go column by column, so that B's fragments are free one after
// the other for the reads of the next block.  Exact: ahead of the last group; B's decoded fragments
// leave no registers for the next ones.
//
// Bound at 8192 x 2048 x 8192, fast, B by tiles: no pipe by itself.  A launch takes 232 to 242 thousand cycles, 108 to
// 119 us, and 125 to 135 in a long row of them (2040 to 2550 TFLOP/s): the clock falls from 2.06 to 1.80 GHz.  The
// matrix pipes are busy 131 thousand of them (54 to 57%), and other vector instructions, nearly all of them the 128
// additions of a block, issue in 82 thousand (34%).  With the sums left to the matrix instruction, without scales, it
// takes 215 thousand, 101 to 116 us: two thirds of the additions run beside matrix instructions.  What the other
// cycles wait for those counters do not tell.  LDS is busy 25%, without conflicts.  By rows each addition takes a product
// of two scales besides (127 to 149 us), and in the exact form the decoding (243 to 273).  Where the
// contraction is short the results' stores show: 8192 x 8192 x 2048 takes 128 to 158 us, some 30 of them 134 MB of
// results that nothing overlaps (one workgroup a CU; a resident grid whose next tile's loads go ahead of the stores
// spilled).
// Earlier forms: a fragment's reads waited for right ahead of its products, and the loads of the next
// block with a tile's scale, 168 us; the barrier ahead of the last group only, 124.  A wave's
// priority raised for half of the waves: 114 to 117.  128 x 128 tiles on four waves: 146.
template <int AF, int BF, bool BTILES, bool EXACT, int BM, int BN, int WM, int WN, int NS>
__global__ __launch_bounds__((BM / WM) * (BN / WN) * 64) void k_f8_gemm(F8GemmArgs g) {
    constexpr int NT = (BM / WM) * (BN / WN) * 64, FM = WM / 16, FN = WN / 16;
    constexpr int ROWS = (BM + BN) * 128, PASS_ROWS = NT / 8, LOADS = (BM + BN) / PASS_ROWS;
    constexpr int STAGE = ROWS + NT * 4;                // a scale for each thread: A's rows, then B's rows or tiles
    static_assert(BM % PASS_ROWS == 0 && BN % PASS_ROWS == 0 && PASS_ROWS % 8 == 0, "whole passes per operand");
    static_assert((BTILES ? BM + 64 : BM + BN) <= NT && kF8Block % WN == 0, "a wave's columns lie in one tile");
    __shared__ __attribute__((aligned(16))) char lds[NS * STAGE];

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
    const uint8_t *a_next, *b_next;
    uint32_t off[LOADS];
#pragma unroll
    for (int i = 0; i < LOADS; ++i) {
        const int r = i * PASS_ROWS + pr;
        off[i] = (uint32_t)(i * PASS_ROWS < BM ? min(r, g.M - 1 - m0) : min(r - BM, g.N - 1 - n0)) * (uint32_t)g.row_bytes +
                 chunk * 16;
    }
    // this thread's scale of a block (a wave's are all A's or all B's), and how far the next block's is
    const bool of_a = wave * 64 < BM;
    const int sr = of_a ? tid : tid - BM;
    const float* s_next;
    const int64_t s_step = of_a ? g.M : BTILES ? 1 : g.N;
    const uint32_t s_off = 4u * (of_a ? (uint32_t)min(sr, g.M - 1 - m0)
                                      : BTILES ? (uint32_t)min(sr, (g.N - 1) / kF8Block - n0 / kF8Block) * (uint32_t)steps
                                               : (uint32_t)min(sr, g.N - 1 - n0));
    auto begin = [&] {
        a_next = g.a + (int64_t)m0 * g.row_bytes;
        b_next = g.b + (int64_t)n0 * g.row_bytes;
        s_next = of_a ? g.a_scales + m0 : BTILES ? g.b_scales + (int64_t)(n0 / kF8Block) * steps : g.b_scales + n0;
    };
    // LOADS + 1 loads of each wave; after the last block they repeat it, into buffers that are not read
    auto load = [&](int buffer, int i) {
        char* to = lds + buffer * STAGE;
        if (i < LOADS) load_to_lds<16>(i * PASS_ROWS < BM ? a_next : b_next, off[i], to + i * NT * 16 + wave * 1024);
        else load_to_lds<4>(s_next, s_off, to + ROWS + wave * 256);
    };
    auto advance = [&](int t) {
        const bool more = t + 1 < steps;
        a_next += more ? kF8Block : 0;
        b_next += more ? kF8Block : 0;
        s_next += more ? s_step : 0;
    };

    f32x4 acc[FM][FN];
    struct Codes {
        u32x4 x, y;
    };
    const int lo = (q ^ (li & 7)) << 4, hi = ((q + 4) ^ (li & 7)) << 4;
    const uint32_t a_at = (wm + li) * 128, b_at = (BM + wn + li) * 128, sa_at = ROWS + (wm + li) * 4;
    const uint32_t sb_at = ROWS + (BM + (BTILES ? wn / kF8Block : wn + 4 * q)) * 4;
    auto read_a = [&](const char* cur, int i) {
        return Codes{*reinterpret_cast<const u32x4*>(cur + a_at + lo + i * 2048), *reinterpret_cast<const u32x4*>(cur + a_at + hi + i * 2048)};
    };
    auto read_b = [&](const char* cur, int j) {
        return Codes{*reinterpret_cast<const u32x4*>(cur + b_at + lo + j * 2048), *reinterpret_cast<const u32x4*>(cur + b_at + hi + j * 2048)};
    };
    auto read_sa = [&](const char* cur, int i) { return *reinterpret_cast<const float*>(cur + sa_at + i * 64); };
    f32x4 sb[BTILES ? 1 : FN];
    auto read_sb = [&](const char* cur) {
        if constexpr (BTILES) {
            sb[0].x = *reinterpret_cast<const float*>(cur + sb_at);
        } else {
#pragma unroll
            for (int j = 0; j < FN; ++j) sb[j] = *reinterpret_cast<const f32x4*>(cur + sb_at + j * 64);
        }
    };
    // acc[i][j] += a product times its scales
    auto add = [&](int i, int j, f32x4 p, float scale) {
#pragma unroll
        for (int r = 0; r < 4; ++r) acc[i][j][r] = __builtin_fmaf(p[r], BTILES ? scale : scale * sb[j][r], acc[i][j][r]);
    };
    auto eight = [](const Codes& c) {
        return i32x8{(int)c.x.x, (int)c.x.y, (int)c.x.z, (int)c.x.w, (int)c.y.x, (int)c.y.y, (int)c.y.z, (int)c.y.w};
    };

    static_assert(FM % 2 == 0, "fragments in pairs");
    Codes a[2], b[FN];
    float sa[2];
    auto halves = [](const Codes& c, auto fmt, float f, u32x4 h[4]) {
        constexpr int F = decltype(fmt)::value;
        h[0] = f8_half8<F>(c.x.x, c.x.y, f); h[1] = f8_half8<F>(c.x.z, c.x.w, f);
        h[2] = f8_half8<F>(c.y.x, c.y.y, f); h[3] = f8_half8<F>(c.y.z, c.y.w, f);
    };
    constexpr std::integral_constant<int, AF> af;
    constexpr std::integral_constant<int, BF> bf;
    // all products, with scales as they are or taken apart
    auto run = [&](auto apart) __attribute__((always_inline)) {
        constexpr bool APART = decltype(apart)::value;
#pragma unroll
        for (int i = 0; i < FM; ++i)
#pragma unroll
            for (int j = 0; j < FN; ++j) acc[i][j] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
        begin();
        if (steps > 0) {
#pragma unroll
            for (int s = 0; s < NS; ++s) {
#pragma unroll
                for (int i = 0; i <= LOADS; ++i) load(s, i);
                advance(s);
                asm volatile("" ::: "memory");              // in this order: the waits count on it
            }
            f8_barrier<(NS - 1) * (LOADS + 1)>();
#pragma unroll
            for (int j = 0; j < FN; ++j) b[j] = read_b(lds, j);
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                a[i] = read_a(lds, i);
                sa[i] = read_sa(lds, i);
            }
            read_sb(lds);
        }
        int buffer = 0;
        for (int t = 0; t < steps; ++t) {
            const char* cur = lds + buffer * STAGE;
            const int after = buffer + 1 == NS ? 0 : buffer + 1;
            const char* next = lds + after * STAGE;
            const f32x4 zero = {0.0f, 0.0f, 0.0f, 0.0f};
            F8Factor<EXACT> fa[2] = {1, 1}, fb[FN];
#pragma unroll
            for (int j = 0; j < FN; ++j) {
                fb[j] = 1;
                if constexpr (APART && !BTILES) {
                    float unused;
                    fb[j] = f8_take<EXACT>(*reinterpret_cast<const float*>(cur + ROWS + (BM + wn + 16 * j + li) * 4), unused);
                    sb[j] = f8_rest<EXACT>(sb[j]);
                }
            }
            if constexpr (APART && BTILES) {
                float rest;
                fb[0] = f8_take<EXACT>(sb[0].x, rest);
                sb[0].x = rest;
#pragma unroll
                for (int j = 1; j < FN; ++j) fb[j] = fb[0];
            }
            auto take_a = [&](int k) {
                if constexpr (APART) fa[k] = f8_take<EXACT>(sa[k], sa[k]);
            };
            auto product = [&](int j, int k) {
                if constexpr (APART) return mfma_f8<BF, AF>(eight(b[j]), eight(a[k]), zero, (int)fb[j], (int)fa[k]);
                else return mfma_f8<BF, AF>(eight(b[j]), eight(a[k]), zero);
            };
            f32x4 p[2][FN];
            float scale[2];
            // the next block has to be there, and every wave to have read this one
            auto turn = [&] {
                f8_barrier<(NS - 2) * (LOADS + 1)>();
                __builtin_amdgcn_sched_barrier(0);
            };
            // B first: a lane then holds four consecutive columns of one output row
            if constexpr (!EXACT) {
#pragma unroll
                for (int i = 0; i < FM - 2; ++i) {
                    take_a(i & 1);
                    scale[i & 1] = BTILES ? sa[i & 1] * sb[0].x : sa[i & 1];
#pragma unroll
                    for (int j = 0; j < FN; ++j) {
                        p[i & 1][j] = product(j, i & 1);
                        if (i > 0) add(i - 1, j, p[(i - 1) & 1][j], scale[(i - 1) & 1]);
                        __builtin_amdgcn_sched_barrier(0);
                    }
                    a[i & 1] = read_a(cur, i + 2);
                    sa[i & 1] = read_sa(cur, i + 2);
                    asm volatile("" ::: "memory");          // the reads stay ahead of the next products
                    __builtin_amdgcn_sched_barrier(0);
                }
                turn();
                float left[2];
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                    take_a(k);
                    left[k] = BTILES ? sa[k] * sb[0].x : sa[k];
                }
                f32x4 r[2][2];
#pragma unroll
                for (int j = 0; j < FN; ++j) {
#pragma unroll
                    for (int k = 0; k < 2; ++k) {
                        r[j & 1][k] = product(j, k);
                        if (j > 0) add(FM - 2 + k, j - 1, r[1 - (j & 1)][k], left[k]);
                        else if constexpr (FM > 2)
#pragma unroll
                            for (int l = k * FN / 2; l < (k + 1) * FN / 2; ++l) add(FM - 3, l, p[(FM - 3) & 1][l], scale[(FM - 3) & 1]);
                        if (k == 1) b[j] = read_b(next, j);
                        if (j + 1 == FN) {
                            a[k] = read_a(next, k);
                            sa[k] = read_sa(next, k);
                        }
#pragma unroll
                        for (int l = (2 * j + k) * (LOADS + 1) / (2 * FN); l < (2 * j + k + 1) * (LOADS + 1) / (2 * FN); ++l) load(buffer, l);
                        asm volatile("" ::: "memory");
                        __builtin_amdgcn_sched_barrier(0);
                    }
                }
#pragma unroll
                for (int k = 0; k < 2; ++k) add(FM - 2 + k, FN - 1, r[(FN - 1) & 1][k], left[k]);
            } else {
                u32x4 bh[FN][4];
#pragma unroll
                for (int j = 0; j < FN; ++j) halves(b[j], bf, (float)fb[j], bh[j]);
#pragma unroll
                for (int i = 0; i < FM; ++i) {
                    take_a(i & 1);
                    scale[i & 1] = BTILES ? sa[i & 1] * sb[0].x : sa[i & 1];
                    u32x4 ah[4];
                    halves(a[i & 1], af, (float)fa[i & 1], ah);
                    if (i + 2 < FM) {
                        a[i & 1] = read_a(cur, i + 2);
                        sa[i & 1] = read_sa(cur, i + 2);
                    }
                    if (i + 1 == FM) {
                        turn();
#pragma unroll
                        for (int l = 0; l <= LOADS; ++l) load(buffer, l);
                    }
                    asm volatile("" ::: "memory");          // the reads stay ahead of the products
                    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
                    for (int h = 0; h < 4; ++h) {
#pragma unroll
                        for (int j = 0; j < FN; ++j) p[i & 1][j] = mfma16<kBF16>(bh[j][h], ah[h], h ? p[i & 1][j] : zero);
#pragma unroll
                        for (int j = h * FN / 4; j < (h + 1) * FN / 4; ++j)
                            if (i > 0) add(i - 1, j, p[(i - 1) & 1][j], scale[(i - 1) & 1]);
                        __builtin_amdgcn_sched_barrier(0);
                    }
                }
#pragma unroll
                for (int j = 0; j < FN; ++j) b[j] = read_b(next, j);
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                    a[k] = read_a(next, k);
                    sa[k] = read_sa(next, k);
                }
                asm volatile("" ::: "memory");
#pragma unroll
                for (int j = 0; j < FN; ++j) add(FM - 1, j, p[(FM - 1) & 1][j], scale[(FM - 1) & 1]);
            }
            read_sb(next);
            advance(t + NS);
            buffer = after;
        }
        f8_barrier<0>();                // no load to LDS is under way, and every wave has read its last block
    };
    run(std::false_type{});
    f8_store(g.accumulate, steps > 0,
             [&] __attribute__((always_inline)) {
#pragma unroll
                 for (int i = 0; i < FM; ++i)
#pragma unroll
                     for (int j = 0; j < FN; j += 2)
                         mx_store_pair(g, m0 + wm + 16 * i + li, n0 + wn + 16 * j, q, acc[i][j], acc[i][j + 1]);
             },
             [&] __attribute__((always_inline)) {
                 return f8_again<BM, NT / 64, BN / WN>(g, acc, m0, wm, wn / WN, n0 + wn, f8_least<AF, BF>(steps),
                                                       reinterpret_cast<uint64_t*>(lds));
             },
             [&] __attribute__((always_inline)) {
                 __syncthreads();
                 run(std::true_type{});
             });
}

// ------------------------------------------------------- few tiles, a long contraction

// As k_f8_gemm for products with fewer tiles than fill the chip, where a block of contraction
// lasts as long as its loads: KS groups of waves share the tile, each taking every KS-th block, so
// that KS blocks are loaded at once, NS - 1 such stages ahead.  The groups' sums meet in LDS, in
// the order of the groups.
template <int AF, int BF, bool BTILES, bool EXACT, int BM, int BN, int WM, int WN, int KS, int NS>
__global__ __launch_bounds__(KS * (BM / WM) * (BN / WN) * 64) void k_f8_split(F8GemmArgs g) {
    constexpr int WAVES = (BM / WM) * (BN / WN), NT = KS * WAVES * 64, FM = WM / 16, FN = WN / 16;
    constexpr int BLOCK = (BM + BN) * 128, PASS_ROWS = NT / 8, PASSES = (BM + BN) / PASS_ROWS, LOADS = KS * PASSES;
    constexpr int SR = BM + (BTILES ? 64 : BN);         // scales of a block: A's rows, then B's rows or tiles
    constexpr int STAGE = KS * BLOCK + NT * 4;
    static_assert(BM % PASS_ROWS == 0 && BN % PASS_ROWS == 0 && PASS_ROWS % 8 == 0, "whole passes per operand");
    static_assert(KS * SR <= NT && kF8Block % WN == 0, "a scale for each thread at most; a wave's columns in one tile");
    constexpr int SUMS = KS * WAVES * FM * FN * 1024;
    static_assert(SUMS + F8Words<BM, NT / 64>::count * 8 <= NS * STAGE, "the sums fit where the codes were");
    __shared__ __attribute__((aligned(16))) char lds[NS * STAGE];

    int tm, tn;
    mx_tile((g.M + BM - 1) / BM, (g.N + BN - 1) / BN, tm, tn);
    const int m0 = tm * BM, n0 = tn * BN;
    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int group = wave / WAVES, part = wave % WAVES;
    const int wm = part % (BM / WM) * WM, wn = part / (BM / WM) * WN;
    const int q = lane >> 4, li = lane & 15;
    const int steps = (int)f8_blocks(g.K), stages = (steps + KS - 1) / KS;

    const int pr = tid >> 3, chunk = (tid & 7) ^ (pr & 7);
    const uint8_t* a0 = g.a + (int64_t)m0 * g.row_bytes;
    const uint8_t* b0 = g.b + (int64_t)n0 * g.row_bytes;
    uint32_t off[PASSES];
#pragma unroll
    for (int i = 0; i < PASSES; ++i) {
        const int r = i * PASS_ROWS + pr;
        off[i] = (uint32_t)(i * PASS_ROWS < BM ? min(r, g.M - 1 - m0) : min(r - BM, g.N - 1 - n0)) * (uint32_t)g.row_bytes +
                 chunk * 16;
    }
    // this thread's scale: of the stage's block sk, of A or B (a wave's are alike)
    const int sk = min(wave * 64 / SR, KS - 1), sw = wave * 64 - sk * SR;
    const bool of_a = sw < BM;
    const int sr = (of_a ? sw : sw - BM) + lane;
    const float* s0 = of_a ? g.a_scales + m0 : BTILES ? g.b_scales + (int64_t)(n0 / kF8Block) * steps : g.b_scales + n0;
    const int64_t s_step = of_a ? g.M : BTILES ? 1 : g.N;
    const uint32_t s_off = 4u * (of_a ? (uint32_t)min(sr, g.M - 1 - m0)
                                      : BTILES ? (uint32_t)min(sr, (g.N - 1) / kF8Block - n0 / kF8Block) * (uint32_t)steps
                                               : (uint32_t)min(sr, g.N - 1 - n0));
    // blocks past the last repeat it, and are not read
    auto issue = [&](int stage) {
        char* to = lds + stage % NS * STAGE;
#pragma unroll
        for (int k = 0; k < KS; ++k) {
            const int64_t block = min(stage * KS + k, steps - 1);
#pragma unroll
            for (int i = 0; i < PASSES; ++i)
                load_to_lds<16>((i * PASS_ROWS < BM ? a0 : b0) + block * kF8Block, off[i], to + k * BLOCK + i * NT * 16 + wave * 1024);
        }
        load_to_lds<4>(s0 + min(stage * KS + sk, steps - 1) * s_step, s_off, to + KS * BLOCK + wave * 256);
    };

    static_assert(FM * FN / 2 == KS && FM % 2 == 0 && FN == 2, "a pair of a wave's fragments for each group");
    f32x4 acc[FM][FN];
    const int lo = (q ^ (li & 7)) << 4, hi = ((q + 4) ^ (li & 7)) << 4;

    f32x4 v[1][FN];
    // all products, with scales as they are or taken apart
    auto run = [&](auto apart) __attribute__((always_inline)) {
        constexpr bool APART = decltype(apart)::value;
#pragma unroll
        for (int i = 0; i < FM; ++i)
#pragma unroll
            for (int j = 0; j < FN; ++j) acc[i][j] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
        for (int s = 0; s < NS - 1 && steps > 0; ++s) {
            issue(s);
            asm volatile("" ::: "memory");                  // in this order: the waits count on it
        }
        for (int s = 0; s < stages; ++s) {
            // the stage is there, and every wave has read the one before, whose buffer is filled anew
            f8_barrier<(NS - 2) * (LOADS + 1)>();
            issue(s + NS - 1);
            if (s * KS + group >= steps) continue;
            const char* cur = lds + s % NS * STAGE + group * BLOCK;
            const float* sc = reinterpret_cast<const float*>(lds + s % NS * STAGE + KS * BLOCK) + group * SR;
            auto read = [&](int row, u32x4& x, u32x4& y) {
                x = *reinterpret_cast<const u32x4*>(cur + (row + li) * 128 + lo);
                y = *reinterpret_cast<const u32x4*>(cur + (row + li) * 128 + hi);
            };
            u32x4 ax[FM], ay[FM], bx[FN], by[FN];
            float sa[FM];
            f32x4 sb[BTILES ? 1 : FN];
#pragma unroll
            for (int j = 0; j < FN; ++j) read(BM + wn + 16 * j, bx[j], by[j]);
#pragma unroll
            for (int i = 0; i < FM; ++i) read(wm + 16 * i, ax[i], ay[i]);
            if constexpr (BTILES) {
                sb[0].x = sc[BM + wn / kF8Block];
            } else {
#pragma unroll
                for (int j = 0; j < FN; ++j) sb[j] = *reinterpret_cast<const f32x4*>(sc + BM + wn + 16 * j + 4 * q);
            }
            F8Factor<EXACT> fa[FM] = {}, fb[FN] = {};
#pragma unroll
            for (int j = 0; j < FN; ++j) {
                fb[j] = 1;
                if constexpr (APART) {
                    float rest;
                    fb[j] = f8_take<EXACT>(BTILES ? sb[0].x : sc[BM + wn + 16 * j + li], rest);
                    if constexpr (!BTILES) sb[j] = f8_rest<EXACT>(sb[j]);
                }
            }
            if constexpr (APART && BTILES) sb[0] = f8_rest<EXACT>(sb[0]);
#pragma unroll
            for (int i = 0; i < FM; ++i) {
                sa[i] = sc[wm + 16 * i + li];
                fa[i] = 1;
                if constexpr (APART) fa[i] = f8_take<EXACT>(sa[i], sa[i]);
                if constexpr (BTILES) sa[i] *= sb[0].x;
            }
            u32x4 bh[EXACT ? FN : 1][4];
            if constexpr (EXACT) {
#pragma unroll
                for (int j = 0; j < FN; ++j) {
                    const float f = (float)fb[j];
                    bh[j][0] = f8_half8<BF>(bx[j].x, bx[j].y, f); bh[j][1] = f8_half8<BF>(bx[j].z, bx[j].w, f);
                    bh[j][2] = f8_half8<BF>(by[j].x, by[j].y, f); bh[j][3] = f8_half8<BF>(by[j].z, by[j].w, f);
                }
            }
#pragma unroll
            for (int i = 0; i < FM; ++i) {
                f32x4 p[FN];
                if constexpr (EXACT) {
                    const float f = (float)fa[i];
                    const u32x4 ah[4] = {f8_half8<AF>(ax[i].x, ax[i].y, f), f8_half8<AF>(ax[i].z, ax[i].w, f),
                                         f8_half8<AF>(ay[i].x, ay[i].y, f), f8_half8<AF>(ay[i].z, ay[i].w, f)};
#pragma unroll
                    for (int j = 0; j < FN; ++j) p[j] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
                    for (int h = 0; h < 4; ++h)
#pragma unroll
                        for (int j = 0; j < FN; ++j) p[j] = mfma16<kBF16>(bh[j][h], ah[h], p[j]);
                } else {
                    const i32x8 a = {(int)ax[i].x, (int)ax[i].y, (int)ax[i].z, (int)ax[i].w,
                                     (int)ay[i].x, (int)ay[i].y, (int)ay[i].z, (int)ay[i].w};
#pragma unroll
                    for (int j = 0; j < FN; ++j) {
                        const i32x8 b = {(int)bx[j].x, (int)bx[j].y, (int)bx[j].z, (int)bx[j].w,
                                         (int)by[j].x, (int)by[j].y, (int)by[j].z, (int)by[j].w};
                        const f32x4 zero = {0.0f, 0.0f, 0.0f, 0.0f};
                        if constexpr (APART) p[j] = mfma_f8<BF, AF>(b, a, zero, (int)fb[j], (int)fa[i]);
                        else p[j] = mfma_f8<BF, AF>(b, a, zero);
                    }
                }
#pragma unroll
                for (int j = 0; j < FN; ++j)
#pragma unroll
                    for (int r = 0; r < 4; ++r) acc[i][j][r] = __builtin_fmaf(p[j][r], BTILES ? sa[i] : sa[i] * sb[j][r], acc[i][j][r]);
            }
        }
        f8_barrier<0>();                // no load to LDS is under way, and every wave has read its last block
        f32x4* sums = reinterpret_cast<f32x4*>(lds);
#pragma unroll
        for (int i = 0; i < FM; ++i)
#pragma unroll
            for (int j = 0; j < FN; ++j) sums[((group * WAVES + part) * FM * FN + i * FN + j) * 64 + lane] = acc[i][j];
        __syncthreads();
        // fragments (i, 0) and (i, 1) of a wave are added up by group i
#pragma unroll
        for (int h = 0; h < FN; ++h) {
            v[0][h] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
            for (int k = 0; k < KS; ++k) v[0][h] += sums[((k * WAVES + part) * FM * FN + group * FN + h) * 64 + lane];
        }
    };
    run(std::false_type{});
    f8_store(g.accumulate, true,
             [&] __attribute__((always_inline)) { mx_store_pair(g, m0 + wm + 16 * group + li, n0 + wn, q, v[0][0], v[0][1]); },
             [&] __attribute__((always_inline)) {
                 return f8_again<BM, NT / 64, BN / WN>(g, v, m0, wm + 16 * group, wn / WN, n0 + wn, f8_least<AF, BF>(steps),
                                                       reinterpret_cast<uint64_t*>(lds + SUMS));
             },
             [&] __attribute__((always_inline)) {
                 __syncthreads();
                 run(std::true_type{});
             });
}

// ------------------------------------------------------------------------ tile choice

// The form that is estimated to take the least time for a block of contraction: `one` us for up to 256
// tiles (one a CU), else `two` for each 512; of the largest form one workgroup fills a CU.  Measured us of whole products with each form, bf16
// results, B by tiles:
//   M x N x K            256 x 256   128 x 128   128 x 64   64 x 64   64 x 64, split
//   8192 x 8192 x 2048   152         185         257        282
//   8192 x 2048 x 8192   117         145         194        225
//   4096 x 4096 x 4096   60          76          103        122
//   2048 x 2048 x 2048               13.9        16.7       20.0
//   1024 x 4096 x 4096   47          26.8        25.8       31.9      39
//   1024 x 2048 x 8192   86          43          28.5       32.6      38
//   512 x 2048 x 2048    27          10.7        8.3        7.5       6.7
//   128 x 2048 x 8192    83          32          21.5       20.3      15.2
//   777 x 1001 x 513                 7.1         5.5        4.6       5.2
// and with fp32 results, B by rows:
//   M x N x K            256 x 128   128 x 64    64 x 64    64 x 64, split
//   8192 x 2048 x 8192   249         303         380
//   4096 x 4096 x 4096   130         161         202
//   1024 x 4096 x 4096   64          42          53         55
//   1024 x 2048 x 8192   117         44          52         50
//   512 x 2048 x 2048    34          13.5        11.8       9.3
//   128 x 2048 x 8192    112         42          37         24.5
//   777 x 1001 x 513                             6.2        6.3
// The split form takes up to 256 small tiles whose contraction is eight blocks or more.
struct F8Form {
    int bm, bn, threads;
    double one, two;
};

inline double f8_estimate(const F8GemmArgs& g, const F8Form& f, int64_t& tiles) {
    tiles = ((int64_t)g.M + f.bm - 1) / f.bm * (((int64_t)g.N + f.bn - 1) / f.bn);
    if (tiles * f.threads > 0xffffffffll) return 1e300;     // more threads than a launch holds
    if (f.bm == 256) return f.one * (double)((tiles + 255) / 256);
    return tiles <= 256 ? f.one : f.two * (double)((tiles + 511) / 512);
}

template <int AF, int BF, bool BTILES, bool EXACT> hipError_t f8_tiled(const F8GemmArgs& g, hipStream_t s) {
    // the first form is the largest one: it holds every product that the entry point lets pass
    constexpr int N = EXACT ? 3 : 4;
    const bool split = f8_blocks(g.K) >= 8;
    const F8Form fast[] = {{256, 256, 512, 1.87, 0}, {128, 128, 512, 0.75, 1.13}, {128, 64, 512, 0.42, 0.80}, {64, 64, 256, split ? 0.24 : 0.40, 0.50}};
    const F8Form exact[] = {{256, 128, 512, 1.90, 0}, {128, 64, 512, 0.69, 1.17}, {64, 64, 256, split ? 0.36 : 0.60, 0.72}};
    const F8Form* forms = EXACT ? exact : fast;
    int best = 0;
    int64_t tiles = 0;
    double least = 1e301;
    for (int i = 0; i < N; ++i) {
        int64_t t;
        const double e = f8_estimate(g, forms[i], t);
        if (e < least) least = e, best = i, tiles = t;
    }
    const dim3 grid((unsigned)tiles), threads(forms[best].threads);
    if (best == N - 1 && split && tiles <= 256)
        hipLaunchKernelGGL((k_f8_split<AF, BF, BTILES, EXACT, 64, 64, 64, 32, 4, 2>), grid, dim3(512), 0, s, g);
    else if constexpr (EXACT) {
        if (best == 0) hipLaunchKernelGGL((k_f8_gemm<AF, BF, BTILES, true, 256, 128, 64, 64, 2>), grid, threads, 0, s, g);
        else if (best == 1) hipLaunchKernelGGL((k_f8_gemm<AF, BF, BTILES, true, 128, 64, 32, 32, 3>), grid, threads, 0, s, g);
        else hipLaunchKernelGGL((k_f8_gemm<AF, BF, BTILES, true, 64, 64, 32, 32, 3>), grid, threads, 0, s, g);
    } else {
        if (best == 0) hipLaunchKernelGGL((k_f8_gemm<AF, BF, BTILES, false, 256, 256, 128, 64, 2>), grid, threads, 0, s, g);
        else if (best == 1) hipLaunchKernelGGL((k_f8_gemm<AF, BF, BTILES, false, 128, 128, 64, 32, 2>), grid, threads, 0, s, g);
        else if (best == 2) hipLaunchKernelGGL((k_f8_gemm<AF, BF, BTILES, false, 128, 64, 32, 32, 3>), grid, threads, 0, s, g);
        else hipLaunchKernelGGL((k_f8_gemm<AF, BF, BTILES, false, 64, 64, 32, 32, 3>), grid, threads, 0, s, g);
    }
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
