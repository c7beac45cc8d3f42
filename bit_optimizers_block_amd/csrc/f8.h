// f8.h -- 8-bit floating-point matrices with an fp32 scale for each block of 128: layout,
// scale rule, element conversions, and the argument blocks of the kernels that read and
// write them.
//
// A block is 128 consecutive elements of a row ("rows") or a tile of 128 x 128 ("tiles").
// Codes lie in rows padded to 128 bytes with zeros: the contraction length of one 8-bit
// matrix instruction and a whole cache line, so a product never has a ragged block.  The
// scales of row blocks lie block by block (a product's tile takes the scales of its rows
// for one block, consecutive ones), those of tiles as the tiles lie.
#pragma once

#include <hip/hip_runtime.h>

#include "mx.h"

namespace bitopt {

constexpr int kF8E4M3 = 0, kF8E5M2 = 1;       // the matrix instruction's own numbers of the formats
constexpr int kF8Tiles = 1;                    // else rows
constexpr int kF8Block = 128;

__host__ __device__ constexpr int64_t f8_blocks(int64_t n) { return (n + kF8Block - 1) / kF8Block; }
__host__ __device__ constexpr int64_t f8_padded(int64_t n) { return f8_blocks(n) * kF8Block; }

struct F8CodecArgs {
    const void* x; int64_t ldx;
    uint8_t* codes; float* scales;       // of x; NULL: not wanted
    uint8_t* codes_t; float* scales_t;   // of its transpose; NULL: not wanted
    int64_t rows, cols;
    void* out; int64_t ldo;              // dequantize
};

// out[m][n] = sum over blocks k of sa[k][m] sb[k][n] sum_j a[m][j] b[n][j]
struct F8GemmArgs {
    const uint8_t* a; const float* a_scales;
    const uint8_t* b; const float* b_scales;
    void* out; int64_t ldo;
    int64_t row_bytes;                   // of a and b: their rows hold the same contraction
    int32_t M, N, K;
    int32_t out_dtype, accumulate;
};

hipError_t launch_f8_quantize(const F8CodecArgs& a, int dtype, int fmt, int blocks, hipStream_t s);
hipError_t launch_f8_dequantize(const F8CodecArgs& a, int dtype, int fmt, int blocks, hipStream_t s);
// fast: on the 8-bit matrix instructions; exact: elements decoded to bf16 (every one is exact in it)
hipError_t launch_f8_fast(const F8GemmArgs& g, int a_fmt, int b_fmt, int b_blocks, hipStream_t s);
hipError_t launch_f8_exact(const F8GemmArgs& g, int a_fmt, int b_fmt, int b_blocks, hipStream_t s);
constexpr int kF8FewRows = 32;
hipError_t launch_f8_few(const F8GemmArgs& g, int a_fmt, int b_fmt, int b_blocks, hipStream_t s);

#ifdef __HIPCC__

// ------------------------------------------------------------------------- device side

template <int FMT> constexpr float kF8Top = FMT == kF8E4M3 ? 448.0f : 57344.0f;

// Factor r = top (1 / amax) of a block from the bits of its largest |x|, both operations rounded,
// with its significand then cut to 13 bits, and the scale 1 / r.  r <= top / amax (1 + 2^-21), also
// where 1 / amax is subnormal, so no element is half a step above the largest one and none
// saturates.  amax counts as top 2^-126 at least: r and 1 / r stay normal numbers, and a block of
// zeros needs no case of its own.
// An infinity or NaN in the block: the scale is NaN and r is zero.
struct F8Scale {
    float r, s;
};
template <int FMT> __device__ __forceinline__ F8Scale f8_scale(uint32_t amax_bits) {
    const float amax = fmaxf(__uint_as_float(amax_bits), kF8Top<FMT> * 0x1p-126f);
    const float r = __uint_as_float(__float_as_uint(1.0f / amax * kF8Top<FMT>) & ~0x7ffu);
    const bool bad = amax_bits >= 0x7f800000u;
    return {bad ? 0.0f : r, bad ? __uint_as_float(0x7fc00000u) : 1.0f / r};
}

// x r for the rounding to eight bits.  With 13 bits of r the product of an fp16 or bf16 value is
// exact in fp32, so its element is rounded once.  An fp32 value's may be rounded onto the border
// of two elements, all of which have even significands in fp32: where that happened, one step
// back towards the exact product puts it on the right side.
template <int DT> __device__ __forceinline__ float f8_scaled(float x, float r) {
    const float p = x * r;
    if constexpr (DT != kF32) return p;
    const float e = __builtin_fmaf(x, r, -p);
    const uint32_t u = __float_as_uint(p);
    const uint32_t back = (int32_t)(__float_as_uint(e) ^ u) < 0 ? u - 1 : u + 1;
    return __uint_as_float(e != 0.0f && (u & 1) == 0 ? back : u);
}

// Four values -> codes (nearest, ties to even).
template <int FMT> __device__ __forceinline__ uint32_t f8_encode4(float a, float b, float c, float d) {
    int r = 0;
    if constexpr (FMT == kF8E4M3) {
        r = __builtin_amdgcn_cvt_pk_fp8_f32(a, b, r, false);
        return (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(c, d, r, true);
    } else {
        r = __builtin_amdgcn_cvt_pk_bf8_f32(a, b, r, false);
        return (uint32_t)__builtin_amdgcn_cvt_pk_bf8_f32(c, d, r, true);
    }
}

// Four codes -> fp32, exact.
template <int FMT> __device__ __forceinline__ void f8_decode4(uint32_t c, float v[4]) {
    f32x2 p, q;
    if constexpr (FMT == kF8E4M3) {
        p = __builtin_amdgcn_cvt_pk_f32_fp8((int)c, false);
        q = __builtin_amdgcn_cvt_pk_f32_fp8((int)c, true);
    } else {
        p = __builtin_amdgcn_cvt_pk_f32_bf8((int)c, false);
        q = __builtin_amdgcn_cvt_pk_f32_bf8((int)c, true);
    }
    v[0] = p.x; v[1] = p.y; v[2] = q.x; v[3] = q.y;
}

// Scales of any size.  The loops multiply a block's sum p by the product of its two scales, which may leave
// fp32's range where p sa sb does not.  Where sa sb overflows, the result is infinite or NaN.  Where it
// is below the normal numbers, a block is off by |p| 2^-150 at most, so the results not below 2^24 times the sum of
// that over all blocks (f8_least) are right.  Of the others those are right whose row of A or row of B is all
// zero.  Where one is left, its tile is taken once more with every scale as f s: f, a power of two, goes into p
// by way of the elements or of the matrix instruction, and the product of two s stays in range.  Results
// that were right keep their bits in that.
// Measured, bf16 results, without and with it: 8192 x 8192 x 2048 127.1 and 128.1 us, 8192 x 2048 x 8192 108.6 and 108.2,
// 512 x 2048 x 2048 7.2 and 7.1; with 2% of A's rows zero 128.6 and 134.5, 108.3 and 110.5, 7.2 and 7.9; all zero 107 and 145.
// Inside the loops it costs more: every scale taken apart 114 and 119 (B by rows 130 and 147, fp32 results 250 and 274), a
// branch to that where a block needs it spills.
template <int AF, int BF> __device__ __forceinline__ float f8_least(int blocks) {
    return (float)blocks * (float)(kF8Block * 0x1p-126 * kF8Top<AF> * kF8Top<BF>);
}
__device__ __forceinline__ bool f8_any(bool v) { return __builtin_amdgcn_ballot_w64(v) != 0; }

// Of the rows of codes whose bits are set, those that hold a code which is neither 0 nor -0; by a whole wave,
// two rows at a time.
__device__ __forceinline__ uint64_t f8_hold(const uint8_t* codes, int64_t bytes, uint64_t rows) {
    uint64_t held = 0;
    while (rows) {
        const uint64_t one = rows & -rows, rest = rows ^ one, two = rest ? rest & -rest : one;
        const uint8_t *p = codes + __builtin_ctzll(one) * bytes, *q = codes + __builtin_ctzll(two) * bytes;
        uint32_t x = 0, y = 0;
        for (int64_t c = 16 * (threadIdx.x & 63); c < bytes; c += 4096)
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const int64_t at = min(c + 1024 * k, bytes - 16);
                const u32x4 v = *gbl(reinterpret_cast<const u32x4*>(p + at)), w = *gbl(reinterpret_cast<const u32x4*>(q + at));
                x |= v.x | v.y | v.z | v.w;
                y |= w.x | w.y | w.z | w.w;
            }
        if (f8_any((x & 0x7f7f7f7fu) != 0)) held |= one;
        if (f8_any((y & 0x7f7f7f7fu) != 0)) held |= two;
        rows &= ~(one | two);
    }
    return held;
}

// Of a wave's 16 R x 16 C results, a lane's four consecutive columns of a row in each tile of 16: the
// smallest of the lane's rows, and whether one is infinite or NaN.  Rows and columns beyond the matrix
// repeat its last ones.
template <int R, int C> __device__ __forceinline__ bool f8_lows(const f32x4 (&v)[R][C], float low[R]) {
    float high = 0.0f;
#pragma unroll
    for (int i = 0; i < R; ++i) {
        low[i] = __builtin_inff();
#pragma unroll
        for (int j = 0; j < C; ++j)
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                low[i] = __builtin_elementwise_minimum(low[i], fabsf(v[i][j][r]));     // NaN where there is one
                high = __builtin_elementwise_maximum(high, fabsf(v[i][j][r]));
            }
    }
    return f8_any(!(high < __builtin_inff()));
}

// The rows of 16 with a lane that says so.
__device__ __forceinline__ uint64_t f8_rows_with(bool v) {
    const uint64_t in = __builtin_amdgcn_ballot_w64(v);
    return (in | in >> 16 | in >> 32 | in >> 48) & 0xffff;
}

// Whether a column from n on holds a code where a result of the rows that are left is below `least`.
template <int R, int C>
__device__ __forceinline__ bool f8_columns(const F8GemmArgs& g, const f32x4 (&v)[R][C], const bool row[R], int n, float least) {
    const int q = (threadIdx.x & 63) >> 4;
    uint64_t cols = 0;
#pragma unroll
    for (int j = 0; j < C; ++j)
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            bool small = false;
#pragma unroll
            for (int i = 0; i < R; ++i) small |= row[i] && fabsf(v[i][j][r]) < least;
            const uint64_t in = __builtin_amdgcn_ballot_w64(small && n + 16 * j + 4 * q + r < g.N);
#pragma unroll
            for (int k = 0; k < 4; ++k) cols |= (uint64_t)((in >> 16 * k & 0xffff) != 0) << (16 * j + 4 * k + r);
        }
    return f8_hold(g.b + (int64_t)n * g.row_bytes, g.row_bytes, cols) != 0;
}

// Whether a workgroup's results have to be taken once more, those of this wave v, from row m0 + wm and column n; it
// is the `part`-th of PARTS waves with the same rows.  words: F8Words<BM, WAVES> of LDS.
template <int BM, int WAVES> struct F8Words {
    static constexpr int rows = (BM + 63) / 64, count = WAVES * (2 * rows + 1);
    static_assert(WAVES * rows <= 64, "a word for each lane");
};
template <int BM, int WAVES, int PARTS, int R, int C>
__device__ __forceinline__ bool f8_again(const F8GemmArgs& g, const f32x4 (&v)[R][C], int m0, int wm, int part, int n, float least,
                                         uint64_t* words) {
    constexpr int W = F8Words<BM, WAVES>::rows;
    constexpr uint64_t kEach = PARTS == 1 ? ~0ull : PARTS == 2 ? 0x5555555555555555ull : 0x1111111111111111ull;
    static_assert(PARTS == 1 || PARTS == 2 || PARTS == 4, "every PARTS-th row");
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), li = lane & 15;
    uint64_t *low_rows = words + WAVES, *zero_rows = low_rows + WAVES * W;
    float low[R];
    const bool bad = f8_lows(v, low);
    bool any = false;
#pragma unroll
    for (int i = 0; i < R; ++i) any |= low[i] < least;
    const bool small = f8_any(any);
    uint64_t mine[W] = {};                              // rows with a result below `least`
    if (__builtin_expect(small, 0)) {
#pragma unroll
        for (int i = 0; i < R; ++i) {
            const uint64_t rows = f8_rows_with(low[i] < least && m0 + wm + 16 * i + li < g.M);
#pragma unroll
            for (int w = 0; w < W; ++w)
                if ((wm + 16 * i) / 64 == w) mine[w] |= rows << (wm + 16 * i) % 64;
        }
        // a row of zeros is one in each of the waves with these rows, which share them out
#pragma unroll
        for (int w = 0; w < W; ++w) {
            const uint64_t own = mine[w] & kEach << part;
            const uint64_t zero = own & ~f8_hold(g.a + (int64_t)(m0 + 64 * w) * g.row_bytes, g.row_bytes, own);
            if (lane == 0) {
                low_rows[wave * W + w] = mine[w];
                zero_rows[wave * W + w] = zero;
            }
        }
    }
    if (lane == 0) words[wave] = (bad ? 2 : 0) | (small ? 1 : 0);
    __syncthreads();
    const uint64_t flags = lane < WAVES ? words[lane] : 0;
    if (__builtin_expect(!f8_any(flags != 0), 1)) return false;
    if (f8_any(flags & 2)) return true;
    // lane W k + w: rows 64 w .. of wave k that are left
    const bool in = lane < WAVES * W && words[lane / W];
    uint64_t zero = in ? zero_rows[lane] : 0;
#pragma unroll
    for (int k = W; k < WAVES * W; k *= 2) zero |= __shfl_xor(zero, k);
    if (!f8_any(in && (low_rows[lane] & ~zero))) return false;
    // and in those, columns that hold a code
    bool row[R];
#pragma unroll
    for (int i = 0; i < R; ++i) {
        const int w = (wm + 16 * i) / 64;
        uint64_t left = 0;
#pragma unroll
        for (int k = 0; k < W; ++k)
            if (k == w) left = mine[k] & ~__shfl(zero, k);
        row[i] = left >> ((wm + 16 * i) % 64 + li) & 1;
    }
    const bool yes = small && f8_columns(g, v, row, n, least);
    __syncthreads();                                    // the flags have been read
    if (lane == 0) words[wave] = yes;
    __syncthreads();
    return f8_any(lane < WAVES && words[lane]);
}

// The same of 16 x 16 results that one wave has.
__device__ __forceinline__ bool f8_again(const F8GemmArgs& g, const f32x4 (&v)[1][1], int m, int n, float least) {
    const int li = threadIdx.x & 15;
    float low[1];
    if (f8_lows(v, low)) return true;
    const uint64_t rows = f8_rows_with(low[0] < least && m + li < g.M);
    if (__builtin_expect(rows == 0, 1)) return false;
    const uint64_t found = f8_hold(g.a + (int64_t)m * g.row_bytes, g.row_bytes, rows);
    const bool row[1] = {(found >> li & 1) != 0};
    return found && f8_columns(g, v, row, n, least);
}

// Results go out before they are looked at, which then runs beside the stores (8192 x 8192 x 2048, an earlier form of
// it, behind them and ahead of them: 134.1 and 136.1 us), and once more where they were taken once more.  Results to
// be added to old ones wait.
template <class Store, class Again, class Redo>
__device__ __forceinline__ void f8_store(bool accumulate, bool look, Store store, Again again, Redo redo) {
    if (!accumulate) store();
    const bool more = look && again();
    if (more) redo();
    if (accumulate || more) store();
}

// A scale as f s for elements that are decoded, which bf16 has to hold with f:
//   |scale|              f        |s|
//   below 2^-63          2^-63    below 1
//   below 2^64           1        from 2^-63 to 2^64
//   the others           2^64     from 1 to 2^64
// No product of two s reaches 2^128, and one below 2^-126 has a result below 2^-150.  A product of
// two elements times fa fb leaves fp32's range only where that of the elements and their scales does.
struct F8Fold {
    float f, s;
};
__device__ __forceinline__ F8Fold f8_fold(float scale) {
    const float a = fabsf(scale), f = a < 0x1p-63f ? 0x1p-63f : a < 0x1p64f ? 1.0f : 0x1p64f;
    return {f, scale * __uint_as_float(0x7f000000u - __float_as_uint(f))};      // of a NaN, s is NaN
}

// The same for the 8-bit matrix instruction, which takes the byte e of 2^(e - 127) for each row: all of the
// exponent, s from 1 to 2 (below where the scale is subnormal).  e = 255 of a NaN makes the result one.
struct F8Parts {
    int e;
    float s;
};
__device__ __forceinline__ F8Parts f8_parts(float scale) {
    const int e = (int)(__float_as_uint(scale) >> 23 & 255u);
    return {e, __builtin_amdgcn_ldexpf(scale, 127 - e)};
}

// Eight codes times f -> bf16, exact: four or three significant bits, exponents from -16 to 15 and f's.
template <int FMT> __device__ __forceinline__ u32x4 f8_half8(uint32_t lo, uint32_t hi, float f = 1.0f) {
    u32x4 r;
    if constexpr (FMT == kF8E4M3) {
        r.x = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, f, false));
        r.y = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, f, true));
        r.z = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, f, false));
        r.w = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, f, true));
    } else {
        r.x = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_bf8(lo, f, false));
        r.y = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_bf8(lo, f, true));
        r.z = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_bf8(hi, f, false));
        r.w = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_bf8(hi, f, true));
    }
    return r;
}

#endif  // __HIPCC__

}  // namespace bitopt
