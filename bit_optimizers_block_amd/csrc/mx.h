// mx.h -- microscaled (MX) matrices: layout, scale rule, element conversions, and the
// argument blocks of the kernels that read and write them.
//
// A row of `cols` values is cut into blocks of 32.  A block is one scale byte s (the
// value 2^(s-127); 255 = NaN) and 32 elements in E2M1 (4 bits) or E4M3 (8 bits).  Rows
// are padded to 128 elements -- the contraction length of one scaled matrix instruction --
// with zero codes and zero scale bytes, so a product never has a ragged block and every
// row of codes starts on a 64-byte line.
#pragma once

#include <hip/hip_runtime.h>

#include "kernels.h"

namespace bitopt {

constexpr int kMxE2M1 = 0, kMxE4M3 = 1;
constexpr int kMxBlock = 32, kMxPad = 128;

__host__ __device__ constexpr int64_t mx_padded(int64_t cols) { return (cols + kMxPad - 1) / kMxPad * kMxPad; }
__host__ __device__ constexpr int64_t mx_code_bytes(int64_t cols, int fmt) {
    return fmt == kMxE2M1 ? mx_padded(cols) / 2 : mx_padded(cols);
}
__host__ __device__ constexpr int64_t mx_scale_bytes(int64_t cols) { return mx_padded(cols) / kMxBlock; }

// ------------------------------------------------------------------- kernel arguments

struct MxCodecArgs {
    const void* x; int64_t ldx;          // quantize: input, elements between rows
    void* out; int64_t ldo;              // dequantize: output
    uint8_t* codes; uint8_t* scales;
    int64_t rows, cols;
};

struct SwigluArgs {
    const void* gate; const void* up; const void* dy;
    void* y; void* dgate; void* dup;
    int64_t ldg, ldu, ldy, lddg, lddu;   // elements between rows; ldy: of y (forward) or dy (backward)
    uint8_t *gate_codes, *gate_scales, *up_codes, *up_scales;
    int64_t rows, cols;
};

// out[m][n] = sum_k A[m][k] B[n][k], fp32 sums, rounded once into out's type.  A is a
// 16-bit matrix (lda elements between rows) or an MX matrix; B is an MX matrix.  Which
// index of each lies along its rows is the kernel's template parameter.
struct MxGemmArgs {
    const void* a; int64_t lda;
    const uint8_t* a_scales;
    const uint8_t* b; const uint8_t* b_scales;
    void* out; int64_t ldo;
    int64_t a_row_bytes, a_row_scales;   // MX operands: bytes between rows of codes / scales
    int64_t b_row_bytes, b_row_scales;
    int32_t M, N, K;
    int32_t out_dtype, accumulate;
};

#ifdef __HIPCC__

// ------------------------------------------------------------------------- device side

typedef uint32_t u32x4a2 __attribute__((ext_vector_type(4), aligned(2)));
typedef uint32_t u32x2a2 __attribute__((ext_vector_type(2), aligned(2)));
typedef float f32x4a4 __attribute__((ext_vector_type(4), aligned(4)));
typedef int i32x8 __attribute__((ext_vector_type(8)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));

// 16 bytes at any address aligned to the element: one load or store (the hardware takes
// unaligned global accesses).  NT: with the non-temporal hint.
template <bool NT = false> __device__ __forceinline__ u32x4 ld16_a2(const void* p) {
    const BITOPT_GLOBAL u32x4a2* q = (const BITOPT_GLOBAL u32x4a2*)p;
    u32x4a2 v;
    if constexpr (NT) v = __builtin_nontemporal_load(q);
    else v = *q;
    return u32x4{v.x, v.y, v.z, v.w};
}
template <bool NT = false> __device__ __forceinline__ void st16_a2(void* p, u32x4 v) {
    const u32x4a2 w = {v.x, v.y, v.z, v.w};
    if constexpr (NT) __builtin_nontemporal_store(w, (BITOPT_GLOBAL u32x4a2*)p);
    else *(BITOPT_GLOBAL u32x4a2*)p = w;
}
__device__ __forceinline__ void st8_a2(void* p, u32x2 v) { *(BITOPT_GLOBAL u32x2a2*)p = u32x2a2{v.x, v.y}; }
template <bool NT = false> __device__ __forceinline__ f32x4 ld16_a4(const float* p) {
    const BITOPT_GLOBAL f32x4a4* q = (const BITOPT_GLOBAL f32x4a4*)p;
    f32x4a4 v;
    if constexpr (NT) v = __builtin_nontemporal_load(q);
    else v = *q;
    return f32x4{v.x, v.y, v.z, v.w};
}
template <bool NT = false> __device__ __forceinline__ void st16_a4(float* p, f32x4 v) {
    const f32x4a4 w = {v.x, v.y, v.z, v.w};
    if constexpr (NT) __builtin_nontemporal_store(w, (BITOPT_GLOBAL f32x4a4*)p);
    else *(BITOPT_GLOBAL f32x4a4*)p = w;
}

// The fp32 operand of the scaled conversions for scale byte s: they read its exponent
// field as an E8M0 byte (0 -> 2^-127, 255 -> NaN).
__device__ __forceinline__ float mx_scale_f32(uint32_t s) { return __uint_as_float(s << 23); }

// Scale byte of a block from the bits of its largest |x|: the smallest 2^e, e >= -127,
// with |x| <= top * 2^e.  top = 1.5 * 2^2 (E2M1) or 1.75 * 2^8 (E4M3), so e is the
// exponent of |x| less top's, plus one when its significand is above top's: no element
// saturates.  A subnormal |x| has exponent field 0, which the bound e >= -127 covers.
// Infinity or NaN anywhere in the block gives 255.
template <int FMT> __device__ __forceinline__ uint32_t mx_scale_byte(uint32_t amax_bits) {
    constexpr int top = FMT == kMxE2M1 ? 2 : 8;
    constexpr uint32_t frac = FMT == kMxE2M1 ? 0x400000u : 0x600000u;
    const int b = (int)(amax_bits >> 23) - top + ((amax_bits & 0x7fffffu) > frac ? 1 : 0);
    return amax_bits >= 0x7f800000u ? 255u : (uint32_t)max(b, 0);
}

// 2^-e for scale byte e + 127 <= 253: exact, and always a normal number.
__device__ __forceinline__ float mx_inverse_scale(uint32_t s) { return __uint_as_float((254u - s) << 23); }

// Four scaled values -> codes (nearest, ties to even; -0 keeps its sign).
__device__ __forceinline__ uint32_t mx_encode4_e2m1(const float v[4]) {
    uint32_t r = 0;
    r = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(r, v[0], v[1], 1.0f, 0);
    return __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(r, v[2], v[3], 1.0f, 1);
}
__device__ __forceinline__ uint32_t mx_encode4_e4m3(const float v[4]) {
    int r = 0;
    r = __builtin_amdgcn_cvt_pk_fp8_f32(v[0], v[1], r, false);
    return (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(v[2], v[3], r, true);
}

// Four codes -> fp32 (exact: the smallest product, 2^-9 * 2^-127, is an fp32 subnormal).
__device__ __forceinline__ void mx_decode4_e2m1(uint32_t c, float s, float v[4]) {
    f32x2 p;
    p = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c, s, 0); v[0] = p.x; v[1] = p.y;
    p = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c, s, 1); v[2] = p.x; v[3] = p.y;
}
__device__ __forceinline__ void mx_decode4_e4m3(uint32_t c, float s, float v[4]) {
    f32x2 p;
    p = __builtin_amdgcn_cvt_scalef32_pk_f32_fp8(c, s, false); v[0] = p.x; v[1] = p.y;
    p = __builtin_amdgcn_cvt_scalef32_pk_f32_fp8(c, s, true); v[2] = p.x; v[3] = p.y;
}

// Codes -> 16-bit values, rounded to nearest even (exact in bf16 above its subnormals;
// fp16 overflows to infinity beyond 65504 and rounds below 2^-14).  8 values in 4 words.
template <int DT> __device__ __forceinline__ u32x4 mx_half8_e2m1(uint32_t c, float s) {
    u32x4 r;
    if constexpr (DT == kBF16) {
        r.x = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(c, s, 0));
        r.y = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(c, s, 1));
        r.z = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(c, s, 2));
        r.w = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(c, s, 3));
    } else {
        r.x = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(c, s, 0));
        r.y = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(c, s, 1));
        r.z = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(c, s, 2));
        r.w = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(c, s, 3));
    }
    return r;
}
template <int DT> __device__ __forceinline__ u32x4 mx_half8_e4m3(uint32_t c0, uint32_t c1, float s) {
    u32x4 r;
    if constexpr (DT == kBF16) {
        r.x = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(c0, s, false));
        r.y = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(c0, s, true));
        r.z = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(c1, s, false));
        r.w = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(c1, s, true));
    } else {
        r.x = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(c0, s, false));
        r.y = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(c0, s, true));
        r.z = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(c1, s, false));
        r.w = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(c1, s, true));
    }
    return r;
}

// Eight 16-bit elements moved d places down (1 <= d <= 7), zeros from above.
__device__ __forceinline__ u32x4 half_shift(u32x4 r, int d) {
#pragma unroll
    for (int w = 0; w < 3; ++w)
        if (d >= 2 * (w + 1)) r = u32x4{r.y, r.z, r.w, 0u};
    // two places a word above; now half of one
    if (d & 1)
        r = u32x4{__builtin_amdgcn_alignbit(r.y, r.x, 16), __builtin_amdgcn_alignbit(r.z, r.y, 16),
                  __builtin_amdgcn_alignbit(r.w, r.z, 16), r.w >> 16};
    return r;
}

// Eight 16-bit elements from any 2-byte-aligned address; the first `n` of them, the rest
// zero, when n < 8.  Where the row holds eight elements up to there (`before` of them precede
// p), they are the last of one load that ends with the row; only shorter rows are read
// element by element, which waits for every element.
template <bool NT = false> __device__ __forceinline__ u32x4 ld_half8(const uint16_t* p, int n, int64_t before) {
    if (n >= 8) return ld16_a2<NT>(p);
    u32x4 r = {0u, 0u, 0u, 0u};
    if (n <= 0) return r;
    if (before + n >= 8) return half_shift(ld16_a2<NT>(p - (8 - n)), 8 - n);
#pragma unroll
    for (int j = 0; j < 8; ++j)
        if (j < n) r[j / 2] |= (uint32_t)gbl(p)[j] << (16 * (j & 1));
    return r;
}

template <int DT> __device__ __forceinline__ f32x4 mfma16(u32x4 a, u32x4 b, f32x4 c) {
    if constexpr (DT == kBF16)
        return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b), c,
                                                       0, 0, 0);
    else
        return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8, a), __builtin_bit_cast(f16x8, b), c, 0,
                                                      0, 0);
}

// Four lane groups q hold dwords d[q] with bytes d[q][0..3]; afterwards group q holds
// d[0..3][q].
__device__ __forceinline__ uint32_t transpose_bytes(uint32_t d, int lane) {
    const auto a = __builtin_amdgcn_permlane32_swap(d, d, false, false);
    // a[0]: the dword of group q % 2, a[1]: of group 2 + q % 2; keep the byte pair q / 2 of both
    const uint32_t pair = __builtin_amdgcn_perm(a[1], a[0], lane & 32 ? 0x07060302u : 0x05040100u);
    const auto b = __builtin_amdgcn_permlane16_swap(pair, pair, false, false);
    // b[0]: rows 0 and 2 of the pair, b[1]: rows 1 and 3; keep byte q % 2 of each row
    return __builtin_amdgcn_perm(b[1], b[0], lane & 16 ? 0x07030501u : 0x06020400u);
}

// Scaled product of 16 x 128 E2M1 codes: lane l holds row l % 16 and block l / 16 of both
// operands, and that block's scale in byte BYTE of sa / sb.
template <int BYTE>
__device__ __forceinline__ f32x4 mfma_e2m1_at(u32x4 a, u32x4 b, f32x4 c, uint32_t sa, uint32_t sb) {
    const i32x8 x = {(int)a.x, (int)a.y, (int)a.z, (int)a.w, 0, 0, 0, 0};
    const i32x8 y = {(int)b.x, (int)b.y, (int)b.z, (int)b.w, 0, 0, 0, 0};
    return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(x, y, c, 4, 4, BYTE, (int)sa, BYTE, (int)sb);
}

// Four consecutive output elements of a row, columns n .. n+3 (those below N), with the
// old values added first when `accumulate`.  Args has out, ldo, out_dtype, accumulate, M and N.
template <class Args> __device__ __forceinline__ void mx_store4(const Args& g, int64_t m, int n, f32x4 v) {
    const int64_t e = m * g.ldo + n;
    const bool whole = n + 4 <= g.N;
    if (g.out_dtype == kF32) {
        float* o = reinterpret_cast<float*>(g.out) + e;
        if (whole) {
            if (g.accumulate) v += ld16_a4(o);
            st16_a4(o, v);
        } else {
#pragma unroll
            for (int j = 0; j < 4; ++j)
                if (n + j < g.N) gbl(o)[j] = g.accumulate ? gbl(o)[j] + v[j] : v[j];
        }
        return;
    }
    uint16_t* o = reinterpret_cast<uint16_t*>(g.out) + e;
    const bool bf = g.out_dtype == kBF16;
    if (g.accumulate) {
#pragma unroll
        for (int j = 0; j < 4; ++j)
            if (n + j < g.N) v[j] += bf ? widen<kBF16>(gbl(o)[j]) : widen<kF16>(gbl(o)[j]);
    }
    const uint32_t lo = bf ? narrow2<kBF16>(v[0], v[1]) : narrow2<kF16>(v[0], v[1]);
    const uint32_t hi = bf ? narrow2<kBF16>(v[2], v[3]) : narrow2<kF16>(v[2], v[3]);
    if (whole) {
        st8_a2(o, u32x2{lo, hi});
    } else {
        if (n < g.N) gbl(o)[0] = (uint16_t)lo;
        if (n + 1 < g.N) gbl(o)[1] = (uint16_t)(lo >> 16);
        if (n + 2 < g.N) gbl(o)[2] = (uint16_t)hi;
    }
}

// Two neighbouring 16 x 16 result tiles of row m, columns n .. n+31: lane group q holds
// columns 4 q .. + 3 of both.  16-bit results are exchanged between neighbouring groups
// first, so a lane stores eight consecutive columns and a row gets whole 64-byte segments.
template <class Args>
__device__ __forceinline__ void mx_store_pair(const Args& g, int64_t m, int n, int q, f32x4 v, f32x4 w) {
    if (g.out_dtype == kF32 || g.accumulate || n + 32 > g.N) {
        if (m >= g.M) return;
        if (n + 4 * q < g.N) mx_store4(g, m, n + 4 * q, v);
        if (n + 16 + 4 * q < g.N) mx_store4(g, m, n + 16 + 4 * q, w);
        return;
    }
    const bool bf = g.out_dtype == kBF16;
    const uint32_t v0 = bf ? narrow2<kBF16>(v[0], v[1]) : narrow2<kF16>(v[0], v[1]);
    const uint32_t v1 = bf ? narrow2<kBF16>(v[2], v[3]) : narrow2<kF16>(v[2], v[3]);
    const uint32_t w0 = bf ? narrow2<kBF16>(w[0], w[1]) : narrow2<kF16>(w[0], w[1]);
    const uint32_t w1 = bf ? narrow2<kBF16>(w[2], w[3]) : narrow2<kF16>(w[2], w[3]);
    // odd groups of the first operand change places with even groups of the second
    const auto a = __builtin_amdgcn_permlane16_swap(v0, w0, false, false);
    const auto b = __builtin_amdgcn_permlane16_swap(v1, w1, false, false);
    // group q: tile q % 2, columns 8 (q / 2) .. + 7
    if (m < g.M)
        st16_a2(reinterpret_cast<uint16_t*>(g.out) + m * g.ldo + n + 16 * (q & 1) + 8 * (q >> 1),
                u32x4{a[0], b[0], a[1], b[1]});
}

// Output tile of a workgroup.  Workgroups go round the 8 XCDs in turn, and each XCD has
// its own L2: give XCD x the x-th contiguous run of tiles, and walk a run in columns of
// four row tiles, so the tiles an XCD works on at once share operand rows (eight: 2% slower).
__device__ __forceinline__ void mx_tile(int tiles_m, int tiles_n, int& tm, int& tn) {
    constexpr int kXcd = 8, kGroup = 4;
    const int n = tiles_m * tiles_n;
    const int x = blockIdx.x % kXcd, i = blockIdx.x / kXcd;
    const int id = x * (n / kXcd) + min(x, n % kXcd) + i;
    const int per = kGroup * tiles_n;
    const int g = id / per, first = g * kGroup;
    const int h = min(kGroup, tiles_m - first);
    tm = first + (id - g * per) % h;
    tn = (id - g * per) / h;
}

#endif  // __HIPCC__

}  // namespace bitopt
