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
constexpr int kF8Rows = 0, kF8Tiles = 1;
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

// Eight codes -> bf16, exact: four or three significant bits, exponents from -16 to 15.
template <int FMT> __device__ __forceinline__ u32x4 f8_half8(uint32_t lo, uint32_t hi) {
    u32x4 r;
    if constexpr (FMT == kF8E4M3) {
        r.x = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, 1.0f, false));
        r.y = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, 1.0f, true));
        r.z = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, 1.0f, false));
        r.w = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, 1.0f, true));
    } else {
        r.x = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_bf8(lo, 1.0f, false));
        r.y = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_bf8(lo, 1.0f, true));
        r.z = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_bf8(hi, 1.0f, false));
        r.w = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_bf8(hi, 1.0f, true));
    }
    return r;
}

#endif  // __HIPCC__

}  // namespace bitopt
