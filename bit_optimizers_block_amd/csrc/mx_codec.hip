// MX codec and SwiGLU with its inputs kept in MX E4M3.
//
// Every kernel here reads and writes each element once and is bound by HBM.  A lane takes
// 16 bytes of a row (four fp32 or eight 16-bit elements), so a wave's loads and stores are
// whole lines; eight or four lanes make a block of 32, and the block maximum meets in DPP
// exchanges, so codes leave the registers without LDS or a second pass.
//
// Hints, us at 8192 x 8192 bf16 and 16384 x 8192 bf16: SwiGLU's tensors are past every cache,
// and streaming them takes the forward pass from 98 to 85 and the backward pass from 99 to
// 84.  dequantize streams its result (E2M1 68 -> 52).  quantize reads what was just computed:
// its loads keep the caches (streaming: 60 -> 58 from HBM, but 8.3 -> 9.2 where 8192 x 2048
// still lies in the Infinity Cache), and so do codes, which the next call reads.
#include "launch.h"
#include "mx_rows.h"

namespace bitopt {

// Codes of this lane's item: bytes per item, and the type that holds them.
template <int DT, int FMT> constexpr int kCodeBytes = FMT == kMxE2M1 ? kPer<DT> / 2 : kPer<DT>;
template <int BYTES> struct CodeWord;
template <> struct CodeWord<2> { using T = uint16_t; };
template <> struct CodeWord<4> { using T = uint32_t; };
template <> struct CodeWord<8> { using T = u32x2; };

// Codes of this lane's item and the scale byte of its block; the block's other elements are
// in the neighbouring lanes of the aligned group of 32 / kPer.
template <int DT, int FMT> __device__ __forceinline__ void encode(const float x[kPer<DT>], uint32_t c[2], uint32_t& scale) {
    // the maximum on bit patterns: |NaN| > infinity > every finite value
    uint32_t m = 0;
#pragma unroll
    for (int j = 0; j < kPer<DT>; ++j) m = max(m, __float_as_uint(x[j]) & 0x7fffffffu);
    m = max(m, (uint32_t)__builtin_amdgcn_mov_dpp((int)m, 0xB1, 0xF, 0xF, true));   // quad_perm 1,0,3,2
    m = max(m, (uint32_t)__builtin_amdgcn_mov_dpp((int)m, 0x4E, 0xF, 0xF, true));   // quad_perm 2,3,0,1
    if constexpr (kPer<DT> == 4)
        m = max(m, (uint32_t)__builtin_amdgcn_mov_dpp((int)m, 0x141, 0xF, 0xF, true));   // row_half_mirror
    scale = mx_scale_byte<FMT>(m);
    const bool bad = scale == 255u;
    const float inv = mx_inverse_scale(bad ? 127u : scale);
    float v[kPer<DT>];
#pragma unroll
    for (int j = 0; j < kPer<DT>; ++j) v[j] = x[j] * inv;
#pragma unroll
    for (int h = 0; h < kPer<DT> / 4; ++h) {
        const uint32_t w = FMT == kMxE2M1 ? mx_encode4_e2m1(v + 4 * h) : mx_encode4_e4m3(v + 4 * h);
        c[h] = bad ? 0u : w;
    }
}

template <int DT, int FMT>
__device__ __forceinline__ void st_codes(uint8_t* codes, uint8_t* scales, int64_t row, int64_t padded, int32_t item,
                                         const uint32_t c[2], uint32_t scale) {
    constexpr int B = kCodeBytes<DT, FMT>, LANES = kMxBlock / kPer<DT>;
    using T = typename CodeWord<B>::T;
    T w;
    if constexpr (B == 8) w = u32x2{c[0], c[1]};
    else if constexpr (FMT == kMxE2M1 && B == 4) w = c[0] | c[1] << 16;
    else w = (T)c[0];
    gbl(reinterpret_cast<T*>(codes))[row * (padded / kPer<DT>) + item] = w;
    if (item % LANES == 0) gbl(scales)[row * (padded / kMxBlock) + item / LANES] = (uint8_t)scale;
}

template <int DT, int FMT>
__device__ __forceinline__ void ld_codes(const uint8_t* codes, const uint8_t* scales, int64_t row, int64_t padded,
                                         int32_t item, float v[kPer<DT>]) {
    using T = typename CodeWord<kCodeBytes<DT, FMT>>::T;
    const float s = mx_scale_f32(gbl(scales)[row * (padded / kMxBlock) + item / (kMxBlock / kPer<DT>)]);
    const T w = gbl(reinterpret_cast<const T*>(codes))[row * (padded / kPer<DT>) + item];
#pragma unroll
    for (int h = 0; h < kPer<DT> / 4; ++h) {
        if constexpr (FMT == kMxE2M1) mx_decode4_e2m1((uint32_t)w >> (16 * h), s, v + 4 * h);
        else if constexpr (kPer<DT> == 4) mx_decode4_e4m3((uint32_t)w, s, v);
        else mx_decode4_e4m3(w[h], s, v + 4 * h);
    }
}

template <int DT, int FMT> __global__ __launch_bounds__(kThreads) void k_mx_quantize(MxCodecArgs a, RowGrid g) {
    const int64_t padded = mx_padded(a.cols);
    for_items(g, a.rows, (int32_t)(padded / kPer<DT>), [&](int64_t row, int32_t item) {
        float v[kPer<DT>];
        uint32_t c[2], s;
        ld_item<DT, false>(a.x, row * a.ldx + kPer<DT> * (int64_t)item, item_elems<DT>(a.cols, item), kPer<DT> * (int64_t)item, v);
        encode<DT, FMT>(v, c, s);
        st_codes<DT, FMT>(a.codes, a.scales, row, padded, item, c, s);
    });
}

template <int DT, int FMT> __global__ __launch_bounds__(kThreads) void k_mx_dequantize(MxCodecArgs a, RowGrid g) {
    const int64_t padded = mx_padded(a.cols);
    for_items(g, a.rows, (int32_t)(padded / kPer<DT>), [&](int64_t row, int32_t item) {
        float v[kPer<DT>];
        ld_codes<DT, FMT>(a.codes, a.scales, row, padded, item, v);
        st_item<DT>(a.out, row * a.ldo + kPer<DT> * (int64_t)item, item_elems<DT>(a.cols, item), v);
    });
}

// 1 / (1 + exp(-g)): 0 and 1 at the infinities.  fp32 results take the library's expf;
// for 16-bit ones exp2 of the rounded product (relative error |g| 2^-24, against half a
// step of 2^-9 or 2^-12) costs a fifth of it.  The reciprocal gives zero for results below
// 2^-126 (g below -87.34): what is lost is below |g| 2^-126 times the other factor.
template <int DT> __device__ __forceinline__ float sigmoid(float g) {
    const float e = DT == kF32 ? expf(-g) : __builtin_amdgcn_exp2f(-1.44269504088896341f * g);
    return __builtin_amdgcn_rcpf(1.0f + e);
}

// y = gate * sigmoid(gate) * up, and both inputs in MX E4M3.  y may lie over gate or up (and in
// the backward pass dgate or dup over dy): a lane reads its item before it writes it, and what the
// last item's load takes from the item before is shifted out.
template <int DT> __global__ __launch_bounds__(kThreads) void k_swiglu_forward(SwigluArgs a, RowGrid g) {
    const int64_t padded = mx_padded(a.cols);
    for_items(g, a.rows, (int32_t)(padded / kPer<DT>), [&](int64_t row, int32_t item) {
        const int n = item_elems<DT>(a.cols, item);
        const int64_t e = kPer<DT> * (int64_t)item;
        float x[kPer<DT>], u[kPer<DT>], y[kPer<DT>];
        uint32_t c[2], s;
        ld_item<DT, true>(a.gate, row * a.ldg + e, n, e, x);
        ld_item<DT, true>(a.up, row * a.ldu + e, n, e, u);
#pragma unroll
        for (int j = 0; j < kPer<DT>; ++j) y[j] = x[j] * sigmoid<DT>(x[j]) * u[j];
        st_item<DT>(a.y, row * a.ldy + e, n, y);
        encode<DT, kMxE4M3>(x, c, s);
        st_codes<DT, kMxE4M3>(a.gate_codes, a.gate_scales, row, padded, item, c, s);
        encode<DT, kMxE4M3>(u, c, s);
        st_codes<DT, kMxE4M3>(a.up_codes, a.up_scales, row, padded, item, c, s);
    });
}

// With s = sigmoid(g): dgate = dy u (s + g s (1 - s)), dup = dy g s, at the saved values.
template <int DT> __global__ __launch_bounds__(kThreads) void k_swiglu_backward(SwigluArgs a, RowGrid g) {
    const int64_t padded = mx_padded(a.cols);
    for_items(g, a.rows, (int32_t)(padded / kPer<DT>), [&](int64_t row, int32_t item) {
        const int n = item_elems<DT>(a.cols, item);
        const int64_t e = kPer<DT> * (int64_t)item;
        float x[kPer<DT>], u[kPer<DT>], d[kPer<DT>], dg[kPer<DT>], du[kPer<DT>];
        ld_item<DT, true>(a.dy, row * a.ldy + e, n, e, d);
        ld_codes<DT, kMxE4M3>(a.gate_codes, a.gate_scales, row, padded, item, x);
        ld_codes<DT, kMxE4M3>(a.up_codes, a.up_scales, row, padded, item, u);
#pragma unroll
        for (int j = 0; j < kPer<DT>; ++j) {
            const float s = sigmoid<DT>(x[j]);
            dg[j] = d[j] * u[j] * s * (1.0f + x[j] * (1.0f - s));
            du[j] = d[j] * x[j] * s;
        }
        st_item<DT>(a.dgate, row * a.lddg + e, n, dg);
        st_item<DT>(a.dup, row * a.lddu + e, n, du);
    });
}

// ------------------------------------------------------------------------- launches

#define BITOPT_MX_LAUNCH(kernel, args)                                              \
    do {                                                                            \
        dim3 grid;                                                                  \
        const RowGrid g = row_grid((args).rows, mx_padded((args).cols) / (dtype == kF32 ? 4 : 8), grid); \
        hipLaunchKernelGGL(HIP_KERNEL_NAME(kernel), grid, dim3(kThreads), 0, s, args, g); \
        return hipGetLastError();                                                   \
    } while (0)

hipError_t launch_mx_quantize(const MxCodecArgs& a, int dtype, int fmt, hipStream_t s) {
    const bool four = fmt == kMxE2M1;
    if (dtype == kF32 && four) BITOPT_MX_LAUNCH((k_mx_quantize<kF32, kMxE2M1>), a);
    if (dtype == kF16 && four) BITOPT_MX_LAUNCH((k_mx_quantize<kF16, kMxE2M1>), a);
    if (dtype == kBF16 && four) BITOPT_MX_LAUNCH((k_mx_quantize<kBF16, kMxE2M1>), a);
    if (dtype == kF32) BITOPT_MX_LAUNCH((k_mx_quantize<kF32, kMxE4M3>), a);
    if (dtype == kF16) BITOPT_MX_LAUNCH((k_mx_quantize<kF16, kMxE4M3>), a);
    BITOPT_MX_LAUNCH((k_mx_quantize<kBF16, kMxE4M3>), a);
}

hipError_t launch_mx_dequantize(const MxCodecArgs& a, int dtype, int fmt, hipStream_t s) {
    const bool four = fmt == kMxE2M1;
    if (dtype == kF32 && four) BITOPT_MX_LAUNCH((k_mx_dequantize<kF32, kMxE2M1>), a);
    if (dtype == kF16 && four) BITOPT_MX_LAUNCH((k_mx_dequantize<kF16, kMxE2M1>), a);
    if (dtype == kBF16 && four) BITOPT_MX_LAUNCH((k_mx_dequantize<kBF16, kMxE2M1>), a);
    if (dtype == kF32) BITOPT_MX_LAUNCH((k_mx_dequantize<kF32, kMxE4M3>), a);
    if (dtype == kF16) BITOPT_MX_LAUNCH((k_mx_dequantize<kF16, kMxE4M3>), a);
    BITOPT_MX_LAUNCH((k_mx_dequantize<kBF16, kMxE4M3>), a);
}

hipError_t launch_swiglu_forward(const SwigluArgs& a, int dtype, hipStream_t s) {
    if (dtype == kF32) BITOPT_MX_LAUNCH(k_swiglu_forward<kF32>, a);
    if (dtype == kF16) BITOPT_MX_LAUNCH(k_swiglu_forward<kF16>, a);
    BITOPT_MX_LAUNCH(k_swiglu_forward<kBF16>, a);
}

hipError_t launch_swiglu_backward(const SwigluArgs& a, int dtype, hipStream_t s) {
    if (dtype == kF32) BITOPT_MX_LAUNCH(k_swiglu_backward<kF32>, a);
    if (dtype == kF16) BITOPT_MX_LAUNCH(k_swiglu_backward<kF16>, a);
    BITOPT_MX_LAUNCH(k_swiglu_backward<kBF16>, a);
}

}  // namespace bitopt
