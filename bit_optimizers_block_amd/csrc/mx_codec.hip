// MX codec and SwiGLU with its inputs kept in MX E4M3.
//
// Every kernel here reads and writes each element once and is bound by HBM.  A lane takes
// eight consecutive elements of a row (a 16-byte load of 16-bit values), four lanes make
// a block of 32, and the block maximum meets in two DPP exchanges, so codes leave the
// registers without LDS or a second pass.
#include <algorithm>

#include "launch.h"
#include "mx.h"

namespace bitopt {

// Lanes along a row: 2^lanes_log2 of a workgroup's 256, the rest of the workgroup takes
// further rows; `steps` row groups per workgroup.
struct RowGrid {
    int32_t lanes_log2, chunks, steps;
};

constexpr int kRowSteps = 4;

static RowGrid row_grid(int64_t rows, int64_t cols, dim3& grid) {
    RowGrid g{};
    const int64_t items = mx_padded(cols) / 8;
    g.lanes_log2 = 4;
    while (g.lanes_log2 < 8 && (int64_t{1} << g.lanes_log2) < items) ++g.lanes_log2;
    g.chunks = (int32_t)((items + (int64_t{1} << g.lanes_log2) - 1) >> g.lanes_log2);
    const int64_t per = kThreads >> g.lanes_log2;
    const int64_t groups = (rows + per - 1) / per;
    g.steps = groups * g.chunks >= 4096 ? kRowSteps : 1;
    grid = dim3((unsigned)g.chunks, (unsigned)std::min<int64_t>((groups + g.steps - 1) / g.steps, 65535));
    return g;
}

// Eight elements of a row as fp32, from any address aligned to the element; zeros from
// element n on.
template <int DT> __device__ __forceinline__ void ld8(const void* base, int64_t e, int n, float v[8]) {
    if constexpr (DT == kF32) {
        const float* p = reinterpret_cast<const float*>(base) + e;
        if (n >= 8) {
            const f32x4 a = ld16_a4(p), b = ld16_a4(p + 4);
#pragma unroll
            for (int j = 0; j < 4; ++j) { v[j] = a[j]; v[4 + j] = b[j]; }
        } else {
#pragma unroll
            for (int j = 0; j < 8; ++j) v[j] = j < n ? gbl(p)[j] : 0.0f;
        }
    } else {
        const u32x4 r = ld_half8(reinterpret_cast<const uint16_t*>(base) + e, n);
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] = widen<DT>(r[j / 2] >> (16 * (j & 1)));
    }
}

template <int DT> __device__ __forceinline__ void st8(void* base, int64_t e, int n, const float v[8]) {
    if constexpr (DT == kF32) {
        float* p = reinterpret_cast<float*>(base) + e;
        if (n >= 8) {
            st16_a4(p, f32x4{v[0], v[1], v[2], v[3]});
            st16_a4(p + 4, f32x4{v[4], v[5], v[6], v[7]});
        } else {
#pragma unroll
            for (int j = 0; j < 8; ++j)
                if (j < n) gbl(p)[j] = v[j];
        }
    } else {
        uint16_t* p = reinterpret_cast<uint16_t*>(base) + e;
        const u32x4 r = {narrow2<DT>(v[0], v[1]), narrow2<DT>(v[2], v[3]), narrow2<DT>(v[4], v[5]),
                         narrow2<DT>(v[6], v[7])};
        if (n >= 8) {
            st16_a2(p, r);
        } else {
#pragma unroll
            for (int j = 0; j < 8; ++j)
                if (j < n) gbl(p)[j] = (uint16_t)(r[j / 2] >> (16 * (j & 1)));
        }
    }
}

// Codes of the eight elements of this lane and the scale byte of its block; the block's
// other elements are in the neighbouring lanes of the aligned group of four.
template <int FMT>
__device__ __forceinline__ void encode8(const float x[8], uint32_t c[FMT == kMxE2M1 ? 1 : 2], uint32_t& scale) {
    // the maximum on bit patterns: |NaN| > infinity > every finite value
    uint32_t m = 0;
#pragma unroll
    for (int j = 0; j < 8; ++j) m = max(m, __float_as_uint(x[j]) & 0x7fffffffu);
    m = max(m, (uint32_t)__builtin_amdgcn_mov_dpp((int)m, 0xB1, 0xF, 0xF, true));   // quad_perm 1,0,3,2
    m = max(m, (uint32_t)__builtin_amdgcn_mov_dpp((int)m, 0x4E, 0xF, 0xF, true));   // quad_perm 2,3,0,1
    scale = mx_scale_byte<FMT>(m);
    const bool bad = scale == 255u;
    const float inv = mx_inverse_scale(bad ? 127u : scale);
    float v[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = x[j] * inv;
    if constexpr (FMT == kMxE2M1) {
        c[0] = bad ? 0u : mx_encode8_e2m1(v);
    } else {
        c[0] = bad ? 0u : mx_encode4_e4m3(v[0], v[1], v[2], v[3]);
        c[1] = bad ? 0u : mx_encode4_e4m3(v[4], v[5], v[6], v[7]);
    }
}

template <int FMT>
__device__ __forceinline__ void st_codes(uint8_t* codes, uint8_t* scales, int64_t row, int64_t padded, int32_t item,
                                         const uint32_t c[FMT == kMxE2M1 ? 1 : 2], uint32_t scale) {
    if constexpr (FMT == kMxE2M1)
        gbl(reinterpret_cast<uint32_t*>(codes))[row * (padded / 8) + item] = c[0];
    else
        gbl(reinterpret_cast<u32x2*>(codes))[row * (padded / 8) + item] = u32x2{c[0], c[1]};
    if ((item & 3) == 0) gbl(scales)[row * (padded / kMxBlock) + item / 4] = (uint8_t)scale;
}

template <int FMT>
__device__ __forceinline__ void ld_codes(const uint8_t* codes, const uint8_t* scales, int64_t row, int64_t padded,
                                         int32_t item, float v[8]) {
    const float s = mx_scale_f32(gbl(scales)[row * (padded / kMxBlock) + item / 4]);
    if constexpr (FMT == kMxE2M1) {
        mx_decode8_e2m1(gbl(reinterpret_cast<const uint32_t*>(codes))[row * (padded / 8) + item], s, v);
    } else {
        const u32x2 c = gbl(reinterpret_cast<const u32x2*>(codes))[row * (padded / 8) + item];
        mx_decode4_e4m3(c.x, s, v);
        mx_decode4_e4m3(c.y, s, v + 4);
    }
}

// Runs f(row, item) for every eight-element item of the padded rows.  All four lanes of a
// block are in or out together (items per row is a multiple of 16).
template <class F> __device__ __forceinline__ void for_items(const RowGrid& g, int64_t rows, int32_t items, F f) {
    const int lanes = 1 << g.lanes_log2;
    const int32_t item = (int32_t)blockIdx.x * lanes + ((int)threadIdx.x & (lanes - 1));
    const int64_t per = kThreads >> g.lanes_log2;
    if (item >= items) return;
    const int64_t stride = per * gridDim.y;
    int64_t row = per * blockIdx.y + (threadIdx.x >> g.lanes_log2);
    for (; row + (kRowSteps - 1) * stride < rows; row += kRowSteps * stride) {
#pragma unroll
        for (int s = 0; s < kRowSteps; ++s) f(row + s * stride, item);
    }
    for (; row < rows; row += stride) f(row, item);
}

__device__ __forceinline__ int item_elems(int64_t cols, int32_t item) {
    return (int)max((int64_t)0, min((int64_t)8, cols - 8 * (int64_t)item));
}

template <int DT, int FMT> __global__ __launch_bounds__(kThreads) void k_mx_quantize(MxCodecArgs a, RowGrid g) {
    const int64_t padded = mx_padded(a.cols);
    for_items(g, a.rows, (int32_t)(padded / 8), [&](int64_t row, int32_t item) {
        float v[8];
        uint32_t c[2], s;
        ld8<DT>(a.x, row * a.ldx + 8 * (int64_t)item, item_elems(a.cols, item), v);
        encode8<FMT>(v, c, s);
        st_codes<FMT>(a.codes, a.scales, row, padded, item, c, s);
    });
}

template <int DT, int FMT> __global__ __launch_bounds__(kThreads) void k_mx_dequantize(MxCodecArgs a, RowGrid g) {
    const int64_t padded = mx_padded(a.cols);
    for_items(g, a.rows, (int32_t)(padded / 8), [&](int64_t row, int32_t item) {
        float v[8];
        ld_codes<FMT>(a.codes, a.scales, row, padded, item, v);
        st8<DT>(a.out, row * a.ldo + 8 * (int64_t)item, item_elems(a.cols, item), v);
    });
}

// 1 / (1 + exp(-g)): 0 and 1 at the infinities.  fp32 results take the library's expf;
// for 16-bit ones exp2 of the rounded product (relative error |g| 2^-24, against half a
// step of 2^-9 or 2^-12) costs a fifth of it.
template <int DT> __device__ __forceinline__ float sigmoid(float g) {
    const float e = DT == kF32 ? expf(-g) : __builtin_amdgcn_exp2f(-1.44269504088896341f * g);
    return __builtin_amdgcn_rcpf(1.0f + e);
}

// y = gate * sigmoid(gate) * up, and both inputs in MX E4M3.
template <int DT> __global__ __launch_bounds__(kThreads) void k_swiglu_forward(SwigluArgs a, RowGrid g) {
    const int64_t padded = mx_padded(a.cols);
    for_items(g, a.rows, (int32_t)(padded / 8), [&](int64_t row, int32_t item) {
        const int n = item_elems(a.cols, item);
        const int64_t e = 8 * (int64_t)item;
        float x[8], u[8], y[8];
        uint32_t c[2], s;
        ld8<DT>(a.gate, row * a.ldg + e, n, x);
        ld8<DT>(a.up, row * a.ldu + e, n, u);
#pragma unroll
        for (int j = 0; j < 8; ++j) y[j] = x[j] * sigmoid<DT>(x[j]) * u[j];
        st8<DT>(a.y, row * a.ldy + e, n, y);
        encode8<kMxE4M3>(x, c, s);
        st_codes<kMxE4M3>(a.gate_codes, a.gate_scales, row, padded, item, c, s);
        encode8<kMxE4M3>(u, c, s);
        st_codes<kMxE4M3>(a.up_codes, a.up_scales, row, padded, item, c, s);
    });
}

// With s = sigmoid(g): dgate = dy u (s + g s (1 - s)), dup = dy g s, at the saved values.
template <int DT> __global__ __launch_bounds__(kThreads) void k_swiglu_backward(SwigluArgs a, RowGrid g) {
    const int64_t padded = mx_padded(a.cols);
    for_items(g, a.rows, (int32_t)(padded / 8), [&](int64_t row, int32_t item) {
        const int n = item_elems(a.cols, item);
        const int64_t e = 8 * (int64_t)item;
        float x[8], u[8], d[8], dg[8], du[8];
        ld8<DT>(a.dy, row * a.ldy + e, n, d);
        ld_codes<kMxE4M3>(a.gate_codes, a.gate_scales, row, padded, item, x);
        ld_codes<kMxE4M3>(a.up_codes, a.up_scales, row, padded, item, u);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const float s = sigmoid<DT>(x[j]);
            dg[j] = d[j] * u[j] * s * (1.0f + x[j] * (1.0f - s));
            du[j] = d[j] * x[j] * s;
        }
        st8<DT>(a.dgate, row * a.lddg + e, n, dg);
        st8<DT>(a.dup, row * a.lddu + e, n, du);
    });
}

// ------------------------------------------------------------------------- launches

#define BITOPT_MX_LAUNCH(kernel, args)                                              \
    do {                                                                            \
        dim3 grid;                                                                  \
        const RowGrid g = row_grid((args).rows, (args).cols, grid);                 \
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
