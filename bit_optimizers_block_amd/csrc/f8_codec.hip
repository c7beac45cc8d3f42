// F8 codec: a matrix to 8 bits, itself, its transpose or both from one reading, and back.
//
// Bound by HBM: the input is read once, the codes written once.  Row blocks alone: a lane takes
// eight elements, sixteen lanes make a block, whose maximum meets in DPP exchanges.  Tiles and
// transposes: a workgroup takes a tile of 128 x 128 into registers, a lane 8 rows by 8 columns;
// sixteen lanes side by side hold a row of the tile, and a lane's eight rows are eight consecutive
// codes of the transpose, which go through LDS to leave in whole lines.  Measured: 8192 x 2048 bf16 by
// rows 10.7 us, 8192 x 8192 bf16 by rows with the transpose 49 (5.2 TB/s), 8192 x 2048 fp32 by tiles
// with the transpose 22.9 (4.4 TB/s); back to fp32 12.4 (6.8 TB/s, part of it from the last-level
// cache).
#include "f8.h"
#include "launch.h"
#include "mx_rows.h"

namespace bitopt {

// The largest of sixteen neighbouring lanes, in all of them.
__device__ __forceinline__ uint32_t max16(uint32_t m) {
    m = max(m, (uint32_t)__builtin_amdgcn_mov_dpp((int)m, 0xB1, 0xF, 0xF, true));    // quad_perm 1,0,3,2
    m = max(m, (uint32_t)__builtin_amdgcn_mov_dpp((int)m, 0x4E, 0xF, 0xF, true));    // quad_perm 2,3,0,1
    m = max(m, (uint32_t)__builtin_amdgcn_mov_dpp((int)m, 0x141, 0xF, 0xF, true));   // row_half_mirror
    return max(m, (uint32_t)__builtin_amdgcn_mov_dpp((int)m, 0x140, 0xF, 0xF, true));  // row_mirror
}

template <int DT, int FMT> __global__ __launch_bounds__(kThreads) void k_f8_rows(F8CodecArgs a, RowGrid g) {
    const int64_t width = f8_padded(a.cols);
    for_items(g, a.rows, (int32_t)(width / 8), [&](int64_t row, int32_t item) {
        const int64_t c = 8 * (int64_t)item;
        float v[8];
        if (a.cols >= 8) {
            Eight<DT> in;
            in.template load<false>(a.x, row * a.ldx, c, a.cols);
            in.values(c + 8 - a.cols, v);
        } else {
#pragma unroll
            for (int j = 0; j < 8; ++j) v[j] = c + j < a.cols ? load1<DT>(a.x, row * a.ldx + c + j) : 0.0f;
        }
        uint32_t m = 0;
#pragma unroll
        for (int j = 0; j < 8; ++j) m = max(m, __float_as_uint(v[j]) & 0x7fffffffu);
        const F8Scale f = f8_scale<FMT>(max16(m));
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] = f8_scaled<DT>(v[j], f.r);
        const u32x2 codes = {f8_encode4<FMT>(v[0], v[1], v[2], v[3]), f8_encode4<FMT>(v[4], v[5], v[6], v[7])};
        *gbl(reinterpret_cast<u32x2*>(a.codes + row * width + c)) = f.r == 0.0f ? u32x2{0u, 0u} : codes;
        if (item % 16 == 0) gbl(a.scales)[item / 16 * a.rows + row] = f.s;
    });
}

template <int DT, int FMT, bool TILES, bool T> __global__ __launch_bounds__(kThreads) void k_f8_quantize(F8CodecArgs a) {
    constexpr int B = kF8Block;
    // the transpose's codes, and before them the maxima of columns of each row group
    __shared__ __attribute__((aligned(16))) uint8_t turned[T ? B * B : 16];
    __shared__ __attribute__((aligned(16))) float factor[T ? B : 4];
    const int tid = threadIdx.x, cg = tid & 15, rg = tid >> 4;
    const int64_t rb = f8_blocks(a.rows), cb = f8_blocks(a.cols);
    const int64_t c0 = (int64_t)blockIdx.x * B, c = c0 + 8 * cg;
    const int n = (int)max((int64_t)0, min((int64_t)8, a.cols - c));
    for (int64_t block = blockIdx.y; block < rb; block += gridDim.y) {
        const int64_t r0 = block * B, r = r0 + 8 * rg;
        float v[8][8];
        if (a.cols >= 8) {
            Eight<DT> in[8];
#pragma unroll
            for (int p = 0; p < 8; ++p) in[p].template load<false>(a.x, min(r + p, a.rows - 1) * a.ldx, c, a.cols);
#pragma unroll
            for (int p = 0; p < 8; ++p) in[p].values(r + p < a.rows ? c + 8 - a.cols : 8, v[p]);
        } else {
#pragma unroll
            for (int p = 0; p < 8; ++p)
#pragma unroll
                for (int j = 0; j < 8; ++j) v[p][j] = r + p < a.rows && j < n ? load1<DT>(a.x, (r + p) * a.ldx + c + j) : 0.0f;
        }
        F8Scale all{};
        if constexpr (TILES) {
            uint32_t m = 0;
#pragma unroll
            for (int p = 0; p < 8; ++p)
#pragma unroll
                for (int j = 0; j < 8; ++j) m = max(m, __float_as_uint(v[p][j]) & 0x7fffffffu);
            m = max16(m);
            m = max(m, (uint32_t)__shfl_xor((int)m, 16));
            m = max(m, (uint32_t)__shfl_xor((int)m, 32));
            uint32_t* wave = reinterpret_cast<uint32_t*>(factor);
            __syncthreads();                // the last tile's maxima have been read
            if ((tid & 63) == 0) wave[tid >> 6] = m;
            __syncthreads();
            all = f8_scale<FMT>(max(max(wave[0], wave[1]), max(wave[2], wave[3])));
            if (tid == 0) {
                if (a.codes) a.scales[block * cb + blockIdx.x] = all.s;
                if (T) a.scales_t[blockIdx.x * rb + block] = all.s;
            }
        }
        if (a.codes) {
            float mine = 0.0f;
#pragma unroll
            for (int p = 0; p < 8; ++p) {
                F8Scale f = all;
                if constexpr (!TILES) {
                    uint32_t m = 0;
#pragma unroll
                    for (int j = 0; j < 8; ++j) m = max(m, __float_as_uint(v[p][j]) & 0x7fffffffu);
                    f = f8_scale<FMT>(max16(m));
                    if (cg == p) mine = f.s;
                }
                if (r + p >= a.rows) continue;
                float w[8];
#pragma unroll
                for (int j = 0; j < 8; ++j) w[j] = f8_scaled<DT>(v[p][j], f.r);
                const u32x2 codes = {f8_encode4<FMT>(w[0], w[1], w[2], w[3]), f8_encode4<FMT>(w[4], w[5], w[6], w[7])};
                *gbl(reinterpret_cast<u32x2*>(a.codes + (r + p) * cb * B + c)) = f.r == 0.0f ? u32x2{0u, 0u} : codes;
            }
            if (!TILES && cg < 8 && r + cg < a.rows) gbl(a.scales)[blockIdx.x * a.rows + r + cg] = mine;
        }
        if constexpr (T) {
            if constexpr (!TILES) {
                uint32_t* maxima = reinterpret_cast<uint32_t*>(turned);
                __syncthreads();            // the last tile's codes have been read
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    uint32_t m = 0;
#pragma unroll
                    for (int p = 0; p < 8; ++p) m = max(m, __float_as_uint(v[p][j]) & 0x7fffffffu);
                    maxima[rg * B + 8 * cg + j] = m;
                }
                __syncthreads();
                if (tid < B) {
                    uint32_t m = 0;
#pragma unroll
                    for (int g = 0; g < 16; ++g) m = max(m, maxima[g * B + tid]);
                    const F8Scale f = f8_scale<FMT>(m);
                    factor[tid] = f.r;
                    if (c0 + tid < a.cols) gbl(a.scales_t)[block * a.cols + c0 + tid] = f.s;
                }
            }
            __syncthreads();
            // column 8 cg + j: its sixteen units of eight rows lie at unit ^ cg
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const float f = TILES ? all.r : factor[8 * cg + j];
                float w[8];
#pragma unroll
                for (int p = 0; p < 8; ++p) w[p] = f8_scaled<DT>(v[p][j], f);
                const u32x2 codes = {f8_encode4<FMT>(w[0], w[1], w[2], w[3]), f8_encode4<FMT>(w[4], w[5], w[6], w[7])};
                *reinterpret_cast<u32x2*>(turned + (8 * cg + j) * B + ((rg ^ cg) << 3)) = f == 0.0f ? u32x2{0u, 0u} : codes;
            }
            __syncthreads();
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int col = i * 32 + (tid >> 3), h = tid & 7, key = col >> 3;
                if (c0 + col >= a.cols) continue;
                const u32x2 lo = *reinterpret_cast<const u32x2*>(turned + col * B + (((2 * h) ^ key) << 3));
                const u32x2 hi = *reinterpret_cast<const u32x2*>(turned + col * B + (((2 * h + 1) ^ key) << 3));
                *gbl(reinterpret_cast<u32x4*>(a.codes_t + (c0 + col) * rb * B + r0 + 16 * h)) = u32x4{lo.x, lo.y, hi.x, hi.y};
            }
        }
    }
}

template <int DT, int FMT> __global__ __launch_bounds__(kThreads) void k_f8_dequantize(F8CodecArgs a, RowGrid g, bool tiles) {
    constexpr int PER = kPer<DT>;
    const int64_t cb = f8_blocks(a.cols);
    for_items(g, a.rows, (int32_t)((a.cols + PER - 1) / PER), [&](int64_t row, int32_t item) {
        const int64_t c = PER * (int64_t)item;
        const int64_t block = c / kF8Block;
        const float s = gbl(a.scales)[tiles ? row / kF8Block * cb + block : block * a.rows + row];
        const uint8_t* p = a.codes + row * cb * kF8Block + c;
        float v[PER];
        if constexpr (PER == 8) {
            const u32x2 w = *gbl(reinterpret_cast<const u32x2*>(p));
            f8_decode4<FMT>(w.x, v);
            f8_decode4<FMT>(w.y, v + 4);
        } else {
            f8_decode4<FMT>(*gbl(reinterpret_cast<const uint32_t*>(p)), v);
        }
#pragma unroll
        for (int j = 0; j < PER; ++j) v[j] *= s;
        st_item<DT>(a.out, row * a.ldo + c, (int)min((int64_t)PER, a.cols - c), v);
    });
}

// ------------------------------------------------------------------------- launches

template <int DT, int FMT> static hipError_t quantize(const F8CodecArgs& a, bool tiles, hipStream_t s) {
    const dim3 grid((unsigned)f8_blocks(a.cols), (unsigned)std::min<int64_t>(f8_blocks(a.rows), 65535));
    if (tiles && a.codes_t) hipLaunchKernelGGL((k_f8_quantize<DT, FMT, true, true>), grid, dim3(kThreads), 0, s, a);
    else if (tiles) hipLaunchKernelGGL((k_f8_quantize<DT, FMT, true, false>), grid, dim3(kThreads), 0, s, a);
    else if (a.codes_t) hipLaunchKernelGGL((k_f8_quantize<DT, FMT, false, true>), grid, dim3(kThreads), 0, s, a);
    else {
        dim3 over;
        const RowGrid g = row_grid(a.rows, f8_padded(a.cols) / 8, over);
        hipLaunchKernelGGL((k_f8_rows<DT, FMT>), over, dim3(kThreads), 0, s, a, g);
    }
    return hipGetLastError();
}

template <int DT, int FMT> static hipError_t dequantize(const F8CodecArgs& a, bool tiles, hipStream_t s) {
    dim3 grid;
    const RowGrid g = row_grid(a.rows, (a.cols + kPer<DT> - 1) / kPer<DT>, grid);
    hipLaunchKernelGGL((k_f8_dequantize<DT, FMT>), grid, dim3(kThreads), 0, s, a, g, tiles);
    return hipGetLastError();
}

hipError_t launch_f8_quantize(const F8CodecArgs& a, int dtype, int fmt, int blocks, hipStream_t s) {
    const bool t = blocks == kF8Tiles, e4 = fmt == kF8E4M3;
    if (dtype == kF32) return e4 ? quantize<kF32, kF8E4M3>(a, t, s) : quantize<kF32, kF8E5M2>(a, t, s);
    if (dtype == kF16) return e4 ? quantize<kF16, kF8E4M3>(a, t, s) : quantize<kF16, kF8E5M2>(a, t, s);
    return e4 ? quantize<kBF16, kF8E4M3>(a, t, s) : quantize<kBF16, kF8E5M2>(a, t, s);
}

hipError_t launch_f8_dequantize(const F8CodecArgs& a, int dtype, int fmt, int blocks, hipStream_t s) {
    const bool t = blocks == kF8Tiles, e4 = fmt == kF8E4M3;
    if (dtype == kF32) return e4 ? dequantize<kF32, kF8E4M3>(a, t, s) : dequantize<kF32, kF8E5M2>(a, t, s);
    if (dtype == kF16) return e4 ? dequantize<kF16, kF8E4M3>(a, t, s) : dequantize<kF16, kF8E5M2>(a, t, s);
    return e4 ? dequantize<kBF16, kF8E4M3>(a, t, s) : dequantize<kBF16, kF8E5M2>(a, t, s);
}

}  // namespace bitopt
