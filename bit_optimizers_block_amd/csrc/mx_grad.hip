// Weight gradient of a linear layer from inputs saved in MX codes, and the product of two
// MX matrices.
#include "launch.h"
#include "mx_gemm.h"

namespace bitopt {

hipError_t launch_mx_grad_weight(const MxGemmArgs& g, int dtype, int fmt, hipStream_t s) {
    const bool four = fmt == kMxE2M1;
    if (dtype == kBF16) return four ? mx_gemm16<kBF16, kAcross16, kAcrossE2M1>(g, s) : mx_gemm16<kBF16, kAcross16, kAcrossE4M3>(g, s);
    return four ? mx_gemm16<kF16, kAcross16, kAcrossE2M1>(g, s) : mx_gemm16<kF16, kAcross16, kAcrossE4M3>(g, s);
}

hipError_t launch_mx_matmul(const MxGemmArgs& g, int a_fmt, int b_fmt, hipStream_t s) {
    if (a_fmt == kMxE2M1 && b_fmt == kMxE2M1)
        return mx_by_tile(
            g,
            [&](dim3 grid) {
                hipLaunchKernelGGL((k_mx_gemm4<256, 256, 128, 64>), grid, dim3(512), 0, s, g);
                return hipGetLastError();
            },
            [&](dim3 grid) {
                hipLaunchKernelGGL((k_mx_gemm4<128, 128, 64, 32>), grid, dim3(512), 0, s, g);
                return hipGetLastError();
            },
            [&](dim3 grid) {
                hipLaunchKernelGGL((k_mx_gemm4<64, 64, 32, 32>), grid, dim3(256), 0, s, g);
                return hipGetLastError();
            });
    if (a_fmt == kMxE2M1) return mx_gemm16<kBF16, kAlongE2M1, kAlongE4M3>(g, s);
    if (b_fmt == kMxE2M1) return mx_gemm16<kBF16, kAlongE4M3, kAlongE2M1>(g, s);
    return mx_gemm16<kBF16, kAlongE4M3, kAlongE4M3>(g, s);
}

}  // namespace bitopt
