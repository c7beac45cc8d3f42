// Products of a linear layer y = x W^T with W or x held in MX codes, tiled.
#include "launch.h"
#include "mx_gemm.h"

namespace bitopt {

hipError_t launch_mx_linear(const MxGemmArgs& g, int dtype, int fmt, hipStream_t s) {
    const bool four = fmt == kMxE2M1;
    if (dtype == kBF16) return four ? mx_gemm16<kBF16, kAlong16, kAlongE2M1>(g, s) : mx_gemm16<kBF16, kAlong16, kAlongE4M3>(g, s);
    return four ? mx_gemm16<kF16, kAlong16, kAlongE2M1>(g, s) : mx_gemm16<kF16, kAlong16, kAlongE4M3>(g, s);
}

hipError_t launch_mx_grad_input(const MxGemmArgs& g, int dtype, int fmt, hipStream_t s) {
    const bool four = fmt == kMxE2M1;
    if (dtype == kBF16) return four ? mx_gemm16<kBF16, kAlong16, kAcrossE2M1>(g, s) : mx_gemm16<kBF16, kAlong16, kAcrossE4M3>(g, s);
    return four ? mx_gemm16<kF16, kAlong16, kAcrossE2M1>(g, s) : mx_gemm16<kF16, kAlong16, kAcrossE4M3>(g, s);
}

}  // namespace bitopt
