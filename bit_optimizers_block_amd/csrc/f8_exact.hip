// Tiled F8 products with fp32 and fp16 results, on the 16-bit matrix instructions.
#include "f8_gemm.h"

namespace bitopt {

hipError_t launch_f8_exact(const F8GemmArgs& g, int a_fmt, int b_fmt, int b_blocks, hipStream_t s) {
    return f8_product<true>(g, a_fmt, b_fmt, b_blocks, s);
}

}  // namespace bitopt
