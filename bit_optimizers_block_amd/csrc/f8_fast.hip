// Tiled F8 products with bf16 results, on the 8-bit matrix instructions.
#include "f8_gemm.h"

namespace bitopt {

hipError_t launch_f8_fast(const F8GemmArgs& g, int a_fmt, int b_fmt, int b_blocks, hipStream_t s) {
    return f8_product<false>(g, a_fmt, b_fmt, b_blocks, s);
}

}  // namespace bitopt
