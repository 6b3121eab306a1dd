// Instantiations of the 8-bit product.
#include "ops_gemm_q8.h"

namespace selscan {

hipError_t launch_gemm_q8(const LaunchGemmQ8& p) {
    if (p.y_bf16) return p.R ? launch_gemm_q8_t<uint16_t, true>(p) : launch_gemm_q8_t<uint16_t, false>(p);
    return p.R ? launch_gemm_q8_t<float, true>(p) : launch_gemm_q8_t<float, false>(p);
}

}  // namespace selscan
