// Instantiations of the norms around a layer.
#include "ops_gnorm.h"

namespace selscan {

int64_t gnorm_groups(int64_t M, int64_t K) {
    const int64_t rows = gnorm_shape(K, false).rows, n = (M + rows - 1) / rows;
    return n < 1024 ? n : 1024;
}

hipError_t launch_gnorm(const LaunchGnorm& p) {
    if (p.bf16) return p.vec ? launch_gnorm_t<uint16_t, true>(p) : launch_gnorm_t<uint16_t, false>(p);
    return p.vec ? launch_gnorm_t<float, true>(p) : launch_gnorm_t<float, false>(p);
}

}  // namespace selscan
