// Instantiations of the norms around a layer.
#include "ops_gnorm.h"

namespace selscan {

int64_t gnorm_groups(int64_t M, int64_t K) {
    // as many workgroups as 256 CUs hold at 8 waves each, so that none waits for another to end
    const GnormShape sh = gnorm_shape(K, false);
    const int64_t n = (M + sh.rows - 1) / sh.rows, waves = sh.threads / 64, most = 256 * (waves <= 8 ? 8 / waves : 1);
    return n < most ? n : most;
}

hipError_t launch_gnorm(const LaunchGnorm& p) {
    if (p.bf16) return p.vec ? launch_gnorm_t<uint16_t, true>(p) : launch_gnorm_t<uint16_t, false>(p);
    return p.vec ? launch_gnorm_t<float, true>(p) : launch_gnorm_t<float, false>(p);
}

}  // namespace selscan
