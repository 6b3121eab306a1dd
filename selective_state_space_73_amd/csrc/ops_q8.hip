// Instantiations of the 8-bit rounding and the norm in front of it.
#include "ops_q8.h"

namespace selscan {

hipError_t launch_q8(const LaunchQ8& p) {
    if (p.bf16) return p.vec ? launch_q8_t<uint16_t, true>(p) : launch_q8_t<uint16_t, false>(p);
    return p.vec ? launch_q8_t<float, true>(p) : launch_q8_t<float, false>(p);
}

}  // namespace selscan
