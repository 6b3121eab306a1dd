// Instantiations of the gated linear recurrence.
#include "ops_glr.h"

namespace selscan {

hipError_t launch_glr(const LaunchGlr& p) {
    if (p.bf16) return p.vec ? launch_glr_t<uint16_t, true>(p) : launch_glr_t<uint16_t, false>(p);
    return p.vec ? launch_glr_t<float, true>(p) : launch_glr_t<float, false>(p);
}

}  // namespace selscan
