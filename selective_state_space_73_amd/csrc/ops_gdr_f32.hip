// Instantiations of the gated delta rule for f32 inputs and outputs.
#include "ops_gdr.h"

namespace selscan {

hipError_t launch_gdr_f32(const LaunchGdr& p) { return launch_gdr_t<float>(p); }

}  // namespace selscan
