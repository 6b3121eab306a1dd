// Instantiations of the gated delta rule for bf16 inputs and outputs.
#include "ops_gdr.h"

namespace selscan {

hipError_t launch_gdr_bf16(const LaunchGdr& p) { return launch_gdr_t<uint16_t>(p); }

}  // namespace selscan
