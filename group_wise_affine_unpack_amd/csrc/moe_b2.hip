// Mixture-of-experts products on 2-bit codes.
#include "moe.h"

namespace qaff {

hipError_t launch_moe_b2(const MoeArgs& a, MoeStep step, hipStream_t s) { return launch_moe_bits<2>(a, step, s); }

}  // namespace qaff
