// Mixture-of-experts products on 4-bit codes.
#include "moe.h"

namespace qaff {

hipError_t launch_moe_b4(const MoeArgs& a, MoeStep step, hipStream_t s) { return launch_moe_bits<4>(a, step, s); }

}  // namespace qaff
