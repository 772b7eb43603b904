// Mixture-of-experts products on 8-bit codes.
#include "moe.h"

namespace qaff {

hipError_t launch_moe_b8(const MoeArgs& a, MoeStep step, hipStream_t s) { return launch_moe_bits<8>(a, step, s); }

}  // namespace qaff
