// Decode attention over caches of 8-bit codes.
#include "paged_attention.h"

namespace qaff {

hipError_t launch_paged_attention_b8(const PagedAttnArgs& a, hipStream_t s) {
  return launch_paged_attention_bits<8>(a, s);
}

}  // namespace qaff
