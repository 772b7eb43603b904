// Decode attention over caches of 2-bit codes.
#include "paged_attention.h"

namespace qaff {

hipError_t launch_paged_attention_b2(const PagedAttnArgs& a, hipStream_t s) {
  return launch_paged_attention_bits<2>(a, s);
}

}  // namespace qaff
