// Decode attention over caches of 4-bit codes.
#include "paged_attention.h"

namespace qaff {

hipError_t launch_paged_attention_b4(const PagedAttnArgs& a, hipStream_t s) {
  return launch_paged_attention_bits<4>(a, s);
}

}  // namespace qaff
