// Decode attention: the code width picks the instantiations.
#include "common.h"

namespace qaff {

hipError_t launch_paged_attention_b2(const PagedAttnArgs& a, hipStream_t s);
hipError_t launch_paged_attention_b4(const PagedAttnArgs& a, hipStream_t s);
hipError_t launch_paged_attention_b8(const PagedAttnArgs& a, hipStream_t s);

hipError_t launch_paged_attention(const PagedAttnArgs& a, hipStream_t s) {
  switch (a.c.bits) {
    case 2: return launch_paged_attention_b2(a, s);
    case 4: return launch_paged_attention_b4(a, s);
    default: return launch_paged_attention_b8(a, s);
  }
}

}  // namespace qaff
