// The cache attention for bf16.
#include "gdn_cache_attention.h"

namespace gdn {

hipError_t launch_attend_bf16(const AttendArgs& a, hipStream_t s) { return attend::launch_attend_t<__bf16>(a, s); }

}  // namespace gdn
