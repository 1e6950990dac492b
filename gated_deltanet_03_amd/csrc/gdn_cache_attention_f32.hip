// The cache attention for f32.
#include "gdn_cache_attention.h"

namespace gdn {

hipError_t launch_attend_f32(const AttendArgs& a, hipStream_t s) { return attend::launch_attend_t<float>(a, s); }

}  // namespace gdn
