// The cache attention for f16.
#include "gdn_cache_attention.h"

namespace gdn {

hipError_t launch_attend_f16(const AttendArgs& a, hipStream_t s) { return attend::launch_attend_t<_Float16>(a, s); }

}  // namespace gdn
