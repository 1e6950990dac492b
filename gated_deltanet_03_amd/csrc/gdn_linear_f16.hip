// Chunked linear-attention prefill for f16 inputs.
#include "gdn_linear_prefill.h"

namespace gdn {

hipError_t launch_linear_prefill_f16(const LinearArgs& a, hipStream_t s) { return linear::launch<_Float16>(a, s); }

}  // namespace gdn
