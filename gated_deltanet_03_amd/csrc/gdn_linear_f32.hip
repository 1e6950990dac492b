// Chunked linear-attention prefill for f32 inputs.
#include "gdn_linear_prefill.h"

namespace gdn {

hipError_t launch_linear_prefill_f32(const LinearArgs& a, hipStream_t s) { return linear::launch<float>(a, s); }

}  // namespace gdn
