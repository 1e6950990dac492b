// Chunked linear-attention prefill for bf16 inputs.
#include "gdn_linear_prefill.h"

namespace gdn {

hipError_t launch_linear_prefill_bf16(const LinearArgs& a, hipStream_t s) { return linear::launch<__bf16>(a, s); }

}  // namespace gdn
