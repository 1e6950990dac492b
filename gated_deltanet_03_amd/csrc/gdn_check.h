// Host-side argument checks shared by the entry points (defined in gdn_api.cpp).
// Each returns GDN_OK or sets the thread's last error and returns its status.
#pragma once

#include <hip/hip_runtime.h>

#include "../../include/gdn.h"

namespace gdn {

gdn_status fail(gdn_status st, const char* fmt, ...);
gdn_status hip_fail(hipError_t e, const char* what);
bool aligned16(const void* p);
bool supported_dim(int32_t d);
size_t elem_size(int32_t dt);
size_t align_up(size_t x, size_t a);
bool overlaps(const void* a, size_t an, const void* b, size_t bn);
gdn_status check_shape(const gdn_shape* sh, const int32_t* cu, int64_t* total_tokens);
gdn_status check_states(const gdn_shape* sh, const float* s0, int64_t stride, const float* s_out);

}  // namespace gdn
