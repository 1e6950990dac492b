// Prefix sum in 64 bits over a wave.
#pragma once

#include "gdn_device.h"

namespace gdn {

// Inclusive prefix sum of x over the wave's lanes, on the VALU: shifts inside
// the rows of 16 lanes, then row ends broadcast to the rows after them.
template <int CTRL, int ROWS>
__device__ __forceinline__ double dpp_or_zero(double x) {
  const uint64_t u = __builtin_bit_cast(uint64_t, x);
  const uint32_t lo = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)(uint32_t)u, CTRL, ROWS, 0xf, false);
  const uint32_t hi = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)(uint32_t)(u >> 32), CTRL, ROWS, 0xf, false);
  return __builtin_bit_cast(double, (uint64_t)hi << 32 | lo);
}

__device__ __forceinline__ double wave_scan64(double x) {
  x += dpp_or_zero<0x111, 0xf>(x);   // row_shr:1
  x += dpp_or_zero<0x112, 0xf>(x);   // row_shr:2
  x += dpp_or_zero<0x114, 0xf>(x);   // row_shr:4
  x += dpp_or_zero<0x118, 0xf>(x);   // row_shr:8
  x += dpp_or_zero<0x142, 0xa>(x);   // row_bcast:15 into rows 1 and 3
  x += dpp_or_zero<0x143, 0xc>(x);   // row_bcast:31 into rows 2 and 3
  return x;
}

}  // namespace gdn
