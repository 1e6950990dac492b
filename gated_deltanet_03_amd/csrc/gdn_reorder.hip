// Rows moved from each entry's source to its own place: states, windows and pages after a beam selection.
//
// A copy, bound by memory.  A thread holds one 16-byte column of all rows of one group: it loads the group's rows
// before it stores any of them, so a group may be permuted in place without a second buffer, and entries that stay
// where they are cost nothing.  Groups of more than 16 rows take narrower columns, so that the rows of one column
// still fit the registers.  4 layers of 32 states of 2 MB, 4 a group, parents at random but in order (221 MB
// to read and write), in place: 54 us, 4.1 TB/s where a copy has 5.1; pages of 128 KB of keys and of values, 8 a group, 16
// groups (35 MB): 11 us.
#include <algorithm>

#include "gdn_cache_internal.h"
#include "gdn_device.h"

namespace gdn {

typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));

template <typename C, int W>
__global__ __launch_bounds__(256) void state_reorder_kernel(ReorderArgs p, int64_t col0, int32_t g0) {
  const int64_t col = col0 + ((int64_t)blockIdx.x * 256 + threadIdx.x) * (int64_t)sizeof(C);
  if (col >= p.row_bytes) return;
  const int64_t g = g0 + (int64_t)blockIdx.y;
  const int32_t* si = p.src_index + g * p.W;
  const int32_t* di = p.dst_index ? p.dst_index + g * p.W : nullptr;
  const int64_t sg = g * p.src_group, last = p.src_group ? p.src_group : p.src_rows;
  const bool same = p.src == p.dst;
  for (int64_t l = blockIdx.z; l < p.layers; l += gridDim.z) {
    const char* src = p.src + l * p.src_layer + col;
    char* dst = p.dst + l * p.dst_layer + col;
    // entry j's rows, if it has any and has to move
    auto rows = [&](int j, int64_t& from, int64_t& to) {
      const int64_t i = si[j];
      from = i + sg;
      to = di ? (int64_t)di[j] : g * p.W + j;
      return i >= 0 && i < last && from < p.src_rows && to >= 0 && to < p.dst_rows && !(same && from == to);
    };
    C x[W];
    int64_t from, to;
#pragma unroll
    for (int j = 0; j < W; ++j)
      if (j < p.W && rows(j, from, to)) x[j] = *reinterpret_cast<const C*>(src + from * p.row_bytes);
#pragma unroll
    for (int j = 0; j < W; ++j)
      if (j < p.W && rows(j, from, to)) *reinterpret_cast<C*>(dst + to * p.row_bytes) = x[j];
  }
}

template <typename C, int W>
static void launch_reorder_w(const ReorderArgs& a, hipStream_t s) {
  const int64_t wgs = (a.row_bytes / (int64_t)sizeof(C) + 255) / 256;
  const unsigned z = (unsigned)std::min<int64_t>(a.layers, 64);
  // a launch has at most kLaunchThreads threads and 65535 groups
  for (int32_t g = 0; g < a.G; g += 65535) {
    const unsigned groups = (unsigned)std::min(65535, a.G - g);
    const int64_t most = std::max<int64_t>(1, kLaunchThreads / 256 / ((int64_t)z * groups));
    for (int64_t w = 0; w < wgs; w += most)
      hipLaunchKernelGGL((state_reorder_kernel<C, W>), dim3((unsigned)std::min(most, wgs - w), groups, z), dim3(256),
                         0, s, a, w * 256 * (int64_t)sizeof(C), g);
  }
}

hipError_t launch_reorder(const ReorderArgs& a, hipStream_t s) {
  prof_begin(K_REORDER, s);
  if (a.W <= 4) launch_reorder_w<u32x4, 4>(a, s);
  else if (a.W <= 8) launch_reorder_w<u32x4, 8>(a, s);
  else if (a.W <= 16) launch_reorder_w<u32x4, 16>(a, s);
  else if (a.W <= 32) launch_reorder_w<u32x2, 32>(a, s);
  else launch_reorder_w<uint32_t, 64>(a, s);
  prof_end(K_REORDER, s);
  return hipGetLastError();
}

}  // namespace gdn
