// Arguments and launchers of the paged cache (append, attention), the beam selection and the reordering of rows.
#pragma once

#include "gdn_ops_internal.h"

namespace gdn {

// What the cache's kernels share.  Rows of the cache are numbered (page * Hkv + head) * page_size + row in it.
struct CacheArgs {
  const int32_t* table;
  const int32_t* lens;
  const int32_t* cu;     // null = dense rows of T tokens
  int32_t N, T, total;   // sequences, tokens per row (dense), token rows
  int32_t Hq, Hkv, d;
  int32_t page_size, num_pages, max_pages;
};

struct AppendArgs {
  CacheArgs c;
  const void* q;         // may be null
  const void* k;
  const void* v;
  int64_t q_stride, k_stride, v_stride;   // elements between tokens
  const float* inv_freq;
  const int32_t* positions;               // null: places in the cache
  const int32_t* pair_axis;               // null: axis 0
  int32_t rotary, interleaved, axes;
  void* q_out;
  void* k_cache;
  void* v_cache;
};

struct AttendArgs {
  CacheArgs c;
  const void* q;
  int64_t q_stride;
  const void* k_cache;
  const void* v_cache;
  void* o;
  float scale_log2;      // scale * log2(e)
  int32_t window;        // 0: none
  int32_t granules;      // 16-row granules of a page
  uint64_t granule_magic;   // ceil(2^32 / granules)
  int32_t few;           // one 32-row tile a workgroup, its waves on different keys
  int32_t slices;        // key slices a head to aim at, 0: tiles are not split
  int32_t units;         // upper bound on (tile, slice) pairs of a head
  float* part_o;         // [units, Hkv, rows of a tile, d]
  float* part_ml;        // [units, Hkv, rows of a tile, 2]
};

struct SelectArgs {
  const void* x;
  int64_t row_stride;
  const float* scores;
  const uint8_t* finished;   // may be null
  int32_t* tokens;
  int32_t* parents;
  float* new_scores;
  uint8_t* new_finished;
  int32_t B, W, K, V;
  int32_t eos, pad;
  int32_t segment, segments; // vocabulary entries of a segment, segments of a row
  float* seg_max;            // [B*W, segments]
  double* seg_sum;           // [B*W, segments]
  uint64_t* best;            // [B*W, segments, K] keys, best first
};

struct ReorderArgs {
  const char* src;
  char* dst;
  int64_t layers, src_layer, dst_layer;   // bytes between layers
  int64_t src_rows, dst_rows, row_bytes, src_group;
  int32_t G, W;
  const int32_t* src_index;
  const int32_t* dst_index;   // may be null
};

// Rows of a tile and the smallest slice of keys: shared by the host's sizes and the kernels.
constexpr int32_t kFewRows = 32, kManyRows = 128;
constexpr int32_t kSliceKeys = 256, kMostSlices = 1024;

hipError_t launch_append(DType dt, const AppendArgs& a, hipStream_t s);
hipError_t launch_attend_f32(const AttendArgs& a, hipStream_t s);
hipError_t launch_attend_f16(const AttendArgs& a, hipStream_t s);
hipError_t launch_attend_bf16(const AttendArgs& a, hipStream_t s);
hipError_t launch_select(DType dt, const SelectArgs& a, hipStream_t s);
hipError_t launch_reorder(const ReorderArgs& a, hipStream_t s);

}  // namespace gdn
