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
  int32_t shares;        // even shares of a head's work, 0: a tile for each workgroup
  int32_t tiles;         // upper bound on a head's tiles
  int32_t unit;          // log2 of the keys of a unit of work
  int32_t extra_drawn;   // what cutting costs, in units of work: where a share is one piece,
  int32_t extra_even;    // and where it is the end of one tile and the beginning of another
  float* part_o;         // [2 shares, Hkv, rows of a tile, d]
  float* part_ml;        // [2 shares, Hkv, rows of a tile, 2]: what the weights were taken against, their sum
  void* cuts;            // [Hkv, shares] of 16 bytes
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

// Sizes that the host's plan and the attention's kernels share: rows of a tile, the fewest keys of a share of few and of
// many rows, the most shares, and by the bytes of one key (rb) the keys of a block, LDS, waves of a workgroup and waves
// a SIMD, which is workgroups a CU.
constexpr int32_t kFewRows = 32, kManyRows = 128;
constexpr int32_t kFewKeys = 128, kManyKeys = 128, kMostShares = 1024;
constexpr int many_keys(int rb) { return rb >= 1024 ? 32 : 64; }
constexpr int many_lds(int rb) { return 4 * many_keys(rb) * rb; }
constexpr int many_waves(int rb) { return rb >= 512 ? 1 : rb >= 256 ? 2 : 3; }
constexpr int few_group(int rb) { return rb >= 1024 ? 2 : 4; }
constexpr int few_lds(int rb) { return few_group(rb) * 64 * rb; }
constexpr int few_waves(int rb) { return rb >= 512 ? 1 : rb >= 256 ? 2 : rb >= 128 ? 3 : 4; }

hipError_t launch_append(DType dt, const AppendArgs& a, hipStream_t s);
hipError_t launch_attend_f32(const AttendArgs& a, hipStream_t s);
hipError_t launch_attend_f16(const AttendArgs& a, hipStream_t s);
hipError_t launch_attend_bf16(const AttendArgs& a, hipStream_t s);
hipError_t launch_select(DType dt, const SelectArgs& a, hipStream_t s);
hipError_t launch_reorder(const ReorderArgs& a, hipStream_t s);

}  // namespace gdn
