// Arguments and launchers of the linear attention, the draft verification and the
// block norms.  They stand apart from gdn_internal.h and gdn_device.h, whose text
// (with the kernels') is what the committed counter summaries are bound to.
#pragma once

#include "gdn_internal.h"

namespace gdn {

// Linear attention with a decay for each head.  Prefill: segments of
// seg_tokens tokens (0: one segment per sequence, no workspace).
struct LinearArgs {
  const void* q;
  const void* k;
  const void* v;
  const float* g;
  int64_t g_stride;      // elements between tokens' log decays: Hv, or 0 (one per head)
  const float* s0;       // may be null (zeros)
  int64_t s0_stride;
  float* s_out;          // may be null
  void* o;
  const int32_t* cu;     // null = dense rows
  int32_t B, T, total;
  int32_t Hq, Hv, dk, dv;
  float scale;
  int32_t first;         // (segment, key head) pair (step: (row, head) pair) of this launch's first workgroup
  // step only
  int32_t cap;
  const int32_t* counts;
  float* su;             // [B, cap, R]
  // prefill only
  int32_t seg_tokens, max_segs;
  float* seg_state;      // [max_segs + B, Hv, dk, dv]: a segment's own state (the first's with the
                         // initial one), then the initial states, in the kernels' order
  float* seg_decay;      // [max_segs, Hv]: its decay
};

constexpr uint32_t kLaunchThreads = 0xffffffffu;   // threads of one launch, at most

constexpr int32_t kVerifyRowMax = 65536;   // entries of a row that one workgroup verifies (no workspace)

struct VerifyArgs {
  const void* p;
  const void* q;         // may be null (deterministic drafts)
  int64_t p_stride, q_stride;
  const int32_t* x;
  const float* u;
  const int32_t* n;      // may be null
  int32_t* tokens;
  int32_t* emit;
  int32_t B, K, V;
  int32_t tile, tiles;   // tiles of `tile` vocabulary entries per row
  double* part;          // [B, tiles] sums of weights
};

struct NormArgs {
  const void* y;
  const void* gate;
  const void* res;
  const void* wpost;
  const void* wnext;
  void* h;
  void* normed;
  int64_t T, row0;       // rows, and the first of this launch
  int32_t D, group, act;
  float scale, eps;
};

// Further ids of the per-kernel event timing.
constexpr KernelId K_LIN_STATE = KernelId(kNumKernels), K_LIN_OUT = KernelId(kNumKernels + 1),
                   K_LIN_WHOLE = KernelId(kNumKernels + 2), K_LIN_STEP = KernelId(kNumKernels + 3),
                   K_VERIFY_SUM = KernelId(kNumKernels + 4), K_VERIFY_DRAW = KernelId(kNumKernels + 5),
                   K_VERIFY_ROW = KernelId(kNumKernels + 6), K_NORM = KernelId(kNumKernels + 7);
constexpr int kAllKernels = kNumKernels + 8;

hipError_t launch_linear_prefill_f32(const LinearArgs& a, hipStream_t s);
hipError_t launch_linear_prefill_f16(const LinearArgs& a, hipStream_t s);
hipError_t launch_linear_prefill_bf16(const LinearArgs& a, hipStream_t s);
hipError_t launch_linear_step(DType dt, const LinearArgs& a, hipStream_t s);
hipError_t launch_verify(DType dt, const VerifyArgs& a, hipStream_t s);
hipError_t launch_norm(DType dt, const NormArgs& a, hipStream_t s);

}  // namespace gdn
