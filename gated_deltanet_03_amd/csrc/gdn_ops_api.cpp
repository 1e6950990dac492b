// C-ABI entry points of the linear attention with decay, the verification of
// drafted tokens and the block norms: host-side validation, workspace sizing
// and dispatch.  Validation runs before any HIP call.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cmath>

#include "../../include/gdn.h"
#include "gdn_check.h"
#include "gdn_ops_internal.h"

using namespace gdn;

namespace {

struct Buf {
  const void* p;
  size_t n;          // bytes
  const char* name;
};

// `out` must not overlap any of `others` (NULL entries are skipped).
gdn_status check_apart(const Buf& out, const Buf* others, int n) {
  if (out.p == nullptr || out.n == 0) return GDN_OK;
  for (int i = 0; i < n; ++i)
    if (others[i].p != nullptr && others[i].n != 0 && overlaps(out.p, out.n, others[i].p, others[i].n))
      return fail(GDN_ERR_INVALID_ARG, "%s overlaps %s", out.name, others[i].name);
  return GDN_OK;
}

bool misaligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) != 0; }

// Tokens per segment of the split prefill, 0 for one segment per sequence.
//
// A segment's workgroup walks its chunks one after another, so (sequence, head)
// pairs alone fill the 256 CUs only from a few hundred on.  From kSlots pairs on,
// two workgroups for each CU, nothing is cut; below that the tokens are cut
//  * into kParts even parts of all heads' tokens, somewhat fewer than kSlots:
//    sequences end inside of parts, so there are up to B * Hv workgroups more, and
//    a second round of a few workgroups costs most of a first one.  Over eleven random
//    lists of 2 to 6 sequences, 8000 to 21000 tokens in all, 8 to 32 heads, mostly
//    d = 128 bf16, 384 / 448 / 480 / 512 / 576 parts took 1.13, 1.04, 1.02, 1.03,
//    1.14 of the best for each;
//  * but not below sqrt(c * longest) tokens: the output pass of a sequence's last
//    segment sums the states of all before it, so fewer tokens a segment make
//    its walk shorter and that sum longer.  Over twelve lists of 1000 to 30000
//    16-bit tokens c = 4, 6, 8, 14, 20 took 1.01, 1.01, 1.03, 1.05, 1.10 of the
//    best for each, over eight fp32 lists, where a token costs more,
//    c = 0.5, 1.5, 3, 5, 7 took 1.02, 1.02, 1.02, 1.06, 1.07.
constexpr int64_t kSlots = 512, kParts = 480;

int32_t segment_tokens(const gdn_shape* sh, int64_t total, bool ragged) {
  const int64_t pairs = (int64_t)sh->B * sh->Hv;
  if (pairs == 0 || pairs >= kSlots) return 0;
  // the longest sequence is not known for ragged input; total bounds it
  const int64_t longest = ragged ? total : sh->T;
  int64_t seg = std::max<int64_t>((total * sh->Hv + kParts - 1) / kParts,
                                  (int64_t)std::sqrt((sh->dtype == GDN_F32 ? 1.5 : 5.0) * (double)longest));
  seg = (seg + 63) / 64 * 64;
  return longest <= 2 * seg ? 0 : (int32_t)seg;
}

int64_t max_segments(const gdn_shape* sh, int64_t total, bool ragged, int32_t seg) {
  if (seg == 0) return sh->B;
  if (!ragged) return (int64_t)sh->B * ((sh->T + seg - 1) / seg);
  return total / seg + sh->B;   // every sequence adds at most one partial (or empty) segment
}

size_t decay_bytes(int64_t segs, int32_t Hv) { return align_up((size_t)segs * Hv * sizeof(float), 256); }

size_t linear_workspace(const gdn_shape* sh, int64_t total, bool ragged) {
  const int32_t seg = segment_tokens(sh, total, ragged);
  if (seg == 0) return 0;
  const int64_t n = max_segments(sh, total, ragged, seg);
  return decay_bytes(n, sh->Hv) + (size_t)(n + sh->B) * sh->Hv * sh->dk * sh->dv * 4;
}

// Token tensors of the linear entry points; fills `ins` (q, k, v, g, initial_state).
gdn_status check_linear(const gdn_shape* sh, const void* q, const void* k, const void* v, const float* g,
                        int64_t g_stride, const float* s0, int64_t s0_stride, const int32_t* cu, const void* o,
                        float* s_out, int64_t* total, Buf ins[6]) {
  gdn_status st = check_shape(sh, cu, total);
  if (st != GDN_OK) return st;
  if (*total > (1LL << 30))   // the kernels' token indices run past the end by a few chunks or one segment
    return fail(GDN_ERR_UNSUPPORTED, "%lld tokens exceed 2^30", (long long)*total);
  if (g_stride != 0 && g_stride != sh->Hv)
    return fail(GDN_ERR_INVALID_ARG, "g_token_stride=%lld must be 0 or Hv=%d", (long long)g_stride, sh->Hv);
  if (*total > 0) {
    const void* ptrs[5] = {q, k, v, g, o};
    const char* names[5] = {"q", "k", "v", "g", "o"};
    for (int i = 0; i < 5; ++i) {
      if (ptrs[i] == nullptr) return fail(GDN_ERR_INVALID_ARG, "%s is NULL", names[i]);
      if (misaligned(ptrs[i], i == 3 ? 4 : 16))
        return fail(GDN_ERR_INVALID_ARG, "%s is not %d-byte aligned", names[i], i == 3 ? 4 : 16);
    }
  }
  if ((st = check_states(sh, s0, s0_stride, s_out)) != GDN_OK) return st;
  if (cu != nullptr && misaligned(cu, 4)) return fail(GDN_ERR_INVALID_ARG, "cu_seqlens is not 4-byte aligned");
  const size_t es = elem_size(sh->dtype), n = (size_t)*total, per = (size_t)sh->Hv * sh->dk * sh->dv * 4;
  ins[0] = {q, n * sh->Hq * sh->dk * es, "q"};
  ins[1] = {k, n * sh->Hq * sh->dk * es, "k"};
  ins[2] = {v, n * sh->Hv * sh->dv * es, "v"};
  ins[3] = {g, (g_stride ? n : (n > 0)) * sh->Hv * 4, "g"};
  ins[4] = {s0, sh->B > 0 ? (size_t)(sh->B - 1) * (size_t)s0_stride * 4 + per : 0, "initial_state"};
  ins[5] = {cu, cu ? (size_t)(sh->B + 1) * 4 : 0, "cu_seqlens"};
  const Buf ob = {o, n * sh->Hv * sh->dv * es, "o"}, fb = {s_out, (size_t)sh->B * per, "final_state"};
  if ((st = check_apart(ob, ins, 6)) != GDN_OK) return st;
  if ((st = check_apart(fb, ins, 4)) != GDN_OK) return st;   // initial_state: check_states
  return check_apart(fb, &ob, 1);
}

LinearArgs linear_args(const gdn_shape* sh, const void* q, const void* k, const void* v, const float* g,
                       int64_t g_stride, const float* s0, int64_t s0_stride, const int32_t* cu, void* o, float* s_out,
                       int64_t total) {
  LinearArgs a{};
  a.q = q; a.k = k; a.v = v; a.g = g; a.g_stride = g_stride;
  a.s0 = s0; a.s0_stride = s0_stride; a.s_out = s_out; a.o = o; a.cu = cu;
  a.B = sh->B; a.T = sh->T; a.total = (int32_t)total;
  a.Hq = sh->Hq; a.Hv = sh->Hv; a.dk = sh->dk; a.dv = sh->dv; a.scale = sh->scale;
  return a;
}

}  // namespace

extern "C" {

size_t gdn_linear_workspace_bytes(const gdn_shape* sh, int32_t ragged) {
  static const int32_t some = 0;
  int64_t total = 0;
  if (check_shape(sh, ragged ? &some : nullptr, &total) != GDN_OK) return (size_t)-1;
  if (total > (1LL << 30)) return fail(GDN_ERR_UNSUPPORTED, "%lld tokens exceed 2^30", (long long)total), (size_t)-1;
  return linear_workspace(sh, total, ragged != 0);
}

gdn_status gdn_linear_prefill(const gdn_shape* sh, const void* q, const void* k, const void* v, const float* g,
                              int64_t g_stride, const float* s0, int64_t s0_stride, const int32_t* cu, void* o,
                              float* s_out, void* ws, size_t ws_bytes, void* stream) {
  int64_t total = 0;
  Buf ins[7];
  gdn_status st = check_linear(sh, q, k, v, g, g_stride, s0, s0_stride, cu, o, s_out, &total, ins);
  if (st != GDN_OK) return st;
  const bool ragged = cu != nullptr;
  LinearArgs a = linear_args(sh, q, k, v, g, g_stride, s0, s0_stride, cu, o, s_out, total);
  a.seg_tokens = segment_tokens(sh, total, ragged);
  const int64_t segs = max_segments(sh, total, ragged, a.seg_tokens);
  if (segs * sh->Hv > 0x3fffffffLL)
    return fail(GDN_ERR_UNSUPPORTED, "too many (segment, head) pairs (%lld)", (long long)segs * sh->Hv);
  a.max_segs = (int32_t)segs;
  const size_t need = linear_workspace(sh, total, ragged);
  if (need > 0) {
    if (ws == nullptr || ws_bytes < need)
      return fail(GDN_ERR_INVALID_ARG, "workspace of %zu bytes is smaller than the %zu required", ws_bytes, need);
    if (!aligned16(ws)) return fail(GDN_ERR_INVALID_ARG, "workspace is not 16-byte aligned");
    const size_t es = elem_size(sh->dtype), per = (size_t)sh->Hv * sh->dk * sh->dv * 4;
    Buf all[8];
    std::copy(ins, ins + 6, all);
    all[6] = {o, (size_t)total * sh->Hv * sh->dv * es, "o"};
    all[7] = {s_out, (size_t)sh->B * per, "final_state"};
    if ((st = check_apart({ws, need, "workspace"}, all, 8)) != GDN_OK) return st;
    a.seg_decay = static_cast<float*>(ws);
    a.seg_state = reinterpret_cast<float*>(static_cast<char*>(ws) + decay_bytes(segs, sh->Hv));
  }
  if (sh->B == 0 || (total == 0 && s_out == nullptr)) return GDN_OK;
  const hipStream_t s = static_cast<hipStream_t>(stream);
  const hipError_t e = sh->dtype == GDN_F32   ? launch_linear_prefill_f32(a, s)
                       : sh->dtype == GDN_F16 ? launch_linear_prefill_f16(a, s)
                                              : launch_linear_prefill_bf16(a, s);
  return e == hipSuccess ? GDN_OK : hip_fail(e, "gdn_linear_prefill launch");
}

gdn_status gdn_linear_step(const gdn_shape* sh, const void* q, const void* k, const void* v, const float* g,
                           int64_t g_stride, const float* s0, int64_t s0_stride, const int32_t* cu, void* o,
                           float* s_out, int32_t cap, const int32_t* counts, float* su, void* stream) {
  int64_t total = 0;
  Buf ins[7];
  gdn_status st = check_linear(sh, q, k, v, g, g_stride, s0, s0_stride, cu, o, s_out, &total, ins);
  if (st != GDN_OK) return st;
  if (cap < 0) return fail(GDN_ERR_INVALID_ARG, "state_update_capacity=%d < 0", cap);
  if (cap > 0) {
    if (counts == nullptr) return fail(GDN_ERR_INVALID_ARG, "capture_count is required when state_update_capacity > 0");
    if (su == nullptr) return fail(GDN_ERR_INVALID_ARG, "state_update is required when state_update_capacity > 0");
    if (misaligned(counts, 4)) return fail(GDN_ERR_INVALID_ARG, "capture_count is not 4-byte aligned");
    if (!aligned16(su)) return fail(GDN_ERR_INVALID_ARG, "state_update is not 16-byte aligned");
    const size_t R = (size_t)sh->Hv + (size_t)sh->Hq * sh->dk + (size_t)sh->Hv * sh->dv;
    Buf all[9];
    std::copy(ins, ins + 6, all);
    all[6] = {o, (size_t)total * sh->Hv * sh->dv * elem_size(sh->dtype), "o"};
    all[7] = {s_out, (size_t)sh->B * sh->Hv * sh->dk * sh->dv * 4, "final_state"};
    all[8] = {counts, (size_t)sh->B * 4, "capture_count"};
    if ((st = check_apart({su, (size_t)sh->B * (size_t)cap * R * 4, "state_update"}, all, 9)) != GDN_OK) return st;
    const Buf cb = {counts, (size_t)sh->B * 4, "capture_count"};
    for (int i = 6; i < 8; ++i)
      if ((st = check_apart(all[i], &cb, 1)) != GDN_OK) return st;
  }
  if (sh->B == 0 || (total == 0 && s_out == nullptr)) return GDN_OK;
  LinearArgs a = linear_args(sh, q, k, v, g, g_stride, s0, s0_stride, cu, o, s_out, total);
  a.cap = cap; a.counts = counts; a.su = su;
  const hipError_t e = launch_linear_step((DType)sh->dtype, a, static_cast<hipStream_t>(stream));
  return e == hipSuccess ? GDN_OK : hip_fail(e, "gdn_linear_step launch");
}

}  // extern "C"

// ---------------------------------------------------------------------------
// Verification of drafted tokens
// ---------------------------------------------------------------------------
namespace {

gdn_status check_verify(const gdn_verify_shape* sh) {
  if (sh == nullptr) return fail(GDN_ERR_INVALID_ARG, "shape is NULL");
  if (sh->B < 0 || sh->K < 0 || sh->V < 1)
    return fail(GDN_ERR_INVALID_ARG, "B=%d and K=%d must be >= 0 and V=%d >= 1", sh->B, sh->K, sh->V);
  if (sh->dtype != GDN_F32 && sh->dtype != GDN_F16 && sh->dtype != GDN_BF16)
    return fail(GDN_ERR_INVALID_ARG, "dtype %d is not a gdn_dtype", sh->dtype);
  if (sh->target_row_stride < sh->V || sh->draft_row_stride < sh->V)
    return fail(GDN_ERR_INVALID_ARG, "row strides %lld, %lld are smaller than V=%d",
                (long long)sh->target_row_stride, (long long)sh->draft_row_stride, sh->V);
  if (sh->B > 65535 || sh->K > 1024) return fail(GDN_ERR_UNSUPPORTED, "B=%d exceeds 65535 or K=%d 1024", sh->B, sh->K);
  if (sh->V > (1 << 24)) return fail(GDN_ERR_UNSUPPORTED, "V=%d exceeds 2^24", sh->V);
  if (sh->target_row_stride > (1LL << 32) || sh->draft_row_stride > (1LL << 32))
    return fail(GDN_ERR_UNSUPPORTED, "row strides above 2^32");
  return GDN_OK;
}

// Vocabulary entries per tile: small enough that one row spreads over many
// workgroups and that finding the token inside its tile is one short scan,
// at most 1024 tiles a row.
int32_t verify_tile(int32_t V) {
  int32_t t = 2048;
  while ((V + t - 1) / t > 1024) t *= 2;
  return t;
}

size_t verify_workspace(const gdn_verify_shape* sh) {
  if (sh->V <= kVerifyRowMax) return 0;
  const int32_t t = verify_tile(sh->V);
  return (size_t)sh->B * ((sh->V + t - 1) / t) * sizeof(double);
}

}  // namespace

extern "C" {

size_t gdn_verify_workspace_bytes(const gdn_verify_shape* sh) {
  return check_verify(sh) == GDN_OK ? verify_workspace(sh) : (size_t)-1;
}

gdn_status gdn_verify_drafts(const gdn_verify_shape* sh, const void* p, const void* q, const int32_t* x,
                             const float* u, const int32_t* n, int32_t* tokens, int32_t* emit, void* ws,
                             size_t ws_bytes, void* stream) {
  gdn_status st = check_verify(sh);
  if (st != GDN_OK) return st;
  if (sh->B == 0) return GDN_OK;
  const size_t es = elem_size(sh->dtype), B = (size_t)sh->B, K = (size_t)sh->K, V = (size_t)sh->V;
  if (p == nullptr || u == nullptr || tokens == nullptr || emit == nullptr || (x == nullptr && K > 0))
    return fail(GDN_ERR_INVALID_ARG, "target_probs, draft_tokens, uniforms, tokens and emit_count are required");
  if (misaligned(p, es) || misaligned(q, es))
    return fail(GDN_ERR_INVALID_ARG, "target_probs / draft_probs are not aligned to their type");
  if (misaligned(x, 4) || misaligned(u, 4) || misaligned(n, 4) || misaligned(tokens, 4) || misaligned(emit, 4))
    return fail(GDN_ERR_INVALID_ARG, "an int32 or fp32 argument is not 4-byte aligned");
  const size_t need = verify_workspace(sh);
  if (need > 0) {
    if (ws == nullptr || ws_bytes < need)
      return fail(GDN_ERR_INVALID_ARG, "workspace of %zu bytes is smaller than the %zu required", ws_bytes, need);
    if (!aligned16(ws)) return fail(GDN_ERR_INVALID_ARG, "workspace is not 16-byte aligned");
  }
  const Buf ins[5] = {{p, ((B * (K + 1) - 1) * (size_t)sh->target_row_stride + V) * es, "target_probs"},
                      {q, K > 0 ? ((B * K - 1) * (size_t)sh->draft_row_stride + V) * es : 0, "draft_probs"},
                      {x, B * K * 4, "draft_tokens"},
                      {u, B * (K + 1) * 4, "uniforms"},
                      {n, B * 4, "draft_count"}};
  const Buf outs[3] = {{tokens, B * (K + 1) * 4, "tokens"}, {emit, B * 4, "emit_count"}, {ws, need, "workspace"}};
  for (int i = 0; i < 3; ++i) {
    if ((st = check_apart(outs[i], ins, 5)) != GDN_OK) return st;
    if ((st = check_apart(outs[i], outs, i)) != GDN_OK) return st;
  }
  VerifyArgs a{};
  a.p = p; a.q = q; a.p_stride = sh->target_row_stride; a.q_stride = sh->draft_row_stride;
  a.x = x; a.u = u; a.n = n; a.tokens = tokens; a.emit = emit;
  a.B = sh->B; a.K = sh->K; a.V = sh->V;
  a.tile = verify_tile(sh->V);
  a.tiles = (sh->V + a.tile - 1) / a.tile;
  a.part = static_cast<double*>(ws);
  const hipError_t e = launch_verify((DType)sh->dtype, a, static_cast<hipStream_t>(stream));
  return e == hipSuccess ? GDN_OK : hip_fail(e, "gdn_verify_drafts launch");
}

// ---------------------------------------------------------------------------
// Norms around a block
// ---------------------------------------------------------------------------
gdn_status gdn_block_norm(const gdn_norm_shape* sh, const void* y, const void* gate, const void* res,
                          const void* wpost, const void* wnext, void* h, void* normed, void* stream) {
  if (sh == nullptr) return fail(GDN_ERR_INVALID_ARG, "shape is NULL");
  if (sh->T < 0 || sh->D < 1)
    return fail(GDN_ERR_INVALID_ARG, "T=%lld must be >= 0 and D=%d >= 1", (long long)sh->T, sh->D);
  if (sh->dtype != GDN_F32 && sh->dtype != GDN_F16 && sh->dtype != GDN_BF16)
    return fail(GDN_ERR_INVALID_ARG, "dtype %d is not a gdn_dtype", sh->dtype);
  if (sh->gate_act < GDN_ACT_NONE || sh->gate_act > GDN_ACT_SIGMOID)
    return fail(GDN_ERR_INVALID_ARG, "gate_act %d is not a gdn_act", sh->gate_act);
  if (sh->group < 1 || sh->D % sh->group != 0)
    return fail(GDN_ERR_INVALID_ARG, "group=%d must be positive and divide D=%d", sh->group, sh->D);
  if (sh->group != sh->D && !supported_dim(sh->group))
    return fail(GDN_ERR_UNSUPPORTED, "group=%d: supported groups are D, 16, 32, 64, 128", sh->group);
  if (sh->D > 16384) return fail(GDN_ERR_UNSUPPORTED, "D=%d exceeds 16384", sh->D);
  if (sh->T > 0x7fffffffLL) return fail(GDN_ERR_UNSUPPORTED, "T=%lld exceeds 2^31-1", (long long)sh->T);
  if (!(sh->eps >= 0.f) || sh->eps == INFINITY) return fail(GDN_ERR_INVALID_ARG, "eps must be finite and >= 0");
  if (!(sh->residual_scale == sh->residual_scale)) return fail(GDN_ERR_INVALID_ARG, "residual_scale is NaN");
  if (sh->T == 0) return GDN_OK;   // empty tensors may have no address
  if ((gate != nullptr) != (sh->gate_act != GDN_ACT_NONE))
    return fail(GDN_ERR_INVALID_ARG, "gate is required with a gate_act other than GDN_ACT_NONE, and only then");
  if ((wnext != nullptr) != (normed != nullptr))
    return fail(GDN_ERR_INVALID_ARG, "next_weight and normed are given together or not at all");
  if (y == nullptr || h == nullptr) return fail(GDN_ERR_INVALID_ARG, "y and h are required");
  const size_t es = elem_size(sh->dtype), n = (size_t)sh->T * sh->D * es;
  const Buf ins[5] = {{y, n, "y"}, {res, n, "residual"}, {gate, n, "gate"},
                      {wpost, (size_t)sh->group * es, "post_weight"}, {wnext, (size_t)sh->D * es, "next_weight"}};
  for (const Buf& b : ins)
    if (misaligned(b.p, es)) return fail(GDN_ERR_INVALID_ARG, "%s is not aligned to its type", b.name);
  if (misaligned(h, es) || misaligned(normed, es))
    return fail(GDN_ERR_INVALID_ARG, "h / normed are not aligned to their type");
  gdn_status st;
  const Buf hb = {h, n, "h"}, nb = {normed, n, "normed"};
  for (int i = 0; i < 5; ++i)   // exactly in place on y or residual is allowed
    if (!(i < 2 && ins[i].p == h) && (st = check_apart(hb, ins + i, 1)) != GDN_OK) return st;
  if ((st = check_apart(nb, ins, 5)) != GDN_OK) return st;
  if ((st = check_apart(nb, &hb, 1)) != GDN_OK) return st;
  NormArgs a{};
  a.y = y; a.gate = gate; a.res = res; a.wpost = wpost; a.wnext = wnext; a.h = h; a.normed = normed;
  a.T = sh->T; a.D = sh->D; a.group = sh->group; a.act = sh->gate_act;
  a.scale = sh->residual_scale; a.eps = sh->eps;
  const hipError_t e = launch_norm((DType)sh->dtype, a, static_cast<hipStream_t>(stream));
  return e == hipSuccess ? GDN_OK : hip_fail(e, "gdn_block_norm launch");
}

}  // extern "C"
