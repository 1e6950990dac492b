// C-ABI entry points of the paged cache (append, attention), the beam selection and the reordering of rows:
// host-side validation, workspace sizing and dispatch.  Validation runs before any HIP call.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cmath>

#include "../../include/gdn.h"
#include "gdn_cache_internal.h"
#include "gdn_check.h"

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

gdn_status check_dtype(int32_t dtype) {
  if (dtype != GDN_F32 && dtype != GDN_F16 && dtype != GDN_BF16)
    return fail(GDN_ERR_INVALID_ARG, "dtype %d is not a gdn_dtype", dtype);
  return GDN_OK;
}

gdn_status check_cache(const gdn_cache_shape* sh, bool ragged, int64_t* tokens) {
  if (sh == nullptr) return fail(GDN_ERR_INVALID_ARG, "shape is NULL");
  if (sh->N < 0 || sh->T < 0) return fail(GDN_ERR_INVALID_ARG, "N=%d and T=%d must be >= 0", sh->N, sh->T);
  if (sh->Hq <= 0 || sh->Hkv <= 0 || sh->Hq % sh->Hkv != 0)
    return fail(GDN_ERR_INVALID_ARG, "Hq=%d must be a positive multiple of Hkv=%d", sh->Hq, sh->Hkv);
  gdn_status st = check_dtype(sh->dtype);
  if (st != GDN_OK) return st;
  if (sh->d != 32 && sh->d != 64 && sh->d != 128 && sh->d != 256)
    return fail(GDN_ERR_UNSUPPORTED, "d=%d: supported head dims of the cache are 32, 64, 128, 256", sh->d);
  if (sh->page_size < 1 || sh->num_pages < 0 || sh->max_pages < 0)
    return fail(GDN_ERR_INVALID_ARG, "page_size=%d must be >= 1, num_pages=%d and max_pages=%d >= 0", sh->page_size,
                sh->num_pages, sh->max_pages);
  if (sh->page_size % 16 != 0 || sh->page_size > 1024)
    return fail(GDN_ERR_UNSUPPORTED, "page_size=%d: supported are multiples of 16 up to 1024", sh->page_size);
  if ((int64_t)sh->max_pages * sh->page_size > (1LL << 26))
    return fail(GDN_ERR_UNSUPPORTED, "max_pages * page_size = %lld exceeds 2^26",
                (long long)sh->max_pages * sh->page_size);
  if ((int64_t)sh->num_pages * sh->page_size > 0x7fffffffLL / sh->Hkv)
    return fail(GDN_ERR_UNSUPPORTED, "the cache has more than 2^31-1 rows");
  if (sh->N > (1 << 20) || sh->Hq > 65535 || sh->Hq / sh->Hkv > 256)
    return fail(GDN_ERR_UNSUPPORTED, "N=%d exceeds 2^20, Hq=%d 65535 or Hq/Hkv 256", sh->N, sh->Hq);
  *tokens = ragged ? (int64_t)sh->T : (int64_t)sh->N * sh->T;
  if (*tokens > (1LL << 30) || *tokens * sh->Hq > 0x7fffffffLL)
    return fail(GDN_ERR_UNSUPPORTED, "%lld tokens of %d heads exceed 2^30 tokens or 2^31-1 rows", (long long)*tokens,
                sh->Hq);
  return GDN_OK;
}

size_t cache_bytes(const gdn_cache_shape* sh) {
  return (size_t)sh->num_pages * sh->Hkv * sh->page_size * sh->d * elem_size(sh->dtype);
}

// Bytes from a [tokens, H, d] tensor's first element to its last one's end.
size_t token_bytes(const gdn_cache_shape* sh, int64_t tokens, int64_t stride, int32_t H) {
  return tokens == 0 ? 0 : ((size_t)(tokens - 1) * stride + (size_t)H * sh->d) * elem_size(sh->dtype);
}

// A token tensor that is read at a stride.
gdn_status check_token_tensor(const gdn_cache_shape* sh, const void* p, int64_t stride, int32_t H, const char* name) {
  if (p == nullptr) return fail(GDN_ERR_INVALID_ARG, "%s is NULL", name);
  if (!aligned16(p)) return fail(GDN_ERR_INVALID_ARG, "%s is not 16-byte aligned", name);
  if (stride < (int64_t)H * sh->d || stride > (1LL << 32) || (stride * (int64_t)elem_size(sh->dtype)) % 16 != 0)
    return fail(GDN_ERR_INVALID_ARG, "%s_token_stride=%lld must be a multiple of 16 bytes, from H * d = %lld up to 2^32",
                name, (long long)stride, (long long)H * sh->d);
  return GDN_OK;
}

// The cache and its tables; fills ins (table, lens, cu).
gdn_status check_tables(const gdn_cache_shape* sh, const void* kc, const void* vc, const int32_t* table,
                        const int32_t* lens, const int32_t* cu, Buf ins[3]) {
  if (sh->num_pages > 0 && (kc == nullptr || vc == nullptr))
    return fail(GDN_ERR_INVALID_ARG, "k_cache and v_cache are required");
  if (!aligned16(kc) || !aligned16(vc)) return fail(GDN_ERR_INVALID_ARG, "k_cache or v_cache is not 16-byte aligned");
  if (lens == nullptr || (table == nullptr && sh->max_pages > 0))
    return fail(GDN_ERR_INVALID_ARG, "block_table and cache_lens are required");
  if (misaligned(table, 4) || misaligned(lens, 4) || misaligned(cu, 4))
    return fail(GDN_ERR_INVALID_ARG, "block_table, cache_lens or cu_seqlens is not 4-byte aligned");
  ins[0] = {table, (size_t)sh->N * sh->max_pages * 4, "block_table"};
  ins[1] = {lens, (size_t)sh->N * 4, "cache_lens"};
  ins[2] = {cu, cu ? ((size_t)sh->N + 1) * 4 : 0, "cu_seqlens"};
  return GDN_OK;
}

CacheArgs cache_args(const gdn_cache_shape* sh, const int32_t* table, const int32_t* lens, const int32_t* cu,
                     int64_t tokens) {
  CacheArgs c{};
  c.table = table; c.lens = lens; c.cu = cu;
  c.N = sh->N; c.T = sh->T; c.total = (int32_t)tokens;
  c.Hq = sh->Hq; c.Hkv = sh->Hkv; c.d = sh->d;
  c.page_size = sh->page_size; c.num_pages = sh->num_pages; c.max_pages = sh->max_pages;
  return c;
}

// How the attention of a call is cut: rows of a tile, shares of a head's work (0: a tile each).
//
// Few rows or many is one choice for a call, by its rows a sequence on average: the host does not know the lengths.
// Tiles of 32 and of 128 rows, 32 on 8 heads of 128, bf16: 16 sequences over 4096 keys with 8 tokens 54 and 67 us, 16
// tokens 55 and 71, 24 tokens 135 and 76; 64 over 1000 keys with 8 tokens 51 and 55, 10 tokens 57 and 55.  Single tokens
// beside a chunk: where the rule takes 32 rows, 64 over 2048 keys and 440 tokens 115 and 126 us, 32 over 4000 and 200 over
// 2000 115 and 127; where it takes 128, 32 over 4000 and 300 over 2000 119 and 131, and 1000 over 4000 190 and 162.
struct Plan {
  int32_t few, shares, rows, unit;
  int64_t tiles;
};

// As many workgroups as the card holds at once share the work evenly.  Tables too narrow for sequences whose cutting
// pays are not cut: then there is no join to launch (2.7 us, also where the kernel finds nothing to cut).  One token, 8
// heads, whole and cut: fp32 of 64 200 keys 11.1 and 14.0 us, 300 keys 13.9 and 14.0, 500 keys 16.3 and 14.0; bf16 of 128
// 300 keys 10.1 and 12.8, 500 keys 11.3 and 12.9, 1000 keys 16.8 and 13.2.
Plan attention_plan(const gdn_cache_shape* sh, int64_t tokens, bool ragged) {
  const int64_t G = sh->Hq / sh->Hkv, rows = tokens * G;
  Plan p{};
  p.few = rows <= (int64_t)kFewRows * sh->N;
  p.rows = p.few ? kFewRows : kManyRows;
  p.tiles = ragged ? rows / p.rows + sh->N : sh->N * (((int64_t)sh->T * G + p.rows - 1) / p.rows);
  const int rb = sh->d * (int)elem_size(sh->dtype), at_once = 256 * (p.few ? few_waves(rb) : many_waves(rb));
  const bool f32 = sh->dtype == GDN_F32;
  if ((int64_t)sh->max_pages * sh->page_size > (p.few ? kFewKeys + (f32 ? 16384 : 49152) / sh->d
                                                      : kManyKeys + (f32 ? 16384 : 81920) / sh->d))
    p.shares = std::max(1, std::min(kMostShares, at_once / sh->Hkv));
  // all tiles with twice the table's keys, and twice that where they are drawn out, stay below 2^30 units
  const int64_t keys = (int64_t)sh->max_pages * sh->page_size + 64 + p.rows;
  while (((p.tiles + sh->N) * ((keys >> p.unit) + 2)) > (1LL << 28)) ++p.unit;
  return p;
}

size_t part_rows(const gdn_cache_shape* sh, const Plan& p) { return (size_t)2 * p.shares * sh->Hkv * p.rows; }
size_t plan_bytes(const gdn_cache_shape* sh, const Plan& p) {
  return part_rows(sh, p) * (sh->d + 2) * 4 + (size_t)p.shares * sh->Hkv * 16;
}

}  // namespace

extern "C" {

// ---------------------------------------------------------------------------
// Paged cache
// ---------------------------------------------------------------------------
gdn_status gdn_cache_append(const gdn_cache_shape* sh, const gdn_append_shape* ap, const void* q, const void* k,
                            const void* v, const float* inv_freq, const int32_t* positions, const int32_t* pair_axis,
                            const int32_t* table, const int32_t* lens, const int32_t* cu, void* q_out, void* kc,
                            void* vc, void* stream) {
  int64_t tokens = 0;
  gdn_status st = check_cache(sh, cu != nullptr, &tokens);
  if (st != GDN_OK) return st;
  if (ap == nullptr) return fail(GDN_ERR_INVALID_ARG, "append is NULL");
  if (ap->rotary < 0 || ap->rotary > sh->d || ap->rotary % 2 != 0)
    return fail(GDN_ERR_INVALID_ARG, "rotary=%d must be even and in [0, d=%d]", ap->rotary, sh->d);
  if (ap->axes < 1 || ap->axes > 8) return fail(GDN_ERR_INVALID_ARG, "axes=%d must be in [1, 8]", ap->axes);
  if (tokens == 0 || sh->N == 0) return GDN_OK;
  if ((inv_freq != nullptr) != (ap->rotary > 0))
    return fail(GDN_ERR_INVALID_ARG, "inv_freq is required with rotary > 0, and only then");
  if ((q != nullptr) != (q_out != nullptr))
    return fail(GDN_ERR_INVALID_ARG, "q and q_out are given together or not at all");
  if (ap->axes > 1 && (positions == nullptr || pair_axis == nullptr))
    return fail(GDN_ERR_INVALID_ARG, "positions and pair_axis are required with %d axes", ap->axes);
  Buf ins[9];
  if ((st = check_tables(sh, kc, vc, table, lens, cu, ins)) != GDN_OK) return st;
  if ((st = check_token_tensor(sh, k, ap->k_token_stride, sh->Hkv, "k")) != GDN_OK) return st;
  if ((st = check_token_tensor(sh, v, ap->v_token_stride, sh->Hkv, "v")) != GDN_OK) return st;
  if (q != nullptr) {
    if ((st = check_token_tensor(sh, q, ap->q_token_stride, sh->Hq, "q")) != GDN_OK) return st;
    if (!aligned16(q_out)) return fail(GDN_ERR_INVALID_ARG, "q_out is not 16-byte aligned");
  }
  if (misaligned(inv_freq, 4) || misaligned(positions, 4) || misaligned(pair_axis, 4))
    return fail(GDN_ERR_INVALID_ARG, "inv_freq, positions or pair_axis is not 4-byte aligned");
  ins[3] = {k, token_bytes(sh, tokens, ap->k_token_stride, sh->Hkv), "k"};
  ins[4] = {v, token_bytes(sh, tokens, ap->v_token_stride, sh->Hkv), "v"};
  ins[5] = {inv_freq, (size_t)ap->rotary / 2 * 4, "inv_freq"};
  ins[6] = {positions, (size_t)ap->axes * tokens * 4, "positions"};
  ins[7] = {pair_axis, (size_t)ap->rotary / 2 * 4, "pair_axis"};
  ins[8] = {q, q ? token_bytes(sh, tokens, ap->q_token_stride, sh->Hq) : 0, "q"};
  const size_t cb = cache_bytes(sh);
  const Buf kb = {kc, cb, "k_cache"}, vb = {vc, cb, "v_cache"};
  const Buf qb = {q_out, q_out ? (size_t)tokens * sh->Hq * sh->d * elem_size(sh->dtype) : 0, "q_out"};
  const bool in_place = q_out == q && ap->q_token_stride == (int64_t)sh->Hq * sh->d;
  if ((st = check_apart(kb, ins, 9)) != GDN_OK) return st;
  if ((st = check_apart(vb, ins, 9)) != GDN_OK) return st;
  if ((st = check_apart(vb, &kb, 1)) != GDN_OK) return st;
  if ((st = check_apart(qb, ins, in_place ? 8 : 9)) != GDN_OK) return st;
  if ((st = check_apart(qb, &kb, 1)) != GDN_OK || (st = check_apart(qb, &vb, 1)) != GDN_OK) return st;
  AppendArgs a{};
  a.c = cache_args(sh, table, lens, cu, tokens);
  a.q = q; a.k = k; a.v = v;
  a.q_stride = ap->q_token_stride; a.k_stride = ap->k_token_stride; a.v_stride = ap->v_token_stride;
  a.inv_freq = inv_freq; a.positions = positions; a.pair_axis = pair_axis;
  a.rotary = ap->rotary; a.interleaved = ap->interleaved != 0; a.axes = ap->axes;
  a.q_out = q_out; a.k_cache = kc; a.v_cache = vc;
  const hipError_t e = launch_append((DType)sh->dtype, a, static_cast<hipStream_t>(stream));
  return e == hipSuccess ? GDN_OK : hip_fail(e, "gdn_cache_append launch");
}

size_t gdn_cache_attention_workspace_bytes(const gdn_cache_shape* sh, int32_t ragged) {
  int64_t tokens = 0;
  if (check_cache(sh, ragged != 0, &tokens) != GDN_OK) return (size_t)-1;
  return tokens == 0 || sh->N == 0 ? 0 : plan_bytes(sh, attention_plan(sh, tokens, ragged != 0));
}

gdn_status gdn_cache_attention(const gdn_cache_shape* sh, const void* q, int64_t q_stride, const void* kc,
                               const void* vc, const int32_t* table, const int32_t* lens, const int32_t* cu,
                               float scale, int32_t window, void* o, void* ws, size_t ws_bytes, void* stream) {
  int64_t tokens = 0;
  gdn_status st = check_cache(sh, cu != nullptr, &tokens);
  if (st != GDN_OK) return st;
  const float scale_log2 = (float)((double)scale * 1.4426950408889634);     // weights are powers of two
  if (!(scale > 0.f) || !(scale_log2 < INFINITY))
    return fail(GDN_ERR_INVALID_ARG, "scale=%g must be > 0 and, times log2(e), finite", (double)scale);
  if (window < 0) return fail(GDN_ERR_INVALID_ARG, "window=%d < 0", window);
  if (tokens == 0 || sh->N == 0) return GDN_OK;
  Buf ins[6];
  if ((st = check_tables(sh, kc, vc, table, lens, cu, ins)) != GDN_OK) return st;
  if ((st = check_token_tensor(sh, q, q_stride, sh->Hq, "q")) != GDN_OK) return st;
  if (o == nullptr) return fail(GDN_ERR_INVALID_ARG, "o is NULL");
  if (!aligned16(o)) return fail(GDN_ERR_INVALID_ARG, "o is not 16-byte aligned");
  const size_t cb = cache_bytes(sh);
  ins[3] = {q, token_bytes(sh, tokens, q_stride, sh->Hq), "q"};
  ins[4] = {kc, cb, "k_cache"};
  ins[5] = {vc, cb, "v_cache"};
  const Buf ob = {o, (size_t)tokens * sh->Hq * sh->d * elem_size(sh->dtype), "o"};
  if ((st = check_apart(ob, ins, 6)) != GDN_OK) return st;
  const Plan plan = attention_plan(sh, tokens, cu != nullptr);
  const size_t need = plan_bytes(sh, plan);
  if (need > 0) {
    if (ws == nullptr || ws_bytes < need)
      return fail(GDN_ERR_INVALID_ARG, "workspace of %zu bytes is smaller than the %zu required", ws_bytes, need);
    if (!aligned16(ws)) return fail(GDN_ERR_INVALID_ARG, "workspace is not 16-byte aligned");
    const Buf wb = {ws, need, "workspace"};
    if ((st = check_apart(wb, ins, 6)) != GDN_OK || (st = check_apart(wb, &ob, 1)) != GDN_OK) return st;
  }
  if ((plan.tiles + plan.shares) * sh->Hkv > (int64_t)(kLaunchThreads / 256))
    return fail(GDN_ERR_UNSUPPORTED, "too many (tile, head) pairs (%lld)", (long long)plan.tiles * sh->Hkv);
  AttendArgs a{};
  a.c = cache_args(sh, table, lens, cu, tokens);
  a.q = q; a.q_stride = q_stride; a.k_cache = kc; a.v_cache = vc; a.o = o;
  a.scale_log2 = scale_log2;
  a.window = std::min(window, 1 << 30);
  a.granules = sh->page_size / 16;
  a.granule_magic = ((1ull << 32) + a.granules - 1) / a.granules;
  a.few = plan.few; a.shares = plan.shares; a.tiles = (int32_t)plan.tiles; a.unit = plan.unit;
  // at a workgroup's rates beside the others': 3 us of few rows' keys; 16 us of many rows' keys, or 40 us where most tiles
  // are cut and written in pieces
  const bool f32 = sh->dtype == GDN_F32;
  a.extra_drawn = ((plan.few ? (f32 ? 8192 : 28672) : (f32 ? 16384 : 81920)) / sh->d) >> plan.unit;
  a.extra_even = plan.few ? a.extra_drawn : (f32 ? 256 : sh->d <= 64 ? 1920 : 1280) >> plan.unit;
  if (need > 0) {
    a.part_o = static_cast<float*>(ws);
    a.part_ml = a.part_o + part_rows(sh, plan) * sh->d;
    a.cuts = a.part_ml + part_rows(sh, plan) * 2;
  }
  const hipStream_t s = static_cast<hipStream_t>(stream);
  const hipError_t e = sh->dtype == GDN_F32   ? launch_attend_f32(a, s)
                       : sh->dtype == GDN_F16 ? launch_attend_f16(a, s)
                                              : launch_attend_bf16(a, s);
  return e == hipSuccess ? GDN_OK : hip_fail(e, "gdn_cache_attention launch");
}

}  // extern "C"

// ---------------------------------------------------------------------------
// Beams
// ---------------------------------------------------------------------------
namespace {

gdn_status check_beam(const gdn_beam_shape* sh) {
  if (sh == nullptr) return fail(GDN_ERR_INVALID_ARG, "shape is NULL");
  if (sh->B < 0 || sh->W < 1 || sh->K < 1 || sh->V < 1)
    return fail(GDN_ERR_INVALID_ARG, "B=%d must be >= 0, W=%d, K=%d and V=%d >= 1", sh->B, sh->W, sh->K, sh->V);
  gdn_status st = check_dtype(sh->dtype);
  if (st != GDN_OK) return st;
  if (sh->row_stride < sh->V)
    return fail(GDN_ERR_INVALID_ARG, "row_stride=%lld is smaller than V=%d", (long long)sh->row_stride, sh->V);
  if (sh->pad_token < 0 || sh->pad_token >= sh->V)
    return fail(GDN_ERR_INVALID_ARG, "pad_token=%d is not in [0, V=%d)", sh->pad_token, sh->V);
  if (sh->W > 64 || sh->K > 64) return fail(GDN_ERR_UNSUPPORTED, "W=%d or K=%d exceeds 64", sh->W, sh->K);
  if (sh->V > (1 << 24)) return fail(GDN_ERR_UNSUPPORTED, "V=%d exceeds 2^24", sh->V);
  if (sh->B > (1 << 20)) return fail(GDN_ERR_UNSUPPORTED, "B=%d exceeds 2^20", sh->B);
  if (sh->row_stride > (1LL << 32)) return fail(GDN_ERR_UNSUPPORTED, "row_stride above 2^32");
  return GDN_OK;
}

// Vocabulary entries a workgroup takes: fewer where the rows alone would leave CUs idle.
int32_t beam_segment(const gdn_beam_shape* sh) {
  const int64_t wgs = (int64_t)sh->B * sh->W * ((sh->V + 8191) / 8192);
  return wgs >= 512 ? 8192 : 2048;
}

struct BeamBytes {
  size_t best, sum, all;
};
BeamBytes beam_bytes(const gdn_beam_shape* sh, int32_t segments) {
  const size_t n = (size_t)sh->B * sh->W * segments;
  BeamBytes b;
  b.best = align_up(n * sh->K * 8, 16);
  b.sum = align_up(n * 8, 16);
  b.all = b.best + b.sum + align_up(n * 4, 16);
  return b;
}

}  // namespace

extern "C" {

size_t gdn_beam_workspace_bytes(const gdn_beam_shape* sh) {
  if (check_beam(sh) != GDN_OK) return (size_t)-1;
  const int32_t seg = beam_segment(sh);
  return sh->B == 0 ? 0 : beam_bytes(sh, (sh->V + seg - 1) / seg).all;
}

gdn_status gdn_beam_select(const gdn_beam_shape* sh, const void* x, const float* scores, const uint8_t* finished,
                           int32_t* tokens, int32_t* parents, float* new_scores, uint8_t* new_finished, void* ws,
                           size_t ws_bytes, void* stream) {
  gdn_status st = check_beam(sh);
  if (st != GDN_OK) return st;
  if (sh->B == 0) return GDN_OK;
  if (x == nullptr || scores == nullptr || tokens == nullptr || parents == nullptr || new_scores == nullptr ||
      new_finished == nullptr)
    return fail(GDN_ERR_INVALID_ARG, "logits, scores, tokens, parents, new_scores and new_finished are required");
  const size_t es = elem_size(sh->dtype), B = (size_t)sh->B, W = (size_t)sh->W, K = (size_t)sh->K;
  if (misaligned(x, es)) return fail(GDN_ERR_INVALID_ARG, "logits are not aligned to their type");
  if (misaligned(scores, 4) || misaligned(tokens, 4) || misaligned(parents, 4) || misaligned(new_scores, 4))
    return fail(GDN_ERR_INVALID_ARG, "an int32 or fp32 argument is not 4-byte aligned");
  const int32_t seg = beam_segment(sh), segments = (sh->V + seg - 1) / seg;
  const BeamBytes need = beam_bytes(sh, segments);
  if (ws == nullptr || ws_bytes < need.all)
    return fail(GDN_ERR_INVALID_ARG, "workspace of %zu bytes is smaller than the %zu required", ws_bytes, need.all);
  if (!aligned16(ws)) return fail(GDN_ERR_INVALID_ARG, "workspace is not 16-byte aligned");
  const Buf ins[3] = {{x, ((B * W - 1) * (size_t)sh->row_stride + (size_t)sh->V) * es, "logits"},
                      {scores, B * W * 4, "scores"},
                      {finished, B * W, "finished"}};
  const Buf outs[5] = {{tokens, B * K * 4, "tokens"}, {parents, B * K * 4, "parents"},
                       {new_scores, B * K * 4, "new_scores"}, {new_finished, B * K, "new_finished"},
                       {ws, need.all, "workspace"}};
  for (int i = 0; i < 5; ++i) {
    if ((st = check_apart(outs[i], ins, 3)) != GDN_OK) return st;
    if ((st = check_apart(outs[i], outs, i)) != GDN_OK) return st;
  }
  SelectArgs a{};
  a.x = x; a.row_stride = sh->row_stride; a.scores = scores; a.finished = finished;
  a.tokens = tokens; a.parents = parents; a.new_scores = new_scores; a.new_finished = new_finished;
  a.B = sh->B; a.W = sh->W; a.K = sh->K; a.V = sh->V; a.eos = sh->eos_token; a.pad = sh->pad_token;
  a.segment = seg; a.segments = segments;
  char* w = static_cast<char*>(ws);
  a.best = reinterpret_cast<uint64_t*>(w);
  a.seg_sum = reinterpret_cast<double*>(w + need.best);
  a.seg_max = reinterpret_cast<float*>(w + need.best + need.sum);
  const hipError_t e = launch_select((DType)sh->dtype, a, static_cast<hipStream_t>(stream));
  return e == hipSuccess ? GDN_OK : hip_fail(e, "gdn_beam_select launch");
}

gdn_status gdn_state_reorder(const gdn_reorder_shape* sh, const void* src, void* dst, const int32_t* si,
                             const int32_t* di, void* stream) {
  if (sh == nullptr) return fail(GDN_ERR_INVALID_ARG, "shape is NULL");
  if (sh->layers < 0 || sh->src_rows < 0 || sh->dst_rows < 0 || sh->row_bytes < 0 || sh->src_group < 0 || sh->G < 0 ||
      sh->W < 0)
    return fail(GDN_ERR_INVALID_ARG, "layers, rows, row_bytes, src_group, G and W must be >= 0");
  if (sh->row_bytes % 16 != 0 || sh->src_layer_stride % 16 != 0 || sh->dst_layer_stride % 16 != 0)
    return fail(GDN_ERR_INVALID_ARG, "row_bytes=%lld and the layer strides must be multiples of 16",
                (long long)sh->row_bytes);
  if (sh->W > 64) return fail(GDN_ERR_UNSUPPORTED, "W=%d exceeds 64", sh->W);
  const int64_t most = 1LL << 40;
  if (sh->row_bytes > most || sh->src_rows > most || sh->dst_rows > most || sh->layers > most ||
      sh->src_group > (1LL << 31) ||
      (sh->row_bytes > 0 && (sh->src_rows > (1LL << 46) / sh->row_bytes || sh->dst_rows > (1LL << 46) / sh->row_bytes)))
    return fail(GDN_ERR_UNSUPPORTED, "rows of more than 2^46 bytes in all");
  if (sh->layers == 0 || sh->G == 0 || sh->W == 0 || sh->row_bytes == 0 || sh->src_rows == 0 || sh->dst_rows == 0)
    return GDN_OK;
  if (src == nullptr || dst == nullptr || si == nullptr)
    return fail(GDN_ERR_INVALID_ARG, "src, dst and src_index are required");
  if (!aligned16(src) || !aligned16(dst)) return fail(GDN_ERR_INVALID_ARG, "src or dst is not 16-byte aligned");
  if (misaligned(si, 4) || misaligned(di, 4)) return fail(GDN_ERR_INVALID_ARG, "an index is not 4-byte aligned");
  const int64_t sb = sh->src_rows * sh->row_bytes, db = sh->dst_rows * sh->row_bytes;
  const int64_t stride_most = (1LL << 62) / sh->layers;
  if (std::llabs(sh->src_layer_stride) > stride_most || std::llabs(sh->dst_layer_stride) > stride_most)
    return fail(GDN_ERR_UNSUPPORTED, "layer strides beyond 2^62 in all");
  if (sh->layers > 1 && std::llabs(sh->dst_layer_stride) < db)
    return fail(GDN_ERR_INVALID_ARG, "dst_layer_stride=%lld is smaller than a layer's %lld bytes",
                (long long)sh->dst_layer_stride, (long long)db);
  const bool in_place = src == dst;
  if (in_place && sh->layers > 1 && sh->src_layer_stride != sh->dst_layer_stride)
    return fail(GDN_ERR_INVALID_ARG, "in place, the layer strides must be equal");
  auto extent = [&](const void* p, int64_t stride, int64_t bytes, const char* name) {
    const int64_t reach = stride * (sh->layers - 1);
    return Buf{static_cast<const char*>(p) + std::min<int64_t>(reach, 0), (size_t)(std::llabs(reach) + bytes), name};
  };
  const Buf s = extent(src, sh->src_layer_stride, sb, "src"), d = extent(dst, sh->dst_layer_stride, db, "dst");
  const size_t n = (size_t)sh->G * sh->W * 4;
  // two layers may be two allocations with the indexes anywhere between them: layer by layer then
  const Buf idx[2] = {{si, n, "src_index"}, {di, di ? n : 0, "dst_index"}};
  gdn_status st;
  if (!in_place && (st = check_apart(d, &s, 1)) != GDN_OK) return st;
  for (int64_t l = 0; l < std::min<int64_t>(sh->layers, 4096); ++l) {
    const Buf one = {static_cast<const char*>(dst) + l * sh->dst_layer_stride, (size_t)db, "dst"};
    if ((st = check_apart(one, idx, 2)) != GDN_OK) return st;
  }
  ReorderArgs a{};
  a.src = static_cast<const char*>(src); a.dst = static_cast<char*>(dst);
  a.layers = sh->layers; a.src_layer = sh->src_layer_stride; a.dst_layer = sh->dst_layer_stride;
  a.src_rows = sh->src_rows; a.dst_rows = sh->dst_rows; a.row_bytes = sh->row_bytes; a.src_group = sh->src_group;
  a.G = sh->G; a.W = sh->W; a.src_index = si; a.dst_index = di;
  const hipError_t e = launch_reorder(a, static_cast<hipStream_t>(stream));
  return e == hipSuccess ? GDN_OK : hip_fail(e, "gdn_state_reorder launch");
}

}  // extern "C"
