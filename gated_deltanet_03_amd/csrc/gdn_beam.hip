// The K best continuations of a beam search: log softmax, scores and selection over beams and vocabulary.
//
//   c(w, v) = (score_w - log sum_u exp(x_wu - m_w)) + (x_wv - m_w),   m_w = max_u x_wu
//
// Bound by reading the logits once.  beam_part_kernel: a workgroup takes a segment of one row into registers, and
// leaves its maximum, its sum of exponentials against that maximum, and its K largest entries in order: within a beam
// that is the order of the logits, whatever the sum turns out to be.  beam_join_kernel: a workgroup for each search
// joins the segments' sums and selects among the K * segments * W entries that are left.
//
// Selection: the K-th largest of a wave's 64 lane maxima, found by bisection over their upper bits with ballots, is a
// bound that at least K entries reach; the entries that reach the highest wave's bound go to a list in LDS, and an
// entry's rank is the number of entries before it.  Lists that do not fit (very many equal entries) are taken one
// maximum at a time.
//
// 16 searches of 8 beams over 131072 tokens, bf16: 16.2 us (the logits alone 6.6 us; by count vector operations, 10 an
// entry, are as long again) and 6.9 us for the join, a chain of latencies; 4 beams over 32003, fp32: 3.8 and 5.1 us.
//
// Sums of exponentials: the difference to the maximum first, so that the exponent's rounding is small where terms are
// large; eight terms a thread in fp32, those in 64 bits.
#include <algorithm>

#include "gdn_cache_internal.h"
#include "gdn_rows.h"
#include "gdn_scan.h"

namespace gdn {

constexpr int kThreads = 256, kList = 1024;

// Floats as integers of the same order (-0 as 0, NaN above or below everything).
__device__ __forceinline__ uint32_t ordered(float x) {
  const uint32_t u = __float_as_uint(x + 0.0f);
  return u ^ ((uint32_t)((int32_t)u >> 31) | 0x80000000u);
}
__device__ __forceinline__ float unordered(uint32_t u) {
  return __uint_as_float(u ^ (~(uint32_t)((int32_t)u >> 31) | 0x80000000u));
}
__device__ __forceinline__ uint64_t ordered64(double x) {
  const uint64_t u = __builtin_bit_cast(uint64_t, x);
  return u ^ ((uint64_t)((int64_t)u >> 63) | 0x8000000000000000ull);
}
__device__ __forceinline__ double unordered64(uint64_t u) {
  return __builtin_bit_cast(double, u ^ (~(uint64_t)((int64_t)u >> 63) | 0x8000000000000000ull));
}

// The upper BITS bits of the k-th largest of the lanes' values (1 <= k <= 64).
template <int BITS>
__device__ __forceinline__ uint32_t kth_of_lanes(uint32_t v, int k) {
  uint32_t t = 0;
#pragma unroll
  for (int b = 31; b >= 32 - BITS; --b) {
    const uint32_t at = t | (1u << b);
    if (__popcll(__ballot(v >= at)) >= k) t = at;
  }
  return t;
}

__device__ __forceinline__ uint32_t wave_max(uint32_t v) {
  auto up = [&](uint32_t o) { v = o > v ? o : v; };
  up(__builtin_amdgcn_update_dpp(0, (int)v, 0xb1, 0xf, 0xf, false));    // lane ^ 1
  up(__builtin_amdgcn_update_dpp(0, (int)v, 0x4e, 0xf, 0xf, false));    // lane ^ 2
  up(__builtin_amdgcn_update_dpp(0, (int)v, 0x141, 0xf, 0xf, false));   // the other four of 8
  up(__builtin_amdgcn_update_dpp(0, (int)v, 0x140, 0xf, 0xf, false));   // the other eight of 16
  const auto a = __builtin_amdgcn_permlane16_swap(v, v, false, false);
  v = a[0] > a[1] ? a[0] : a[1];
  const auto b = __builtin_amdgcn_permlane32_swap(v, v, false, false);
  return b[0] > b[1] ? b[0] : b[1];
}

__device__ __forceinline__ uint64_t wave_max64(uint64_t v) {
#pragma unroll
  for (int m = 1; m < 64; m <<= 1) {
    const uint64_t o = __shfl_xor(v, m);
    v = o > v ? o : v;
  }
  return v;
}

__device__ __forceinline__ double wave_sum64(double v) {
  const uint64_t u = __builtin_bit_cast(uint64_t, wave_scan64(v));
  const uint32_t lo = __builtin_amdgcn_readlane((int)(uint32_t)u, 63);
  return __builtin_bit_cast(double, (uint64_t)(uint32_t)__builtin_amdgcn_readlane((int)(u >> 32), 63) << 32 | lo);
}

// Entries of a segment as keys: the logit's order, then the lower index first.
__device__ __forceinline__ uint64_t entry_key(float x, int v) { return (uint64_t)ordered(x) << 32 | (uint32_t)~v; }

__device__ __forceinline__ uint64_t lane_value64(uint64_t v, int lane) {
  return (uint64_t)(uint32_t)__builtin_amdgcn_readlane((int)(v >> 32), lane) << 32 |
         (uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)v, lane);
}

// Entries of a list of n <= 64, by rank: body(rank, key, place) for the wave's share of them, every `waves`-th, a ballot
// each (a loop over the list in every thread: 2.9 us for 30 entries, so 0.6).
template <typename B>
__device__ __forceinline__ void by_rank(const uint64_t* list, const uint32_t* from, int n, int wave, int waves,
                                        B&& body) {
  const int lane = threadIdx.x & 63;
  const uint64_t k = lane < n ? list[lane] : 0;
  const uint32_t f = from && lane < n ? from[lane] : 0;
  for (int i = wave; i < n; i += waves) {
    const uint64_t ki = lane_value64(k, i);
    const uint32_t fi = (uint32_t)__builtin_amdgcn_readlane((int)f, i);
    const int rank = __popcll(__ballot(k > ki || (k == ki && f > fi)));
    if (lane == 0) body(rank, ki, fi);
  }
}

// How many of a list's n entries come before one: larger keys, or equal ones with the larger place.
template <bool PLACES>
__device__ __forceinline__ int rank_of(const uint64_t* list, const uint32_t* from, int n, uint64_t k, uint32_t f) {
  int rank = 0, o = 0;
  for (; o + 8 <= n; o += 8) {
#pragma unroll
    for (int i = 0; i < 8; ++i) rank += list[o + i] > k || (PLACES && list[o + i] == k && from[o + i] > f);
  }
  for (; o < n; ++o) rank += list[o] > k || (PLACES && list[o] == k && from[o] > f);
  return rank;
}

// NV 16-byte vectors a thread: NV * 256 * (16 / sizeof(T)) entries a segment.
template <typename T, int NV>
__global__ __launch_bounds__(kThreads, 8) void beam_part_kernel(SelectArgs p, int64_t row0) {
  constexpr int E = Vec16<T>::N;
  __shared__ uint64_t list[kList];
  __shared__ uint32_t wave_top[4], wave_kth[4];
  __shared__ double wave_sum[4];
  __shared__ int count;
  __shared__ uint64_t top_key[4];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int64_t row = row0 + blockIdx.y;
  const int seg = blockIdx.x, v0 = seg * p.segment;
  const T* x = static_cast<const T*>(p.x) + row * p.row_stride;
  Vec16<T> q[NV];
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    const int v = v0 + (j * kThreads + tid) * E;
    if (v + E <= p.V) {
      __builtin_memcpy(q[j].e, x + v, 16);
    } else {
#pragma unroll
      for (int i = 0; i < E; ++i) q[j].e[i] = v + i < p.V ? x[v + i] : Elem<T>::from_f(-INFINITY);
    }
  }
  if (p.finished && p.finished[row]) return;      // (asked for beside the entries) the join reads nothing of it
  if (tid == 0) count = 0;
  // The entries stay packed: the compiler would keep them widened from one pass to the next, in twice the registers.
  auto repack = [&] {
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      uint4 u = __builtin_bit_cast(uint4, q[j]);
      asm volatile("" : "+v"(u.x), "+v"(u.y), "+v"(u.z), "+v"(u.w));
      q[j] = __builtin_bit_cast(Vec16<T>, u);
    }
  };
  float top = -INFINITY;                         // (NaN does not show here, but in the sum)
#pragma unroll
  for (int j = 0; j < NV; ++j)
#pragma unroll
    for (int i = 0; i < E; ++i) top = fmaxf(top, q[j].f(i));
  repack();
  const uint32_t mine = ordered(top);
  const uint32_t kth = kth_of_lanes<16>(mine, p.K), wtop = wave_max(mine);
  if (lane == 0) wave_top[wave] = wtop, wave_kth[wave] = kth;
  __syncthreads();
  uint32_t m = wave_top[0], bound = wave_kth[0];
#pragma unroll
  for (int w = 1; w < 4; ++w) {
    m = wave_top[w] > m ? wave_top[w] : m;
    bound = wave_kth[w] > bound ? wave_kth[w] : bound;
  }
  const int64_t at = row * p.segments + seg;
  const float most = unordered(m);
  const uint32_t void_key = ordered(-INFINITY);
  if (bound <= void_key) bound = void_key + 1;   // -infinity is no entry
  const float least = unordered(bound);
  double sum = 0.0;
  if (most == -INFINITY) {                       // differences would be NaN where entries are -infinity
#pragma unroll
    for (int j = 0; j < NV; ++j)
#pragma unroll
      for (int i = 0; i < E; ++i)
        if (q[j].f(i) != q[j].f(i)) sum = NAN;
  } else {
    uint32_t reach[(NV * E + 31) / 32] = {};     // which of the thread's entries reach the bound
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      float part = 0.f;
#pragma unroll
      for (int i = 0; i < E; ++i) {
        const float f = q[j].f(i);
        part += __builtin_amdgcn_exp2f((f - most) * 1.44269504f);
        if (f >= least) reach[(j * E + i) / 32] |= 1u << (j * E + i) % 32;
      }
      sum += (double)part;
    }
#pragma unroll
    for (int r = 0; r < (NV * E + 31) / 32; ++r)
      for (uint32_t left = reach[r]; left != 0; left &= left - 1) {
        const int k = r * 32 + __ffs(left) - 1, v = v0 + (k / E * kThreads + tid) * E + k % E;
        const int n = atomicAdd(&count, 1);
        if (n < kList) list[n] = entry_key(Elem<T>::to_f(x[v]), v);   // read again: registers cannot be indexed
      }
  }
  sum = wave_sum64(sum);
  if (lane == 0) wave_sum[wave] = sum;
  __syncthreads();
  sum = (wave_sum[0] + wave_sum[1]) + (wave_sum[2] + wave_sum[3]);
  const bool wrong = !(sum < INFINITY) || most == INFINITY;
  if (tid == 0) {                                // NaN tells the join that the beam is absent
    p.seg_max[at] = wrong ? NAN : most;
    p.seg_sum[at] = sum;
  }
  const int n = wrong ? 0 : count;
  uint64_t* best = p.best + at * p.K;
  if (n <= 64) {
    by_rank(list, nullptr, n, wave, 4, [&](int rank, uint64_t k, uint32_t) {
      if (rank < p.K) best[rank] = k;
    });
    if (tid >= n && tid < p.K) best[tid] = 0;
    return;
  }
  if (n <= kList) {
    for (int i = tid; i < n; i += kThreads) {
      const uint64_t k = list[i];
      const int rank = rank_of<false>(list, nullptr, n, k, 0);
      if (rank < p.K) best[rank] = k;
    }
    return;
  }
  uint64_t last = ~0ull;                         // one maximum below the last one at a time, read again
  for (int r = 0; r < p.K; ++r) {
    uint64_t k = 0;
    for (int v = v0 + tid; v < min(v0 + p.segment, p.V); v += kThreads) {
      const uint64_t e = entry_key(Elem<T>::to_f(x[v]), v);
      if (e < last && e > k && (uint32_t)(e >> 32) > void_key) k = e;
    }
    k = wave_max64(k);
    if (lane == 0) top_key[wave] = k;
    __syncthreads();
    k = top_key[0];
#pragma unroll
    for (int w = 1; w < 4; ++w) k = top_key[w] > k ? top_key[w] : k;
    if (tid == 0) best[r] = k;
    last = k;
    __syncthreads();
  }
}

// One workgroup a search.  A thread holds up to kHeld of the entries, loaded before the sums are joined; only searches
// with more entries (very large vocabularies, many beams) read the others again from memory.
constexpr int kJoin = 1024, kWaves = kJoin / 64, kHeld = 4;

__global__ __launch_bounds__(kJoin) void beam_join_kernel(SelectArgs p) {
  __shared__ double start[64];                   // score minus log of the sum; NaN: absent
  __shared__ double high[64];                    // the maximum, apart: the log would drown in one of -1e38
  __shared__ uint8_t done[64];
  __shared__ uint64_t key[kList];
  __shared__ uint32_t from[kList];
  __shared__ int count;
  __shared__ uint64_t top_key[kWaves];
  __shared__ uint32_t top_from[kWaves];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int64_t b = blockIdx.x;
  if (tid == 0) count = 0;
  // entry i: the (i % (K * segments))-th of beam i / (K * segments)
  const int per = p.K * p.segments, all = per * p.W;
  uint64_t held[kHeld];
#pragma unroll
  for (int h = 0; h < kHeld; ++h) {
    const int i = tid + h * kJoin;
    held[h] = i < all ? p.best[b * all + i] : 0;
  }
  for (int w = wave; w < p.W; w += kWaves) {     // sums: a wave a beam
    const int64_t row = b * p.W + w;
    const float score = p.scores[row];
    const bool fin = p.finished && p.finished[row];
    double log_sum = 0.0;
    float m = -INFINITY;
    bool wrong = !(fabsf(score) < INFINITY);
    if (!fin) {
      for (int s = lane; s < p.segments; s += 64) {
        const float f = p.seg_max[row * p.segments + s];
        wrong |= f != f;
        m = fmaxf(m, f);
      }
      m = unordered(wave_max(ordered(m)));
      double sum = 0.0;
      for (int s = lane; s < p.segments; s += 64) {
        const float f = p.seg_max[row * p.segments + s];
        if (f > -INFINITY) sum += p.seg_sum[row * p.segments + s] * exp((double)f - (double)m);
      }
      sum = wave_sum64(sum);
      wrong = __ballot(wrong) != 0 || m == -INFINITY;
      log_sum = log(sum);
    }
    if (lane == 0) {
      start[w] = wrong ? (double)NAN : (double)score - log_sum;
      high[w] = m;
      done[w] = fin;
    }
  }
  __syncthreads();

  // entry i as a score's order and a place: 0 if it is none
  auto candidate = [&](int i, uint64_t e, uint64_t& k, uint32_t& f) {
    const int w = i / per;
    k = 0;
    f = 0;
    const double s = start[w];
    if (s != s) return;
    if (done[w]) {
      if (i != w * per) return;
      k = ordered64(s);
      f = (uint32_t)~((w << 24) | p.pad);
      return;
    }
    if (e == 0) return;
    k = ordered64(s + ((double)unordered((uint32_t)(e >> 32)) - high[w]));
    f = (uint32_t)~((w << 24) | (int)~(uint32_t)e);   // token below 2^24, beam below 2^6: lower flat index, larger f
  };
  uint64_t hk[kHeld];
  uint32_t hf[kHeld];
#pragma unroll
  for (int h = 0; h < kHeld; ++h) {
    hk[h] = 0, hf[h] = 0;
    if (tid + h * kJoin < all) candidate(tid + h * kJoin, held[h], hk[h], hf[h]);
  }
  // body(key, place) of every entry of this thread
  auto each = [&](auto&& body) {
#pragma unroll
    for (int h = 0; h < kHeld; ++h) body(hk[h], hf[h]);
    for (int i = tid + kHeld * kJoin; i < all; i += kJoin) {
      uint64_t k;
      uint32_t f;
      candidate(i, p.best[b * all + i], k, f);
      body(k, f);
    }
  };
  // The lists are in order: the K-th largest of 64 maxima of their first entries, the same in every wave, is a bound
  // that K entries reach (in fp32: rounding keeps the order).
  auto coarse = [](uint64_t k) { return k ? ordered((float)unordered64(k)) : 0u; };
  uint32_t mine = 0;
  for (int l = lane; l < p.W * p.segments; l += 64) {
    uint64_t k;
    uint32_t f;
    candidate(l * p.K, p.best[b * all + (int64_t)l * p.K], k, f);
    const uint32_t h = coarse(k);
    mine = h > mine ? h : mine;
  }
  const uint32_t bound = kth_of_lanes<32>(mine, p.K);
  each([&](uint64_t k, uint32_t f) {
    if (k != 0 && coarse(k) >= bound) {
      const int n = atomicAdd(&count, 1);
      if (n < kList) key[n] = k, from[n] = f;
    }
  });
  __syncthreads();
  const int n = count;
  auto put = [&](int r, uint64_t k, uint32_t f) {
    const int64_t o = b * p.K + r;
    const uint32_t u = ~f;
    const int w = (int)(u >> 24), v = (int)(u & 0xffffff);
    p.tokens[o] = k ? v : -1;
    p.parents[o] = k ? w : -1;
    p.new_scores[o] = k ? (float)unordered64(k) : -INFINITY;
    p.new_finished[o] = !k || done[w] || v == p.eos;
  };
  if (n <= 64) {
    by_rank(key, from, n, wave, kWaves, [&](int rank, uint64_t k, uint32_t f) {
      if (rank < p.K) put(rank, k, f);
    });
    if (tid >= n && tid < p.K) put(tid, 0, ~0u);
    return;
  }
  if (n <= kList) {
    if (tid < n) {
      const uint64_t k = key[tid];
      const uint32_t f = from[tid];
      const int rank = rank_of<true>(key, from, n, k, f);
      if (rank < p.K) put(rank, k, f);
    }
    return;
  }
  uint64_t last = ~0ull;
  uint32_t last_f = ~0u;
  for (int r = 0; r < p.K; ++r) {
    uint64_t k = 0;
    uint32_t f = 0;
    each([&](uint64_t ki, uint32_t fi) {
      if ((ki < last || (ki == last && fi < last_f)) && (ki > k || (ki == k && fi > f))) k = ki, f = fi;
    });
    const uint64_t wk = wave_max64(k);
    const uint32_t wf = wave_max(k == wk ? f : 0);
    if (lane == 0) top_key[wave] = wk, top_from[wave] = wf;
    __syncthreads();
    k = top_key[0], f = top_from[0];
#pragma unroll
    for (int w = 1; w < kWaves; ++w)
      if (top_key[w] > k || (top_key[w] == k && top_from[w] > f)) k = top_key[w], f = top_from[w];
    if (tid == 0) put(r, k, f);
    last = k, last_f = f;
    __syncthreads();
  }
}

template <typename T>
static hipError_t launch_select_t(const SelectArgs& a, hipStream_t s) {
  constexpr int E = Vec16<T>::N;
  prof_begin(K_SELECT_PART, s);
  const int64_t rows = (int64_t)a.B * a.W;
  const int64_t most = std::min<int64_t>(65535, kLaunchThreads / kThreads / a.segments);
  for (int64_t r = 0; r < rows; r += most) {
    const dim3 grid((unsigned)a.segments, (unsigned)std::min(most, rows - r));
    if (a.segment == 2048) hipLaunchKernelGGL((beam_part_kernel<T, 8 / E>), grid, dim3(kThreads), 0, s, a, r);
    else hipLaunchKernelGGL((beam_part_kernel<T, 32 / E>), grid, dim3(kThreads), 0, s, a, r);
  }
  prof_end(K_SELECT_PART, s);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  prof_begin(K_SELECT_JOIN, s);
  hipLaunchKernelGGL(beam_join_kernel, dim3((unsigned)a.B), dim3(kJoin), 0, s, a);
  prof_end(K_SELECT_JOIN, s);
  return hipGetLastError();
}

hipError_t launch_select(DType dt, const SelectArgs& a, hipStream_t s) {
  switch (dt) {
    case DType::F32: return launch_select_t<float>(a, s);
    case DType::F16: return launch_select_t<_Float16>(a, s);
    case DType::BF16: return launch_select_t<__bf16>(a, s);
  }
  return hipErrorInvalidValue;
}

}  // namespace gdn
