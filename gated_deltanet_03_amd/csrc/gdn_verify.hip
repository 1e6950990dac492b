// Verification of drafted tokens against the target's probabilities.
//
// Up to 65536 entries one kernel, a workgroup a row (verify_row): tiles of one
// wave's 512 entries are summed, the tile that holds u * sum(w) is found among the
// at most 128 sums and scanned by one wave.
//
// Beyond, two kernels.  verify_sum: one workgroup per (tile of the vocabulary,
// row) finds how many drafts the row accepts (a gather of at most K pairs), then
// sums the tiles' weights w = max(p_a - q_a, 0) (or p_a).  verify_draw: one
// workgroup per row scans the tiles' sums, finds the tile that holds u * sum(w),
// and scans that tile alone.
//
// Only one row of p and one of q are read; one tile is read again, from the
// cache.  Bound by memory for a batch, by the call's host time for one row.
//
// Sums in 64 bits: a vocabulary of 10^5 entries puts the borders between tokens
// 10^-5 apart, and sums in 32 bits, whose order depends on the split, would
// place one token in a hundred wrongly.
//
// Calls measured, fp32, inputs new to the caches: one row of 32003 8.7 us in one
// kernel, bound by its host time, 12.1 in two; 64 rows of 32768 8.6 and 11.7, of 65536
// 12.6 and 12.8, 128 rows of 65536 15.7 and 17.8.  64 rows of 131072 take 18.0 us
// (64 MB), 18.4 with four tiles a workgroup; 256 rows of them 49.3 and 52.7.  The
// token is picked by ballots: with atomics on LDS the second kernel took 25 us.
#include "gdn_ops_internal.h"
#include "gdn_rows.h"
#include "gdn_scan.h"

namespace gdn {

constexpr int VT = 256;              // threads
constexpr int VPT = 8;               // consecutive entries a thread
constexpr int VSUB = VT * VPT;       // entries per pass of a workgroup
constexpr int VMAXT = 1024;          // tiles a row, at most

// Number of accepted drafts of row b among its first n (every lane of the wave).
template <typename T>
__device__ __forceinline__ int accepted(const VerifyArgs& p, int b, int n) {
  const int lane = threadIdx.x & 63;
  for (int i0 = 0; i0 < n; i0 += 64) {
    const int i = i0 + lane;
    bool ok = true;
    if (i < n) {
      const int x = p.x[(size_t)b * p.K + i];
      ok = false;
      if (x >= 0 && x < p.V) {
        const size_t rp = (size_t)b * (p.K + 1) + i, rq = (size_t)b * p.K + i;
        const double px = (double)Elem<T>::to_f(static_cast<const T*>(p.p)[rp * (size_t)p.p_stride + x]);
        const double qx =
            p.q ? (double)Elem<T>::to_f(static_cast<const T*>(p.q)[rq * (size_t)p.q_stride + x]) : 1.0;
        ok = (double)p.u[rp] * qx < px;   // exact: 24 x 24 bits
      }
    }
    const uint64_t bad = __ballot(!ok);
    if (bad) return i0 + (int)__builtin_ctzll(bad);
  }
  return n;
}

__device__ __forceinline__ int drafts_of(const VerifyArgs& p, int b) {
  const int n = p.n ? p.n[b] : p.K;
  return n > p.K ? p.K : n;
}

// The weights of row b after `a` accepted drafts.
template <typename T>
struct Weights {
  const T* pr;
  const T* qr;       // null: nothing subtracted
  int drop;          // entry of weight 0 (a refused deterministic draft), or -1
  __device__ __forceinline__ Weights(const VerifyArgs& p, int b, int a, bool refused) {
    pr = static_cast<const T*>(p.p) + ((size_t)b * (p.K + 1) + a) * (size_t)p.p_stride;
    qr = refused && p.q ? static_cast<const T*>(p.q) + ((size_t)b * p.K + a) * (size_t)p.q_stride : nullptr;
    drop = refused && !p.q ? p.x[(size_t)b * p.K + a] : -1;
  }
  struct Raw {
    Vec16<T> p[VPT / Vec16<T>::N], q[VPT / Vec16<T>::N];
  };
  // Entries base .. base+VPT-1, all inside the row.
  __device__ __forceinline__ void fetch(int base, Raw& r) const {
    constexpr int N = Vec16<T>::N;
#pragma unroll
    for (int j = 0; j < VPT / N; ++j) __builtin_memcpy(r.p[j].e, pr + base + j * N, 16);
    if (qr)
#pragma unroll
      for (int j = 0; j < VPT / N; ++j) __builtin_memcpy(r.q[j].e, qr + base + j * N, 16);
  }
  __device__ __forceinline__ void weigh(int base, const Raw& r, double* w) const {
    constexpr int N = Vec16<T>::N;
#pragma unroll
    for (int j = 0; j < VPT; ++j) {
      const double x = (double)r.p[j / N].f(j % N);
      const double d = qr ? x - (double)r.q[j / N].f(j % N) : x;
      w[j] = d > 0.0 && d < __builtin_inf() && base + j != drop ? d : 0.0;
    }
  }
  // Weights base .. base+VPT-1 of a row that ends at `end`.
  __device__ __forceinline__ void load(int base, int end, double* w) const {
    constexpr int N = Vec16<T>::N;
    Raw r;
    if (base + VPT <= end) {
      fetch(base, r);
    } else {
#pragma unroll
      for (int j = 0; j < VPT / N; ++j) {
        r.p[j] = load_vec(pr, base + j * N, end);
        if (qr) r.q[j] = load_vec(qr, base + j * N, end);
      }
    }
    weigh(base, r, w);
  }
};

// Inclusive scan over the workgroup's threads and the total.
__device__ __forceinline__ double block_scan(double x, double* lds, double& total) {
  const int wave = threadIdx.x >> 6;
  x = wave_scan64(x);
  __syncthreads();
  if ((threadIdx.x & 63) == 63) lds[wave] = x;
  __syncthreads();
  total = 0.0;
  double before = 0.0;
#pragma unroll
  for (int w = 0; w < VT / 64; ++w) {
    if (w == wave) before = total;
    total += lds[w];
  }
  return before + x;
}

// One candidate of a thread, in index order over the threads: an index (-1:
// none) and the sum before it.
struct Pick {
  int at = -1;
  double before = 0.0;
};

struct PickLds {
  int hit[VT / 64], last[VT / 64];
  double hit_before[VT / 64], last_before[VT / 64];
};

// The first `hit` of the workgroup, else its last `last` (found = false).
__device__ __forceinline__ Pick block_pick(const Pick& hit, const Pick& last, PickLds& lds, bool& found) {
  const int wave = threadIdx.x >> 6;
  const uint64_t h = __ballot(hit.at >= 0), l = __ballot(last.at >= 0);
  const int hs = h ? (int)__builtin_ctzll(h) : 0, ls = l ? 63 - (int)__builtin_clzll(l) : 0;
  const int lane = threadIdx.x & 63;
  __syncthreads();   // the last call's reads are done
  if (lane == hs) {
    lds.hit[wave] = hit.at;
    lds.hit_before[wave] = hit.before;
  }
  if (lane == ls) {
    lds.last[wave] = last.at;
    lds.last_before[wave] = last.before;
  }
  __syncthreads();
  Pick best;
#pragma unroll
  for (int w = 0; w < VT / 64; ++w)
    if (lds.last[w] >= 0) best = {lds.last[w], lds.last_before[w]};
  found = false;
#pragma unroll
  for (int w = VT / 64 - 1; w >= 0; --w)
    if (lds.hit[w] >= 0) {
      best = {lds.hit[w], lds.hit_before[w]};
      found = true;
    }
  return best;
}

template <typename T>
__device__ __forceinline__ double tile_sum(const Weights<T>& wt, const VerifyArgs& p, int tile) {
  const int end = min(p.V, (tile + 1) * p.tile);
  double s = 0.0;
  for (int e = tile * p.tile + (int)threadIdx.x * VPT; e < end; e += VSUB) {
    double w[VPT];
    wt.load(e, p.V, w);
#pragma unroll
    for (int i = 0; i < VPT; ++i) s += w[i];
  }
  return s;
}

template <typename T>
__global__ __launch_bounds__(VT) void verify_sum_kernel(VerifyArgs p) {
  __shared__ double lds[VT / 64];
  const int tile = blockIdx.x, b = blockIdx.y, tid = threadIdx.x;
  const int n = drafts_of(p, b);
  if (n < 0) {
    if (tile == 0 && tid == 0) p.emit[b] = 0;
    return;
  }
  const int a = accepted<T>(p, b, n);
  if (tile == 0 && tid == 0) p.emit[b] = a + 1;
  const double s = wave_scan64(tile_sum(Weights<T>(p, b, a, a < n), p, tile));
  if ((tid & 63) == 63) lds[tid >> 6] = s;
  __syncthreads();
  if (tid == 0) {
    double total = 0.0;
#pragma unroll
    for (int w = 0; w < VT / 64; ++w) total += lds[w];
    p.part[(size_t)b * p.tiles + tile] = total;
  }
}

template <typename T>
__global__ __launch_bounds__(VT) void verify_draw_kernel(VerifyArgs p) {
  __shared__ double lds[VT / 64];
  __shared__ double part[VMAXT];
  __shared__ PickLds picks;
  const int b = blockIdx.x, tid = threadIdx.x;
  const int a = p.emit[b] - 1;
  const size_t tok = (size_t)b * (p.K + 1);
  for (int i = tid; i <= p.K; i += VT)
    if (i != a) p.tokens[tok + i] = i < a ? p.x[(size_t)b * p.K + i] : -1;
  if (a < 0) return;
  const bool refused = a < drafts_of(p, b);
  Weights<T> wt(p, b, a, refused);
  for (int t = tid; t < p.tiles; t += VT) part[t] = p.part[(size_t)b * p.tiles + t];
  __syncthreads();

  // prefix sums of the tiles in order; each thread owns TPT neighbours
  constexpr int TPT = VMAXT / VT;
  double total, upto;
  auto scan_tiles = [&] {
    double s = 0.0;
#pragma unroll
    for (int i = 0; i < TPT; ++i) s += tid * TPT + i < p.tiles ? part[tid * TPT + i] : 0.0;
    upto = block_scan(s, lds, total) - s;
  };
  scan_tiles();
  if (refused && !(total > 0.0)) {   // p <= q everywhere: draw from p itself
    wt.qr = nullptr;
    wt.drop = -1;
    for (int t = 0; t < p.tiles; ++t) {
      double x;
      block_scan(tile_sum(wt, p, t), lds, x);
      if (tid == 0) part[t] = x;
    }
    __syncthreads();
    scan_tiles();
  }
  if (!(total > 0.0)) {
    if (tid == 0) p.tokens[tok + a] = -1;
    return;
  }
  const double u = (double)p.u[tok + p.K];
  const double r = (u > 0.0 ? u : 0.0) * total;
  bool found;
  Pick hit, last;
  double c = upto;
#pragma unroll
  for (int i = 0; i < TPT; ++i) {
    const int t = tid * TPT + i;
    if (t < p.tiles && part[t] > 0.0) {
      last = {t, c};
      if (hit.at < 0 && c + part[t] > r) hit = last;
      c += part[t];
    }
  }
  const Pick tile = block_pick(hit, last, picks, found);   // total > 0: there is one
  double start = tile.before;
  const int end = min(p.V, (tile.at + 1) * p.tile);
  int token = -1;
  for (int e0 = tile.at * p.tile; e0 < end; e0 += VSUB) {
    const int e = e0 + tid * VPT;
    double w[VPT], s = 0.0, sub;
    wt.load(e, end, w);
#pragma unroll
    for (int i = 0; i < VPT; ++i) s += w[i];
    c = start + (block_scan(s, lds, sub) - s);
    hit = last = Pick{};
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      if (w[i] > 0.0) {
        last.at = e + i;
        c += w[i];
        if (hit.at < 0 && c > r) hit.at = e + i;
      }
    }
    const Pick v = block_pick(hit, last, picks, found);
    if (v.at >= 0) token = v.at;
    if (found) break;
    start += sub;
  }
  if (tid == 0) p.tokens[tok + a] = token;
}

constexpr int VROW_WAVES = 16, VROW_PASS = VROW_WAVES * 64 * VPT;   // entries a pass of a row's workgroup

template <typename T>
__global__ __launch_bounds__(64 * VROW_WAVES) void verify_row_kernel(VerifyArgs p) {
  constexpr int MAXT = kVerifyRowMax / (64 * VPT), AHEAD = 4;
  static_assert(MAXT == 128, "two tiles a lane");
  __shared__ double part[MAXT];
  const int b = blockIdx.x, tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const size_t tok = (size_t)b * (p.K + 1);
  const int n = drafts_of(p, b);
  const int a = n < 0 ? -1 : accepted<T>(p, b, n);
  if (tid == 0) p.emit[b] = a + 1;
  for (int i = tid; i <= p.K; i += 64 * VROW_WAVES)
    if (i != a) p.tokens[tok + i] = i < a ? p.x[(size_t)b * p.K + i] : -1;
  if (a < 0) return;
  const bool refused = a < n;
  Weights<T> wt(p, b, a, refused);
  double s0, s1, upto, total;
  // sums of the tiles, their prefix sums (each lane owns two neighbours) and the total
  auto sums = [&] {
    for (int e0 = 0; e0 < p.V; e0 += AHEAD * VROW_PASS) {
      if (e0 + AHEAD * VROW_PASS <= p.V) {
        typename Weights<T>::Raw raw[AHEAD];
#pragma unroll
        for (int i = 0; i < AHEAD; ++i) wt.fetch(e0 + i * VROW_PASS + tid * VPT, raw[i]);
#pragma unroll
        for (int i = 0; i < AHEAD; ++i) {
          const int e = e0 + i * VROW_PASS + tid * VPT;
          double w[VPT], s = 0.0;
          wt.weigh(e, raw[i], w);
#pragma unroll
          for (int j = 0; j < VPT; ++j) s += w[j];
          s = wave_scan64(s);
          if (lane == 63) part[e / (64 * VPT)] = s;
        }
      } else {
        for (int e = e0 + tid * VPT; e - lane * VPT < p.V; e += VROW_PASS) {   // as long as the wave has entries
          double w[VPT], s = 0.0;
          wt.load(e, p.V, w);
#pragma unroll
          for (int j = 0; j < VPT; ++j) s += w[j];
          s = wave_scan64(s);
          if (lane == 63) part[e / (64 * VPT)] = s;
        }
      }
    }
    __syncthreads();
    const int tiles = (p.V + 64 * VPT - 1) / (64 * VPT);
    s0 = 2 * lane < tiles ? part[2 * lane] : 0.0;
    s1 = 2 * lane + 1 < tiles ? part[2 * lane + 1] : 0.0;
    const double upto_all = wave_scan64(s0 + s1);
    upto = upto_all - (s0 + s1);
    total = __shfl(upto_all, 63);
  };
  sums();
  if (refused && !(total > 0.0)) {   // p <= q everywhere: draw from p itself
    wt.qr = nullptr;
    wt.drop = -1;
    __syncthreads();
    sums();
  }
  if (wave != 0) return;
  int token = -1;
  if (total > 0.0) {
    const double u = (double)p.u[tok + p.K];
    const double r = (u > 0.0 ? u : 0.0) * total;
    const bool h0 = s0 > 0.0 && upto + s0 > r, h1 = s1 > 0.0 && upto + s0 + s1 > r;
    const uint64_t hit = __ballot(h0 || h1), some = __ballot(s0 > 0.0 || s1 > 0.0);
    const int src = hit ? (int)__builtin_ctzll(hit) : 63 - (int)__builtin_clzll(some);   // total > 0: some
    const bool second = hit ? !h0 : s1 > 0.0;
    const int e = (2 * src + (int)__shfl((int)second, src)) * 64 * VPT + lane * VPT;
    const double start = __shfl(second ? upto + s0 : upto, src);
    double w[VPT], s = 0.0;
    wt.load(e, p.V, w);
#pragma unroll
    for (int j = 0; j < VPT; ++j) s += w[j];
    double c = start + (wave_scan64(s) - s);
    int first = -1, last = -1;
#pragma unroll
    for (int j = 0; j < VPT; ++j)
      if (w[j] > 0.0) {
        last = e + j;
        c += w[j];
        if (first < 0 && c > r) first = e + j;
      }
    const uint64_t f = __ballot(first >= 0), l = __ballot(last >= 0);
    if (f) token = __shfl(first, (int)__builtin_ctzll(f));
    else if (l) token = __shfl(last, 63 - (int)__builtin_clzll(l));
  }
  if (lane == 0) p.tokens[tok + a] = token;
}

template <typename T>
static hipError_t launch_verify_t(const VerifyArgs& a, hipStream_t s) {
  if (a.V <= kVerifyRowMax) {
    prof_begin(K_VERIFY_ROW, s);
    hipLaunchKernelGGL((verify_row_kernel<T>), dim3(a.B), dim3(64 * VROW_WAVES), 0, s, a);
    prof_end(K_VERIFY_ROW, s);
    return hipGetLastError();
  }
  prof_begin(K_VERIFY_SUM, s);
  hipLaunchKernelGGL((verify_sum_kernel<T>), dim3(a.tiles, a.B), dim3(VT), 0, s, a);
  prof_end(K_VERIFY_SUM, s);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  prof_begin(K_VERIFY_DRAW, s);
  hipLaunchKernelGGL((verify_draw_kernel<T>), dim3(a.B), dim3(VT), 0, s, a);
  prof_end(K_VERIFY_DRAW, s);
  return hipGetLastError();
}

hipError_t launch_verify(DType dt, const VerifyArgs& a, hipStream_t s) {
  switch (dt) {
    case DType::F32: return launch_verify_t<float>(a, s);
    case DType::F16: return launch_verify_t<_Float16>(a, s);
    case DType::BF16: return launch_verify_t<__bf16>(a, s);
  }
  return hipErrorInvalidValue;
}

}  // namespace gdn
