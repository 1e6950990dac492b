// Verification of drafted tokens against the target's probabilities.
//
// Two kernels.  verify_sum: one workgroup per (tile of the vocabulary, row)
// finds how many drafts the row accepts (a gather of at most K pairs), then sums
// the tile's weights w = max(p_a - q_a, 0) (or p_a) in 64 bits.  verify_draw:
// one workgroup per row scans the tiles' sums, finds the tile that holds
// u * sum(w), and scans that tile alone.  Only one row of p and one of q are
// read; the second kernel re-reads one tile from the cache.  Bound by memory for
// a batch, by the latency of two launches for one row.
//
// Sums in 64 bits: a vocabulary of 10^5 entries puts the borders between tokens
// 10^-5 apart, and sums in 32 bits, whose order depends on the split, would
// place one token in a hundred wrongly.
#include "gdn_internal.h"
#include "gdn_rows.h"

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
  __device__ __forceinline__ void load(int base, int V, double* w) const {
    constexpr int N = Vec16<T>::N;
#pragma unroll
    for (int j = 0; j < VPT; j += N) {
      const Vec16<T> pv = load_vec(pr, base + j, V);
      Vec16<T> qv{};
      if (qr) qv = load_vec(qr, base + j, V);
#pragma unroll
      for (int i = 0; i < N; ++i) {
        const double d = qr ? (double)pv.f(i) - (double)qv.f(i) : (double)pv.f(i);
        w[j + i] = d > 0.0 && d < __builtin_inf() && base + j + i != drop ? d : 0.0;
      }
    }
  }
};

__device__ __forceinline__ double wave_scan(double x) {   // inclusive, over the wave's lanes
  const int lane = threadIdx.x & 63;
#pragma unroll
  for (int d = 1; d < 64; d *= 2) {
    const double y = __shfl_up(x, d);
    if (lane >= d) x += y;
  }
  return x;
}

// Inclusive scan over the workgroup's threads and the total.
__device__ __forceinline__ double block_scan(double x, double* lds, double& total) {
  const int wave = threadIdx.x >> 6;
  x = wave_scan(x);
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
  const int tile = blockIdx.x, b = blockIdx.y;
  const int n = drafts_of(p, b);
  if (n < 0) {
    if (tile == 0 && threadIdx.x == 0) p.emit[b] = 0;
    return;
  }
  const int a = accepted<T>(p, b, n);
  if (tile == 0 && threadIdx.x == 0) p.emit[b] = a + 1;
  const Weights<T> wt(p, b, a, a < n);
  double total;
  block_scan(tile_sum(wt, p, tile), lds, total);
  if (threadIdx.x == 0) p.part[(size_t)b * p.tiles + tile] = total;
}

template <typename T>
__global__ __launch_bounds__(VT) void verify_draw_kernel(VerifyArgs p) {
  __shared__ double lds[VT / 64];
  __shared__ double part[VMAXT];
  __shared__ int first, last;
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
  if (tid == 0) {
    first = p.tiles;
    last = -1;
  }
  __syncthreads();
  double start = 0.0;
  {
    double c = upto;
#pragma unroll
    for (int i = 0; i < TPT; ++i) {
      const int t = tid * TPT + i;
      if (t < p.tiles && part[t] > 0.0) {
        if (c + part[t] > r) atomicMin(&first, t);
        atomicMax(&last, t);
        c += part[t];
      }
    }
  }
  __syncthreads();
  const int tile = first < p.tiles ? first : last;
  __syncthreads();
  if (tid == 0) {
    first = p.V;
    last = -1;
  }
  // sum of the tiles before it, in the order of the scan above
  if (tid == tile / TPT) {
    double c = upto;
    for (int t = tid * TPT; t < tile; ++t) c += part[t];
    lds[0] = c;
  }
  __syncthreads();
  start = lds[0];
  __syncthreads();
  const int end = min(p.V, (tile + 1) * p.tile);
  for (int e0 = tile * p.tile; e0 < end; e0 += VSUB) {
    const int e = e0 + tid * VPT;
    double w[VPT], s = 0.0, sub;
    wt.load(e, end, w);
#pragma unroll
    for (int i = 0; i < VPT; ++i) s += w[i];
    double c = start + (block_scan(s, lds, sub) - s);
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      if (w[i] > 0.0) {
        c += w[i];
        if (c > r) atomicMin(&first, e + i);
        atomicMax(&last, e + i);
      }
    }
    start += sub;
  }
  __syncthreads();
  if (tid == 0) p.tokens[tok + a] = first < p.V ? first : last;
}

template <typename T>
static hipError_t launch_verify_t(const VerifyArgs& a, hipStream_t s) {
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
