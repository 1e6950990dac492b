// Norms before and after a block, fused with its gate, residual and scale.
//
//   n = y * rsqrt(mean_group(y^2) + eps) * w_post,  m = n * act(gate),
//   h = residual + scale * m,  normed = h * rsqrt(mean_D(h^2) + eps) * w_next
//
// Bound by memory: every input is read once and every output written once.  A
// row is held in the registers of WPR waves (NPT 16-byte vectors a lane), all
// its loads issued before the first reduction; the second norm works on the
// registers.  Group sums of up to 32 lanes stay inside a wave; only sums over
// a whole row of several waves go through LDS (one barrier each).
//
// Few vectors a lane, many waves a row: 8192 x 4096 bf16 with everything (335 MB)
// took 175 us with one wave a row, 121 with two, 79 with four, 66 with eight
// (one row each, no looping) on repeated inputs; looping with the row's loads marked
// as read once, and with other inputs each call, 63: 5.3 TB/s, where a 1 GiB copy
// reaches 5.2.
#include <algorithm>

#include "gdn_ops_internal.h"
#include "gdn_rows.h"

namespace gdn {

template <int WPR>
__device__ __forceinline__ float row_sum(float x, float* lds, int wave_in_row) {
  x = group_sum(x, 64);
  if constexpr (WPR > 1) {
    if ((threadIdx.x & 63) == 0) lds[wave_in_row] = x;
    lds_barrier();
    x = 0.f;
#pragma unroll
    for (int w = 0; w < WPR; ++w) x += lds[w];
  }
  return x;
}

// LOOP: the workgroup takes every gridDim.x-th row, issues the next row's loads
// before it works on this one and keeps the weights in registers.
template <typename T, int NPT, int WPR, int RPW, bool LOOP>
__global__ __launch_bounds__(64 * WPR * RPW) void block_norm_kernel(NormArgs p) {
  constexpr int VEC = Vec16<T>::N;
  // [row parity][norm]: a wave still summing one row's parts must not meet the next row's
  __shared__ float red[2][2][WPR];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int wr = wave % WPR, rw = wave / WPR;
  int64_t row = p.row0 + (int64_t)blockIdx.x * RPW + rw;
  if (RPW > 1 && row >= p.T) return;   // RPW > 1 only with WPR = 1: no barrier follows
  const int64_t step = (int64_t)gridDim.x * RPW;
  const int D = p.D;
  const T* wp = static_cast<const T*>(p.wpost);
  const T* wn = static_cast<const T*>(p.wnext);
  const bool gated = p.act != 0, res = p.res != nullptr, post = wp != nullptr, next = wn != nullptr;
  const bool whole = p.group == D;

  struct Row {
    Vec16<T> y[NPT], g[NPT], r[NPT];
  };
  auto load_row = [&](int64_t at, Row& x) {
    const T* y = static_cast<const T*>(p.y) + (size_t)at * D;
    const T* g = static_cast<const T*>(p.gate) + (size_t)at * D;
    const T* r = static_cast<const T*>(p.res) + (size_t)at * D;
#pragma unroll
    for (int j = 0; j < NPT; ++j) {
      const int e = (j * 64 * WPR + wr * 64 + lane) * VEC;
      if (LOOP && e + VEC <= D) {
        x.y[j] = load_vec_once(y + e);
        if (gated) x.g[j] = load_vec_once(g + e);
        if (res) x.r[j] = load_vec_once(r + e);
      } else {
        x.y[j] = load_vec(y, e, D);
        if (gated) x.g[j] = load_vec(g, e, D);
        if (res) x.r[j] = load_vec(r, e, D);
      }
    }
  };
  auto store_row = [&](void* base, int e, const float* x) {
    T* r = static_cast<T*>(base) + (size_t)row * D;
    if (e < D) store_vec(r, e, D, x);
  };

  Row cur;
  load_row(row, cur);
  Vec16<T> wv[NPT], nv[NPT];
#pragma unroll
  for (int j = 0; j < NPT; ++j) {
    const int e = (j * 64 * WPR + wr * 64 + lane) * VEC;
    if (post) wv[j] = whole ? load_vec(wp, e, D) : load_vec(wp, e % p.group, p.group);
    if (next) nv[j] = load_vec(wn, e, D);
  }
  for (int parity = 0;; parity ^= 1) {
    Row ahead;
    const bool more = LOOP && row + step < p.T;
    if (more) load_row(row + step, ahead);
    float h[NPT][VEC], rs[NPT];
    if (post) {
      float sq[NPT], all = 0.f;
#pragma unroll
      for (int j = 0; j < NPT; ++j) {
        sq[j] = 0.f;
#pragma unroll
        for (int i = 0; i < VEC; ++i) sq[j] = fmaf(cur.y[j].f(i), cur.y[j].f(i), sq[j]);
        all += sq[j];
      }
      if (whole) {
        const float r = rsqrtf(row_sum<WPR>(all, red[parity][0], wr) / (float)D + p.eps);
#pragma unroll
        for (int j = 0; j < NPT; ++j) rs[j] = r;
      } else {
#pragma unroll
        for (int j = 0; j < NPT; ++j)
          rs[j] = rsqrtf(group_sum(sq[j], p.group / VEC) / (float)p.group + p.eps);
      }
    }
    float ss = 0.f;
#pragma unroll
    for (int j = 0; j < NPT; ++j) {
      const int e = (j * 64 * WPR + wr * 64 + lane) * VEC;
#pragma unroll
      for (int i = 0; i < VEC; ++i) {
        float x = cur.y[j].f(i);
        if (post) x *= rs[j] * wv[j].f(i);
        if (gated) {
          const float z = cur.g[j].f(i);
          const float s = 1.f / (1.f + __expf(-z));
          x *= p.act == 1 ? z * s : s;
        }
        x *= p.scale;
        if (res) x += cur.r[j].f(i);
        h[j][i] = x;
        ss = fmaf(x, x, ss);
      }
      store_row(p.h, e, h[j]);
    }
    if (next) {
      const float r = rsqrtf(row_sum<WPR>(ss, red[parity][1], wr) / (float)D + p.eps);
#pragma unroll
      for (int j = 0; j < NPT; ++j) {
        float x[VEC];
#pragma unroll
        for (int i = 0; i < VEC; ++i) x[i] = h[j][i] * r * nv[j].f(i);
        store_row(p.normed, (j * 64 * WPR + wr * 64 + lane) * VEC, x);
      }
    }
    if (!more) return;
    cur = ahead;
    row += step;
  }
}

// Workgroups of a call that loops over its rows: 16 for each CU.
constexpr int64_t kNormWg = 4096;

template <typename T, int NPT, int WPR>
static void launch_norm_w(const NormArgs& a, hipStream_t s) {
  constexpr int RPW = WPR == 1 ? 4 : 1;
  const int64_t wgs = (a.T + RPW - 1) / RPW;
  const dim3 block(64 * WPR * RPW);
  if constexpr (NPT == 1) {   // two rows of more vectors do not fit the registers of 16 waves
    if (wgs > kNormWg) {
      hipLaunchKernelGGL((block_norm_kernel<T, NPT, WPR, RPW, true>), dim3((unsigned)kNormWg), block, 0, s, a);
      return;
    }
  }
  const int64_t most = kLaunchThreads / block.x;
  for (int64_t w = 0; w < wgs; w += most) {
    NormArgs b = a;
    b.row0 = w * RPW;
    hipLaunchKernelGGL((block_norm_kernel<T, NPT, WPR, RPW, false>), dim3((unsigned)std::min(most, wgs - w)), block, 0,
                       s, b);
  }
}

// Waves and vectors a lane for a row of nv vectors.
template <typename T>
static hipError_t launch_norm_t(const NormArgs& a, hipStream_t s) {
  const int nv = (a.D + Vec16<T>::N - 1) / Vec16<T>::N;
  prof_begin(K_NORM, s);
  if (nv <= 64) launch_norm_w<T, 1, 1>(a, s);
  else if (nv <= 128) launch_norm_w<T, 1, 2>(a, s);
  else if (nv <= 256) launch_norm_w<T, 1, 4>(a, s);
  else if (nv <= 512) launch_norm_w<T, 1, 8>(a, s);
  else if (nv <= 1024) launch_norm_w<T, 1, 16>(a, s);
  else if (nv <= 2048) launch_norm_w<T, 2, 16>(a, s);
  else if constexpr (sizeof(T) == 4) launch_norm_w<T, 4, 16>(a, s);   // D <= 16384
  prof_end(K_NORM, s);
  return hipGetLastError();
}

hipError_t launch_norm(DType dt, const NormArgs& a, hipStream_t s) {
  switch (dt) {
    case DType::F32: return launch_norm_t<float>(a, s);
    case DType::F16: return launch_norm_t<_Float16>(a, s);
    case DType::BF16: return launch_norm_t<__bf16>(a, s);
  }
  return hipErrorInvalidValue;
}

}  // namespace gdn
