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
#include "gdn_internal.h"
#include "gdn_rows.h"

namespace gdn {

template <int WPR>
__device__ __forceinline__ float row_sum(float x, float* lds, int wave_in_row, int row_in_wg) {
  x = group_sum(x, 64);
  if constexpr (WPR > 1) {
    if ((threadIdx.x & 63) == 0) lds[row_in_wg * WPR + wave_in_row] = x;
    __syncthreads();
    x = 0.f;
#pragma unroll
    for (int w = 0; w < WPR; ++w) x += lds[row_in_wg * WPR + w];
  }
  return x;
}

template <typename T, int NPT, int WPR, int RPW>
__global__ __launch_bounds__(64 * WPR * RPW) void block_norm_kernel(NormArgs p) {
  constexpr int VEC = Vec16<T>::N;
  __shared__ float red[2][WPR * RPW];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int wr = wave % WPR, rw = wave / WPR;
  const int64_t row = (int64_t)blockIdx.x * RPW + rw;
  if (RPW > 1 && row >= p.T) return;   // RPW > 1 only with WPR = 1: no barrier follows
  const int D = p.D;
  const size_t off = (size_t)row * D;
  const T* yr = static_cast<const T*>(p.y) + off;
  const T* gr = static_cast<const T*>(p.gate) + off;
  const T* rr = static_cast<const T*>(p.res) + off;
  const T* wp = static_cast<const T*>(p.wpost);
  const T* wn = static_cast<const T*>(p.wnext);
  const bool gated = p.act != 0, res = p.res != nullptr, post = wp != nullptr, next = wn != nullptr;
  const bool whole = p.group == D;

  Vec16<T> yv[NPT], gv[NPT], rv[NPT], wv[NPT];
#pragma unroll
  for (int j = 0; j < NPT; ++j) {
    const int e = (j * 64 * WPR + wr * 64 + lane) * VEC;
    yv[j] = load_vec(yr, e, D);
    if (gated) gv[j] = load_vec(gr, e, D);
    if (res) rv[j] = load_vec(rr, e, D);
    if (post) wv[j] = whole ? load_vec(wp, e, D) : load_vec(wp, e % p.group, p.group);
  }
  float h[NPT][VEC], rs[NPT];
  if (post) {
    float sq[NPT], all = 0.f;
#pragma unroll
    for (int j = 0; j < NPT; ++j) {
      sq[j] = 0.f;
#pragma unroll
      for (int i = 0; i < VEC; ++i) sq[j] = fmaf(yv[j].f(i), yv[j].f(i), sq[j]);
      all += sq[j];
    }
    if (whole) {
      const float r = rsqrtf(row_sum<WPR>(all, red[0], wr, rw) / (float)D + p.eps);
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
      float x = yv[j].f(i);
      if (post) x *= rs[j] * wv[j].f(i);
      if (gated) {
        const float z = gv[j].f(i);
        const float s = 1.f / (1.f + __expf(-z));
        x *= p.act == 1 ? z * s : s;
      }
      x *= p.scale;
      if (res) x += rv[j].f(i);
      h[j][i] = x;
      ss = fmaf(x, x, ss);
    }
    if (e < D) store_vec(static_cast<T*>(p.h) + off, e, D, h[j]);
  }
  if (!next) return;
  const float r = rsqrtf(row_sum<WPR>(ss, red[1], wr, rw) / (float)D + p.eps);
#pragma unroll
  for (int j = 0; j < NPT; ++j) {
    const int e = (j * 64 * WPR + wr * 64 + lane) * VEC;
    if (e >= D) continue;
    const Vec16<T> w = load_vec(wn, e, D);
    float x[VEC];
#pragma unroll
    for (int i = 0; i < VEC; ++i) x[i] = h[j][i] * r * w.f(i);
    store_vec(static_cast<T*>(p.normed) + off, e, D, x);
  }
}

template <typename T, int NPT, int WPR>
static void launch_norm_w(const NormArgs& a, hipStream_t s) {
  constexpr int RPW = WPR == 1 ? 4 : 1;
  hipLaunchKernelGGL((block_norm_kernel<T, NPT, WPR, RPW>), dim3((unsigned)((a.T + RPW - 1) / RPW)),
                     dim3(64 * WPR * RPW), 0, s, a);
}

// Waves and vectors a lane for a row of nv vectors.
template <typename T>
static hipError_t launch_norm_t(const NormArgs& a, hipStream_t s) {
  const int nv = (a.D + Vec16<T>::N - 1) / Vec16<T>::N;
  prof_begin(K_NORM, s);
  if (nv <= 64) launch_norm_w<T, 1, 1>(a, s);
  else if (nv <= 128) launch_norm_w<T, 2, 1>(a, s);
  else if (nv <= 256) launch_norm_w<T, 1, 4>(a, s);
  else if (nv <= 512) launch_norm_w<T, 2, 4>(a, s);
  else if (nv <= 1024) launch_norm_w<T, 1, 16>(a, s);
  else if (nv <= 2048) launch_norm_w<T, 2, 16>(a, s);
  else launch_norm_w<T, 4, 16>(a, s);
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
