// Token-by-token linear attention with a decay for each head, with capture of
// the (decay, key, value) records.
//
//   S <- alpha S + k v^T,  o = scale S^T q   (S after the update)
//
// Bound by memory: the fp32 state is read and written once a call, whatever the
// number of tokens.  A workgroup owns [dk x CW] of one (row, head) state, CW = 32
// columns where dv allows (whole 128-byte lines); its waves own 32 rows each,
// a lane RPL adjacent rows of 4 columns.  There is no reduction before the
// update (unlike the delta rule), so a token's only coupling is the sum over dk
// of o: over the lanes of a column on the VALU, over the waves through LDS
// once per TB tokens.
//
// Measured at 32 heads of d = 128, bf16: 64 rows of one token 40.5 us (270 MB at
// 6.6 TB/s back to back, part of it from the last-level cache; 49 us, 5.5 TB/s, with
// other inputs each time), one row 3.9 us (5.2), 8 rows of 1 to 7 tokens with records
// 9.4 us (11.4): there each token's loads wait inside of the token loop.
#include <algorithm>

#include "gdn_device.h"
#include "gdn_ops_internal.h"

namespace gdn {

constexpr int TB = 8;   // tokens between two sums over the waves

template <int CPL>
__device__ __forceinline__ float sum_column(float x) {   // over the lanes sharing lane % CPL
  if constexpr (CPL <= 4) x += __builtin_amdgcn_update_dpp(0.f, x, 0x124, 0xf, 0xf, false);   // row_ror:4
  x += __builtin_amdgcn_update_dpp(0.f, x, 0x128, 0xf, 0xf, false);                           // row_ror:8
  const auto a = __builtin_amdgcn_permlane16_swap(__float_as_uint(x), __float_as_uint(x), false, false);
  x = __uint_as_float(a[0]) + __uint_as_float(a[1]);
  const auto b = __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(x), false, false);
  return __uint_as_float(b[0]) + __uint_as_float(b[1]);
}

template <typename T, int DK, int CW>
__global__ __launch_bounds__(64 * (DK >= 32 ? DK / 32 : 1)) void linear_step_kernel(LinearArgs p) {
  constexpr int NW = DK >= 32 ? DK / 32 : 1;        // waves
  constexpr int CPL = CW / 4, RG = 64 / CPL;        // lanes across the columns, down the rows
  constexpr int RPL = DK / NW / RG;                 // rows a lane
  static_assert(RPL >= 1, "more lanes than rows");
  __shared__ __align__(16) float part[TB][NW][CW];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int cg = lane % CPL, rg = lane / CPL;
  const int nsl = p.dv / CW;
  const int slice = (int)(blockIdx.x % nsl), pair = p.first + (int)(blockIdx.x / nsl);
  const int b = pair / p.Hv, h = pair % p.Hv, G = p.Hv / p.Hq, hk = h / G;
  const int col = slice * CW + cg * 4, row0 = wave * (DK / NW) + rg * RPL;
  const size_t sidx = (size_t)row0 * p.dv + col;

  f32x4 S[RPL];
  if (p.s0 != nullptr) {
    const float* s0 = p.s0 + (int64_t)b * p.s0_stride + (size_t)h * DK * p.dv + sidx;
#pragma unroll
    for (int r = 0; r < RPL; ++r) S[r] = *reinterpret_cast<const f32x4*>(s0 + (size_t)r * p.dv);
  } else {
#pragma unroll
    for (int r = 0; r < RPL; ++r) S[r] = f32x4{0.f, 0.f, 0.f, 0.f};
  }
  int t0, t1;
  seq_range(p.cu, p.T, p.total, b, t0, t1);
  int ncap = 0;
  if (p.cap > 0) {
    const int lim = min(p.cap, t1 - t0), c = p.counts[b];
    ncap = c < 0 ? 0 : min(c, lim);
  }
  const T* qp = static_cast<const T*>(p.q);
  const T* kp = static_cast<const T*>(p.k);
  const T* vp = static_cast<const T*>(p.v);
  T* op = static_cast<T*>(p.o);
  const size_t R = (size_t)p.Hv + (size_t)p.Hq * DK + (size_t)p.Hv * p.dv;

  for (int tb = t0; tb < t1; tb += TB) {
    const int nt = min(TB, t1 - tb);
    for (int u = 0; u < nt; ++u) {
      const size_t t = (size_t)(tb + u);
      float kr[RPL], qr[RPL], vr[4];
      load_row_f32<T, RPL>(kp + (t * p.Hq + hk) * DK + row0, kr);
      load_row_f32<T, RPL>(qp + (t * p.Hq + hk) * DK + row0, qr);
      load_row_f32<T, 4>(vp + (t * p.Hv + h) * p.dv + col, vr);
      const float a = expf(p.g[t * (size_t)p.g_stride + h]);
      f32x4 o = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int r = 0; r < RPL; ++r)
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          S[r][c] = fmaf(kr[r], vr[c], a * S[r][c]);   // the replay's order
          o[c] = fmaf(S[r][c], qr[r], o[c]);
        }
#pragma unroll
      for (int c = 0; c < 4; ++c) o[c] = sum_column<CPL>(o[c]);
      if (rg == 0) *reinterpret_cast<f32x4*>(&part[u][wave][cg * 4]) = o;
      const int c = tb + u - t0;
      if (c < ncap) {
        float* rec = p.su + ((size_t)b * p.cap + c) * R;
        if (slice == 0 && threadIdx.x == 0) rec[h] = a;
        if (slice == 0 && cg == 0 && h % G == 0) {
#pragma unroll
          for (int r = 0; r < RPL; ++r) rec[p.Hv + (size_t)hk * DK + row0 + r] = kr[r];
        }
        if (wave == 0 && rg == 0) {
#pragma unroll
          for (int j = 0; j < 4; ++j) rec[p.Hv + (size_t)p.Hq * DK + (size_t)h * p.dv + col + j] = vr[j];
        }
      }
    }
    lds_barrier();
    for (int i = threadIdx.x; i < nt * CW; i += 64 * NW) {
      const int u = i / CW, c = i % CW;
      float o = 0.f;
#pragma unroll
      for (int w = 0; w < NW; ++w) o += part[u][w][c];
      op[((size_t)(tb + u) * p.Hv + h) * p.dv + slice * CW + c] = Elem<T>::from_f(p.scale * o);
    }
    lds_barrier();
  }
  if (p.s_out != nullptr) {
    float* so = p.s_out + ((size_t)b * p.Hv + h) * DK * p.dv + sidx;
#pragma unroll
    for (int r = 0; r < RPL; ++r)
      __builtin_nontemporal_store(S[r], reinterpret_cast<f32x4*>(so + (size_t)r * p.dv));
  }
}

template <typename T, int DK, int CW>
static void launch_step_w(const LinearArgs& a, hipStream_t s) {
  constexpr int NW = DK >= 32 ? DK / 32 : 1;
  const int64_t pairs = (int64_t)a.B * a.Hv, nsl = a.dv / CW, most = kLaunchThreads / (64 * NW) / nsl;
  for (int64_t first = 0; first < pairs; first += most) {
    LinearArgs b = a;
    b.first = (int32_t)first;
    hipLaunchKernelGGL((linear_step_kernel<T, DK, CW>), dim3((unsigned)(std::min(most, pairs - first) * nsl)),
                       dim3(64 * NW), 0, s, b);
  }
}

template <typename T, int DK>
static void launch_step_dk(const LinearArgs& a, hipStream_t s) {
  if (a.dv % 32 == 0) launch_step_w<T, DK, 32>(a, s);
  else launch_step_w<T, DK, 16>(a, s);
}

template <typename T>
static hipError_t launch_step_t(const LinearArgs& a, hipStream_t s) {
  prof_begin(K_LIN_STEP, s);
  switch (a.dk) {
    case 16: launch_step_dk<T, 16>(a, s); break;
    case 32: launch_step_dk<T, 32>(a, s); break;
    case 64: launch_step_dk<T, 64>(a, s); break;
    default: launch_step_dk<T, 128>(a, s); break;
  }
  prof_end(K_LIN_STEP, s);
  return hipGetLastError();
}

hipError_t launch_linear_step(DType dt, const LinearArgs& a, hipStream_t s) {
  switch (dt) {
    case DType::F32: return launch_step_t<float>(a, s);
    case DType::F16: return launch_step_t<_Float16>(a, s);
    case DType::BF16: return launch_step_t<__bf16>(a, s);
  }
  return hipErrorInvalidValue;
}

}  // namespace gdn
