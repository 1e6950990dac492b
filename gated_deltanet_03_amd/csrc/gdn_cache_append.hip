// New keys (rotated by their positions) and values into their pages, queries rotated beside them.
//
//   a_j = position * inv_freq_j,  (x1, x2) -> (x1 cos a_j - x2 sin a_j, x1 sin a_j + x2 cos a_j)
//
// Bound by memory: every row is read and written once.  A workgroup takes a few tokens: it finds their places, puts
// the cosine and sine of each pair into LDS (once for all heads) and then streams the heads' rows through registers,
// 16 bytes at a time.  14,286 tokens of 20 rows of 256, a quarter rotated, bf16: 61 us (4.8 TB/s; a copy has 5.1); one
// token's 48 rows of 128 3.2 us.
//
// A turn count a / 2 pi of some 10^5 keeps too few bits of its fraction in fp32, so it is taken in fp64 and reduced to
// an eighth of a turn there; the rest is a Taylor series in fp32 of at most pi/4 = 0.785: through x^9 / 9! and
// x^8 / 8! it leaves 0.785^11 / 11! = 2e-9 and 0.785^10 / 10! = 2.5e-8 (2^-25), below an fp32 rounding.
#include <algorithm>

#include "gdn_cache_device.h"
#include "gdn_rows.h"

namespace gdn {

__device__ __forceinline__ float2 cos_sin(int position, float inv_freq) {
  const double turns = (double)position * (double)inv_freq * 0.15915494309189533577;   // 1 / (2 pi)
  const double quarters = 4.0 * (turns - __builtin_rint(turns));                       // in [-2, 2]
  const double whole = __builtin_rint(quarters);
  const float x = (float)((quarters - whole) * 1.5707963267948966192), y = x * x;
  float s = fmaf(y, 2.75573192e-6f, -1.98412698e-4f);
  s = fmaf(y, s, 8.33333333e-3f);
  s = fmaf(y, s, -1.66666667e-1f);
  s = fmaf(x * y, s, x);
  float c = fmaf(y, 2.48015873e-5f, -1.38888889e-3f);
  c = fmaf(y, c, 4.16666667e-2f);
  c = fmaf(y, c, -0.5f);
  c = fmaf(y, c, 1.0f);
  const int k = (int)whole & 3;
  const float a = (k & 1) ? s : c, b = (k & 1) ? c : s;
  return make_float2((k == 1 || k == 2) ? -a : a, (k & 2) ? -b : b);
}

constexpr int kAppendTokens = 4;     // tokens of a workgroup
constexpr int kMaxPairs = 128;       // d / 2 at most

// E: elements of a piece, 16 bytes of them, or 1 where the rotated part does not divide into such pieces.
template <typename T, int E>
__global__ __launch_bounds__(256) void cache_append_kernel(AppendArgs p, int32_t token0) {
  __shared__ float2 trig[kAppendTokens][kMaxPairs];
  __shared__ int64_t place[kAppendTokens];   // the token's row of head 0, -1: on no page
  __shared__ int32_t known[kAppendTokens];   // whether the token belongs to a sequence
  struct Piece { T e[E]; };
  const CacheArgs& c = p.c;
  const int tid = threadIdx.x, half = p.rotary / 2;
  const int t0 = token0 + (int)blockIdx.x * kAppendTokens;
  {
    const int w = tid >> 6, t = t0 + w;     // a wave finds one token's place
    int s = -1;
    if (t < c.total) s = c.cu ? find_sequence(c.cu, c.N, t) : t / c.T;
    int at = 0;
    if (s >= 0) {
      int b, e;
      seq_range(c.cu, c.T, c.total, s, b, e);
      at = c.lens[s] - (e - t);
    }
    if ((tid & 63) == 0) {
      int64_t row = -1;
      if (s >= 0 && at >= 0 && at < c.max_pages * c.page_size) {
        const int page = c.table[(int64_t)s * c.max_pages + at / c.page_size];
        if (page >= 0 && page < c.num_pages)
          row = (int64_t)page * c.Hkv * c.page_size + at % c.page_size;
      }
      place[w] = row;
      known[w] = s >= 0;
    }
    if (s >= 0) {
      for (int j = tid & 63; j < half; j += 64) {
        int pos = at;
        if (p.positions) {
          int axis = p.pair_axis ? p.pair_axis[j] : 0;
          axis = axis < 0 ? 0 : (axis >= p.axes ? p.axes - 1 : axis);
          pos = p.positions[(int64_t)axis * c.total + t];
        }
        trig[w][j] = cos_sin(pos, p.inv_freq[j]);
      }
    }
  }
  __syncthreads();

  // rows of one token: the queries, the keys, the values; items of a row: its pairs of pieces, then single pieces
  const int turned = half / E, kept = (c.d - p.rotary) / E, plain = c.d / E;
  const int heads = (p.q ? c.Hq : 0) + c.Hkv;
  const int rotated = heads * (turned + kept), items = rotated + c.Hkv * plain;
  for (int i = (int)blockIdx.y * 256 + tid; i < items * kAppendTokens; i += 256 * (int)gridDim.y) {
    const int w = i / items, k = i - w * items, t = t0 + w;
    if (!known[w]) continue;
    const T* src;
    T* dst;
    int item;
    if (k < rotated) {
      int h = k / (turned + kept);
      item = k - h * (turned + kept);
      if (p.q && h < c.Hq) {
        src = static_cast<const T*>(p.q) + t * p.q_stride + h * c.d;
        dst = static_cast<T*>(p.q_out) + ((int64_t)t * c.Hq + h) * c.d;
      } else {
        if (p.q) h -= c.Hq;
        if (place[w] < 0) continue;
        src = static_cast<const T*>(p.k) + t * p.k_stride + h * c.d;
        dst = static_cast<T*>(p.k_cache) + (place[w] + (int64_t)h * c.page_size) * c.d;
      }
      if (item < turned) {
        const int j = item * E;
        Piece a, b, x, y;
        if (p.interleaved) {   // pieces 2 item and 2 item + 1 hold pairs j .. j + E - 1
          __builtin_memcpy(&a, src + 2 * j, sizeof(Piece));
          __builtin_memcpy(&b, src + 2 * j + E, sizeof(Piece));
          if constexpr (E == 1) {
            const float2 r = trig[w][j];
            const float u = Elem<T>::to_f(a.e[0]), v = Elem<T>::to_f(b.e[0]);
            x.e[0] = Elem<T>::from_f(u * r.x - v * r.y);
            y.e[0] = Elem<T>::from_f(u * r.y + v * r.x);
          } else {
#pragma unroll
            for (int n = 0; n < E / 2; ++n) {
              const float2 r = trig[w][j + n], r2 = trig[w][j + E / 2 + n];
              float u = Elem<T>::to_f(a.e[2 * n]), v = Elem<T>::to_f(a.e[2 * n + 1]);
              x.e[2 * n] = Elem<T>::from_f(u * r.x - v * r.y);
              x.e[2 * n + 1] = Elem<T>::from_f(u * r.y + v * r.x);
              u = Elem<T>::to_f(b.e[2 * n]), v = Elem<T>::to_f(b.e[2 * n + 1]);
              y.e[2 * n] = Elem<T>::from_f(u * r2.x - v * r2.y);
              y.e[2 * n + 1] = Elem<T>::from_f(u * r2.y + v * r2.x);
            }
          }
          __builtin_memcpy(dst + 2 * j, &x, sizeof(Piece));
          __builtin_memcpy(dst + 2 * j + E, &y, sizeof(Piece));
        } else {
          __builtin_memcpy(&a, src + j, sizeof(Piece));
          __builtin_memcpy(&b, src + half + j, sizeof(Piece));
#pragma unroll
          for (int n = 0; n < E; ++n) {
            const float2 r = trig[w][j + n];
            const float u = Elem<T>::to_f(a.e[n]), v = Elem<T>::to_f(b.e[n]);
            x.e[n] = Elem<T>::from_f(u * r.x - v * r.y);
            y.e[n] = Elem<T>::from_f(u * r.y + v * r.x);
          }
          __builtin_memcpy(dst + j, &x, sizeof(Piece));
          __builtin_memcpy(dst + half + j, &y, sizeof(Piece));
        }
        continue;
      }
      item = p.rotary + (item - turned) * E;
    } else {
      const int h = (k - rotated) / plain;
      if (place[w] < 0) continue;
      item = (k - rotated - h * plain) * E;
      src = static_cast<const T*>(p.v) + t * p.v_stride + h * c.d;
      dst = static_cast<T*>(p.v_cache) + (place[w] + (int64_t)h * c.page_size) * c.d;
    }
    Piece a;
    __builtin_memcpy(&a, src + item, sizeof(Piece));
    __builtin_memcpy(dst + item, &a, sizeof(Piece));
  }
}

template <typename T, int E>
static void launch_append_e(const AppendArgs& a, hipStream_t s) {
  const int64_t wgs = ((int64_t)a.c.total + kAppendTokens - 1) / kAppendTokens;
  // few tokens: their heads are spread over workgroups
  const int64_t rows = (a.q ? a.c.Hq : 0) + 2 * (int64_t)a.c.Hkv;
  const int64_t parts = std::max<int64_t>(1, std::min(512 / wgs, rows * (a.c.d / E) * kAppendTokens / 256));
  const int64_t most = kLaunchThreads / 256 / parts;
  for (int64_t w = 0; w < wgs; w += most)
    hipLaunchKernelGGL((cache_append_kernel<T, E>), dim3((unsigned)std::min(most, wgs - w), (unsigned)parts), dim3(256),
                       0, s, a, (int32_t)(w * kAppendTokens));
}

template <typename T>
static hipError_t launch_append_t(const AppendArgs& a, hipStream_t s) {
  constexpr int E = 16 / (int)sizeof(T);
  prof_begin(K_APPEND, s);
  if (a.rotary % (2 * E) == 0) launch_append_e<T, E>(a, s);
  else launch_append_e<T, 1>(a, s);
  prof_end(K_APPEND, s);
  return hipGetLastError();
}

hipError_t launch_append(DType dt, const AppendArgs& a, hipStream_t s) {
  switch (dt) {
    case DType::F32: return launch_append_t<float>(a, s);
    case DType::F16: return launch_append_t<_Float16>(a, s);
    case DType::BF16: return launch_append_t<__bf16>(a, s);
  }
  return hipErrorInvalidValue;
}

}  // namespace gdn
