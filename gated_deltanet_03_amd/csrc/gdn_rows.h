// Row helpers of the verification and norm kernels: 16-byte vectors at any
// element alignment, and sums over aligned groups of lanes.
#pragma once

#include "gdn_device.h"

namespace gdn {

// 16 bytes of T.  Rows of odd widths start anywhere, so the access assumes
// only the element's alignment (global memory takes unaligned 16-byte accesses).
template <typename T>
struct Vec16 {
  static constexpr int N = 16 / (int)sizeof(T);
  T e[N];
  __device__ __forceinline__ float f(int i) const { return Elem<T>::to_f(e[i]); }
};

// Entries base .. base+N-1 of a row of `len`; those past its end are 0.
template <typename T>
__device__ __forceinline__ Vec16<T> load_vec(const T* __restrict__ row, int base, int len) {
  Vec16<T> v;
  if (base + Vec16<T>::N <= len) {
    __builtin_memcpy(v.e, row + base, 16);
  } else {
#pragma unroll
    for (int i = 0; i < Vec16<T>::N; ++i) v.e[i] = base + i < len ? row[base + i] : Elem<T>::from_f(0.f);
  }
  return v;
}

template <typename T>
__device__ __forceinline__ void store_vec(T* __restrict__ row, int base, int len, const float* x) {
  Vec16<T> v;
#pragma unroll
  for (int i = 0; i < Vec16<T>::N; ++i) v.e[i] = Elem<T>::from_f(x[i]);
  if (base + Vec16<T>::N <= len) {
    __builtin_memcpy(row + base, v.e, 16);
  } else {
#pragma unroll
    for (int i = 0; i < Vec16<T>::N; ++i)
      if (base + i < len) row[base + i] = v.e[i];
  }
}

// 16 bytes inside a row that nothing reads again: not kept in the caches.
template <typename T>
__device__ __forceinline__ Vec16<T> load_vec_once(const T* __restrict__ p) {
  typedef uint32_t u32x4 __attribute__((ext_vector_type(4), aligned(2)));
  const u32x4 x = __builtin_nontemporal_load(reinterpret_cast<const u32x4*>(p));
  return __builtin_bit_cast(Vec16<T>, x);
}

// Sum over aligned groups of `lanes` lanes (a power of two up to 64,
// wave-uniform), left in every lane of the group.
__device__ __forceinline__ float group_sum(float x, int lanes) {
  if (lanes > 1) x += __builtin_amdgcn_update_dpp(0.f, x, 0xb1, 0xf, 0xf, false);    // lane ^ 1
  if (lanes > 2) x += __builtin_amdgcn_update_dpp(0.f, x, 0x4e, 0xf, 0xf, false);    // lane ^ 2
  if (lanes > 4) x += __builtin_amdgcn_update_dpp(0.f, x, 0x141, 0xf, 0xf, false);   // the other four of 8
  if (lanes > 8) x += __builtin_amdgcn_update_dpp(0.f, x, 0x140, 0xf, 0xf, false);   // the other eight of 16
  if (lanes > 16) {
    const auto a = __builtin_amdgcn_permlane16_swap(__float_as_uint(x), __float_as_uint(x), false, false);
    x = __uint_as_float(a[0]) + __uint_as_float(a[1]);
  }
  if (lanes > 32) {
    const auto b = __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(x), false, false);
    x = __uint_as_float(b[0]) + __uint_as_float(b[1]);
  }
  return x;
}

}  // namespace gdn
