// Attention of new tokens over a paged cache, causal, with shared key heads.
//
//   o_i = sum_j exp(scale q_i . k_j) v_j / sum_j exp(scale q_i . k_j),   p_i - window < j <= p_i
//
// One pass over the keys with a running maximum m and sum l; a row is one (token, query head) pair, and the rows of one
// key head lie together (row = token * G + head in the group), so that a tile of rows shares every key it reads.
//
// Both products run transposed on 32x32 matrix instructions: scores S^T = K Q^T (lane: query l % 32, its keys
// 8 (i / 4) + 4 (l / 32) + i % 4 in 16 accumulators) and O^T += V^T P^T.  A lane so holds all its keys' scores of one
// query: maximum and sum are taken in the lane and over one exchange with lane ^ 32, the factors of the running
// maximum are one number a lane, and the weights are already the second product's operand: its contraction index is
// permuted to the order in which the accumulators hold the keys, and V's operand is read in the same order (transposed
// LDS reads for 16-bit types).
//
// Keys and values come from global memory to LDS without passing registers (16 bytes a lane).  What is absent (keys
// past the sequence's or the tile's end or before its window, numbers that are no page) is loaded from a block of zeros.
//
// m follows the maximum only when that has grown by more than 2^8: exp(s - m) is then at most 2^8, which 16-bit
// operands hold, and most tiles leave the output accumulators alone.
#pragma once

#include <algorithm>

#include "gdn_cache_device.h"
#include "gdn_rows.h"

namespace gdn {
namespace attend {

typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef short s16x4 __attribute__((ext_vector_type(4)));

static __device__ uint4 zeros16[1];

// One wave instruction: every lane copies 16 bytes from base + voff, or from its own address, to lds + 16 * lane.
// Written out because the compiler would wait for all loads in flight before any LDS read after the builtin.
__device__ __forceinline__ void dma16(uint32_t voff, const void* base, uint32_t lds) {
  asm volatile("s_mov_b32 m0, %2\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %0, %1" ::"v"(voff), "s"(base), "s"(lds)
               : "memory");
}
__device__ __forceinline__ void dma16(const void* src, uint32_t lds) {
  asm volatile("s_mov_b32 m0, %1\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %0, off" ::"v"(src), "s"(lds) : "memory");
}
template <int N>
__device__ __forceinline__ void wait_loads() {   // all but the last N
  asm volatile("s_waitcnt vmcnt(%0)" ::"n"(N) : "memory");
}

__device__ __forceinline__ s16x4 read_tr16(const unsigned char* p) {
  return __builtin_amdgcn_ds_read_tr16_b64_v4i16((__attribute__((address_space(3))) s16x4*)p);
}

__device__ __forceinline__ float other_half_max(float x) {
  const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(x), false, false);
  return fmaxf(__uint_as_float(r[0]), __uint_as_float(r[1]));
}
__device__ __forceinline__ float other_half_sum(float x) {
  const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(x), false, false);
  return __uint_as_float(r[0]) + __uint_as_float(r[1]);
}

// 16-byte pieces of an LDS row are stored at piece ^ f(row).
// Keys: 16-byte reads of one piece in 32 rows; 8 rows on each other's heels meet distinct eighths of 128 bytes, 16 rows
// distinct sixteenths of 256.
template <int PPR>
__device__ __forceinline__ int key_swizzle(int r) {
  if constexpr (PPR >= 16) return r & 15;
  else if constexpr (PPR == 8) return ((r >> 1) & 3) | (((r ^ (r >> 3)) & 1) << 2);
  else return (r >> 1) & 3;
}
// Values, 16-bit: transposed reads of 4 rows x 32 bytes by 16 lanes, x 64 bytes by 32.
// Values, fp32: 4-byte reads of 128 bytes of rows r and r + 4.
template <int ES, int PPR>
__device__ __forceinline__ int value_swizzle(int r) {
  if constexpr (ES == 4) return PPR >= 16 ? ((r >> 2) & 1) << 3 : 0;
  else if constexpr (PPR >= 16) return (0xca60 >> ((r & 3) << 2)) & 15;   // 0, 6, 10, 12
  else if constexpr (PPR == 8) return (r & 3) << 1;
  else return ((r >> 1) & 1) << 1;
}

// Which tile, slice of keys and sequence a workgroup has.
struct Unit {
  int s, tile, slice, slices;
  int b, L, lens;        // first token, new tokens, keys of the sequence
};

// Tiles and keys of sequence s (0 tiles: nothing to do).
template <int ROWS>
__device__ __forceinline__ void sequence_size(const AttendArgs& a, int G, int s, int& b, int& L, int& lens, int& tiles,
                                              int& span) {
  b = L = lens = tiles = span = 0;
  if (s < a.c.N) {
    int e;
    seq_range(a.c.cu, a.c.T, a.c.total, s, b, e);
    L = e - b;
    lens = min(max(a.c.lens[s], -(1 << 30)), 1 << 30);
    tiles = (int)(((int64_t)L * G + ROWS - 1) / ROWS);
    const int room = a.c.max_pages * a.c.page_size;
    span = lens < 0 ? 0 : (lens < room ? lens : room);
    if (a.window > 0) {   // one tile sees no more than this
      const int64_t most = (int64_t)a.window + ROWS / G + 1;
      if (span > most) span = (int)most;
    }
  }
}

// Keys of a slice: the work of all tiles over the slices aimed at, at least kSliceKeys.
template <int ROWS>
__device__ __forceinline__ int slice_keys(const AttendArgs& a, int G) {
  const int lane = threadIdx.x & 63;
  int64_t all = 0;
  for (int s = lane; s < a.c.N; s += 64) {
    int b, L, lens, tiles, span;
    sequence_size<ROWS>(a, G, s, b, L, lens, tiles, span);
    all += (int64_t)tiles * span;
  }
#pragma unroll
  for (int m = 1; m < 64; m <<= 1) all += __shfl_xor(all, m);
  const int64_t k = (all + a.slices - 1) / a.slices;
  return (int)(k < kSliceKeys ? kSliceKeys : (k + 127) / 128 * 128);
}

// The u-th (sequence, tile, slice) of a head; false past the last one.  The whole wave calls it.
template <int ROWS>
__device__ __forceinline__ bool find_unit(const AttendArgs& a, int G, int u, Unit& r) {
  const int lane = threadIdx.x & 63;
  const int keys = a.slices ? slice_keys<ROWS>(a, G) : 0x7fffff00;
  int before = 0;
  for (int s0 = 0; s0 < a.c.N; s0 += 64) {
    int b, L, lens, tiles, span;
    sequence_size<ROWS>(a, G, s0 + lane, b, L, lens, tiles, span);
    const int slices = span > keys ? (span + keys - 1) / keys : 1, mine = tiles * slices;
    int upto = mine;
#pragma unroll
    for (int m = 1; m < 64; m <<= 1) {
      const int o = __shfl_up(upto, m);
      if (lane >= m) upto += o;
    }
    const int total = __builtin_amdgcn_readlane(upto, 63);
    if (u < before + total) {
      const int j = __ffsll((unsigned long long)__ballot(u < before + upto)) - 1;
      const int rest = u - before - (__builtin_amdgcn_readlane(upto, j) - __builtin_amdgcn_readlane(mine, j));
      r.s = s0 + j;
      r.b = __builtin_amdgcn_readlane(b, j);
      r.L = __builtin_amdgcn_readlane(L, j);
      r.lens = __builtin_amdgcn_readlane(lens, j);
      r.slices = __builtin_amdgcn_readlane(slices, j);
      // a sequence's last tiles see the most keys: first
      r.tile = __builtin_amdgcn_readlane(tiles, j) - 1 - rest / r.slices;
      r.slice = rest % r.slices;
      return true;
    }
    before += total;
  }
  return false;
}

template <typename T> struct Op;
template <> struct Op<__bf16> {
  using V = bf16x8;
  static __device__ __forceinline__ f32x16 mma(const V& a, const V& b, const f32x16& c) {
    return __builtin_amdgcn_mfma_f32_32x32x16_bf16(a, b, c, 0, 0, 0);
  }
};
template <> struct Op<_Float16> {
  using V = f16x8;
  static __device__ __forceinline__ f32x16 mma(const V& a, const V& b, const f32x16& c) {
    return __builtin_amdgcn_mfma_f32_32x32x16_f16(a, b, c, 0, 0, 0);
  }
};

// One wave's 32 queries: their operands, output accumulators, maximum and sum.
template <typename T, int D>
struct Wave {
  static constexpr int ES = (int)sizeof(T), PPR = D * ES / 16, RB = D * ES, E = 16 / ES;
  static constexpr bool F32 = ES == 4;
  static constexpr int QN = D / (2 * E);            // 16-byte pieces of a query a lane holds
  static constexpr int DT = D / 32;
  uint4 q[QN];
  f32x16 o[DT];
  float m, mc, l;      // m in score units, mc = m * scale (0 while m = -infinity), l of this lane's keys
  int lo, hi;          // the keys this lane's query sees: lo <= key <= hi

  __device__ __forceinline__ void init() {
#pragma unroll
    for (int t = 0; t < DT; ++t)
#pragma unroll
      for (int i = 0; i < 16; ++i) o[t][i] = 0.f;
    m = -INFINITY;
    mc = l = 0.f;
  }

  // Query row `src` (all lanes of a pair read theirs); pieces 2 s + l / 32.
  __device__ __forceinline__ void load_query(const T* src) {
    const int h = (threadIdx.x >> 5) & 1;
#pragma unroll
    for (int s = 0; s < QN; ++s) q[s] = *reinterpret_cast<const uint4*>(src + (2 * s + h) * E);
  }

  // Scores of 32 keys, rows r0 .. r0 + 31 of the LDS tile.
  __device__ __forceinline__ f32x16 scores(const unsigned char* K, int r0) const {
    const int lane = threadIdx.x & 63, h = lane >> 5, r = lane & 31;
    const int f = key_swizzle<PPR>(r);
    f32x16 s;
#pragma unroll
    for (int i = 0; i < 16; ++i) s[i] = 0.f;
#pragma unroll
    for (int t = 0; t < QN; ++t) {
      const uint4 k = *reinterpret_cast<const uint4*>(K + (r0 + r) * RB + (((2 * t + h) ^ f) << 4));
      if constexpr (F32) {
        const f32x4 a = __builtin_bit_cast(f32x4, k), b = __builtin_bit_cast(f32x4, q[t]);
#pragma unroll
        for (int e = 0; e < 4; ++e) s = __builtin_amdgcn_mfma_f32_32x32x2f32(a[e], b[e], s, 0, 0, 0);
      } else {
        s = Op<T>::mma(__builtin_bit_cast(typename Op<T>::V, k), __builtin_bit_cast(typename Op<T>::V, q[t]), s);
      }
    }
    return s;
  }

  // -infinity where the query does not see the key; key0: key of row 0, gone: bit g set where 16 rows have no page.
  static __device__ __forceinline__ int key_of(int i) {
    return 8 * (i >> 2) + (i & 3) + 4 * (((int)threadIdx.x >> 5) & 1);
  }
  __device__ __forceinline__ void mask(f32x16& s, int key0, int gone) const {
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      const int k = key0 + key_of(i);
      if (k < lo || k > hi || ((gone >> (i >> 3)) & 1)) s[i] = -INFINITY;
    }
  }

  // The running maximum takes `top` (of this lane's keys) in.
  __device__ __forceinline__ void raise(float top, float c, float slack) {
    top = other_half_max(top);
    if (__ballot(top > m + slack || (m == -INFINITY && top > m)) == 0) return;
    const float n = fmaxf(m, top);
    const float f = n == -INFINITY ? 1.f : __builtin_amdgcn_exp2f((m - n) * c);
    m = n;
    mc = n == -INFINITY ? 0.f : n * c;
    l *= f;
#pragma unroll
    for (int t = 0; t < DT; ++t)
#pragma unroll
      for (int i = 0; i < 16; ++i) o[t][i] *= f;
  }

  // Scores to weights.
  __device__ __forceinline__ void weigh(f32x16& s, float c) {
    float part = 0.f;
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      s[i] = __builtin_amdgcn_exp2f(fmaf(s[i], c, -mc));
      part += s[i];
    }
    l += part;
  }

  // V's operand for 16 keys (rows r0 .. r0 + 15) and 32 columns, in the weights' order.
  static __device__ __forceinline__ uint4 value_operand(const unsigned char* V, int r0, int t) {
    const int lane = threadIdx.x & 63, h = lane >> 5, g = (lane >> 4) & 1;
    const int r = 4 * h + ((lane & 15) >> 2);
    const int piece = (4 * t + 2 * g + ((lane & 3) >> 1)) ^ value_swizzle<ES, PPR>(r);
    const unsigned char* at = V + (r0 + r) * RB + (piece << 4) + ((lane & 1) << 3);
    const uint2 a = __builtin_bit_cast(uint2, read_tr16(at)), b = __builtin_bit_cast(uint2, read_tr16(at + 8 * RB));
    return make_uint4(a.x, a.y, b.x, b.y);
  }
  // One fp32 value: column 32 t + l % 32 of the lane's i-th key.
  static __device__ __forceinline__ float value_at(const unsigned char* V, int r0, int t, int i) {
    const int lane = threadIdx.x & 63;
    const int r = r0 + key_of(i), col = 32 * t + (lane & 31);
    return *reinterpret_cast<const float*>(V + r * RB + (((col >> 2) ^ value_swizzle<ES, PPR>(r)) << 4) +
                                           ((col & 3) << 2));
  }

  // Two weights of the lane's keys 8 s .. 8 s + 7, rounded to T.
  static __device__ __forceinline__ uint4 weight_operand(const f32x16& p, int s) {
    union { T e[8]; uint4 u; } w;
#pragma unroll
    for (int j = 0; j < 8; ++j) w.e[j] = Elem<T>::from_f(p[8 * s + j]);
    return w.u;
  }

  // o += V^T P^T over 32 keys.
  __device__ __forceinline__ void add_values(const unsigned char* V, int r0, const f32x16& p) {
    if constexpr (F32) {
#pragma unroll
      for (int t = 0; t < DT; ++t)
#pragma unroll
        for (int i = 0; i < 16; ++i)
          o[t] = __builtin_amdgcn_mfma_f32_32x32x2f32(value_at(V, r0, t, i), p[i], o[t], 0, 0, 0);
    } else {
#pragma unroll
      for (int s = 0; s < 2; ++s) {
        const auto w = __builtin_bit_cast(typename Op<T>::V, weight_operand(p, s));
#pragma unroll
        for (int t = 0; t < DT; ++t)
          o[t] = Op<T>::mma(__builtin_bit_cast(typename Op<T>::V, value_operand(V, r0 + 16 * s, t)), w, o[t]);
      }
    }
  }

  // Which of 32 rows of values hold an infinity or NaN.
  static __device__ __forceinline__ uint32_t not_finite(const unsigned char* V, int r0) {
    constexpr int LANES = PPR < 64 ? PPR : 64, PER = 64 / LANES;   // lanes of a row, rows at once
    const int lane = threadIdx.x & 63;
    uint32_t rows = 0;
    for (int r = 0; r < 32; r += PER) {
      const uint4 x = *reinterpret_cast<const uint4*>(V + (r0 + r) * RB + lane * 16);
      const uint32_t w[4] = {x.x, x.y, x.z, x.w};
      bool bad = false;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        if constexpr (F32) {
          bad |= (w[i] & 0x7f800000u) == 0x7f800000u;
        } else {
          constexpr uint32_t X = __is_same(T, __bf16) ? 0x7f80u : 0x7c00u;
          bad |= (w[i] & X) == X || (w[i] & (X << 16)) == (X << 16);
        }
      }
      const uint64_t b = __ballot(bad);
#pragma unroll
      for (int k = 0; k < PER; ++k)
        if ((b >> (k * LANES)) & (LANES == 64 ? ~0ull : (1ull << LANES) - 1)) rows |= 1u << (r + k);
    }
    return rows;
  }

  // The same for tiles of which a query may see a part, with infinities or NaN in rows `bad`: those rows enter the
  // products as zeros and are added key by key to the queries that see them.
  __device__ __forceinline__ void add_values_apart(const unsigned char* V, int r0, const f32x16& p, uint32_t bad,
                                                   int key0, int gone) {
    const int lane = threadIdx.x & 63, h = lane >> 5;
#pragma unroll
    for (int t = 0; t < DT; ++t) {
      if constexpr (F32) {
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          const float v = value_at(V, r0, t, i);
          o[t] = __builtin_amdgcn_mfma_f32_32x32x2f32(((bad >> key_of(i)) & 1) ? 0.f : v, p[i], o[t], 0, 0, 0);
        }
      } else {
#pragma unroll
        for (int s = 0; s < 2; ++s) {
          union { uint16_t e[8]; uint4 u; } v;
          v.u = value_operand(V, r0 + 16 * s, t);
#pragma unroll
          for (int j = 0; j < 8; ++j)
            if ((bad >> key_of(8 * s + j)) & 1) v.e[j] = 0;
          o[t] = Op<T>::mma(__builtin_bit_cast(typename Op<T>::V, v.u),
                            __builtin_bit_cast(typename Op<T>::V, weight_operand(p, s)), o[t]);
        }
      }
    }
    for (uint32_t left = bad; left != 0; left &= left - 1) {
      const int k = __ffs(left) - 1, key = key0 + k;
      float w = 0.f;      // its weight, in the lanes of half (k / 4) % 2
#pragma unroll
      for (int i = 0; i < 16; ++i)
        if (i == (k >> 3) * 4 + (k & 3)) w = F32 ? p[i] : Elem<T>::to_f(Elem<T>::from_f(p[i]));
      w = __shfl(w, (lane & 31) + 32 * ((k >> 2) & 1));
      const bool sees = key >= lo && key <= hi && !((gone >> (k >> 4)) & 1);
      const int r = r0 + k;
#pragma unroll
      for (int t = 0; t < DT; ++t) {
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          const int col = 32 * t + 8 * (i >> 2) + 4 * h + (i & 3);
          const T v = *reinterpret_cast<const T*>(V + r * RB + (((col / E) ^ value_swizzle<ES, PPR>(r)) << 4) +
                                                  (col % E) * ES);
          if (sees) o[t][i] += w * Elem<T>::to_f(v);
        }
      }
    }
  }
};

// Page numbers of 64 granules of 16 keys, one a lane, as rows of the cache (-1: no page).
struct Pages {
  int first;      // first granule held
  int row;        // this lane's
  uint64_t none;  // lanes without a page
};

template <typename A>
__device__ __forceinline__ void load_pages(const A& a, const int32_t* __restrict__ table, int head, int g0, Pages& p) {
  const int g = g0 + (int)(threadIdx.x & 63);
  // g * (ceil(2^32 / n)) >> 32 = g / n: the error g (n - 1) / (n 2^32) is below 1 / n for g < 2^32 / n
  const int page = (int)(((uint64_t)(uint32_t)g * a.granule_magic) >> 32), sub = g - page * a.granules;
  int row = -1;
  if (page < a.c.max_pages) {
    const int n = table[page];
    if (n >= 0 && n < a.c.num_pages) row = (n * a.c.Hkv + head) * a.c.page_size + sub * 16;
  }
  p.first = g0;
  p.row = row;
  p.none = __ballot(row < 0);
}

// Copies NR rows of keys (or values) from key `key` on (a multiple of NR, inside of one granule or NR a multiple of
// 16) to LDS; rows outside of [beg, end) and without a page as zeros.
template <int ES, int D, int NR, bool VALUES>
__device__ __forceinline__ void stage_rows(const void* cache, const Pages& pg, int key, int beg, int end, uint32_t lds) {
  constexpr int RB = D * ES, PPR = RB / 16, RPI = 64 / PPR > 0 ? 64 / PPR : 1;   // rows an instruction
  static_assert(PPR <= 64, "a row is at most one instruction");
  const int lane = threadIdx.x & 63;
  constexpr int GR = NR < 16 ? NR : 16;      // rows of one granule
#pragma unroll
  for (int g = 0; g < NR / GR; ++g) {
    const int at = key + g * 16;
    const int row = __builtin_amdgcn_readlane(pg.row, ((at >> 4) - pg.first) & 63);
    const bool whole = row >= 0 && at >= beg && at + GR <= end;
    const char* base = static_cast<const char*>(cache) + ((int64_t)row + (at & 15)) * RB;
#pragma unroll
    for (int n = 0; n < GR / RPI; ++n) {
      const int r = n * RPI + lane / PPR;          // row of the granule's part
      const int tr = (at & 15) + r + 16 * g;       // (swizzles go by the row's number modulo 16)
      const int piece = (lane % PPR) ^ (VALUES ? value_swizzle<ES, PPR>(tr) : key_swizzle<PPR>(tr));
      const uint32_t off = (uint32_t)(r * RB + piece * 16);
      const uint32_t to = lds + (uint32_t)((g * 16 + n * RPI) * RB);
      if (whole) {
        dma16(off, base, to);
      } else {
        const bool in = row >= 0 && at + r >= beg && at + r < end;
        dma16(in ? static_cast<const void*>(base + off) : static_cast<const void*>(zeros16), to);
      }
    }
  }
}


// A tile's rows and keys.
template <int ROWS>
struct Tile {
  int R, row0, room, pmin, pmax, beg, end, b, lens, L;
  __device__ __forceinline__ Tile(const AttendArgs& a, int G, const Unit& u) {
    R = u.L * G;
    row0 = u.tile * ROWS;
    b = u.b, lens = u.lens, L = u.L;
    room = min(max(lens, 0), a.c.max_pages * a.c.page_size);
    pmin = lens - L + row0 / G;
    pmax = lens - L + min(row0 + ROWS - 1, R - 1) / G;
    beg = a.window > 0 ? max(0, pmin - a.window + 1) : 0;
    end = min(pmax + 1, room);
  }
};

// Row n of the tile (clamped to the last one): its query, output row and the keys it sees.
template <typename T, int D, int ROWS>
__device__ __forceinline__ int64_t set_row(const AttendArgs& a, int G, int head, const Tile<ROWS>& t, int n,
                                           Wave<T, D>& w) {
  const int r = min(t.row0 + n, t.R - 1), token = r / G, g = r - token * G;
  const int p = t.lens - t.L + token;
  w.hi = min(p, t.room - 1);
  w.lo = a.window > 0 ? max(0, p - a.window + 1) : 0;
  w.load_query(static_cast<const T*>(a.q) + (int64_t)(t.b + token) * a.q_stride + (head * G + g) * D);
  return ((int64_t)(t.b + token) * a.c.Hq + head * G + g) * D;
}

template <typename T>
__device__ __forceinline__ void store_final(T* dst, float x, float y, float z, float u, float l) {
  const float f = 1.f / l;
  if (l == 0.f) store4<T>(dst, 0.f, 0.f, 0.f, 0.f);
  else store4<T>(dst, x * f, y * f, z * f, u * f);
}

// Many rows: four waves of 32 rows, the same keys.  Tiles of KT keys are double buffered; a tile's loads are issued one
// tile ahead, and the one barrier a tile also says that nobody reads the other buffer any more.
template <typename T, int D>
struct ManyShape {
  static constexpr int RB = D * (int)sizeof(T);
  static constexpr int KT = RB >= 1024 ? 32 : 64;
  static constexpr int NS = KT / 32, BYTES = 4 * KT * RB;
  static constexpr int WAVES = BYTES <= 81920 ? 2 : 1;   // a SIMD
};

template <typename T, int D>
__global__ __launch_bounds__(256, (ManyShape<T, D>::WAVES)) void cache_attention_many_kernel(AttendArgs a) {
  using S = ManyShape<T, D>;
  constexpr int KT = S::KT, RB = S::RB, ES = (int)sizeof(T), NR = KT / 4;
  extern __shared__ __align__(16) unsigned char smem[];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int G = a.c.Hq / a.c.Hkv, head = (int)(blockIdx.x % a.c.Hkv), unit = (int)(blockIdx.x / a.c.Hkv);
  Unit u;
  if (!find_unit<kManyRows>(a, G, unit, u)) return;
  const Tile<kManyRows> t(a, G, u);
  Wave<T, D> w;
  w.init();
  const int mine = wave * 32 + (lane & 31);
  const int64_t out = set_row(a, G, head, t, mine, w);
  const int key_first = t.beg & ~(KT - 1);
  const int tiles = t.end > t.beg ? (t.end - key_first + KT - 1) / KT : 0, per = (tiles + u.slices - 1) / u.slices;
  const int tb = u.slice * per, te = min(tiles, tb + per);
  const float c = a.scale_log2, slack = 8.f / c;
  const int32_t* table = a.c.table + (int64_t)u.s * a.c.max_pages;
  const uint32_t lds = (uint32_t)(uintptr_t)(__attribute__((address_space(3))) unsigned char*)smem;
  Pages pg;
  pg.first = -0x40000000;
  auto stage = [&](int i, int buf) {
    const int key = key_first + i * KT;
    if ((key >> 4) - pg.first >= 64) load_pages(a, table, head, key >> 4, pg);
    const uint32_t at = lds + (uint32_t)(buf * 2 * KT * RB + wave * NR * RB);
    stage_rows<ES, D, NR, false>(a.k_cache, pg, key + wave * NR, t.beg, t.end, at);
    stage_rows<ES, D, NR, true>(a.v_cache, pg, key + wave * NR, t.beg, t.end, at + KT * RB);
    return (int)((pg.none >> ((key >> 4) - pg.first)) & ((1 << (KT / 16)) - 1));
  };
  int gone = 0;
  if (tb < te) gone = stage(tb, 0);
  for (int i = tb; i < te; ++i) {
    const int buf = (i - tb) & 1, key = key_first + i * KT, absent = gone;
    wait_loads<0>();
    lds_barrier();
    if (i + 1 < te) gone = stage(i + 1, buf ^ 1);
    const unsigned char* K = smem + buf * 2 * KT * RB;
    const unsigned char* V = K + KT * RB;
    f32x16 s[S::NS];
#pragma unroll
    for (int n = 0; n < S::NS; ++n) s[n] = w.scores(K, 32 * n);
    const bool part = key + KT - 1 > min(t.pmin, t.room - 1) || (a.window > 0 && key < t.pmax - a.window + 1) || absent;
    if (part) {
#pragma unroll
      for (int n = 0; n < S::NS; ++n) w.mask(s[n], key + 32 * n, absent >> (2 * n));
    }
    float top = -INFINITY;
#pragma unroll
    for (int n = 0; n < S::NS; ++n)
#pragma unroll
      for (int j = 0; j < 16; ++j) top = fmaxf(top, s[n][j]);
    w.raise(top, c, slack);
#pragma unroll
    for (int n = 0; n < S::NS; ++n) w.weigh(s[n], c);
#pragma unroll
    for (int n = 0; n < S::NS; ++n) {
      const uint32_t bad = part ? w.not_finite(V, 32 * n) : 0;
      if (__builtin_expect(bad != 0, 0)) w.add_values_apart(V, 32 * n, s[n], bad, key + 32 * n, absent >> (2 * n));
      else w.add_values(V, 32 * n, s[n]);
    }
  }
  const float l = other_half_sum(w.l);
  if (t.row0 + mine >= t.R) return;
  const int h = lane >> 5;
  if (u.slices == 1) {
    T* o = static_cast<T*>(a.o) + out;
#pragma unroll
    for (int k = 0; k < D / 32; ++k)
#pragma unroll
      for (int j = 0; j < 4; ++j)
        store_final(o + 32 * k + 8 * j + 4 * h, w.o[k][4 * j], w.o[k][4 * j + 1], w.o[k][4 * j + 2], w.o[k][4 * j + 3], l);
  } else {
    const int64_t slot = ((int64_t)unit * a.c.Hkv + head) * kManyRows + mine;
    float* o = a.part_o + slot * D;
#pragma unroll
    for (int k = 0; k < D / 32; ++k)
#pragma unroll
      for (int j = 0; j < 4; ++j)
        store4<float>(o + 32 * k + 8 * j + 4 * h, w.o[k][4 * j], w.o[k][4 * j + 1], w.o[k][4 * j + 2], w.o[k][4 * j + 3]);
    if (h == 0) *reinterpret_cast<float2*>(a.part_ml + slot * 2) = make_float2(w.m, l);
  }
}

// Few rows: one tile of 32 rows, each wave on its own 32 keys at a time with its own piece of LDS and no barrier: once
// a tile's keys have been read the next ones are on their way, once its values have been read the next values.
template <typename T, int D>
struct FewShape {
  static constexpr int RB = D * (int)sizeof(T), NW = RB >= 1024 ? 2 : 4;
  static constexpr int BYTES = NW * 64 * RB, WAVES = BYTES <= 81920 ? 2 : 1;
};

template <typename T, int D>
__global__ __launch_bounds__((64 * FewShape<T, D>::NW), (FewShape<T, D>::WAVES))
void cache_attention_few_kernel(AttendArgs a) {
  using S = FewShape<T, D>;
  constexpr int RB = S::RB, ES = (int)sizeof(T), NW = S::NW, NI = 32 * RB / 1024;
  extern __shared__ __align__(16) unsigned char smem[];
  __shared__ float2 ml[NW][32];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int G = a.c.Hq / a.c.Hkv, head = (int)(blockIdx.x % a.c.Hkv), unit = (int)(blockIdx.x / a.c.Hkv);
  Unit u;
  if (!find_unit<kFewRows>(a, G, unit, u)) return;
  const Tile<kFewRows> t(a, G, u);
  Wave<T, D> w;
  w.init();
  set_row(a, G, head, t, lane & 31, w);
  const int key_first = t.beg & ~31;
  const int tiles = t.end > t.beg ? (t.end - key_first + 31) / 32 : 0, per = (tiles + u.slices - 1) / u.slices;
  const int tb = u.slice * per, te = min(tiles, tb + per);
  const float c = a.scale_log2, slack = 8.f / c;
  const int32_t* table = a.c.table + (int64_t)u.s * a.c.max_pages;
  const unsigned char* K = smem + wave * 64 * RB;
  const unsigned char* V = K + 32 * RB;
  const uint32_t ldsK = (uint32_t)(uintptr_t)(__attribute__((address_space(3))) unsigned char*)smem + wave * 64 * RB;
  Pages pg;
  pg.first = -0x40000000;
  auto pages_for = [&](int i) {
    const int g = (key_first >> 4) + 2 * i;
    if (g - pg.first >= 64) load_pages(a, table, head, g, pg);
    return (int)((pg.none >> (g - pg.first)) & 3);
  };
  int i = tb + wave, gone = 0;
  if (i < te) {
    gone = pages_for(i);
    stage_rows<ES, D, 32, false>(a.k_cache, pg, key_first + 32 * i, t.beg, t.end, ldsK);
    stage_rows<ES, D, 32, true>(a.v_cache, pg, key_first + 32 * i, t.beg, t.end, ldsK + 32 * RB);
  }
  for (; i < te; i += NW) {
    const int key = key_first + 32 * i, absent = gone, next = i + NW;
    wait_loads<NI>();                              // the keys: the values were issued after them
    f32x16 s = w.scores(K, 0);
    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
    if (next < te) {
      gone = pages_for(next);
      stage_rows<ES, D, 32, false>(a.k_cache, pg, key_first + 32 * next, t.beg, t.end, ldsK);
    }
    const bool part = key + 31 > min(t.pmin, t.room - 1) || (a.window > 0 && key < t.pmax - a.window + 1) || absent;
    if (part) w.mask(s, key, absent);
    float top = -INFINITY;
#pragma unroll
    for (int j = 0; j < 16; ++j) top = fmaxf(top, s[j]);
    w.raise(top, c, slack);
    w.weigh(s, c);
    if (next < te) wait_loads<NI>();               // the values: the next keys were issued after them
    else wait_loads<0>();
    const uint32_t bad = part ? w.not_finite(V, 0) : 0;
    if (__builtin_expect(bad != 0, 0)) w.add_values_apart(V, 0, s, bad, key, absent);
    else w.add_values(V, 0, s);
    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
    if (next < te) stage_rows<ES, D, 32, true>(a.v_cache, pg, key_first + 32 * next, t.beg, t.end, ldsK + 32 * RB);
  }
  // join the waves: everyone's accumulators in LDS (pieces of 16 bytes at piece ^ row % 8)
  const float l = other_half_sum(w.l);
  const int h = lane >> 5, row = lane & 31;
  if (h == 0) ml[wave][row] = make_float2(w.m, l);
  __syncthreads();                                 // and nobody reads keys or values any more
  float4* O = reinterpret_cast<float4*>(smem);
#pragma unroll
  for (int k = 0; k < D / 32; ++k)
#pragma unroll
    for (int j = 0; j < 4; ++j)
      O[(wave * 32 + row) * (D / 4) + ((8 * k + 2 * j + h) ^ (row & 7))] =
          make_float4(w.o[k][4 * j], w.o[k][4 * j + 1], w.o[k][4 * j + 2], w.o[k][4 * j + 3]);
  __syncthreads();
  const int rows = min(kFewRows, t.R - t.row0);
  const int64_t slot = ((int64_t)unit * a.c.Hkv + head) * kFewRows;
  for (int k = threadIdx.x; k < rows * (D / 4); k += 64 * NW) {
    const int r = k / (D / 4), piece = k % (D / 4);
    float m = -INFINITY;
#pragma unroll
    for (int v = 0; v < NW; ++v) m = fmaxf(m, ml[v][r].x);
    float4 sum = make_float4(0.f, 0.f, 0.f, 0.f);
    float tot = 0.f;
#pragma unroll
    for (int v = 0; v < NW; ++v) {
      const float2 x = ml[v][r];
      const float f = x.x == -INFINITY ? 0.f : __builtin_amdgcn_exp2f((x.x - m) * c);
      const float4 p = O[(v * 32 + r) * (D / 4) + (piece ^ (r & 7))];
      sum.x += f * p.x, sum.y += f * p.y, sum.z += f * p.z, sum.w += f * p.w;
      tot += f * x.y;
    }
    if (u.slices == 1) {
      const int token = (t.row0 + r) / G, g = t.row0 + r - token * G;
      T* o = static_cast<T*>(a.o) + ((int64_t)(t.b + token) * a.c.Hq + head * G + g) * D + 4 * piece;
      store_final(o, sum.x, sum.y, sum.z, sum.w, tot);
    } else {
      *reinterpret_cast<float4*>(a.part_o + (slot + r) * D + 4 * piece) = sum;
      if (piece == 0) *reinterpret_cast<float2*>(a.part_ml + (slot + r) * 2) = make_float2(m, tot);
    }
  }
}

// Joins the slices of a row: a workgroup a row, groups of D / 4 threads on every few slices.
template <typename T, int D, int ROWS>
__global__ __launch_bounds__(256) void cache_attention_join_kernel(AttendArgs a, int64_t row0) {
  constexpr int PIECES = D / 4, GROUPS = 256 / PIECES;
  __shared__ float weight[kMostSlices];
  __shared__ float4 sums[GROUPS][PIECES];
  __shared__ float red[8];
  const int lane = threadIdx.x & 63, G = a.c.Hq / a.c.Hkv;
  const int64_t at = row0 + blockIdx.x;             // (tile, head, row of the tile)
  const int n = (int)(at % ROWS), head = (int)(at / ROWS % a.c.Hkv), want = (int)(at / ROWS / a.c.Hkv);
  // the want-th tile, and how many (tile, slice) pairs come before it
  const int keys = slice_keys<ROWS>(a, G);
  int before = 0, units = 0, slices = 0, first = 0, tile = 0, b = 0, L = 0;
  bool found = false;
  for (int s0 = 0; s0 < a.c.N && !found; s0 += 64) {
    int bb, LL, lens, tiles, span;
    sequence_size<ROWS>(a, G, s0 + lane, bb, LL, lens, tiles, span);
    const int sl = span > keys ? (span + keys - 1) / keys : 1;
    int upto = tiles, upto_units = tiles * sl;
#pragma unroll
    for (int m = 1; m < 64; m <<= 1) {
      const int o = __shfl_up(upto, m), o2 = __shfl_up(upto_units, m);
      if (lane >= m) upto += o, upto_units += o2;
    }
    const int total = __builtin_amdgcn_readlane(upto, 63);
    if (want < before + total) {
      const int j = __ffsll((unsigned long long)__ballot(want < before + upto)) - 1;
      const int tl = __builtin_amdgcn_readlane(tiles, j);
      slices = __builtin_amdgcn_readlane(sl, j);
      const int rest = want - before - (__builtin_amdgcn_readlane(upto, j) - tl);
      first = units + __builtin_amdgcn_readlane(upto_units, j) - tl * slices + rest * slices;
      tile = tl - 1 - rest;
      b = __builtin_amdgcn_readlane(bb, j);
      L = __builtin_amdgcn_readlane(LL, j);
      found = true;
    }
    before += total;
    units += __builtin_amdgcn_readlane(upto_units, 63);
  }
  const int r = tile * ROWS + n;
  // (malformed offsets may count more pairs than there is room for)
  if (!found || slices < 2 || r >= L * G || first + slices > a.units) return;
  auto slot = [&](int s) { return ((int64_t)(first + s) * a.c.Hkv + head) * ROWS + n; };
  float m = -INFINITY;
  for (int s = threadIdx.x; s < slices; s += 256) {
    const float x = a.part_ml[slot(s) * 2];
    weight[s] = x;
    m = fmaxf(m, x);
  }
#pragma unroll
  for (int k = 1; k < 64; k <<= 1) m = fmaxf(m, __shfl_xor(m, k));
  if (lane == 0) red[threadIdx.x >> 6] = m;
  __syncthreads();
  m = fmaxf(fmaxf(red[0], red[1]), fmaxf(red[2], red[3]));
  float l = 0.f;
  for (int s = threadIdx.x; s < slices; s += 256) {
    const float x = weight[s], f = x == -INFINITY ? 0.f : __builtin_amdgcn_exp2f((x - m) * a.scale_log2);
    weight[s] = f;
    l += f * a.part_ml[slot(s) * 2 + 1];
  }
#pragma unroll
  for (int k = 1; k < 64; k <<= 1) l += __shfl_xor(l, k);
  if (lane == 0) red[4 + (threadIdx.x >> 6)] = l;
  __syncthreads();
  l = (red[4] + red[5]) + (red[6] + red[7]);
  const int piece = threadIdx.x % PIECES, group = threadIdx.x / PIECES;
  float4 sum = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
  for (int s = group; s < slices; s += GROUPS) {
    const float4 p = *reinterpret_cast<const float4*>(a.part_o + slot(s) * D + 4 * piece);
    const float f = weight[s];
    sum.x += f * p.x, sum.y += f * p.y, sum.z += f * p.z, sum.w += f * p.w;
  }
  sums[group][piece] = sum;
  __syncthreads();
  if (group != 0) return;
#pragma unroll
  for (int k = 1; k < GROUPS; ++k) {
    const float4 p = sums[k][piece];
    sum.x += p.x, sum.y += p.y, sum.z += p.z, sum.w += p.w;
  }
  const int token = r / G, g = r - token * G;
  store_final(static_cast<T*>(a.o) + ((int64_t)(b + token) * a.c.Hq + head * G + g) * D + 4 * piece, sum.x, sum.y,
              sum.z, sum.w, l);
}

template <typename K>
static hipError_t allow_lds(K kernel, int bytes) {
  return bytes > 65536 ? hipFuncSetAttribute(reinterpret_cast<const void*>(kernel),
                                             hipFuncAttributeMaxDynamicSharedMemorySize, bytes)
                       : hipSuccess;
}

template <typename T, int D>
static hipError_t launch_attend_d(const AttendArgs& a, int64_t tiles, hipStream_t s) {
  const unsigned wgs = (unsigned)((int64_t)a.units * a.c.Hkv);
  prof_begin(K_ATTEND, s);
  hipError_t e;
  if (a.few) {
    using S = FewShape<T, D>;
    e = allow_lds(cache_attention_few_kernel<T, D>, S::BYTES);
    if (e != hipSuccess) return e;
    hipLaunchKernelGGL((cache_attention_few_kernel<T, D>), dim3(wgs), dim3(64 * S::NW), S::BYTES, s, a);
  } else {
    using S = ManyShape<T, D>;
    e = allow_lds(cache_attention_many_kernel<T, D>, S::BYTES);
    if (e != hipSuccess) return e;
    hipLaunchKernelGGL((cache_attention_many_kernel<T, D>), dim3(wgs), dim3(256), S::BYTES, s, a);
  }
  prof_end(K_ATTEND, s);
  if ((e = hipGetLastError()) != hipSuccess || a.slices == 0) return e;
  prof_begin(K_ATTEND_JOIN, s);
  const int64_t rows = tiles * a.c.Hkv * (a.few ? kFewRows : kManyRows), most = kLaunchThreads / 256;
  for (int64_t r = 0; r < rows; r += most) {
    const dim3 grid((unsigned)std::min(most, rows - r));
    if (a.few) hipLaunchKernelGGL((cache_attention_join_kernel<T, D, kFewRows>), grid, dim3(256), 0, s, a, r);
    else hipLaunchKernelGGL((cache_attention_join_kernel<T, D, kManyRows>), grid, dim3(256), 0, s, a, r);
  }
  prof_end(K_ATTEND_JOIN, s);
  return hipGetLastError();
}

template <typename T>
static hipError_t launch_attend_t(const AttendArgs& a, hipStream_t s) {
  const int64_t tiles = a.units - a.slices;
  switch (a.c.d) {
    case 32: return launch_attend_d<T, 32>(a, tiles, s);
    case 64: return launch_attend_d<T, 64>(a, tiles, s);
    case 128: return launch_attend_d<T, 128>(a, tiles, s);
    case 256: return launch_attend_d<T, 256>(a, tiles, s);
  }
  return hipErrorInvalidValue;
}

}  // namespace attend
}  // namespace gdn
