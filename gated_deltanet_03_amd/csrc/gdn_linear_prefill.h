// Chunked prefill of linear attention with a decay for each head (kernels;
// instantiated for one input type by each gdn_linear_<type>.hip).
//
// Inside a chunk of C tokens with cumulative log decays G_i:
//
//   o_i   = scale [ e^{G_i} S^T q_i + sum_{j <= i} e^{G_i - G_j} (q_i . k_j) v_j ]
//   S_out = e^{G_C} S + sum_j e^{G_C - G_j} k_j v_j^T
//
// Long sequences are cut into segments (few sequences and heads would leave most
// CUs idle).  Pass kState gives each segment's own state, the first's with the
// initial one; pass kOut sums those before its segment, walks it for the outputs,
// and writes the final state after the last.  Without segments one pass, kWhole,
// does both.
//
// A workgroup walks the chunks of one (segment, value head, column slice) with
// the fp32 state in the registers of its waves: each wave owns all dk rows of its
// own 16*NT columns.  Everything is 16x16 MFMA tiles:
//   * S is carried in accumulators; two of its tiles are directly an operand of
//     S^T Q (their dk rows permuted inside each 32-row block so that Q's and K's
//     operands are contiguous 16-byte reads);
//   * the scores come out as P^T = K Q^T, in the form of an operand of V^T P^T;
//     each wave computes some tiles and hands them to the others through LDS in
//     fragment order and fp32 (for fp16 they are brought into its range by a power
//     of two a query when they are read: q . k alone may be far outside of it);
//   * o^T is accumulated, so a lane holds adjacent columns of one token and
//     writes them with one access;
//   * K^T and V operands (contraction over tokens) come from transpose reads of
//     the row-major tiles.
// Two barriers a chunk: before the first, all products that read the tiles
// (scores, S^T Q, the state's update) while later chunks' loads are in flight;
// after it, V^T P^T on registers once the next tiles are stored.
//
// The state's update uses e^{G_C - G_j} v_j split into parts of the input type
// (three for bf16, two for fp16), so the carried state keeps fp32 accuracy.  The
// state and the scores are two parts each where they are operands of o (2^-16 of a
// term for bf16, 2^-22 for fp16: o is rounded once, at its end; one part each made
// its error 1.4 times that rounding and took 155 us instead of 178 on the 14286
// tokens below).  kOut's own walk, which ends in no final state, takes two bf16
// parts of the decayed v (2^-16 again).  For fp16 a power of two brings each column
// of these operands into its range, so that no column depends on its neighbours.
//
// Log decays are summed in 64 bits.  A decay between two tokens of one 16-token
// tile is the exponential of a difference of coarse parts (multiples of 1/64,
// exact) and fine parts: in a long chunk of strong decays |G| reaches thousands
// while neighbouring G_i - G_j are small.  Between tiles it is the product of two
// factors that are both at most 1, from the tile's start to the query and from
// the key to the tile's start.  A decay below e^-128 is 0 in fp32, so g is clamped
// there and -infinity needs no special case.
//
// What bounds it: 14286 ragged tokens x 32 heads, d = 128, bf16 take 178 us, 62 of
// them the state pass; the passes move 245 and 421 MB, 47 and 81 us as a copy.  In the
// output pass a wave's 32-token chunk is about 610 VALU, 75 MFMA and 50 LDS
// instructions, and VALU, MFMA and LDS are busy 49, 24 and 23 % of the time (41, 31 and
// 31 in the state pass): conversions and decays, then latencies, with two waves a
// SIMD (232 to 250 VGPRs) to hide them.  A third wave a SIMD spills.  Before the
// operands were in two parts (output pass 97 us) chunks re-read from the cache were
// no faster, bank-conflict-free tiles gained 1 %, and one column tile a wave (twice
// the waves and LDS reads) took 122 us, four 119 us.
#pragma once

#include <algorithm>

#include "gdn_device.h"
#include "gdn_mfma.h"
#include "gdn_ops_internal.h"
#include "gdn_scan.h"

namespace gdn {
namespace linear {

typedef short s16x4 __attribute__((ext_vector_type(4)));

// Within each group of 16 lanes, lane i receives element i % 4 of the 8-byte
// pieces addressed by lanes 4j + i / 4, j = 0..3 (as its element j).
__device__ __forceinline__ s16x4 lds_read_tr(const void* p) {
  return __builtin_amdgcn_ds_read_tr16_b64_v4i16((__attribute__((address_space(3))) s16x4*)p);
}

__device__ __forceinline__ float max_groups(float x) {   // over the lanes of equal lane % 16, x >= 0
  const auto a = __builtin_amdgcn_permlane16_swap(__float_as_uint(x), __float_as_uint(x), false, false);
  x = fmaxf(__uint_as_float(a[0]), __uint_as_float(a[1]));
  const auto b = __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(x), false, false);
  return fmaxf(__uint_as_float(b[0]), __uint_as_float(b[1]));
}

__device__ __forceinline__ double lane64(double x, int lane) {
  const uint64_t u = __builtin_bit_cast(uint64_t, x);
  const uint32_t lo = __builtin_amdgcn_readlane((int)(uint32_t)u, lane);
  const uint32_t hi = __builtin_amdgcn_readlane((int)(u >> 32), lane);
  return __builtin_bit_cast(double, (uint64_t)hi << 32 | lo);
}

// Exponent shift that brings |x| <= m into [2^13, 2^15) (0 for m = 0 or not finite).
__device__ __forceinline__ int shift_for(float m) {
  if (!(m > 0.f) || m > 3.0e38f) return 0;
  const int e = 14 - ilogbf(m);
  return e < -100 ? -100 : (e > 100 ? 100 : e);
}

__device__ __forceinline__ f32x4 shifted(const f32x4& x, int sh) {   // x * 2^sh
  return f32x4{ldexpf(x[0], sh), ldexpf(x[1], sh), ldexpf(x[2], sh), ldexpf(x[3], sh)};
}

// Segment `seg`: its sequence and tokens, its number in the sequence and whether
// it is the last.  An empty sequence has one empty segment.  False past the end.
struct Segment {
  int s, t0, t1, j;
  bool last;
};

__device__ __forceinline__ bool find_segment(const LinearArgs& p, int seg, Segment& x) {
  if (p.seg_tokens == 0) {
    x.s = seg;
    x.j = 0;
    x.last = true;
    seq_range(p.cu, p.T, p.total, seg, x.t0, x.t1);
    return true;
  }
  const int L = p.seg_tokens;
  if (p.cu == nullptr) {
    const int per = (p.T + L - 1) / L;
    x.s = seg / per;
    x.j = seg % per;
    x.last = x.j == per - 1;
    x.t0 = x.s * p.T + x.j * L;
    x.t1 = min(x.t0 + L, (x.s + 1) * p.T);
    return true;
  }
  const int lane = threadIdx.x & 63;
  int base = 0;
  for (int s0 = 0; s0 < p.B; s0 += 64) {
    int a = 0, b = 0;
    if (s0 + lane < p.B) clamp_range(p.cu[s0 + lane], p.cu[s0 + lane + 1], p.total, a, b);
    const int n = s0 + lane < p.B ? max(1, (b - a + L - 1) / L) : 0;
    int incl = n;
#pragma unroll
    for (int d = 1; d < 64; d *= 2) {
      const int y = __shfl_up(incl, d);
      if (lane >= d) incl += y;
    }
    const uint64_t hit = __ballot(base + incl > seg);
    if (hit) {
      const int f = (int)__builtin_ctzll(hit);
      const int count = __builtin_amdgcn_readlane(n, f);
      x.s = s0 + f;
      x.j = seg - (base + __builtin_amdgcn_readlane(incl, f) - count);
      x.last = x.j == count - 1;
      x.t0 = __builtin_amdgcn_readlane(a, f) + x.j * L;
      x.t1 = min(x.t0 + L, __builtin_amdgcn_readlane(b, f));
      return true;
    }
    base += __builtin_amdgcn_readlane(incl, 63);
  }
  return false;
}

// dk index of row m of state tile t (16 rows a tile): tiles 2b and 2b+1 hold the
// block's rows so that a lane's 8 contraction slots are 8 adjacent dk.
template <int DK>
__device__ __forceinline__ int state_row(int t, int m) {
  if constexpr (DK < 32) return m;
  else return 32 * (t >> 1) + 8 * (m >> 2) + 4 * (t & 1) + (m & 3);
}

// Column of row m of column tile n (counted over all of dv): with at least two
// tiles, a lane's rows 4g..4g+3 of tiles 2b and 2b+1 are 8 adjacent columns.
// The same map as the rows', so that it does not depend on how tiles are dealt
// to waves: the passes may deal them differently.
__device__ __forceinline__ int state_col(int dv, int n, int m) { return dv < 32 ? m : state_row<32>(n, m); }

// A chunk's decays; the state pass keeps only the first two.
template <int C, bool STATE>
struct Decays {
  static constexpr int O = STATE ? 4 : C, RT = C / 16;
  __align__(16) float w[C];              // e^{G_last - G_i}
  __align__(16) float gamma[4];          // e^{G_last}
  __align__(16) float hi[O];             // coarse and fine part of G_i
  __align__(16) float lo[O];
  __align__(16) float eg[O];             // e^{G_i}
  __align__(16) float row[O];            // e^{G_i - G_s}, s the last token before i's tile
  __align__(16) float col[STATE ? 4 : 8 * RT * (RT - 1)];   // at col_at(t) + j: e^{G_{16t-1} - G_j}, j < 16t
};

// First of the 16t column factors of query tile t >= 1.
__device__ __forceinline__ constexpr int col_at(int t) { return 8 * t * (t - 1); }

// One wave: the decays of a chunk from lane i's log decay (0 past the end);
// returns their sum.
template <int C, bool STATE>
__device__ __forceinline__ double fill_decays(float g, Decays<C, STATE>& d) {
  const int lane = threadIdx.x & 63;
  const double x = wave_scan64(lane < C ? (double)(g < -128.f ? -128.f : g) : 0.0);
  const double end = lane64(x, C - 1);
  if (lane < C) d.w[lane] = expf((float)(end - x));
  if (lane == 0) d.gamma[0] = expf((float)end);
  if constexpr (!STATE) {
    constexpr int RT = C / 16;
    double start = 0.0;
#pragma unroll
    for (int t = 1; t < RT; ++t) {
      const double at = lane64(x, 16 * t - 1);
      if (lane >= 16 * t) start = at;
      if (lane < 16 * t) d.col[col_at(t) + lane] = __expf((float)(at - x));
    }
    if (lane < C) {
      const float hi = rintf((float)x * 64.f) * 0.015625f;
      d.hi[lane] = hi;
      d.lo[lane] = (float)(x - (double)hi);
      d.eg[lane] = expf((float)x);
      d.row[lane] = __expf((float)(x - start));
    }
  }
  return end;
}

// Fragments of P: row tile i holds i / 2 + 1 blocks of 32 keys.
__device__ __forceinline__ constexpr int p_frag(int i, int b) { return (i + 1) * (i + 1) / 4 + b; }

// A row-major tile of W columns in LDS.  16-bit rows are unpadded; the 16-byte
// pieces of row r are permuted by an exclusive or with a value that makes both
// the 16 rows of one piece (row_frag) and the 4 rows x 4 pieces of a transpose
// read (token_frag) fall on different banks.
template <typename T, int W>
struct Tile {
  static constexpr int P = W * (int)sizeof(T) / 16;             // pieces a row
  static constexpr int STRIDE = sizeof(T) == 2 ? W : W + 4;
  static __device__ __forceinline__ int at(int r, int c) {
    if constexpr (sizeof(T) == 4) return r * STRIDE + c;
    const int q = r >> 2 & 3;
    const int x = P == 16 ? (r & 3) << 2 | q : P == 8 ? (r & 2) << 1 | q : P == 4 ? q : r >> 3 & 1;
    return r * STRIDE + ((c >> 3 ^ x) << 3) + (c & 7);
  }
};

template <typename T, int C, int DK, int NT, int NW, bool STATE>
struct Smem {
  static constexpr int CW = 16 * NT * NW;
  __align__(16) T k[C * Tile<T, DK>::STRIDE];
  __align__(16) T v[C * Tile<T, CW>::STRIDE];
  __align__(16) T q[STATE ? 8 : C * Tile<T, DK>::STRIDE];
  __align__(16) float p[STATE ? 4 : p_frag(C / 16, 0) * 512];
  Decays<C, STATE> d[2];
};

// A (or, transposed, B) operand of rows 16*tile.. over dk block kb.
template <typename T, int DK>
__device__ __forceinline__ Frag<T> row_frag(const T* base, int tile, int kb) {
  const int lane = threadIdx.x & 63, i16 = lane & 15, g4 = lane >> 4;
  const T* r = base + 16 * tile * Tile<T, DK>::STRIDE + Tile<T, DK>::at(i16, DK >= 32 ? 32 * kb + 8 * g4 : 4 * g4);
  if constexpr (DK >= 32) {
    return load_frag_8<T>(r);
  } else {
    Frag<T> f = zero_frag<T>();
    if constexpr (sizeof(T) == 4) {
      f.lo = *reinterpret_cast<const f32x4*>(r);
    } else {
      const auto a = *reinterpret_cast<const typename Half4<T>::type*>(r);
      f.v[0] = a[0]; f.v[1] = a[1]; f.v[2] = a[2]; f.v[3] = a[3];
    }
    return f;
  }
}

// Operand over the 32 tokens of block tb for column tile `c0..`: slot 8g + j is
// token 32tb + 4g + j (j < 4) or 32tb + 16 + 4g + j - 4.  `cols(m)`: column of row m.
template <typename T, int W, typename F>
__device__ __forceinline__ Frag<T> token_frag(const T* base, int tb, F cols) {
  using M = Tile<T, W>;
  const int lane = threadIdx.x & 63, i16 = lane & 15, g4 = lane >> 4;
  Frag<T> f;
  if constexpr (sizeof(T) == 4) {
    const int c = cols(i16);
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      f.lo[q] = base[M::at(32 * tb + 4 * g4 + q, c)];
      f.hi[q] = base[M::at(32 * tb + 16 + 4 * g4 + q, c)];
    }
  } else {
    // lane i addresses token i / 4 and the four columns of rows 4 (i % 4) ..
    const T* a = base + 32 * tb * M::STRIDE + M::at(4 * g4 + (i16 >> 2), cols(4 * (i16 & 3)));
    const s16x4 x = lds_read_tr(a), y = lds_read_tr(a + 16 * M::STRIDE);
    union { s16x4 s[2]; decltype(f.v) v; } u;
    u.s[0] = x;
    u.s[1] = y;
    f.v = u.v;
  }
  return f;
}

template <typename T>
__device__ __forceinline__ float frag_get(const Frag<T>& f, int i) {
  if constexpr (sizeof(T) == 4) return i < 4 ? f.lo[i & 3] : f.hi[i & 3];
  else return Elem<T>::to_f(f.v[i]);
}

// Parts of the decayed v of a fragment: one fp32; bf16 three, or two where only
// outputs follow; fp16 two.
enum class Pass { kState, kOut, kWhole };   // segment states; outputs from given states; both (no segments)
template <typename T, Pass P>
constexpr int kParts = sizeof(T) == 4 ? 1 : (__is_same(T, __bf16) && P != Pass::kOut ? 3 : 2);

// Parts of the state and of the scores as operands of o.
template <typename T>
constexpr int kOperandParts = sizeof(T) == 4 ? 1 : 2;

template <typename T, int N>
__device__ __forceinline__ void split(const float* x, Frag<T>* part) {
  if constexpr (sizeof(T) == 4) {
    part[0].lo = f32x4{x[0], x[1], x[2], x[3]};
    part[0].hi = f32x4{x[4], x[5], x[6], x[7]};
  } else {
    typedef T T2 __attribute__((ext_vector_type(2)));   // pairs: one conversion instruction for two
    typedef float f32x2 __attribute__((ext_vector_type(2)));
#pragma unroll
    for (int j = 0; j < 8; j += 2) {
      f32x2 r = {x[j], x[j + 1]};
#pragma unroll
      for (int n = 0; n < N; ++n) {
        const T2 h = __builtin_convertvector(r, T2);
        part[n].v[j] = h[0];
        part[n].v[j + 1] = h[1];
        r -= __builtin_convertvector(h, f32x2);
      }
    }
  }
}

template <typename T, int N>
__device__ __forceinline__ void split(const f32x4& lo, const f32x4& hi, Frag<T>* part) {
  const float x[8] = {lo[0], lo[1], lo[2], lo[3], hi[0], hi[1], hi[2], hi[3]};
  split<T, N>(x, part);
}

// A fragment of f(index) in each slot.
template <typename T, typename F>
__device__ __forceinline__ Frag<T> make_slots(F f) {
  Frag<T> y;
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const float v = f(j);
    if constexpr (sizeof(T) == 2) y.v[j] = Elem<T>::from_f(v);
    else if (j < 4) y.lo[j & 3] = v;
    else y.hi[j & 3] = v;
  }
  return y;
}

// Two waves a SIMD; one for the narrow output pass with few workgroups (at most two of two
// waves a CU), which keeps a 64-token chunk on its way in 72 registers.
template <Pass PASS, int C, int NW>
constexpr int kWaves = PASS == Pass::kOut && C == 64 && NW <= 2 ? 1 : 2;

template <typename T, int C, int DK, int NT, int NW, Pass PASS>
__global__ __launch_bounds__(64 * NW, (kWaves<PASS, C, NW>)) void linear_chunk_kernel(LinearArgs p) {
  constexpr bool STATE = PASS == Pass::kState;
  using SM = Smem<T, C, DK, NT, NW, STATE>;
  constexpr int CW = SM::CW, THREADS = 64 * NW;
  using KT = Tile<T, DK>;
  using VT = Tile<T, CW>;
  constexpr int RT = C / 16, NTB = C / 32;                    // token tiles and 32-token blocks
  constexpr int NST = DK / 16, NKB = DK >= 32 ? DK / 32 : 1;  // state row tiles, dk blocks
  constexpr int PER = 16 / (int)sizeof(T), KP = DK / PER, VP = CW / PER;   // 16-byte pieces a row
  constexpr int NKL = (C * KP + THREADS - 1) / THREADS, NVL = (C * VP + THREADS - 1) / THREADS;
  constexpr int KR = THREADS / KP, VR = THREADS / VP;         // rows between a thread's pieces
  static_assert(THREADS % KP == 0 && THREADS % VP == 0, "");
  constexpr int NP = kParts<T, PASS>, OP = kOperandParts<T>;
  __shared__ SM sm;

  // XCD-aware order: the workgroups that share one segment's keys get ids equal mod 8
  const int G = p.Hv / p.Hq, nsl = p.dv / CW, share = G * nsl;
  const int unit = p.first + (int)(blockIdx.x >> 3) / share * 8 + (int)(blockIdx.x & 7);
  if (unit >= p.max_segs * p.Hq) return;
  const int seg = unit / p.Hq, hk = unit % p.Hq, sub = (int)(blockIdx.x >> 3) % share;
  const int h = hk * G + sub / nsl, slice = sub % nsl;
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int i16 = lane & 15, g4 = lane >> 4;
  Segment sg;
  if (!find_segment(p, seg, sg)) return;
  const int s = __builtin_amdgcn_readfirstlane(sg.s), t0 = __builtin_amdgcn_readfirstlane(sg.t0),
            t1 = __builtin_amdgcn_readfirstlane(sg.t1), sj = __builtin_amdgcn_readfirstlane(sg.j);
  const size_t per = (size_t)DK * p.dv, krow = (size_t)p.Hq * DK, vrow = (size_t)p.Hv * p.dv;
  const T* qp = static_cast<const T*>(p.q) + (size_t)hk * DK;
  const T* kp = static_cast<const T*>(p.k) + (size_t)hk * DK;
  const T* vp = static_cast<const T*>(p.v) + (size_t)h * p.dv + slice * CW;
  const int tile0 = wave * NT;   // this wave's first column tile in the slice

  // state tile (t, n): lane holds rows 4g..4g+3 of the tile, column i16
  f32x4 S[NST][NT];
  auto slot_at = [&](int slot, int t, int n) {   // the workspace's states are kept in this order
    return reinterpret_cast<f32x4*>(p.seg_state + ((size_t)slot * p.Hv + h) * per) +
           (t * (p.dv / 16) + slice * (CW / 16) + tile0 + n) * 64 + lane;
  };
  auto seg_at = [&](int j, int t, int n) { return slot_at(seg - sj + j, t, n); };
  auto state_at = [&](int t, int n, int e) {
    return (size_t)h * per + (size_t)state_row<DK>(t, 4 * g4 + e) * p.dv + slice * CW + state_col(CW, tile0 + n, i16);
  };
  const float* s0 = p.s0 != nullptr ? p.s0 + (int64_t)s * p.s0_stride : nullptr;
  float* so = p.s_out != nullptr ? p.s_out + (size_t)s * p.Hv * per : nullptr;
  const float* decay = p.seg_decay + (size_t)(seg - sj) * p.Hv + h;   // of this sequence's segments
#pragma unroll
  for (int t = 0; t < NST; ++t)
#pragma unroll
    for (int n = 0; n < NT; ++n) S[t][n] = f32x4{0.f, 0.f, 0.f, 0.f};
  if (sj == 0 && s0 != nullptr) {
    // kOut takes kState's copy: in place, the initial state may be overwritten by
    // the final one, which another workgroup writes
#pragma unroll
    for (int t = 0; t < NST; ++t)
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        if constexpr (PASS == Pass::kOut) {
          S[t][n] = *slot_at(p.max_segs + s, t, n);
        } else {
#pragma unroll
          for (int e = 0; e < 4; ++e) S[t][n][e] = s0[state_at(t, n, e)];
          if constexpr (STATE) *slot_at(p.max_segs + s, t, n) = S[t][n];
        }
      }
  }
  if constexpr (PASS == Pass::kOut) {
    // the state before this segment, from those of the segments before it (the
    // first of which includes the initial state), and after the last the final one
    constexpr int AHEAD = 4, TG = NST * NT > 8 ? 8 / NT : NST;   // 8 tiles of 4 segments in flight
#pragma unroll
    for (int tg = 0; tg < NST; tg += TG) {
      for (int j0 = 0; j0 < sj; j0 += AHEAD) {
        f32x4 own[AHEAD][TG][NT];
#pragma unroll
        for (int j = 0; j < AHEAD; ++j)
          if (j0 + j < sj)
#pragma unroll
            for (int t = 0; t < TG; ++t)
#pragma unroll
              for (int n = 0; n < NT; ++n) own[j][t][n] = *seg_at(j0 + j, tg + t, n);
#pragma unroll
        for (int j = 0; j < AHEAD; ++j)
          if (j0 + j < sj) {
            const float f = decay[(size_t)(j0 + j) * p.Hv];
#pragma unroll
            for (int t = 0; t < TG; ++t)
#pragma unroll
              for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int e = 0; e < 4; ++e)
                  S[tg + t][n][e] = j0 + j > 0 ? fmaf(f, S[tg + t][n][e], own[j][t][n][e]) : own[j][t][n][e];
          }
      }
    }
    if (sg.last && so != nullptr) {
      const float f = decay[(size_t)sj * p.Hv];
#pragma unroll
      for (int t = 0; t < NST; ++t)
#pragma unroll
        for (int n = 0; n < NT; ++n) {
          const f32x4 own = *seg_at(sj, t, n);
#pragma unroll
          for (int e = 0; e < 4; ++e) so[state_at(t, n, e)] = sj > 0 ? fmaf(f, S[t][n][e], own[e]) : own[e];
        }
    }
  }

  // A chunk's tiles on their way through registers, two chunks ahead where two
  // sets fit.  Every fetch issues the same loads (past the end those of the last
  // row), so that waiting for one set does not wait for the next.
  struct Set {
    uint4 k[NKL], q[STATE ? 1 : NKL], v[NVL];
  };
  constexpr bool DEEP = !STATE && 2 * NKL + NVL <= 8;   // the state pass: slower with it (74 us against 62)
  const uint32_t krow_b = (uint32_t)(krow * sizeof(T)), vrow_b = (uint32_t)(vrow * sizeof(T));
  const uint32_t koff = (uint32_t)(tid / KP) * krow_b, voff = (uint32_t)(tid / VP) * vrow_b;
  auto piece = [](const T* base, uint32_t off) {
    return *reinterpret_cast<const uint4*>(reinterpret_cast<const char*>(base) + off);
  };
  auto fetch = [&](int c0, Set& x) {
    c0 = min(c0, t1 - 1);
    const uint32_t last = (uint32_t)(min(C, t1 - c0) - 1);
    const T *kc = kp + (size_t)c0 * krow, *qc = qp + (size_t)c0 * krow, *vc = vp + (size_t)c0 * vrow;
#pragma unroll
    for (int i = 0; i < NKL; ++i) {
      const uint32_t off = min(koff + (uint32_t)(i * KR) * krow_b, last * krow_b) + tid % KP * 16;
      x.k[i] = piece(kc, off);
      if constexpr (!STATE) x.q[i] = piece(qc, off);
    }
#pragma unroll
    for (int i = 0; i < NVL; ++i)
      x.v[i] = piece(vc, min(voff + (uint32_t)(i * VR) * vrow_b, last * vrow_b) + tid % VP * 16);
  };
  auto stage = [&](int c0, Set& x) {
    if (t1 - c0 < C) {   // rows past the end are 0
#pragma unroll
      for (int i = 0; i < NKL; ++i) {
        const bool in = tid / KP + i * KR < t1 - c0;
        x.k[i] = in ? x.k[i] : uint4{0, 0, 0, 0};
        if constexpr (!STATE) x.q[i] = in ? x.q[i] : uint4{0, 0, 0, 0};
      }
#pragma unroll
      for (int i = 0; i < NVL; ++i) x.v[i] = tid / VP + i * VR < t1 - c0 ? x.v[i] : uint4{0, 0, 0, 0};
    }
#pragma unroll
    for (int i = 0; i < NKL; ++i) {
      const int r = tid / KP + i * KR;
      if (C * KP % THREADS == 0 || r < C) {
        *reinterpret_cast<uint4*>(&sm.k[KT::at(r, tid % KP * PER)]) = x.k[i];
        if constexpr (!STATE) *reinterpret_cast<uint4*>(&sm.q[KT::at(r, tid % KP * PER)]) = x.q[i];
      }
    }
#pragma unroll
    for (int i = 0; i < NVL; ++i) {
      const int r = tid / VP + i * VR;
      if (C * VP % THREADS == 0 || r < C) *reinterpret_cast<uint4*>(&sm.v[VT::at(r, tid % VP * PER)]) = x.v[i];
    }
  };
  // wave 0 turns log decays into decays one chunk ahead
  double gsum = 0.0;
  auto load_g = [&](int c0) {
    return lane < C && c0 + lane < t1 ? p.g[(size_t)(c0 + lane) * (size_t)p.g_stride + h] : 0.f;
  };
  float gnext = 0.f;
  Set xa, xb;
  if (t0 < t1) {
    float g0 = 0.f;
    if (wave == 0) {
      g0 = load_g(t0);
      gnext = load_g(t0 + C);
    }
    fetch(t0, xa);
    if constexpr (DEEP) fetch(t0 + C, xb);
    if (wave == 0) gsum += fill_decays<C, STATE>(g0, sm.d[0]);
    stage(t0, xa);
  }
  lds_barrier();
  // one chunk, `next` holding the one after it and `free` taking the one fetched
  auto chunk = [&](int c0, int par, Set& next, Set& free) __attribute__((always_inline)) {
    const int len = min(C, t1 - c0);
    const bool more = c0 + C < t1;
    const auto& D = sm.d[par];
    // the log decays first: once the tiles are staged they have arrived too
    const float g1 = gnext;
    if (wave == 0) gnext = load_g(c0 + 2 * C);
    fetch(c0 + (DEEP ? 2 * C : C), free);
    if (wave == 0 && more) gsum += fill_decays<C, STATE>(g1, sm.d[par ^ 1]);

    // V operands of this wave's columns
    Frag<T> vf[NTB][NT];
#pragma unroll
    for (int b = 0; b < NTB; ++b)
#pragma unroll
      for (int n = 0; n < NT; ++n)
        vf[b][n] = token_frag<T, CW>(sm.v, b, [&](int m) { return state_col(CW, tile0 + n, m); });

    f32x4 acc[STATE ? 1 : RT][NT];
    if constexpr (!STATE) {
      // this wave's tiles of the decayed scores (wave 0 has the decays to do)
      for (int it = NW - 1 - wave; it < RT * (RT + 1) / 2; it += NW) {
        const int i = it < 1 ? 0 : it < 3 ? 1 : it < 6 ? 2 : 3, j = it - i * (i + 1) / 2;   // j <= i
        f32x4 pt = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int kb = 0; kb < NKB; ++kb) {
          const Frag<T> qf = row_frag<T, DK>(sm.q, i, kb), kf = row_frag<T, DK>(sm.k, j, kb);
          if constexpr (DK >= 32) mma<T>(pt, kf, qf);
          else mma_lo<T>(pt, kf, qf);
        }
        // lane holds (key 16j + 4g + e, query 16i + i16)
        if (j < i) {
          const float row = D.row[16 * i + i16];
          const f32x4 col = *reinterpret_cast<const f32x4*>(&D.col[col_at(i) + 16 * j + 4 * g4]);
#pragma unroll
          for (int e = 0; e < 4; ++e) pt[e] *= row * col[e];
        } else {
          const float ih = D.hi[16 * i + i16], il = D.lo[16 * i + i16];
          const f32x4 jh = *reinterpret_cast<const f32x4*>(&D.hi[16 * j + 4 * g4]);
          const f32x4 jl = *reinterpret_cast<const f32x4*>(&D.lo[16 * j + 4 * g4]);
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const float d = (ih - jh[e]) + (il - jl[e]);
            pt[e] = 4 * g4 + e <= i16 ? pt[e] * __expf(d) : 0.f;
          }
        }
        // half a fragment; the last row tile's other half is 0
        float* half = &sm.p[p_frag(i, j >> 1) * 512 + 256 * (j & 1) + lane * 4];
        *reinterpret_cast<f32x4*>(half) = pt;
        if (j == i && (j & 1) == 0) *reinterpret_cast<f32x4*>(half + 256) = f32x4{0.f, 0.f, 0.f, 0.f};
      }
      // the state's part of o; fp16: each column is brought into range by a power of two
      int sh[NT];
      if constexpr (__is_same(T, _Float16)) {
#pragma unroll
        for (int n = 0; n < NT; ++n) {
          float m = 0.f;
#pragma unroll
          for (int t = 0; t < NST; ++t)
#pragma unroll
            for (int e = 0; e < 4; ++e) m = fmaxf(m, fabsf(S[t][n][e]));
          sh[n] = shift_for(max_groups(m));
        }
      }
#pragma unroll
      for (int i = 0; i < RT; ++i)
#pragma unroll
        for (int n = 0; n < NT; ++n) acc[i][n] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int b = 0; b < NKB; ++b) {
        Frag<T> sf[NT][OP];
#pragma unroll
        for (int n = 0; n < NT; ++n) {
          f32x4 lo = S[DK >= 32 ? 2 * b : 0][n], hi = {0.f, 0.f, 0.f, 0.f};
          if constexpr (DK >= 32) hi = S[2 * b + 1][n];
          if constexpr (__is_same(T, _Float16)) {
            lo = shifted(lo, sh[n]);
            hi = shifted(hi, sh[n]);
          }
          split<T, OP>(lo, hi, sf[n]);
        }
#pragma unroll
        for (int i = 0; i < RT; ++i) {
          const Frag<T> qf = row_frag<T, DK>(sm.q, i, b);
#pragma unroll
          for (int q = 0; q < OP; ++q)
#pragma unroll
            for (int n = 0; n < NT; ++n) {
              if constexpr (DK >= 32) mma<T>(acc[i][n], sf[n][q], qf);
              else mma_lo<T>(acc[i][n], sf[n][q], qf);
            }
        }
      }
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        f32x4 down = {1.f, 1.f, 1.f, 1.f};   // a lane's outputs are columns 4g.. of a tile
        if constexpr (__is_same(T, _Float16)) {
#pragma unroll
          for (int e = 0; e < 4; ++e) down[e] = ldexpf(1.f, -__shfl(sh[n], 4 * g4 + e));
        }
#pragma unroll
        for (int i = 0; i < RT; ++i) acc[i][n] *= D.eg[16 * i + i16] * down;
      }
    }

    // S = gamma S + K^T (w v)
    if (STATE || more || PASS == Pass::kWhole) {
      float x[NTB][NT][8];
      float m[NT] = {};   // fp16: each column is brought into range by a power of two
#pragma unroll
      for (int b = 0; b < NTB; ++b) {
        const f32x4 w0 = *reinterpret_cast<const f32x4*>(&D.w[32 * b + 4 * g4]);
        const f32x4 w1 = *reinterpret_cast<const f32x4*>(&D.w[32 * b + 16 + 4 * g4]);
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            x[b][n][j] = (j < 4 ? w0[j & 3] : w1[j & 3]) * frag_get<T>(vf[b][n], j);
            if constexpr (__is_same(T, _Float16)) m[n] = fmaxf(m[n], fabsf(x[b][n][j]));
          }
      }
      int sh[NT];
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        float gamma = D.gamma[0];
        if constexpr (__is_same(T, _Float16)) {
          sh[n] = shift_for(max_groups(m[n]));
          gamma = ldexpf(gamma, sh[n]);
        }
#pragma unroll
        for (int t = 0; t < NST; ++t) S[t][n] *= gamma;
      }
#pragma unroll
      for (int b = 0; b < NTB; ++b) {
        Frag<T> part[NT][NP];
#pragma unroll
        for (int n = 0; n < NT; ++n) {
          if constexpr (__is_same(T, _Float16)) {
#pragma unroll
            for (int j = 0; j < 8; ++j) x[b][n][j] = ldexpf(x[b][n][j], sh[n]);
          }
          split<T, NP>(x[b][n], part[n]);
        }
#pragma unroll
        for (int t = 0; t < NST; ++t) {
          const Frag<T> kt = token_frag<T, DK>(sm.k, b, [&](int r) { return state_row<DK>(t, r); });
#pragma unroll
          for (int q = 0; q < NP; ++q)
#pragma unroll
            for (int n = 0; n < NT; ++n) mma<T>(S[t][n], kt, part[n][q]);
        }
      }
      if constexpr (__is_same(T, _Float16)) {
#pragma unroll
        for (int t = 0; t < NST; ++t)
#pragma unroll
          for (int n = 0; n < NT; ++n) S[t][n] = shifted(S[t][n], -sh[n]);
      }
    }
    lds_barrier();   // the tiles are read, P is written
    if (more) stage(c0 + C, next);

    // V^T P^T runs over whole blocks of 32 tokens with P = 0 after the query: 0 times an
    // infinity or a NaN would carry it back to the queries before it.  Such values (rare;
    // found by a product with 0) are taken out of V here, and what they reach is set to NaN
    // below.
    uint64_t lost = 0;
    uint32_t lost_v[NTB][NT];   // bit j: slot j of this lane
    if constexpr (!STATE) {
      f32x4 zero = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int b = 0; b < NTB; ++b)
#pragma unroll
        for (int n = 0; n < NT; ++n) mma<T>(zero, vf[b][n], zero_frag<T>());
      lost = __ballot(zero[0] + zero[1] + zero[2] + zero[3] != 0.f);
      if (__builtin_expect(lost != 0, 0)) {
#pragma unroll
        for (int b = 0; b < NTB; ++b)
#pragma unroll
          for (int n = 0; n < NT; ++n) {
            lost_v[b][n] = 0;
            const Frag<T> raw = vf[b][n];
            vf[b][n] = make_slots<T>([&](int j) {
              const float x = frag_get<T>(raw, j);
              const bool fine = fabsf(x) < __builtin_inff();
              lost_v[b][n] |= (fine ? 0u : 1u) << j;
              return fine ? x : 0.f;
            });
          }
      }
    }
    if constexpr (!STATE) {
      T* orow = static_cast<T*>(p.o) + ((size_t)c0 + i16) * vrow + (size_t)h * p.dv + slice * CW;
#pragma unroll
      for (int i = 0; i < RT; ++i) {
        f32x4 pt[NTB][2];
#pragma unroll
        for (int b = 0; b <= i / 2; ++b)
#pragma unroll
          for (int e = 0; e < 2; ++e)
            pt[b][e] = *reinterpret_cast<const f32x4*>(&sm.p[p_frag(i, b) * 512 + 256 * e + lane * 4]);
        // fp16: each query's scores are brought into range by a power of two
        int sh = 0;
        if constexpr (__is_same(T, _Float16)) {
          float m = 0.f;
#pragma unroll
          for (int b = 0; b <= i / 2; ++b)
#pragma unroll
            for (int e = 0; e < 4; ++e) m = fmaxf(m, fmaxf(fabsf(pt[b][0][e]), fabsf(pt[b][1][e])));
          sh = shift_for(max_groups(m));
        }
        f32x4 pv[NT];
#pragma unroll
        for (int n = 0; n < NT; ++n) pv[n] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int b = 0; b <= i / 2; ++b) {
          Frag<T> pf[OP];
          if constexpr (__is_same(T, _Float16)) split<T, OP>(shifted(pt[b][0], sh), shifted(pt[b][1], sh), pf);
          else split<T, OP>(pt[b][0], pt[b][1], pf);
#pragma unroll
          for (int q = 0; q < OP; ++q)
#pragma unroll
            for (int n = 0; n < NT; ++n) mma<T>(pv[n], vf[b][n], pf[q]);
        }
#pragma unroll
        for (int n = 0; n < NT; ++n) acc[i][n] += __is_same(T, _Float16) ? shifted(pv[n], -sh) : pv[n];
        if (__builtin_expect(lost != 0, 0)) {   // counts the values taken out up to each query
          int last = lane;
          asm volatile("" : "+v"(last));        // (its masks are not kept in registers over the chunks)
          last = 16 * i + (last & 15) - 4 * (last >> 4);
#pragma unroll
          for (int n = 0; n < NT; ++n) {
            f32x4 hits = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int b = 0; b <= i / 2; ++b)
              mma<T>(hits, make_slots<T>([&](int j) { return lost_v[b][n] >> j & 1 ? 1.f : 0.f; }),
                     make_slots<T>([&](int j) { return 32 * b + (j < 4 ? j : 12 + j) <= last ? 1.f : 0.f; }));
#pragma unroll
            for (int e = 0; e < 4; ++e)
              if (hits[e] > 0.f) acc[i][n][e] = __builtin_nanf("");
          }
        }
        // lane holds token 16i + i16, columns state_col(4g..4g+3) of each tile
        if (16 * i + i16 < len) {
          T* at = orow + (size_t)(16 * i) * vrow;
          if constexpr (NT == 2 && sizeof(T) == 2) {
            const Frag<T> f = make_frag<T>(p.scale * acc[i][0], p.scale * acc[i][1]);
            store_frag_native<T>(at + state_col(CW, tile0, 4 * g4), f);
          } else {
#pragma unroll
            for (int n = 0; n < NT; ++n) {
              const f32x4 x = p.scale * acc[i][n];
              store4<T>(at + state_col(CW, tile0 + n, 4 * g4), x[0], x[1], x[2], x[3]);
            }
          }
        }
      }
    }
    lds_barrier();
  };
  Set& other = DEEP ? xb : xa;
  for (int c0 = t0; c0 < t1; c0 += 2 * C) {
    chunk(c0, 0, other, xa);
    if (c0 + C < t1) chunk(c0 + C, 1, xa, other);
  }

  if constexpr (STATE) {
    if (tid == 0 && slice == 0) p.seg_decay[(size_t)seg * p.Hv + h] = expf((float)gsum);
#pragma unroll
    for (int t = 0; t < NST; ++t)
#pragma unroll
      for (int n = 0; n < NT; ++n) *seg_at(sj, t, n) = S[t][n];
  } else if constexpr (PASS == Pass::kWhole) {
    if (so != nullptr) {
#pragma unroll
      for (int t = 0; t < NST; ++t)
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int e = 0; e < 4; ++e) so[state_at(t, n, e)] = S[t][n][e];
    }
  }
}

template <typename T, int C, int DK, int NT, int NW, Pass P>
static hipError_t run_pass(KernelId id, const LinearArgs& a, hipStream_t s) {
  const int64_t units = ((int64_t)a.max_segs * a.Hq + 7) / 8 * 8;
  const int64_t share = (a.Hv / a.Hq) * (a.dv / (16 * NT * NW)), most = kLaunchThreads / (64 * NW) / share / 8 * 8;
  prof_begin(id, s);
  for (int64_t u = 0; u < units; u += most) {
    LinearArgs b = a;
    b.first = (int32_t)u;
    hipLaunchKernelGGL((linear_chunk_kernel<T, C, DK, NT, NW, P>), dim3((unsigned)(std::min(most, units - u) * share)),
                       dim3(64 * NW), 0, s, b);
  }
  prof_end(id, s);
  return hipGetLastError();
}

// TILES column tiles a workgroup, NT a wave in the output pass (whose chunks
// are COUT tokens), else one.
template <typename T, int DK, int TILES, int NT, int COUT>
static hipError_t launch_tiles(const LinearArgs& a, hipStream_t s) {
  constexpr int C = sizeof(T) == 2 ? 64 : 32;
  if (a.seg_tokens == 0) return run_pass<T, C, DK, 1, TILES, Pass::kWhole>(K_LIN_WHOLE, a, s);
  const hipError_t e = run_pass<T, C, DK, 1, TILES, Pass::kState>(K_LIN_STATE, a, s);
  return e == hipSuccess ? run_pass<T, COUT, DK, NT, TILES / NT, Pass::kOut>(K_LIN_OUT, a, s) : e;
}

// Up to 256 (segment, head) pairs leave CUs idle: half the columns a workgroup,
// one column tile a wave (1000 tokens x 8 heads of 128, bf16: 24 us, 31 us without).
// In fp32 the matrix units bound a workgroup, so up to 512 (20 x 150 tokens x 8 heads
// of 64 x 128: 44 us, 55 us without).  Over thirteen 16-bit lists of lengths
// 0, 128, 256, 512 pairs took 1.05, 1.03, 1.01, 1.01 of the best for each, over ten
// fp32 lists 0, 256, 512, 700 took 1.05, 1.02, 1.01, 1.01.
template <typename T, int DK, int DV>
static hipError_t launch_d(const LinearArgs& a, hipStream_t s) {
  if constexpr (DV >= 64) {
    constexpr int COUT = sizeof(T) == 2 ? 64 : 32;
    if ((int64_t)a.max_segs * a.Hv <= (sizeof(T) == 4 ? 512 : 256))
      return launch_tiles<T, DK, DV / 32, 1, COUT>(a, s);
  }
  constexpr int NT = sizeof(T) == 2 && DV >= 64 ? 2 : 1;
  return launch_tiles<T, DK, DV / 16, NT, 32>(a, s);
}

template <typename T, int DK>
static hipError_t launch_dk(const LinearArgs& a, hipStream_t s) {
  switch (a.dv) {
    case 16: return launch_d<T, DK, 16>(a, s);
    case 32: return launch_d<T, DK, 32>(a, s);
    case 64: return launch_d<T, DK, 64>(a, s);
    case 128: return launch_d<T, DK, 128>(a, s);
  }
  return hipErrorInvalidValue;
}

template <typename T>
static hipError_t launch(const LinearArgs& a, hipStream_t s) {
  switch (a.dk) {
    case 16: return launch_dk<T, 16>(a, s);
    case 32: return launch_dk<T, 32>(a, s);
    case 64: return launch_dk<T, 64>(a, s);
    case 128: return launch_dk<T, 128>(a, s);
  }
  return hipErrorInvalidValue;
}

}  // namespace linear
}  // namespace gdn
