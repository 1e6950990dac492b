// Chunked prefill of linear attention with a decay for each head (kernels;
// instantiated for one input type by each gdn_linear_<type>.hip).
//
// Inside a chunk of C tokens with cumulative log decays G_i:
//
//   o_i   = scale [ e^{G_i} S^T q_i + sum_{j <= i} e^{G_i - G_j} (q_i . k_j) v_j ]
//   S_out = e^{G_C} S + sum_j e^{G_C - G_j} k_j v_j^T
//
// A workgroup walks the chunks of one (segment, value head) with the fp32 state
// in the registers of its waves: each wave owns all dk rows of its own 16*NT
// columns, so the waves share only the staged q, k, v tiles.  Everything is
// 16x16 MFMA tiles:
//   * S is carried in accumulators; two of its tiles are directly the B operand
//     of Q*S (their dk rows permuted inside each 32-row block so that Q's and
//     K's operands are contiguous 16-byte reads);
//   * P^T = K Q^T comes out as the A operand of P*V without a shuffle, at the
//     price that each wave computes the (lower) scores itself;
//   * K^T and V operands (contraction over tokens) come from transpose reads of
//     the row-major tiles.
// The state's update uses e^{G_C - G_j} v_j split into parts of the input type
// (three for bf16, two scaled ones for fp16), so the carried state keeps fp32
// accuracy; the state and the scores are rounded to 16 bits where they are
// operands of o.
//
// Log decays are summed in 64 bits and kept as a coarse part (a multiple of
// 1/64, whose differences are exact) and a fine part: in a long chunk of strong
// decays |G| reaches thousands while neighbouring G_i - G_j are small.  A decay
// below e^-128 is 0 in fp32, so g is clamped there and -infinity needs no
// special case.
#pragma once

#include "gdn_device.h"
#include "gdn_internal.h"
#include "gdn_mfma.h"

namespace gdn {
namespace linear {

typedef short s16x4 __attribute__((ext_vector_type(4)));

// Within each group of 16 lanes, lane i receives element i % 4 of the 8-byte
// pieces addressed by lanes 4j + i / 4, j = 0..3 (as its element j).
__device__ __forceinline__ s16x4 lds_read_tr(const void* p) {
  return __builtin_amdgcn_ds_read_tr16_b64_v4i16((__attribute__((address_space(3))) s16x4*)p);
}

template <typename T> constexpr int kChunk = sizeof(T) == 2 ? 64 : 32;

__device__ __forceinline__ float max_all(float x) {   // over the wave
#pragma unroll
  for (int d = 1; d < 64; d *= 2) x = fmaxf(x, __shfl_xor(x, d));
  return x;
}

// Exponent shift that brings |x| <= m into [2^13, 2^15) (0 for m = 0 or not finite).
__device__ __forceinline__ int shift_for(float m) {
  if (!(m > 0.f) || m > 3.0e38f) return 0;
  const int e = 14 - ilogbf(m);
  return e < -100 ? -100 : (e > 100 ? 100 : e);
}

// Sequence and token range of segment `seg` (false past the last one).
__device__ __forceinline__ bool segment_range(const LinearArgs& p, int seg, int& s, int& t0, int& t1, bool& last) {
  last = true;
  if (p.seg_tokens == 0) {
    s = seg;
    seq_range(p.cu, p.T, p.total, s, t0, t1);
    return true;
  }
  const int L = p.seg_tokens;
  if (p.cu == nullptr) {
    const int per = (p.T + L - 1) / L;
    s = seg / per;
    const int first = s * p.T + (seg % per) * L;
    t0 = first;
    t1 = min(first + L, (s + 1) * p.T);
    return true;
  }
  const int lane = threadIdx.x & 63;
  int base = 0;
  for (int s0 = 0; s0 < p.B; s0 += 64) {
    int a = 0, b = 0;
    if (s0 + lane < p.B) clamp_range(p.cu[s0 + lane], p.cu[s0 + lane + 1], p.total, a, b);
    const int n = (b - a + L - 1) / L;
    int incl = n;
#pragma unroll
    for (int d = 1; d < 64; d *= 2) {
      const int y = __shfl_up(incl, d);
      if (lane >= d) incl += y;
    }
    const uint64_t hit = __ballot(base + incl > seg);
    if (hit) {
      const int f = (int)__builtin_ctzll(hit);
      const int j = seg - (base + __shfl(incl, f) - __shfl(n, f));
      const int begin = __shfl(a, f), end = __shfl(b, f);
      s = s0 + f;
      t0 = begin + j * L;
      t1 = min(t0 + L, end);
      return true;
    }
    base += __shfl(incl, 63);
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

template <typename T, int DK, int NT, int NW>
struct Smem {
  static constexpr int C = kChunk<T>, DV = 16 * NT * NW;
  static constexpr int PAD = 16 / (int)sizeof(T);
  static constexpr int KS = DK + PAD, VS = DV + PAD;   // row strides
  __align__(16) T q[C * KS];
  __align__(16) T k[C * KS];
  __align__(16) T v[C * VS];
  __align__(16) float hi[C];     // coarse and fine part of G_i
  __align__(16) float lo[C];
  __align__(16) float w[C];      // e^{G_last - G_i}
  __align__(16) float eg[C];     // e^{G_i}
  float gamma;                   // e^{G_last}
};

// A (or, transposed, B) operand of rows 16*tile.. over dk block kb.
template <typename T, int DK>
__device__ __forceinline__ Frag<T> row_frag(const T* base, int stride, int tile, int kb) {
  const int lane = threadIdx.x & 63, i16 = lane & 15, g4 = lane >> 4;
  const T* r = base + (16 * tile + i16) * stride;
  if constexpr (DK >= 32) {
    return load_frag_8<T>(r + 32 * kb + 8 * g4);
  } else {
    Frag<T> f = zero_frag<T>();
    if constexpr (sizeof(T) == 4) {
      f.lo = *reinterpret_cast<const f32x4*>(r + 4 * g4);
    } else {
      const auto a = *reinterpret_cast<const typename Half4<T>::type*>(r + 4 * g4);
      f.v[0] = a[0]; f.v[1] = a[1]; f.v[2] = a[2]; f.v[3] = a[3];
    }
    return f;
  }
}

// Operand over the 32 tokens of block tb for column tile `c0..`: slot 8g + j is
// token 32tb + 4g + j (j < 4) or 32tb + 16 + 4g + j - 4.  `cols(m)`: column of row m.
template <typename T, typename F>
__device__ __forceinline__ Frag<T> token_frag(const T* base, int stride, int tb, F cols) {
  const int lane = threadIdx.x & 63, i16 = lane & 15, g4 = lane >> 4;
  Frag<T> f;
  if constexpr (sizeof(T) == 4) {
    const int c = cols(i16);
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      f.lo[q] = base[(32 * tb + 4 * g4 + q) * stride + c];
      f.hi[q] = base[(32 * tb + 16 + 4 * g4 + q) * stride + c];
    }
  } else {
    // lane i addresses token i / 4 and the four columns of rows 4 (i % 4) ..
    const int c = cols(4 * (i16 & 3));
    const T* a = base + (32 * tb + 4 * g4 + (i16 >> 2)) * stride + c;
    const s16x4 x = lds_read_tr(a), y = lds_read_tr(a + 16 * stride);
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

// Parts of the decayed v of a fragment: one fp32, three bf16, two fp16.
template <typename T> constexpr int kParts = sizeof(T) == 4 ? 1 : (__is_same(T, __bf16) ? 3 : 2);

template <typename T>
__device__ __forceinline__ void split(const float* x, Frag<T>* part) {
  if constexpr (sizeof(T) == 4) {
    part[0].lo = f32x4{x[0], x[1], x[2], x[3]};
    part[0].hi = f32x4{x[4], x[5], x[6], x[7]};
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      float r = x[j];
#pragma unroll
      for (int n = 0; n < kParts<T>; ++n) {
        part[n].v[j] = Elem<T>::from_f(r);
        r -= Elem<T>::to_f(part[n].v[j]);
      }
    }
  }
}

// Walks the chunks of one (segment, head).  STATE: only the segment's own state
// and decay (for the split); else the outputs, from the state before it.
template <typename T, int DK, int NT, int NW, bool STATE>
__global__ __launch_bounds__(64 * NW) void linear_chunk_kernel(LinearArgs p) {
  using SM = Smem<T, DK, NT, NW>;
  constexpr int C = SM::C, DV = SM::DV, KS = SM::KS, VS = SM::VS, THREADS = 64 * NW;
  constexpr int RT = C / 16, NTB = C / 32;                    // token tiles and 32-token blocks
  constexpr int NST = DK / 16, NKB = DK >= 32 ? DK / 32 : 1;  // state row tiles, dk blocks
  constexpr int PER = 16 / (int)sizeof(T), KP = DK / PER, VP = DV / PER;   // 16-byte pieces a row
  constexpr int NKL = (C * KP + THREADS - 1) / THREADS, NVL = (C * VP + THREADS - 1) / THREADS;
  __shared__ SM sm;

  // XCD-aware order: the value heads that share one segment's keys get ids equal mod 8
  const int G = p.Hv / p.Hq;
  const int unit = (int)(blockIdx.x >> 3) / G * 8 + (int)(blockIdx.x & 7);
  if (unit >= p.max_segs * p.Hq) return;
  const int seg = unit / p.Hq, hk = unit % p.Hq, h = hk * G + (int)(blockIdx.x >> 3) % G;
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int i16 = lane & 15, g4 = lane >> 4;
  int s, t0, t1;
  bool last;
  if (!segment_range(p, seg, s, t0, t1, last)) return;
  s = __builtin_amdgcn_readfirstlane(s);
  t0 = __builtin_amdgcn_readfirstlane(t0);
  t1 = __builtin_amdgcn_readfirstlane(t1);
  const size_t per = (size_t)DK * DV;
  const T* qp = static_cast<const T*>(p.q) + (size_t)hk * DK;
  const T* kp = static_cast<const T*>(p.k) + (size_t)hk * DK;
  const T* vp = static_cast<const T*>(p.v) + (size_t)h * DV;
  T* op = static_cast<T*>(p.o) + (size_t)h * DV;
  const int col0 = wave * 16 * NT;

  // state tile (t, n): lane holds rows 4g..4g+3 of the tile, column i16
  f32x4 S[NST][NT];
  const float* sin = nullptr;
  if constexpr (!STATE)
    sin = p.seg_tokens != 0 ? p.seg_state + ((size_t)seg * p.Hv + h) * per
          : p.s0 != nullptr ? p.s0 + (int64_t)s * p.s0_stride + (size_t)h * per : nullptr;
#pragma unroll
  for (int t = 0; t < NST; ++t)
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int e = 0; e < 4; ++e)
        S[t][n][e] = sin != nullptr ? sin[(size_t)state_row<DK>(t, 4 * g4 + e) * DV + col0 + 16 * n + i16] : 0.f;
  double gsum = 0.0;

  uint4 kreg[NKL], qreg[NKL], vreg[NVL];
  float greg = 0.f;
  auto fetch = [&](int c0) {
    const int len = min(C, t1 - c0);
#pragma unroll
    for (int i = 0; i < NKL; ++i) {
      const int x = tid + i * THREADS, r = x / KP, pc = x % KP;
      const bool in = r < len;
      const size_t off = (size_t)(c0 + (in ? r : 0)) * p.Hq * DK + pc * PER;
      kreg[i] = in ? *reinterpret_cast<const uint4*>(kp + off) : uint4{0, 0, 0, 0};
      if constexpr (!STATE) qreg[i] = in ? *reinterpret_cast<const uint4*>(qp + off) : uint4{0, 0, 0, 0};
    }
#pragma unroll
    for (int i = 0; i < NVL; ++i) {
      const int x = tid + i * THREADS, r = x / VP, pc = x % VP;
      const bool in = r < len;
      const size_t off = (size_t)(c0 + (in ? r : 0)) * p.Hv * DV + pc * PER;
      vreg[i] = in ? *reinterpret_cast<const uint4*>(vp + off) : uint4{0, 0, 0, 0};
    }
    if (tid < C) greg = tid < len ? p.g[(size_t)(c0 + tid) * (size_t)p.g_stride + h] : 0.f;
  };

  if (t0 < t1) fetch(t0);
  for (int c0 = t0; c0 < t1; c0 += C) {
    const int len = min(C, t1 - c0);
    lds_barrier();   // the last chunk's reads of the tiles are done
#pragma unroll
    for (int i = 0; i < NKL; ++i) {
      const int x = tid + i * THREADS, r = x / KP, pc = x % KP;
      if (C * KP % THREADS == 0 || r < C) {
        *reinterpret_cast<uint4*>(&sm.k[r * KS + pc * PER]) = kreg[i];
        if constexpr (!STATE) *reinterpret_cast<uint4*>(&sm.q[r * KS + pc * PER]) = qreg[i];
      }
    }
#pragma unroll
    for (int i = 0; i < NVL; ++i) {
      const int x = tid + i * THREADS, r = x / VP, pc = x % VP;
      if (C * VP % THREADS == 0 || r < C) *reinterpret_cast<uint4*>(&sm.v[r * VS + pc * PER]) = vreg[i];
    }
    if (wave == 0) {   // cumulative log decays
      double x = lane < C ? (double)(greg < -128.f ? -128.f : greg) : 0.0;
#pragma unroll
      for (int d = 1; d < C; d *= 2) {
        const double y = __shfl_up(x, d);
        if (lane >= d) x += y;
      }
      const double end = __shfl(x, C - 1);
      gsum += end;
      if (lane < C) {
        const float hi = rintf((float)x * 64.f) * 0.015625f;
        sm.hi[lane] = hi;
        sm.lo[lane] = (float)(x - (double)hi);
        sm.w[lane] = expf((float)(end - x));
        sm.eg[lane] = expf((float)x);
      }
      if (lane == 0) sm.gamma = expf((float)end);
    }
    lds_barrier();
    if (c0 + C < t1) fetch(c0 + C);

    // V operands of this wave's columns
    Frag<T> vf[NTB][NT];
#pragma unroll
    for (int b = 0; b < NTB; ++b)
#pragma unroll
      for (int n = 0; n < NT; ++n)
        vf[b][n] = token_frag<T>(sm.v, VS, b, [&](int m) { return col0 + 16 * n + m; });

    if constexpr (!STATE) {
      // state operands; fp16 ones scaled by a power of two into its range
      int sh = 0;
      if constexpr (__is_same(T, _Float16)) {
        float m = 0.f;
#pragma unroll
        for (int t = 0; t < NST; ++t)
#pragma unroll
          for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int e = 0; e < 4; ++e) m = fmaxf(m, fabsf(S[t][n][e]));
        sh = shift_for(max_all(m));
      }
      const float up = ldexpf(1.f, sh), down = ldexpf(1.f, -sh);
      Frag<T> sf[NKB][NT];
#pragma unroll
      for (int b = 0; b < NKB; ++b)
#pragma unroll
        for (int n = 0; n < NT; ++n) {
          f32x4 lo = S[DK >= 32 ? 2 * b : 0][n], hi = DK >= 32 ? S[DK >= 32 ? 2 * b + 1 : 0][n] : f32x4{0.f, 0.f, 0.f, 0.f};
          if constexpr (__is_same(T, _Float16)) {
            lo *= up;
            hi *= up;
          }
          sf[b][n] = make_frag<T>(lo, hi);
        }
#pragma unroll
      for (int i = 0; i < RT; ++i) {
        Frag<T> qf[NKB];
#pragma unroll
        for (int b = 0; b < NKB; ++b) qf[b] = row_frag<T, DK>(sm.q, KS, i, b);
        f32x4 acc[NT];
        const f32x4 eg = *reinterpret_cast<const f32x4*>(&sm.eg[16 * i + 4 * g4]);
#pragma unroll
        for (int n = 0; n < NT; ++n) {
          acc[n] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
          for (int b = 0; b < NKB; ++b) {
            if constexpr (DK >= 32) mma<T>(acc[n], qf[b], sf[b][n]);
            else mma_lo<T>(acc[n], qf[b], sf[b][n]);
          }
          acc[n] *= eg * down;
        }
        const float ih = sm.hi[16 * i + i16], il = sm.lo[16 * i + i16];
#pragma unroll
        for (int b = 0; b <= i / 2; ++b) {
          f32x4 pt[2];
#pragma unroll
          for (int u = 0; u < 2; ++u) {
            const int j = 2 * b + u;
            pt[u] = f32x4{0.f, 0.f, 0.f, 0.f};
            if (j > i) continue;
#pragma unroll
            for (int kb = 0; kb < NKB; ++kb) {
              const Frag<T> kf = row_frag<T, DK>(sm.k, KS, j, kb);
              if constexpr (DK >= 32) mma<T>(pt[u], kf, qf[kb]);
              else mma_lo<T>(pt[u], kf, qf[kb]);
            }
            // lane holds (key 16j + 4g + e, query 16i + i16)
            const f32x4 jh = *reinterpret_cast<const f32x4*>(&sm.hi[16 * j + 4 * g4]);
            const f32x4 jl = *reinterpret_cast<const f32x4*>(&sm.lo[16 * j + 4 * g4]);
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const float d = (ih - jh[e]) + (il - jl[e]);
              pt[u][e] = j < i || 4 * g4 + e <= i16 ? pt[u][e] * __expf(d) : 0.f;
            }
          }
          const Frag<T> pf = make_frag<T>(pt[0], pt[1]);
#pragma unroll
          for (int n = 0; n < NT; ++n) mma<T>(acc[n], pf, vf[b][n]);
        }
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const int r = 16 * i + 4 * g4 + e;
            if (r < len)
              op[(size_t)(c0 + r) * p.Hv * DV + col0 + 16 * n + i16] = Elem<T>::from_f(p.scale * acc[n][e]);
          }
      }
    }

    // S = gamma S + K^T (w v)
    float x[NTB][NT][8];
    float m = 0.f;
#pragma unroll
    for (int b = 0; b < NTB; ++b) {
      const f32x4 w0 = *reinterpret_cast<const f32x4*>(&sm.w[32 * b + 4 * g4]);
      const f32x4 w1 = *reinterpret_cast<const f32x4*>(&sm.w[32 * b + 16 + 4 * g4]);
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          x[b][n][j] = (j < 4 ? w0[j & 3] : w1[j & 3]) * frag_get<T>(vf[b][n], j);
          m = fmaxf(m, fabsf(x[b][n][j]));
        }
    }
    float up = 1.f, down = 1.f;
    if constexpr (__is_same(T, _Float16)) {
      const int sh = shift_for(max_all(m));
      up = ldexpf(1.f, sh);
      down = ldexpf(1.f, -sh);
    }
    const float gamma = sm.gamma * up;
#pragma unroll
    for (int t = 0; t < NST; ++t)
#pragma unroll
      for (int n = 0; n < NT; ++n) S[t][n] *= gamma;
#pragma unroll
    for (int b = 0; b < NTB; ++b) {
      Frag<T> part[NT][kParts<T>];
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        if constexpr (__is_same(T, _Float16)) {
#pragma unroll
          for (int j = 0; j < 8; ++j) x[b][n][j] *= up;
        }
        split<T>(x[b][n], part[n]);
      }
#pragma unroll
      for (int t = 0; t < NST; ++t) {
        const Frag<T> kt = token_frag<T>(sm.k, KS, b, [&](int r) { return state_row<DK>(t, r); });
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int q = 0; q < kParts<T>; ++q) mma<T>(S[t][n], kt, part[n][q]);
      }
    }
    if constexpr (__is_same(T, _Float16)) {
#pragma unroll
      for (int t = 0; t < NST; ++t)
#pragma unroll
        for (int n = 0; n < NT; ++n) S[t][n] *= down;
    }
  }

  float* sout = nullptr;
  if constexpr (STATE) {
    sout = p.seg_state + ((size_t)seg * p.Hv + h) * per;
    if (tid == 0) p.seg_decay[(size_t)seg * p.Hv + h] = gsum;
  } else if (p.seg_tokens == 0 && p.s_out != nullptr) {
    sout = p.s_out + ((size_t)s * p.Hv + h) * per;
  }
  if (sout != nullptr) {
#pragma unroll
    for (int t = 0; t < NST; ++t)
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int e = 0; e < 4; ++e)
          sout[(size_t)state_row<DK>(t, 4 * g4 + e) * DV + col0 + 16 * n + i16] = S[t][n][e];
  }
}

// Replaces each segment's own state by the state before it, and writes the
// final states: element-wise recurrences over the segments of a sequence.
template <typename T>
__global__ __launch_bounds__(256) void linear_carry_kernel(LinearArgs p) {
  const size_t per = (size_t)p.dk * p.dv;
  const int nblk = (int)((per / 4 + 255) / 256);
  const int blk = (int)(blockIdx.x % nblk), pair = (int)(blockIdx.x / nblk);
  const int s = pair / p.Hv, h = pair % p.Hv, L = p.seg_tokens;
  int first = 0, n = 0;
  if (p.cu == nullptr) {
    n = (p.T + L - 1) / L;
    first = s * n;
  } else {
    const int lane = threadIdx.x & 63;
    for (int i0 = 0; i0 <= s; i0 += 64) {
      int a = 0, b = 0;
      if (i0 + lane <= s) clamp_range(p.cu[i0 + lane], p.cu[i0 + lane + 1], p.total, a, b);
      int c = (b - a + L - 1) / L;
      const int mine = __shfl(c, s - i0 < 64 ? s - i0 : 63);
#pragma unroll
      for (int d = 1; d < 64; d *= 2) c += __shfl_xor(c, d);
      first += c;
      n = mine;
    }
    first -= n;
  }
  n = min(n, p.max_segs - first);
  const size_t e = ((size_t)blk * 256 + threadIdx.x) * 4;
  if (e >= per) return;
  f32x4 S = {0.f, 0.f, 0.f, 0.f};
  if (p.s0 != nullptr) S = *reinterpret_cast<const f32x4*>(p.s0 + (int64_t)s * p.s0_stride + (size_t)h * per + e);
  for (int j = 0; j < n; ++j) {
    const size_t at = (size_t)(first + j) * p.Hv + h;
    f32x4* x = reinterpret_cast<f32x4*>(p.seg_state + at * per + e);
    const f32x4 own = *x;
    *x = S;
    const float a = expf((float)p.seg_decay[at]);
#pragma unroll
    for (int i = 0; i < 4; ++i) S[i] = fmaf(a, S[i], own[i]);
  }
  if (p.s_out != nullptr) *reinterpret_cast<f32x4*>(p.s_out + ((size_t)s * p.Hv + h) * per + e) = S;
}

template <typename T, int DK, int NT, int NW>
static hipError_t launch_w(const LinearArgs& a, hipStream_t s) {
  const long long units = (long long)a.max_segs * a.Hq;
  const dim3 grid((unsigned)((units + 7) / 8 * 8 * (a.Hv / a.Hq))), block(64 * NW);
  hipError_t e;
  if (a.seg_tokens != 0) {
    prof_begin(K_LIN_STATE, s);
    hipLaunchKernelGGL((linear_chunk_kernel<T, DK, NT, NW, true>), grid, block, 0, s, a);
    prof_end(K_LIN_STATE, s);
    if ((e = hipGetLastError()) != hipSuccess) return e;
    prof_begin(K_LIN_CARRY, s);
    const long long nblk = ((long long)a.dk * a.dv / 4 + 255) / 256;
    hipLaunchKernelGGL((linear_carry_kernel<T>), dim3((unsigned)(nblk * a.B * a.Hv)), dim3(256), 0, s, a);
    prof_end(K_LIN_CARRY, s);
    if ((e = hipGetLastError()) != hipSuccess) return e;
  }
  prof_begin(K_LIN_OUT, s);
  hipLaunchKernelGGL((linear_chunk_kernel<T, DK, NT, NW, false>), grid, block, 0, s, a);
  prof_end(K_LIN_OUT, s);
  return hipGetLastError();
}

template <typename T, int DK>
static hipError_t launch_dk(const LinearArgs& a, hipStream_t s) {
  switch (a.dv) {
    case 16: return launch_w<T, DK, 1, 1>(a, s);
    case 32: return launch_w<T, DK, 1, 2>(a, s);
    case 64: return launch_w<T, DK, 1, 4>(a, s);
    case 128: return launch_w<T, DK, 2, 4>(a, s);
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
