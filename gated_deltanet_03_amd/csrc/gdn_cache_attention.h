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
// m follows the maximum only when that has grown by more than 2^8 (fp16: 2^6): exp(s - m) is then at most that, which
// 16-bit operands hold, and most tiles leave the output accumulators alone.  In fp16 weights are taken 2^7 times as
// large, so up to 2^13 of 2^16: its numbers end at 2^-24, and many keys with small weights may outweigh the largest
// (131072 keys of 2^-25 of it hold 2^-8 of the sum, and were 0); so the smallest is 2^-31 of the maximum's weight.
// 2048 tokens over 16384 keys, 32 heads of 64: 358 us without, 360 so, 361 with growth of 2^4 and weights 2^8 times.
#pragma once

#include <algorithm>
#include <type_traits>

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
               : "memory", "m0");
}
__device__ __forceinline__ void dma16(const void* src, uint32_t lds) {
  asm volatile("s_mov_b32 m0, %1\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %0, off" ::"v"(src), "s"(lds) : "memory", "m0");
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
__device__ __forceinline__ constexpr int key_swizzle(int r) {
  if constexpr (PPR >= 16) return r & 15;
  else if constexpr (PPR == 8) return ((r >> 1) & 3) | (((r ^ (r >> 3)) & 1) << 2);
  else return (r >> 1) & 3;
}
// Values, 16-bit: transposed reads of 4 rows x 32 bytes by 16 lanes, x 64 bytes by 32.
// Values, fp32: 4-byte reads of 128 bytes of rows r and r + 4.
template <int ES, int PPR>
__device__ __forceinline__ constexpr int value_swizzle(int r) {
  if constexpr (ES == 4) return PPR >= 16 ? ((r >> 2) & 1) << 3 : 0;
  else if constexpr (PPR >= 16) return (0xca60 >> ((r & 3) << 2)) & 15;   // 0, 6, 10, 12
  else if constexpr (PPR == 8) return (r & 3) << 1;
  else return ((r >> 1) & 1) << 1;
}

__device__ __forceinline__ int scalar(int x) { return __builtin_amdgcn_readfirstlane(x); }
__device__ __forceinline__ int lane_value(int x, int lane) { return __builtin_amdgcn_readlane(x, lane); }

// x / n and its ceiling where that is below 2^20: the reciprocal's product is less than one off.
__device__ __forceinline__ int quotient(int x, int n) {
  const int q = (int)((float)x * __builtin_amdgcn_rcpf((float)n)), r = x - q * n;
  return q + (r >= n) - (r < 0);
}
__device__ __forceinline__ int quotient_up(int x, int n) { return quotient(x + n - 1, n); }

// Inclusive prefix sum over the wave's lanes.
__device__ __forceinline__ int wave_scan(int x) {
  x += __builtin_amdgcn_update_dpp(0, x, 0x111, 0xf, 0xf, false);   // row_shr:1
  x += __builtin_amdgcn_update_dpp(0, x, 0x112, 0xf, 0xf, false);
  x += __builtin_amdgcn_update_dpp(0, x, 0x114, 0xf, 0xf, false);
  x += __builtin_amdgcn_update_dpp(0, x, 0x118, 0xf, 0xf, false);
  x += __builtin_amdgcn_update_dpp(0, x, 0x142, 0xa, 0xf, false);   // row_bcast:15 into rows 1 and 3
  x += __builtin_amdgcn_update_dpp(0, x, 0x143, 0xc, 0xf, false);   // row_bcast:31 into rows 2 and 3
  return x;
}
__device__ __forceinline__ int wave_max(int x) {   // of numbers that are not negative
  x = max(x, __builtin_amdgcn_update_dpp(0, x, 0x111, 0xf, 0xf, false));
  x = max(x, __builtin_amdgcn_update_dpp(0, x, 0x112, 0xf, 0xf, false));
  x = max(x, __builtin_amdgcn_update_dpp(0, x, 0x114, 0xf, 0xf, false));
  x = max(x, __builtin_amdgcn_update_dpp(0, x, 0x118, 0xf, 0xf, false));
  x = max(x, __builtin_amdgcn_update_dpp(0, x, 0x142, 0xa, 0xf, false));
  x = max(x, __builtin_amdgcn_update_dpp(0, x, 0x143, 0xc, 0xf, false));
  return lane_value(x, 63);
}
__device__ __forceinline__ int wave_sum(int x) { return lane_value(wave_scan(x), 63); }

// How the work of one head is laid out.
//
// The tiles of all sequences lie on one line, a tile about as long as the keys it sees and what starting one costs,
// in units of 2^unit keys that the host chooses so that the line is shorter than 2^30: v_i = first + step * i for
// tile i of a sequence, never more than twice the table's keys. The first workgroups take whole tiles, one each; what
// is left of the line is cut into `shares` even pieces, whatever the sequences' lengths are: the rest of one tile, whole
// tiles, the beginning of one more. Pieces that are not whole tiles go to the workspace and are joined.
//
// Nothing is cut where that would end no later.  Whole tiles end with the longest one, or with as many rounds as
// there are tiles for a share, of average ones; cut ones with an even share and what the pieces and their join cost:
// 3 us with few rows, 16 us with many where a share is one piece, else 40 us (128 rows of 128 in fp32 are 64 KB,
// written and read again by every share).  Few rows wait for memory, which fewer workgroups than fit keep busy too:
// there only the longest tile counts (256 tokens over 100 to 1103 keys of 8 heads of 128, bf16: 145 us cut, 121
// whole).  A prompt of 2000 tokens, 32 on 8 heads of 128, bf16: 94 us cut, 68 whole; 1000 tokens over 4000 keys: 94
// us cut, 108 whole; 4000 over 8000: 432 cut, 408 whole.
//
// Many rows: workgroups that walk one head's keys side by side read them from the cache they share, and pieces that
// begin anywhere do not (16384 keys of 8 heads, 512 tiles of 128 rows, bf16: 677 us cut evenly, 563 whole). So whole
// rounds of `shares` tiles stay whole, the last ones of a sequence, which see the most keys, first; with three rounds
// or more nothing is cut. Tiles longer than 5/4 of an even share are always cut, so that one long sequence does not
// outlast all others.
//
// Where shares are many times the tiles, tiles are drawn out to whole numbers of shares: a share is then one piece,
// and a second one's start (plan, page numbers, first loads: 6 us) costs more than the longer shares. A share is a
// multiple `run` of the step there, so that tile i has ceil((ceil(first / step) + i) / run) of them, whose sum and
// its inverse have a closed form.
//
// Borders between shares that come within a 16th of a share of a tile's end are moved there.
struct Piece {
  int s, b, L, lens, tile;
  int at, length;          // the tile's start and length on the line
};

// What all workgroups of a call agree on.
struct Shares {
  int longest;             // of the tiles that may stay whole
  int whole;               // tiles that stay whole
  int rest, share;         // length of the line that is left, and of a share of it
  int drawn;               // tiles are whole numbers of shares: of how many steps a share is, 0: they are not
};

// What the work is laid out from.
struct Work {
  const int32_t* cu;
  const int32_t* lens;
  int N, T, total, G, room, window, tiles, shares, unit, extra_drawn, extra_even;
};

template <bool FEW>
struct Line {
  static constexpr int ROWS = FEW ? kFewRows : kManyRows;
  const Work& a;
  int base;                // sequences base .. base + 63 are loaded, one a lane
  int b, L, lens, tiles;
  int first, step;

  __device__ __forceinline__ explicit Line(const Work& work) : a(work), base(-1) {}

  __device__ __forceinline__ void load(int s0) {
    if (s0 == base) return;
    base = s0;
    const int s = s0 + (int)(threadIdx.x & 63);
    b = L = lens = tiles = first = step = 0;
    if (s < a.N) {
      int e;
      seq_range(a.cu, a.T, a.total, s, b, e);
      L = e - b;
      lens = min(max(a.lens[s], 0), 1 << 30);     // (below 0 no token has a place, as with 0)
      tiles = (int)(((int64_t)L * a.G + ROWS - 1) / ROWS);
      const int old = min(max(lens - L, 0), a.room), more = ROWS / a.G + 1;
      const bool inside = a.window > 0 && a.window < old;
      first = (((inside ? a.window : old) + 64 + more) >> a.unit) + 1;
      step = inside ? 0 : more >> a.unit;
      // No tile sees more keys than the table has; `step`, rounded up, goes beyond that by itself (at most twice as far
      // in 128 rows), and new tokens behind the table's end without a limit: then all tiles count as the table.
      const int most = ((a.room + 64 + more) >> a.unit) + 1;
      if (first + (int64_t)step * (tiles - 1) > 2 * most) first = most, step = 0;
    }
  }

  // i tiles of a sequence.
  static __device__ __forceinline__ int tiles_length(int first, int step, int i) {
    return first * i + (int)((int64_t)step * (((int64_t)i * (i - 1)) >> 1));
  }
  // The lane's sequence without its last `kept` tiles.
  __device__ __forceinline__ int length(int kept, const Shares& sh) const {
    if (sh.drawn) {
      if (__ballot(tiles > 1) == 0) return tiles * Drawn(first, step, sh).q * sh.share;
      return tiles > 0 ? Drawn(first, step, sh).shares(tiles) * sh.share : 0;
    }
    return tiles_length(first, step, tiles - kept);
  }

  // Drawn out: tile i of a sequence has q + floor((i + r) / run) shares.
  struct Drawn {
    int run, q, r;
    __device__ __forceinline__ Drawn(int first, int step, const Shares& sh) : run(1 << 30), r(0) {
      if (step != 0) {
        const int a = up(first, step) + sh.drawn - 1;
        run = sh.drawn, q = quotient(a, run), r = a - q * run;
      } else {
        q = quotient_up(first, sh.share);
      }
    }
    // The shares of i tiles; g(r + i) of them lie in whole runs.
    __device__ __forceinline__ int shares(int i) const {
      const int g = quotient(r + i, run);
      return i * q + run * (g * (g - 1) / 2) + (r + i - g * run) * g;
    }
    // The tile in which share x lies: of those from tile run * g - r on with q + g shares each, g nearly by the
    // quadratic's root, then exactly.
    __device__ __forceinline__ int tile(int x) const {
      auto before = [&](int g) { return (run * g - r) * q + run * (g * (g - 1) / 2); };
      int g = 0;
      if (run < 1 << 30) {
        const float v = (float)q - 0.5f, w = 2.f * (float)(r * q + x) * __builtin_amdgcn_rcpf((float)run);
        g = max((int)(__builtin_amdgcn_sqrtf(v * v + w) - v), 0);
        while (g > 0 && before(g) > x) --g;
        while (before(g + 1) <= x) ++g;
      }
      return run * g - r + quotient(x - before(g), q + g);
    }
  };
  static __device__ __forceinline__ int up(int x, int n) { return (int)(((uint32_t)x + (uint32_t)n - 1) / (uint32_t)n); }

  // How many of the lane's tiles may stay whole, however many others do.
  __device__ __forceinline__ int may_be_whole(int longest) const {
    return first + step * (tiles - 1) <= longest ? tiles : 0;
  }

  __device__ __forceinline__ Shares share_out() {
    Shares r{0, 0, 0, 1, 0};
    int all = 0, count = 0, longest = 0;
    for (int s = 0; s < a.N; s += 64) {
      load(s);
      all += wave_sum(tiles_length(first, step, tiles));
      count += wave_sum(min(tiles, a.tiles + 1));
      longest = max(longest, wave_max(tiles > 0 ? first + step * (tiles - 1) : 0));
      if (count > a.tiles) return r;      // offsets that overlap: more tiles than the line has room for, no work at all
    }
    const int even = up(all, a.shares), least = max((FEW ? kFewKeys : kManyKeys) >> a.unit, 1);
    r.rest = all;
    r.share = max(least, even);
    const bool drawn = count * 4 <= a.shares;
    const int extra = drawn ? a.extra_drawn : a.extra_even;
    bool none = longest <= r.share + extra;
    if constexpr (!FEW) {
      if (none && count > a.shares) {       // whole tiles take rounds of average ones, or end with short ones
        const int rounds = quotient_up(count, a.shares);
        if (up(all, count) * rounds > even + extra) {
          int brief = 0;
          for (int s = 0; s < a.N; s += 64) {
            load(s);
            brief += wave_sum(first > extra ? 0 : step > 0 ? min((extra - first) / step + 1, tiles) : tiles);
          }
          none = brief >= count - (rounds - 1) * a.shares;
        }
      }
    }
    if constexpr (FEW) {
      if (none) {
        r.longest = longest;
        r.whole = count;
        r.rest = 0;
      }
    }
    if (!none && drawn) {
      // a tile has at most (its length + a step) / share + 1 shares
      const int steps = max((ROWS / a.G + 1) >> a.unit, 1);
      r.drawn = up(max(least, up(all + count * steps, a.shares - count)), steps);
      r.share = r.drawn * steps;
      r.rest = 0;
      for (int s = 0; s < a.N; s += 64) {
        load(s);
        r.rest += wave_sum(length(0, r));
      }
    } else if constexpr (!FEW) {
      r.longest = none ? longest : even + even / 4;
      int may = 0, sure = 0;
      for (int s = 0; s < a.N; s += 64) {
        load(s);
        const int w = may_be_whole(r.longest);
        may += wave_sum(w);
        sure += wave_sum(tiles - w);
      }
      const int rounds = may / a.shares;
      r.whole = none || (sure == 0 && rounds >= 3) ? may : rounds * a.shares;
      int before = 0;
      r.rest = 0;
      for (int s = 0; s < a.N; s += 64) {
        load(s);
        const int mine = may_be_whole(r.longest), upto = before + wave_scan(mine);
        r.rest += wave_sum(length(min(max(r.whole - (upto - mine), 0), mine), r));
        before = lane_value(upto, 63);
      }
      r.share = max(least, up(r.rest, a.shares));
    }
    return r;
  }

  // The tile number `pos` of those that are whole (WHOLE; of all tiles if nothing is shared), or the sequence and tile
  // at `pos` of what is left.
  template <bool WHOLE>
  __device__ __forceinline__ bool find(const Shares& sh, int pos, Piece& p) {
    int tiles_before = 0, before = 0;
    for (int s0 = 0; s0 < a.N; s0 += 64) {
      load(s0);
      int kept = 0;
      if (a.shares == 0) {
        kept = tiles;
      } else if (!FEW || WHOLE) {     // (of few rows all are whole, or none)
        const int may = may_be_whole(sh.longest), upto = tiles_before + wave_scan(may);
        kept = min(max(sh.whole - (upto - may), 0), may);
        tiles_before = lane_value(upto, 63);
      }
      const int mine = WHOLE ? kept : length(kept, sh), upto = before + wave_scan(mine), total = lane_value(upto, 63);
      if (pos < total) {
        const int j = __ffsll((unsigned long long)__ballot(pos < upto)) - 1;
        const int rest = pos - lane_value(upto - mine, j), n = lane_value(tiles, j);
        const int cut = n - lane_value(kept, j);     // tiles that are not whole
        const int f = lane_value(first, j), st = lane_value(step, j);
        int i = 0, at = 0, length = 1;
        if constexpr (WHOLE) {
          i = max(n - 1 - rest, 0);                  // a sequence's last tiles see the most keys: first
        } else {
          if (sh.drawn) {
            const Drawn x(f, st, sh);
            length = x.q * sh.share;
            if (n > 1) {
              i = x.tile(quotient(rest, sh.share));
              at = x.shares(i) * sh.share;
              length = x.shares(i + 1) * sh.share - at;
            }
          } else {
            if (cut > 1) {        // f i + st i (i - 1) / 2 <= rest, nearly by the quadratic's root, then exactly
              float x = (float)rest * __builtin_amdgcn_rcpf((float)f);
              if (st != 0) {
                const float s = __builtin_amdgcn_rcpf((float)st), v = (float)f * s - 0.5f;
                x = __builtin_amdgcn_sqrtf(v * v + 2.f * (float)rest * s) - v;
              }
              i = min(max((int)x, 0), cut - 1);
              while (i > 0 && tiles_length(f, st, i) > rest) --i;
              while (i + 1 < cut && tiles_length(f, st, i + 1) <= rest) ++i;
            }
            at = tiles_length(f, st, i);
            length = f + st * i;
          }
        }
        p.s = s0 + j;
        p.b = lane_value(b, j);
        p.L = lane_value(L, j);
        p.lens = lane_value(lens, j);
        p.tile = i;
        p.at = pos - rest + at;
        p.length = length;
        return true;
      }
      before = total;
    }
    return false;
  }
};

// What the join of a tile cut between workgroups j - 1 and j needs: its rows, and its pieces begin .. end - 1 (of them
// the one numbered 0 is the end of share j - 1, k that of share j - 1 + k).  Nothing to join: end - begin < 2.
struct Cut {
  int b, L, tile;
  short begin, end;
};

// Borders near a tile's end lie there.
__device__ __forceinline__ int border(int x, int length, int share) {
  const int near = share >> 4;
  return x >= length ? length : (x < near ? 0 : (length - x < near ? length : x));
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
  // How far scores may grow above m, and what weights are more than exp(s - m), as powers of two.
  static constexpr bool F16 = __is_same(T, _Float16);
  static constexpr float SLACK = F16 ? 6.f : 8.f, MORE = F16 ? 7.f : 0.f;
  uint4 q[QN];
  f32x16 o[DT];
  float m, mc, l;      // m in score units, mc = m * scale - MORE (0 while m = -infinity), l of this lane's keys
  int lo, hi;          // the keys this lane's query sees: lo <= key <= hi
  int lane;

  __device__ __forceinline__ void init(int lane_) {
    lane = lane_;
#pragma unroll
    for (int t = 0; t < DT; ++t)
#pragma unroll
      for (int i = 0; i < 16; ++i) o[t][i] = 0.f;
    m = -INFINITY;
    mc = l = 0.f;
  }

  // Query row `src` (all lanes of a pair read theirs); pieces 2 s + l / 32.
  __device__ __forceinline__ void load_query(const T* src) {
    const int h = lane >> 5;
#pragma unroll
    for (int s = 0; s < QN; ++s) q[s] = *reinterpret_cast<const uint4*>(src + (2 * s + h) * E);
  }

  // Piece t of 32 keys' operand: rows r0 .. r0 + 31 of the LDS tile; and its products, added to their scores.
  __device__ __forceinline__ uint4 key_piece(const unsigned char* K, int r0, int t) const {
    const int h = lane >> 5, r = lane & 31;
    return *reinterpret_cast<const uint4*>(K + (r0 + r) * RB + (((2 * t + h) ^ key_swizzle<PPR>(r)) << 4));
  }
  __device__ __forceinline__ void add_product(f32x16& s, const uint4& k, int t) const {
    if constexpr (F32) {
      const f32x4 a = __builtin_bit_cast(f32x4, k), b = __builtin_bit_cast(f32x4, q[t]);
#pragma unroll
      for (int e = 0; e < 4; ++e) s = __builtin_amdgcn_mfma_f32_32x32x2f32(a[e], b[e], s, 0, 0, 0);
    } else {
      s = Op<T>::mma(__builtin_bit_cast(typename Op<T>::V, k), __builtin_bit_cast(typename Op<T>::V, q[t]), s);
    }
  }
  static __device__ __forceinline__ f32x16 zeros() {
    f32x16 s;
#pragma unroll
    for (int i = 0; i < 16; ++i) s[i] = 0.f;
    return s;
  }

  // Scores of 32 keys.  fp32 adds two products at a time, d / 2 roundings in a row: four sums instead of one bring the
  // error of o against 64 bits from 4.6e-7 to 2.8e-7 (d = 64) and 9.0e-7 to 3.7e-7 (256), for 1% of the time.
  // Where they are made in turn with exponentials, two: 8.4e-7 to 5.2e-7 (300 tokens over 700 keys, d = 256) for 0.3 to
  // 0.9% of the time; four would bring 3.9e-7, but cost 2 to 4% in vector operations there.
  template <int N>
  struct Sums {
    f32x16 s[N];
    __device__ __forceinline__ Sums() {
#pragma unroll
      for (int n = 0; n < N; ++n) s[n] = zeros();
    }
    __device__ __forceinline__ void join(int i) {      // key i's, left in s[0]
      if constexpr (N > 1) s[0][i] += s[1][i];
      if constexpr (N > 2) s[0][i] += s[2][i] + s[3][i];
    }
  };
  __device__ __forceinline__ f32x16 scores(const unsigned char* K, int r0) const {
    constexpr int SUMS = !F32 ? 1 : D <= 32 ? 2 : 4;
    Sums<SUMS> x;
#pragma unroll
    for (int t = 0; t < QN; ++t) add_product(x.s[t % SUMS], key_piece(K, r0, t), t);
#pragma unroll
    for (int i = 0; i < 16; ++i) x.join(i);
    return x.s[0];
  }

  // -infinity where the query does not see the key; key0: key of row 0, gone: bit g set where 16 rows have no page.
  __device__ __forceinline__ int key_of(int i) const {
    return 8 * (i >> 2) + (i & 3) + 4 * (lane >> 5);
  }
  __device__ __forceinline__ void mask(f32x16& s, int key0, int gone) const {
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      const int k = key0 + key_of(i);
      if (k < lo || k > hi || ((gone >> (i >> 3)) & 1)) s[i] = -INFINITY;
    }
  }

  // The running maximum takes `top` (of this lane's keys) in.  Weights are taken against mc as rounded, so the factors
  // between maxima are too (contracted, or of (m - n) * scale, they would be off by 2^-24 of the maximum itself).
  __device__ __forceinline__ void raise(float top, float c, float slack) {
#pragma clang fp contract(off)
    top = other_half_max(top);
    if (__ballot(top > m + slack || (m == -INFINITY && top > m)) == 0) return;
    const float n = fmaxf(m, top), nc = n * c - MORE;
    const float f = m == -INFINITY ? 1.f : __builtin_amdgcn_exp2f(mc - nc);
    m = n;
    mc = n == -INFINITY ? 0.f : nc;
    l *= f;
#pragma unroll
    for (int t = 0; t < DT; ++t)
#pragma unroll
      for (int i = 0; i < 16; ++i) o[t][i] *= f;
  }

  // What the weights were taken against, -infinity without a key.
  __device__ __forceinline__ float against() const { return m == -INFINITY ? -INFINITY : mc; }

  // Weights of 32 keys as operands: fp32, or rounded to T, which is what the 16-bit matrix instructions take (fp32 ones
  // are a sixteenth as fast).  Summed as rounded, the error of o against 64 bits is 1.35 times (bf16; fp16 1.15) that of
  // rounding o alone; a second product with what rounding takes off would bring it there, for half as many matrix
  // operations again.
  struct Weights {
    uint4 u[F32 ? 4 : 2];
    __device__ __forceinline__ float at(int i) const {
      if constexpr (F32) return __builtin_bit_cast(f32x4, u[i >> 2])[i & 3];
      else return Elem<T>::to_f(__builtin_bit_cast(typename Op<T>::V, u[i >> 3])[i & 7]);
    }
    // Weights i, i + 1 are made here: the compiler would else move them behind the branches that follow.
    __device__ __forceinline__ void pin(int i) {
      uint32_t* x = &u[0].x;
      if constexpr (F32) asm volatile("" : "+v"(x[i]), "+v"(x[i + 1]));
      else asm volatile("" : "+v"(x[i >> 1]));
    }
  };
  // Two scores to weights.
  __device__ __forceinline__ void weigh_two(Weights& w, const f32x16& s, int i, float c) const {
    const float a = __builtin_amdgcn_exp2f(fmaf(s[i], c, -mc)), b = __builtin_amdgcn_exp2f(fmaf(s[i + 1], c, -mc));
    uint32_t* u = &w.u[0].x;
    if constexpr (F32) {
      u[i] = __float_as_uint(a);
      u[i + 1] = __float_as_uint(b);
    } else {
      typedef float f32x2 __attribute__((ext_vector_type(2)));
      typedef T two __attribute__((ext_vector_type(2)));
      u[i >> 1] = __builtin_bit_cast(uint32_t, __builtin_convertvector(f32x2{a, b}, two));
    }
  }
  __device__ __forceinline__ Weights weigh(const f32x16& s, float c) const {
    Weights w;
#pragma unroll
    for (int i = 0; i < 16; i += 2) weigh_two(w, s, i, c);
    return w;
  }
  // Adds weights i, i + 1 to x, as they enter the product: what rounding does to a weight acts above and below the line.
  // For 16-bit types in one instruction: over 1.5 million random sums it rounded once, to the nearest, in 95 to 100% of
  // cases by range, and else was off by at most 1 unit of the last place (bf16), 1.4 or 2^-37 (fp16), downwards.  Sums
  // of 16 weights are made so and then added to l in fp32.
  static __device__ __forceinline__ float add_two(float x, const Weights& w, int i) {
    const uint32_t* u = &w.u[0].x;
    if constexpr (F32) {
      return x + __uint_as_float(u[i]) + __uint_as_float(u[i + 1]);
    } else {
      typedef T two __attribute__((ext_vector_type(2)));
      const two ones = {(T)1.f, (T)1.f};
      if constexpr (__is_same(T, __bf16))
        return __builtin_amdgcn_fdot2_f32_bf16(__builtin_bit_cast(two, u[i >> 1]), ones, x, false);
      else
        return __builtin_amdgcn_fdot2(__builtin_bit_cast(two, u[i >> 1]), ones, x, false);
    }
  }
  static __device__ __forceinline__ float sum(const Weights& w) {
    float x = 0.f;
#pragma unroll
    for (int i = 0; i < 16; i += 2) x = add_two(x, w, i);
    return x;
  }

  // V's operand for 16 keys (rows r0 .. r0 + 15) and 32 columns, in the weights' order.
  __device__ __forceinline__ uint4 value_operand(const unsigned char* V, int r0, int t) const {
    const int h = lane >> 5, g = (lane >> 4) & 1;
    const int r = 4 * h + ((lane & 15) >> 2);
    const int piece = (4 * t + 2 * g + ((lane & 3) >> 1)) ^ value_swizzle<ES, PPR>(r);
    const unsigned char* at = V + (r0 + r) * RB + (piece << 4) + ((lane & 1) << 3);
    const uint2 a = __builtin_bit_cast(uint2, read_tr16(at)), b = __builtin_bit_cast(uint2, read_tr16(at + 8 * RB));
    return make_uint4(a.x, a.y, b.x, b.y);
  }
  // One fp32 value: column 32 t + l % 32 of the lane's i-th key.
  __device__ __forceinline__ float value_at(const unsigned char* V, int r0, int t, int i) const {
    const int r = r0 + key_of(i), col = 32 * t + (lane & 31);
    return *reinterpret_cast<const float*>(V + r * RB + (((col >> 2) ^ value_swizzle<ES, PPR>(r)) << 4) +
                                           ((col & 3) << 2));
  }

  // o += V^T P^T over 32 keys in PARTS parts: part k = (keys, columns) of 16 x 32, or one key's 32 columns a lane.
  static constexpr int PARTS = (F32 ? 16 : 2) * DT;
  using Value = typename std::conditional<F32, float, uint4>::type;
  __device__ __forceinline__ Value value_part(const unsigned char* V, int r0, int k) const {
    if constexpr (F32) return value_at(V, r0, k % DT, k / DT);
    else return value_operand(V, r0 + 16 * (k / DT), k % DT);
  }
  __device__ __forceinline__ void add_part(const Value& v, const Weights& p, int k) {
    if constexpr (F32)
      o[k % DT] = __builtin_amdgcn_mfma_f32_32x32x2f32(v, p.at(k / DT), o[k % DT], 0, 0, 0);
    else
      o[k % DT] = Op<T>::mma(__builtin_bit_cast(typename Op<T>::V, v), __builtin_bit_cast(typename Op<T>::V, p.u[k / DT]),
                             o[k % DT]);
  }
  __device__ __forceinline__ void add_values(const unsigned char* V, int r0, const Weights& p) {
#pragma unroll
    for (int k = 0; k < PARTS; ++k) add_part(value_part(V, r0, k), p, k);
  }

  // Whether 32 rows of values hold no infinity or NaN: the largest of all without signs.
  __device__ __forceinline__ bool finite(const unsigned char* V, int r0) const {
    typedef unsigned short u16x2 __attribute__((ext_vector_type(2)));
    uint32_t top = 0;
#pragma unroll 8
    for (int n = 0; n < RB / 32; ++n) {
      const uint4 x = *reinterpret_cast<const uint4*>(V + r0 * RB + n * 1024 + lane * 16);
      const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        if constexpr (F32) {
          top = max(top, w[i] & 0x7fffffffu);
        } else {
          top = __builtin_bit_cast(uint32_t, __builtin_elementwise_max(__builtin_bit_cast(u16x2, top),
                                                                       __builtin_bit_cast(u16x2, w[i] & 0x7fff7fffu)));
        }
      }
    }
    constexpr uint32_t X = __is_same(T, _Float16) ? 0x7c00u : 0x7f80u;
    const bool bad = F32 ? top >= 0x7f800000u : (top & 0xffffu) >= X || top >> 16 >= X;
    return __ballot(bad) == 0;
  }

  // Which of 32 rows of values hold an infinity or NaN.
  __device__ __forceinline__ uint32_t not_finite(const unsigned char* V, int r0) const {
    constexpr int LANES = PPR < 64 ? PPR : 64, PER = 64 / LANES;   // lanes of a row, rows at once
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

  // Rows of values with infinities or NaN, in a tile of which a query may see a part: a weight of 0 would not keep them
  // out of the product.  They are added key by key to the queries that see them; clear_rows() then takes them out.
  __device__ __forceinline__ void add_rows(const unsigned char* V, int r0, const Weights& p, uint32_t bad, int key0,
                                           int gone) {
    const int h = lane >> 5;
    for (uint32_t left = bad; left != 0; left &= left - 1) {
      const int k = __ffs(left) - 1, key = key0 + k;
      float w = 0.f;      // its weight, in the lanes of half (k / 4) % 2
#pragma unroll
      for (int i = 0; i < 16; ++i)
        if (i == (k >> 3) * 4 + (k & 3)) w = p.at(i);
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
  __device__ __forceinline__ void clear_rows(unsigned char* V, int r0, uint32_t bad) const {
    for (uint32_t left = bad; left != 0; left &= left - 1) {
      const int r = r0 + __ffs(left) - 1;
      for (int x = lane; x < PPR; x += 64) *reinterpret_cast<uint4*>(V + r * RB + x * 16) = make_uint4(0, 0, 0, 0);
    }
  }
};

// Page numbers of 64 granules of 16 keys, one a lane, as rows of the cache (-1: no page).
struct Pages {
  int first;      // first granule held
  int row;        // this lane's
  uint64_t none;  // lanes without a page
};

__device__ __forceinline__ void load_pages(const AttendArgs& a, const int32_t* __restrict__ table, int head, int g0,
                                           int lane, Pages& p) {
  const int g = g0 + lane;
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

// Copies NR rows of keys (or values) from key `key` on to LDS, rows outside of [beg, end) and without a page as zeros.
// Either NR and key are multiples of 16, or all NR rows from key on lie in one granule, at the same rows of it each time.
//
// An instruction copies 1024 bytes of LDS in order, so which piece of which row a lane fetches is a matter of its own
// address.  The swizzles are linear over exclusive or: instruction n's place is the first one's, with a constant.
template <int ES, int D, int NR, bool VALUES>
struct Stage {
  static constexpr int RB = D * ES, PPR = RB / 16, RPI = 64 / PPR;     // rows an instruction
  static constexpr int GR = NR < 16 ? NR : 16;                         // rows of one granule
  static_assert(PPR <= 64 && GR % RPI == 0, "a row is at most one instruction, a granule whole ones");
  int lane;
  uint32_t place;          // of the lane's piece in instruction 0, from the first row on

  static __device__ __forceinline__ constexpr int swizzle(int r) {
    return VALUES ? value_swizzle<ES, PPR>(r) : key_swizzle<PPR>(r);
  }
  // sub: the first row's number in its granule
  __device__ __forceinline__ Stage(int lane_, int sub) : lane(lane_) {
    const int r = lane / PPR;
    place = (uint32_t)(r * RB + (((lane % PPR) ^ swizzle(r) ^ swizzle(sub)) << 4));
  }
  __device__ __forceinline__ void operator()(const void* cache, const Pages& pg, int key, int beg, int end,
                                             uint32_t lds) const {
#pragma unroll
    for (int g = 0; g < NR / GR; ++g) {
      const int at = key + g * 16;
      const int granule = __builtin_amdgcn_readlane(pg.row, ((at >> 4) - pg.first) & 63);
      const bool there = granule >= 0;
      const int row = granule + (GR < 16 ? at & 15 : 0);     // (of no page: no row, whatever is added)
      const char* base = static_cast<const char*>(cache) + (int64_t)row * RB;
      const uint32_t to = lds + (uint32_t)(g * 16 * RB);
      if (there && at >= beg && at + GR <= end) {
#pragma unroll
        for (int n = 0; n < GR / RPI; ++n)
          dma16((place ^ (uint32_t)(swizzle(n * RPI) << 4)) + n * 1024, base, to + n * 1024);
      } else {
#pragma unroll
        for (int n = 0; n < GR / RPI; ++n) {
          const int k = at + n * RPI + lane / PPR;
          const char* src = base + (place ^ (uint32_t)(swizzle(n * RPI) << 4)) + n * 1024;
          dma16(there && k >= beg && k < end ? static_cast<const void*>(src) : static_cast<const void*>(zeros16),
                to + n * 1024);
        }
      }
    }
  }
};

// A tile's rows and keys.
template <int ROWS>
struct Tile {
  int R, row0, room, pmin, pmax, beg, end, b, lens, L;
  __device__ __forceinline__ Tile(const AttendArgs& a, int G, const Piece& u) {
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

// The lane, hidden from the compiler: what a piece computes from it is not kept in registers for the next piece.
__device__ __forceinline__ int fresh_lane() {
  int lane = threadIdx.x & 63;
  asm volatile("" : "+v"(lane));
  return lane & 63;
}

// A workgroup's next piece: the part [from, to) of a tile's length.
struct Next {
  Piece u;
  int from, to;
  Shares sh;
  int pos, end, slot;    // the share's next place and its end; the piece's slot of the workspace
  Cut cut;
  int j, state;          // share; kTile, kPart, or kNone: nothing left
};
enum { kNone, kTile, kPart };

// Finds workgroup j's first piece (first), or the one after the last.  Not inlined: the kernels' registers are full, and
// what this computes would be kept in them over the pieces.
template <bool FEW>
__device__ __attribute__((noinline)) void plan_piece(Work w, int j, bool first,
                                                     __attribute__((address_space(3))) Next* k) {
  // arguments come in vector registers: as scalars again, branches on them are branches
  const uint64_t cu = (uint64_t)w.cu, lens = (uint64_t)w.lens;
  auto address = [](uint64_t x) {
    return reinterpret_cast<const int32_t*>((uint64_t)(uint32_t)scalar((int)(x >> 32)) << 32 | (uint32_t)scalar((int)x));
  };
  const Work a{address(cu), address(lens), scalar(w.N), scalar(w.T), scalar(w.total), scalar(w.G), scalar(w.room),
               scalar(w.window), scalar(w.tiles), scalar(w.shares), scalar(w.unit), scalar(w.extra_drawn),
               scalar(w.extra_even)};
  j = scalar(j);
  first = scalar(first) != 0;
  Line<FEW> line(a);
  Shares sh{0, 0, 0, 1, 0};
  int pos = 0, end = 0;
  bool tile = a.shares == 0;
  if (!first) {
    sh = Shares{scalar(k->sh.longest), scalar(k->sh.whole), scalar(k->sh.rest), scalar(k->sh.share), scalar(k->sh.drawn)};
    pos = scalar(k->pos);
    end = scalar(k->end);
    j = scalar(k->j);
  } else if (!tile) {
    sh = line.share_out();
    if (j >= sh.whole + a.shares) {                  // the grid has room for more whole tiles
      k->state = kNone;
      k->j = -1;
      return;
    }
    tile = j < sh.whole;
    if (!tile) j -= sh.whole;
    const int64_t at = (int64_t)j * sh.share;
    pos = (int)min(at, (int64_t)sh.rest);
    end = (int)min(at + sh.share, (int64_t)sh.rest);
  }
  Piece u{0, 0, 0, 0, 0, 0, 0};
  int from = 0, to = 1, state = kNone, slot = 0;
  Cut cut{0, 0, 0, 0, 0};
  if (tile) {
    if (line.template find<true>(sh, j, u)) state = kTile;
    // where there are no workgroups behind the shares, the cuts of the last ones, none, are written here
    j = FEW && a.tiles <= a.shares ? a.shares - sh.whole + j : -1;
  } else {
    while (pos < end && line.template find<false>(sh, pos, u)) {
      from = pos - u.at;
      to = min(u.length, end - u.at);
      slot = 2 * j + (from == 0);
      if (first && from > 0 && u.at >= pos - sh.share) {
        const int last = u.at + u.length;
        const int n = quotient(last - 1, sh.share);                // the share that ends the tile
        const int begin = border(from, u.length, sh.share) == 0;
        const int over = border(n * sh.share - u.at, u.length, sh.share) == u.length;
        cut = Cut{u.b, u.L, u.tile, (short)begin, (short)(n - j + 2 - over)};
      }
      first = false;
      pos = u.at + to;
      from = border(from, u.length, sh.share);
      to = border(to, u.length, sh.share);
      if (to > from) {
        state = kPart;
        break;
      }
    }
  }
  k->u.s = u.s, k->u.b = u.b, k->u.L = u.L, k->u.lens = u.lens, k->u.tile = u.tile;
  k->u.length = u.length, k->from = from, k->to = to, k->pos = pos, k->end = end, k->slot = slot;
  k->sh.longest = sh.longest, k->sh.whole = sh.whole, k->sh.rest = sh.rest, k->sh.share = sh.share;
  k->sh.drawn = sh.drawn;
  k->cut.b = cut.b, k->cut.L = cut.L, k->cut.tile = cut.tile, k->cut.begin = cut.begin, k->cut.end = cut.end;
  k->j = j, k->state = state;
}

// A workgroup's tile, or its share's pieces one after another: body(piece, from, to, whole, slot) for the part
// [from, to) of a tile's length; pieces that are not whole tiles have a slot of the workspace.  Without shares every
// workgroup has a tile.
template <bool FEW, typename B>
__device__ __forceinline__ void walk(const AttendArgs& a, int G, int head, int j, B&& body) {
  __shared__ Next k;
  const int wave = scalar(threadIdx.x >> 6);
  const Work work{a.c.cu, a.c.lens, a.c.N, a.c.T, a.c.total, G, a.c.max_pages * a.c.page_size, a.window, a.tiles, a.shares,
                  a.unit, a.extra_drawn, a.extra_even};
  for (bool first = true;; first = false) {
    // One wave for all: the others would only get in its way.  (k may be written: all have read the last one's before
    // a barrier in body.)
    if (wave == 0) plan_piece<FEW>(work, j, first, (__attribute__((address_space(3))) Next*)&k);
    lds_barrier();
    const int state = scalar(k.state), share = scalar(k.j);
    if (first && share >= 0 && threadIdx.x == 0) static_cast<Cut*>(a.cuts)[head * a.shares + share] = k.cut;
    if (state == kNone) return;
    const Piece u{scalar(k.u.s), scalar(k.u.b), scalar(k.u.L), scalar(k.u.lens), scalar(k.u.tile), 0, scalar(k.u.length)};
    const int from = scalar(k.from), to = scalar(k.to);
    body(u, from, to, state == kTile || (from == 0 && to == u.length), scalar(k.slot));
    if (state == kTile) return;
  }
}

// The blocks of `n` that the part [from, to) of a tile's length is: the same function of a border on both its sides.
__device__ __forceinline__ void part_blocks(int n, const Piece& u, int from, int to, int& b, int& e) {
  const float blocks = (float)n / (float)u.length;
  b = scalar(min((int)((float)from * blocks), n));
  e = to == u.length ? n : scalar(min((int)((float)to * blocks), n));
}

// Many rows: four waves of 32 rows, the same keys, in blocks of KT of them.  Keys and values have two buffers each; a
// block's loads are issued one block ahead.  The one barrier a block says that its loads have landed and that nobody
// reads the buffers that the next ones go to.
//
// Bound by the matrix unit and the vector unit's exponentials in turn: 44 and 42% busy with heads of 128, LDS 22% and
// free of conflicts.  2048 new tokens over 16384 keys, bf16: 32 heads of 128 522 us (987 TFLOP/s; a large matrix product
// has 1221), of 64 352 us (730, as many exponentials for half the products), 16 heads of 256 580 us (888); 1024 over
// 4096 fp32, 32 heads of 128 562 us (107 of 138).
//
// Where the registers leave one wave a SIMD (D = 256, fp32 from D = 128 on), nothing fills the matrix unit while that wave
// makes weights: keys are loaded two blocks ahead and multiplied one block ahead, in turn with the exponentials of the
// block before (2048 new tokens over 16384 keys, 16 heads of 256, bf16: 780 -> 596 us).  With two waves or more the
// other wave does that, and the plain order needs fewer registers (D = 128: 542 us plain, 552 in turn).  There, waves
// that multiply go first (542 -> 522 us).
template <typename T, int D>
struct ManyShape {
  static constexpr int RB = D * (int)sizeof(T), KT = many_keys(RB), NS = KT / 32;
  static constexpr bool ALONE = many_waves(RB) == 1;     // one wave a SIMD
};

template <typename T, int D>
__global__ __launch_bounds__(256, (many_waves(D * (int)sizeof(T)))) void cache_attention_many_kernel(AttendArgs a) {
  using S = ManyShape<T, D>;
  constexpr int KT = S::KT, RB = S::RB, ES = (int)sizeof(T), NR = KT / 4;
  extern __shared__ __align__(16) unsigned char smem[];
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int G = a.c.Hq / a.c.Hkv, head = (int)(blockIdx.x % a.c.Hkv);
  const float c = a.scale_log2, slack = Wave<T, D>::SLACK / c;
  const uint32_t lds = (uint32_t)(uintptr_t)(__attribute__((address_space(3))) unsigned char*)smem;
  walk<false>(a, G, head, (int)(blockIdx.x / a.c.Hkv), [&](const Piece& u, int from, int to, bool whole, int slot) {
    const int lane = fresh_lane(), h = lane >> 5;
    const Tile<kManyRows> t(a, G, u);
    Wave<T, D> w;
    w.init(lane);
    const int mine = wave * 32 + (lane & 31);
    const int64_t out = set_row(a, G, head, t, mine, w);
    const int key_first = t.beg & ~(KT - 1);
    int tb, te;
    part_blocks(t.end > t.beg ? (t.end - key_first + KT - 1) / KT : 0, u, from, to, tb, te);
    const int32_t* table = a.c.table + (int64_t)u.s * a.c.max_pages;
    const Stage<ES, D, NR, false> stage_k(lane, wave * NR & 15);
    const Stage<ES, D, NR, true> stage_v(lane, wave * NR & 15);
    // keys run one block ahead of values (ALONE): a page window each
    Pages kp, vp;
    kp.first = vp.first = -0x40000000;
    auto stage_keys = [&](int i) {
      const int key = key_first + i * KT;
      if ((key >> 4) - kp.first >= 64) load_pages(a, table, head, key >> 4, lane, kp);
      stage_k(a.k_cache, kp, key + wave * NR, t.beg, t.end, lds + (uint32_t)((i & 1) * KT * RB + wave * NR * RB));
      return (int)((kp.none >> ((key >> 4) - kp.first)) & ((1 << (KT / 16)) - 1));
    };
    auto stage_values = [&](int i) {
      const int key = key_first + i * KT;
      if ((key >> 4) - vp.first >= 64) load_pages(a, table, head, key >> 4, lane, vp);
      stage_v(a.v_cache, vp, key + wave * NR, t.beg, t.end, lds + (uint32_t)((2 + (i & 1)) * KT * RB + wave * NR * RB));
    };
    // whether some row of the tile does not see some of block i's keys
    auto partly = [&](int i, int absent) {
      const int key = key_first + i * KT;
      return key + KT - 1 > min(t.pmin, t.room - 1) || (a.window > 0 && key < t.pmax - a.window + 1) || absent;
    };
    f32x16 s[S::NS];
    auto mask = [&](int i, int absent) {
#pragma unroll
      for (int n = 0; n < S::NS; ++n) w.mask(s[n], key_first + i * KT + 32 * n, absent >> (2 * n));
    };
    lds_barrier();                                 // nobody reads the last piece's blocks any more
    auto clean = [&](int i, int absent, typename Wave<T, D>::Weights (&p)[S::NS]) {
      unsigned char* V = smem + (2 + (i & 1)) * KT * RB;
#pragma unroll
      for (int n = 0; n < S::NS; ++n) {
        if (__builtin_expect(!w.finite(V, 32 * n), 0)) {       // the same for all four waves
          const uint32_t bad = w.not_finite(V, 32 * n);
          w.add_rows(V, 32 * n, p[n], bad, key_first + i * KT + 32 * n, absent >> (2 * n));
          lds_barrier();
          w.clear_rows(V, 32 * n, bad);                        // all waves write the same zeros
          lds_barrier();
        }
      }
    };
    auto highest = [&] {
      float top = -INFINITY;
#pragma unroll
      for (int n = 0; n < S::NS; ++n)
#pragma unroll
        for (int j = 0; j < 16; ++j) top = fmaxf(top, s[n][j]);
      return top;
    };
    if constexpr (!S::ALONE) {
      int ahead = 0;                               // keys without a page in the next block
      if (tb < te) {
        ahead = stage_keys(tb);
        stage_values(tb);
      }
      for (int i = tb; i < te; ++i) {
        const int absent = ahead;
        wait_loads<0>();
        lds_barrier();
        if (i + 1 < te) {
          ahead = stage_keys(i + 1);
          stage_values(i + 1);
        }
        __builtin_amdgcn_s_setprio(1);
#pragma unroll
        for (int n = 0; n < S::NS; ++n) s[n] = w.scores(smem + (i & 1) * KT * RB, 32 * n);
        __builtin_amdgcn_s_setprio(0);
        const bool part = partly(i, absent);
        if (part) mask(i, absent);
        w.raise(highest(), c, slack);
        typename Wave<T, D>::Weights p[S::NS];
#pragma unroll
        for (int n = 0; n < S::NS; ++n) {
          p[n] = w.weigh(s[n], c);
          w.l += Wave<T, D>::sum(p[n]);
        }
        if (part) clean(i, absent, p);
        __builtin_amdgcn_s_setprio(1);
#pragma unroll
        for (int n = 0; n < S::NS; ++n) w.add_values(smem + (2 + (i & 1)) * KT * RB, 32 * n, p[n]);
        __builtin_amdgcn_s_setprio(0);
      }
    } else {
      int absent = 0, ahead = 0;                     // keys without a page in blocks i, i + 1
      if (tb < te) {
        absent = stage_keys(tb);
        stage_values(tb);
        if (tb + 1 < te) ahead = stage_keys(tb + 1);
        wait_loads<0>();
        lds_barrier();
#pragma unroll
        for (int n = 0; n < S::NS; ++n) s[n] = w.scores(smem + (tb & 1) * KT * RB, 32 * n);
        if (partly(tb, absent)) mask(tb, absent);
      }
      float top = highest();
      // Block i: its scores are there.  The next block's are computed beside its weights, and their maximum beside its
      // products with the values, a product and a few vector operations in turn: the compiler left to itself puts all
      // products before all exponentials, and neither unit works while the other does.
      auto step = [&](int i, auto more) {
        using W = Wave<T, D>;
        constexpr int AHEAD = 3;                     // LDS reads in flight
        constexpr int SUMS = W::F32 ? 2 : 1;
        unsigned char* V = smem + (2 + (i & 1)) * KT * RB;
        const unsigned char* K = smem + ((i + 1) & 1) * KT * RB;
        w.raise(top, c, slack);
        typename W::template Sums<SUMS> x[S::NS];
        typename W::Weights p[S::NS];
        if constexpr (more.value) {
          constexpr int N = S::NS * W::QN, PAIRS = 8 * S::NS;
          uint4 k[AHEAD + 1];
#pragma unroll
          for (int t = 0; t < AHEAD; ++t) k[t] = w.key_piece(K, 32 * (t / W::QN), t % W::QN);
#pragma unroll
          for (int t = 0; t < N; ++t) {
            if (t + AHEAD < N)
              k[(t + AHEAD) % (AHEAD + 1)] = w.key_piece(K, 32 * ((t + AHEAD) / W::QN), (t + AHEAD) % W::QN);
            w.add_product(x[t / W::QN].s[t % SUMS], k[t % (AHEAD + 1)], t % W::QN);
#pragma unroll
            for (int e = t * PAIRS / N; e < (t + 1) * PAIRS / N; ++e) {
              w.weigh_two(p[e / 8], s[e / 8], e % 8 * 2, c);
              p[e / 8].pin(e % 8 * 2);
            }
            __builtin_amdgcn_sched_barrier(0);
          }
        } else {
#pragma unroll
          for (int n = 0; n < S::NS; ++n) p[n] = w.weigh(s[n], c);
        }
        if (partly(i, absent)) clean(i, absent, p);
        constexpr int N = S::NS * W::PARTS, PAIRS = 8 * S::NS;
        typename W::Value v[AHEAD + 1];
        float part[S::NS], high = -INFINITY;
#pragma unroll
        for (int n = 0; n < S::NS; ++n) part[n] = 0.f;
#pragma unroll
        for (int t = 0; t < AHEAD; ++t) v[t] = w.value_part(V, 32 * (t / W::PARTS), t % W::PARTS);
#pragma unroll
        for (int t = 0; t < N; ++t) {
          if (t + AHEAD < N)
            v[(t + AHEAD) % (AHEAD + 1)] = w.value_part(V, 32 * ((t + AHEAD) / W::PARTS), (t + AHEAD) % W::PARTS);
          w.add_part(v[t % (AHEAD + 1)], p[t / W::PARTS], t % W::PARTS);
#pragma unroll
          for (int e = t * PAIRS / N; e < (t + 1) * PAIRS / N; ++e) {
            part[e / 8] = W::add_two(part[e / 8], p[e / 8], e % 8 * 2);
            if constexpr (more.value) {
              x[e / 8].join(e % 8 * 2);
              x[e / 8].join(e % 8 * 2 + 1);
              high = fmaxf(fmaxf(high, x[e / 8].s[0][e % 8 * 2]), x[e / 8].s[0][e % 8 * 2 + 1]);
            }
            asm volatile("" : "+v"(part[e / 8]), "+v"(high));
          }
          __builtin_amdgcn_sched_barrier(0);
        }
#pragma unroll
        for (int n = 0; n < S::NS; ++n) w.l += part[n];
        if constexpr (more.value) {
#pragma unroll
          for (int n = 0; n < S::NS; ++n) s[n] = x[n].s[0];
          top = high;
        }
      };
      for (int i = tb; i + 1 < te; ++i) {
        if (i > tb) wait_loads<0>();
        lds_barrier();                               // (at first: all have read block tb's keys, the next go there)
        int then = 0;
        if (i + 2 < te) then = stage_keys(i + 2);
        stage_values(i + 1);
        step(i, std::true_type{});
        absent = ahead;
        ahead = then;
        if (partly(i + 1, absent)) {
          mask(i + 1, absent);
          top = highest();
        }
      }
      if (tb < te) {
        if (tb + 1 < te) {
          wait_loads<0>();
          lds_barrier();
        }
        step(te - 1, std::false_type{});
      }
    }
    const float l = other_half_sum(w.l);
    if (t.row0 + mine >= t.R) return;
    if (whole) {
      T* o = static_cast<T*>(a.o) + out;
#pragma unroll
      for (int k = 0; k < D / 32; ++k)
#pragma unroll
        for (int j = 0; j < 4; ++j)
          store_final(o + 32 * k + 8 * j + 4 * h, w.o[k][4 * j], w.o[k][4 * j + 1], w.o[k][4 * j + 2], w.o[k][4 * j + 3], l);
    } else {
      const int64_t at = ((int64_t)slot * a.c.Hkv + head) * kManyRows + mine;
      float* o = a.part_o + at * D;
#pragma unroll
      for (int k = 0; k < D / 32; ++k)
#pragma unroll
        for (int j = 0; j < 4; ++j)
          store4<float>(o + 32 * k + 8 * j + 4 * h, w.o[k][4 * j], w.o[k][4 * j + 1], w.o[k][4 * j + 2], w.o[k][4 * j + 3]);
      if (h == 0) *reinterpret_cast<float2*>(a.part_ml + at * 2) = make_float2(w.against(), l);
    }
  });
}

// Few rows: one tile of 32 rows, each wave on its own 32 keys at a time with its own piece of LDS and no barrier: once
// a tile's keys have been read the next ones are on their way, once its values have been read the next values.  Bound by
// reading the cache: one token over 131001 keys of 2 heads of 256, bf16, 54 us (4.9 TB/s), 32 tokens over 600 to 32011
// keys of 8 heads of 128 98 us (5.2).  Short ones by latency: 3 us until the work is found, 3 us to the first keys.
template <typename T, int D>
__global__ __launch_bounds__((64 * few_group(D * (int)sizeof(T))), (few_waves(D * (int)sizeof(T))))
void cache_attention_few_kernel(AttendArgs a) {
  constexpr int RB = D * (int)sizeof(T), ES = (int)sizeof(T), NW = few_group(RB), NI = 32 * RB / 1024;
  extern __shared__ __align__(16) unsigned char smem[];
  __shared__ float2 ml[NW][32];
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int G = a.c.Hq / a.c.Hkv, head = (int)(blockIdx.x % a.c.Hkv);
  const float c = a.scale_log2, slack = Wave<T, D>::SLACK / c;
  unsigned char* K = smem + wave * 64 * RB;
  unsigned char* V = K + 32 * RB;
  const uint32_t ldsK = (uint32_t)(uintptr_t)(__attribute__((address_space(3))) unsigned char*)smem + wave * 64 * RB;
  walk<true>(a, G, head, (int)(blockIdx.x / a.c.Hkv), [&](const Piece& u, int from, int to, bool whole, int slot) {
    const int lane = fresh_lane();
    const Tile<kFewRows> t(a, G, u);
    Wave<T, D> w;
    w.init(lane);
    const int key_first = t.beg & ~31;
    int tb, te;
    part_blocks(t.end > t.beg ? (t.end - key_first + 31) / 32 : 0, u, from, to, tb, te);
    const int32_t* table = a.c.table + (int64_t)u.s * a.c.max_pages;
    const Stage<ES, D, 32, false> stage_k(lane, 0);
    const Stage<ES, D, 32, true> stage_v(lane, 0);
    Pages pg;
    pg.first = -0x40000000;
    auto pages_for = [&](int i) {
      const int g = (key_first >> 4) + 2 * i;
      if (g - pg.first >= 64) load_pages(a, table, head, g, lane, pg);
      return (int)((pg.none >> (g - pg.first)) & 3);
    };
    int i = tb + wave, gone = 0;
    if (i < te) {
      gone = pages_for(i);
      stage_k(a.k_cache, pg, key_first + 32 * i, t.beg, t.end, ldsK);
      stage_v(a.v_cache, pg, key_first + 32 * i, t.beg, t.end, ldsK + 32 * RB);
    }
    set_row(a, G, head, t, lane & 31, w);
    for (; i < te; i += NW) {
      const int key = key_first + 32 * i, absent = gone, next = i + NW;
      wait_loads<NI>();                              // the keys: the values were issued after them
      f32x16 s = w.scores(K, 0);
      asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
      if (next < te) {
        gone = pages_for(next);
        stage_k(a.k_cache, pg, key_first + 32 * next, t.beg, t.end, ldsK);
      }
      const bool part = key + 31 > min(t.pmin, t.room - 1) || (a.window > 0 && key < t.pmax - a.window + 1) || absent;
      if (part) w.mask(s, key, absent);
      float top = -INFINITY;
#pragma unroll
      for (int j = 0; j < 16; ++j) top = fmaxf(top, s[j]);
      w.raise(top, c, slack);
      const auto p = w.weigh(s, c);
      w.l += Wave<T, D>::sum(p);
      if (next < te) wait_loads<NI>();               // the values: the next keys were issued after them
      else wait_loads<0>();
      if (part && __builtin_expect(!w.finite(V, 0), 0)) {
        const uint32_t bad = w.not_finite(V, 0);
        w.add_rows(V, 0, p, bad, key, absent);
        w.clear_rows(V, 0, bad);
        asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
      }
      w.add_values(V, 0, p);
      asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
      if (next < te) stage_v(a.v_cache, pg, key_first + 32 * next, t.beg, t.end, ldsK + 32 * RB);
    }
    // join the waves: everyone's accumulators in LDS (pieces of 16 bytes at piece ^ row % 8)
    const float l = other_half_sum(w.l);
    const int h = lane >> 5, row = lane & 31;
    if (h == 0) ml[wave][row] = make_float2(w.against(), l);
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
    const int64_t at = ((int64_t)slot * a.c.Hkv + head) * kFewRows;
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
        const float f = x.x == -INFINITY ? 0.f : __builtin_amdgcn_exp2f(x.x - m);
        const float4 p = O[(v * 32 + r) * (D / 4) + (piece ^ (r & 7))];
        sum.x += f * p.x, sum.y += f * p.y, sum.z += f * p.z, sum.w += f * p.w;
        tot += f * x.y;
      }
      if (whole) {
        const int token = (t.row0 + r) / G, g = t.row0 + r - token * G;
        T* o = static_cast<T*>(a.o) + ((int64_t)(t.b + token) * a.c.Hq + head * G + g) * D + 4 * piece;
        store_final(o, sum.x, sum.y, sum.z, sum.w, tot);
      } else {
        *reinterpret_cast<float4*>(a.part_o + (at + r) * D + 4 * piece) = sum;
        if (piece == 0) *reinterpret_cast<float2*>(a.part_ml + (at + r) * 2) = make_float2(m, tot);
      }
    }
    __syncthreads();                                 // the next piece may overwrite all of it
  });
}

// Joins the pieces of tiles that lie in several shares.  Bound by latency: workgroups x / Hkv, of as many as there are
// tiles at most, find their cut among those of all shares by one load a thread (a workgroup for each share instead, most
// of them with nothing to do: 8.4 us for 13 tiles, 8 heads and 96 shares, so 4.5).  A tile's rows go round among
// gridDim.y workgroups; a thread has 4 columns of a row and every few pieces of it (a running maximum and sum over them),
// the groups of pieces are joined in LDS, in their order.  2 tiles of 128 pieces of 8 rows of 256: 6.4 us.
constexpr int kJoinThreads = 1024;
static_assert(kJoinThreads >= kMostShares, "a thread for each share");

template <typename T, int D, int ROWS>
__global__ __launch_bounds__(kJoinThreads) void cache_attention_join_kernel(AttendArgs a) {
  constexpr int COLS = D / 4, AT_ONCE = 8;
  __shared__ float2 ml[kJoinThreads];
  __shared__ float4 sums[kJoinThreads];
  __shared__ int cuts[kJoinThreads / 64], found;
  const int G = a.c.Hq / a.c.Hkv, head = (int)(blockIdx.x % a.c.Hkv), mine_of_all = (int)(blockIdx.x / a.c.Hkv);
  const Cut* all = static_cast<const Cut*>(a.cuts) + head * a.shares;
  {
    const int s = threadIdx.x, lane = s & 63, wave = s >> 6;
    bool cut = false;
    if (s < a.shares) cut = all[s].end - all[s].begin >= 2;
    const uint64_t b = __ballot(cut);
    if (lane == 0) cuts[wave] = __popcll(b);
    if (s == 0) found = -1;
    __syncthreads();
    int rank = mine_of_all - __popcll(b & ((1ull << lane) - 1));
    for (int w = 0; w < wave; ++w) rank -= cuts[w];
    if (cut && rank == 0) found = s;
    __syncthreads();
  }
  const int j = scalar(found);
  if (j < 0) return;
  const Cut cut = all[j];
  const int row0 = cut.tile * ROWS, rows = min(ROWS, cut.L * G - row0), turn = (int)gridDim.y;
  const int mine = (rows - (int)blockIdx.y + turn - 1) / turn, items = mine * COLS;
  if (items <= 0) return;
  const int groups = max(1, min(kJoinThreads / items, (cut.end - cut.begin + AT_ONCE - 1) / AT_ONCE));
  const int group = threadIdx.x / items;
  for (int base = 0; base < items; base += kJoinThreads) {      // more than once only with one group
    const int item = base + (groups > 1 ? (int)threadIdx.x - group * items : (int)threadIdx.x);
    const bool on = groups > 1 ? group < groups : item < items;
    const int n = (int)blockIdx.y + item / COLS * turn, col = item % COLS * 4;
    float m = -INFINITY, l = 0.f;
    float4 sum = make_float4(0.f, 0.f, 0.f, 0.f);
    if (on) {
      auto at = [&](int k) {
        return ((int64_t)(k == 0 ? 2 * (j - 1) + 1 : 2 * (j - 1 + k)) * a.c.Hkv + head) * ROWS + n;
      };
      const int first = cut.begin + (groups > 1 ? group : 0);
      for (int k0 = first; k0 < cut.end; k0 += AT_ONCE * groups) {
        float2 x[AT_ONCE];
        float4 p[AT_ONCE];
        float top = m;
#pragma unroll
        for (int i = 0; i < AT_ONCE; ++i) {
          const int k = k0 + i * groups;
          x[i] = make_float2(-INFINITY, 0.f);
          p[i] = make_float4(0.f, 0.f, 0.f, 0.f);
          if (k < cut.end) {
            x[i] = *reinterpret_cast<const float2*>(a.part_ml + at(k) * 2);
            p[i] = *reinterpret_cast<const float4*>(a.part_o + at(k) * D + col);
          }
        }
#pragma unroll
        for (int i = 0; i < AT_ONCE; ++i) top = fmaxf(top, x[i].x);
        const float f = m == -INFINITY ? 0.f : __builtin_amdgcn_exp2f(m - top);
        sum.x *= f, sum.y *= f, sum.z *= f, sum.w *= f;
        l *= f;
        m = top;
#pragma unroll
        for (int i = 0; i < AT_ONCE; ++i) {
          const float w = x[i].x == -INFINITY ? 0.f : __builtin_amdgcn_exp2f(x[i].x - m);
          sum.x += w * p[i].x, sum.y += w * p[i].y, sum.z += w * p[i].z, sum.w += w * p[i].w;
          l += w * x[i].y;
        }
      }
    }
    if (groups > 1) {
      ml[threadIdx.x] = make_float2(m, l);
      sums[threadIdx.x] = sum;
      __syncthreads();
      if (group != 0) return;
      for (int g = 1; g < groups; ++g) m = fmaxf(m, ml[g * items + item].x);
      l = 0.f;
      sum = make_float4(0.f, 0.f, 0.f, 0.f);
      for (int g = 0; g < groups; ++g) {
        const float2 x = ml[g * items + item];
        const float4 p = sums[g * items + item];
        const float w = x.x == -INFINITY ? 0.f : __builtin_amdgcn_exp2f(x.x - m);
        sum.x += w * p.x, sum.y += w * p.y, sum.z += w * p.z, sum.w += w * p.w;
        l += w * x.y;
      }
    }
    if (on) {
      const int token = (row0 + n) / G, g = row0 + n - token * G;
      store_final(static_cast<T*>(a.o) + ((int64_t)(cut.b + token) * a.c.Hq + head * G + g) * D + col, sum.x, sum.y,
                  sum.z, sum.w, l);
    }
  }
}

template <typename K>
static hipError_t allow_lds(K kernel, int bytes) {
  return bytes > 65536 ? hipFuncSetAttribute(reinterpret_cast<const void*>(kernel),
                                             hipFuncAttributeMaxDynamicSharedMemorySize, bytes)
                       : hipSuccess;
}

template <typename T, int D>
static hipError_t launch_attend_d(const AttendArgs& a, hipStream_t s) {
  constexpr int RB = D * (int)sizeof(T);
  // few rows and no more tiles: shares alone; else some tiles or all are taken whole before them
  const unsigned shares = (unsigned)((int64_t)a.shares * a.c.Hkv), tiles = (unsigned)((int64_t)a.tiles * a.c.Hkv);
  const unsigned wgs = a.few && a.tiles <= a.shares ? shares : tiles + shares;
  prof_begin(K_ATTEND, s);
  hipError_t e;
  if (a.few) {
    e = allow_lds(cache_attention_few_kernel<T, D>, few_lds(RB));
    if (e != hipSuccess) return e;
    hipLaunchKernelGGL((cache_attention_few_kernel<T, D>), dim3(wgs), dim3(64 * few_group(RB)), few_lds(RB), s, a);
  } else {
    e = allow_lds(cache_attention_many_kernel<T, D>, many_lds(RB));
    if (e != hipSuccess) return e;
    hipLaunchKernelGGL((cache_attention_many_kernel<T, D>), dim3(wgs), dim3(256), many_lds(RB), s, a);
  }
  prof_end(K_ATTEND, s);
  if ((e = hipGetLastError()) != hipSuccess || a.shares < 2) return e;
  prof_begin(K_ATTEND_JOIN, s);
  const unsigned cuts = std::min(shares, tiles);
  const dim3 grid(cuts, std::max(1u, std::min(8u, 256 / cuts)));       // one workgroup a CU
  if (a.few) hipLaunchKernelGGL((cache_attention_join_kernel<T, D, kFewRows>), grid, dim3(kJoinThreads), 0, s, a);
  else hipLaunchKernelGGL((cache_attention_join_kernel<T, D, kManyRows>), grid, dim3(kJoinThreads), 0, s, a);
  prof_end(K_ATTEND_JOIN, s);
  return hipGetLastError();
}

template <typename T>
static hipError_t launch_attend_t(const AttendArgs& a, hipStream_t s) {
  switch (a.c.d) {
    case 32: return launch_attend_d<T, 32>(a, s);
    case 64: return launch_attend_d<T, 64>(a, s);
    case 128: return launch_attend_d<T, 128>(a, s);
    case 256: return launch_attend_d<T, 256>(a, s);
  }
  return hipErrorInvalidValue;
}

}  // namespace attend
}  // namespace gdn
