// Work lists of the products over rows grouped by expert. The row counts live
// on the device, so the blocks of a launch find their own tiles.
#pragma once

#include "device.h"

namespace moe {

// Walks tiles t = t0, t0 + step, .. (ascending) over the experts that have
// more than `lo` and at most `hi` rows, each with ceil(rows / bt) * per tiles.
// Every wave walks by itself: it holds the row ranges of 64 experts, one a
// lane, and their running tile counts, so a lookup is a ballot and the offsets
// are read once per 64 experts. No LDS, no barrier, no list in memory.
// Offsets are cut to [0, N] and to ascending order, so whatever they hold no
// tile reaches past row N.
struct GroupTile {
  int expert;  // local expert
  int beg;     // its first row
  int rows;    // its rows
  int tile;    // tile within the expert, 0 .. ceil(rows / bt) * per - 1
};

// Experts with at most this many rows go to narrow tiles, others to tiles of 256
// rows (the kernels' files have the measurements).
constexpr int kNarrowRows = 128;

struct GroupWalk {
  // How far one walk has come: the chunk of 64 experts it is in, and the tiles
  // of the experts before.
  struct Place {
    int c0 = 0, before = 0;
  };

  const int* off;
  int L, N, per, shift, lo, hi;
  int c0, total;         // the chunk held, and its tiles
  int beg, rows, upto;   // this lane's expert; upto: running count of tiles with it

  __device__ __forceinline__ int tiles_of(int r) const {
    return r > lo && r <= hi ? ((r + (1 << shift) - 1) >> shift) * per : 0;
  }
  // The rows of this lane's expert of the chunk at `first`.
  __device__ __forceinline__ int range(int first, int* b) {
    const int i = first + (int)(threadIdx.x % kWave);
    *b = 0;
    if (i >= L) return 0;
    *b = max(0, min(off[i], N));
    return max(*b, min(off[i + 1], N)) - *b;
  }
  __device__ __forceinline__ void load(int first) {
    c0 = first;
    rows = range(first, &beg);
    upto = wave_inclusive_sum(tiles_of(rows));
    total = __builtin_amdgcn_readlane(upto, kWave - 1);
  }
  // bt: rows to a tile, a power of two.
  __device__ __forceinline__ void start(const int* offsets, int num_local, int n, int per_pass,
                                        int bt, int more_than, int at_most) {
    off = offsets;
    L = num_local;
    N = n;
    per = per_pass;
    shift = 31 - __builtin_clz(bt);
    lo = more_than;
    hi = at_most;
    load(0);
  }
  // Right behind start(): whether the experts with at most `most` rows (if
  // there are others) cost `blocks` blocks no further round of tiles where they
  // are taken along with the others: `per` tiles for an expert of up to
  // kNarrowRows rows, and for each 256 of one with more. (Not asked for more
  // than 512 experts: each 64 are a trip to memory.)
  __device__ __forceinline__ bool rounds_hold(int most, int per, int blocks) {
    if (L > 8 * kWave) return false;
    int few = 0, tiles = 0;
    for (int c = 0, b, r = rows; c < L; c += kWave) {
      if (c > 0) r = range(c, &b);
      few += __popcll(__ballot(r > 0 && r <= most));
      const int n = r <= most ? 0 : r <= kNarrowRows ? 1 : (r + 255) / 256;
      tiles += __builtin_amdgcn_readlane(wave_inclusive_sum(n), kWave - 1);
    }
    // (N M < 2^31: 32 bits hold all of these)
    const uint32_t t = tiles * per, more = few * per;
    return t > 0 && more <= (t + blocks - 1) / blocks * blocks - t;
  }
  // False past the last tile. `t` is wave-uniform and never goes down for a
  // Place. Several Places may walk; the chunk is read again where they are in
  // different ones.
  __device__ __forceinline__ bool find(Place& p, int t, GroupTile* out) {
    if (c0 != p.c0) load(p.c0);
    while (t - p.before >= total) {
      if (p.c0 + kWave >= L) return false;
      p.before += total;
      p.c0 += kWave;
      load(p.c0);
    }
    const int at = t - p.before;
    const int j = __ffsll((unsigned long long)__ballot(upto > at)) - 1;
    out->expert = c0 + j;
    out->beg = __builtin_amdgcn_readlane(beg, j);
    out->rows = __builtin_amdgcn_readlane(rows, j);
    out->tile = at - (__builtin_amdgcn_readlane(upto, j) - tiles_of(out->rows));
    return true;
  }
};

constexpr int kAnyRows = 0x7FFFFFFF;

// The three products. A block computes D[r, c] = sum over kk of A[r, kk] B[c, kk]
// with r the output's contiguous index (four consecutive r per lane are one
// store):
//   forward   r = m  c = n  kk = k   A = W[e]       B = x rows      y[n, m]
//   dx        r = k  c = n  kk = m   A = W[e]^T     B = dy rows     dx[n, k]
//   dw        r = k  c = m  kk = n   A = x rows^T   B = dy rows^T   dw[e][m, k]
enum class Product { kForward, kDx, kDw };

// Division by a number that the host knows: m = floor((2^32 - 1) / d), and for
// n < 2^31 the high half of n m is n / d or one less.
struct Divisor {
  uint32_t d, m;
};
inline Divisor divisor(uint32_t d) { return Divisor{d, 0xFFFFFFFFu / d}; }
__device__ __forceinline__ int divide(int n, const Divisor& v) {
  uint32_t q = __umulhi((uint32_t)n, v.m);
  if ((uint32_t)n - q * v.d >= v.d) ++q;
  return (int)q;
}

struct GroupedArgs {
  const uint16_t* x;    // forward, dw: [T, K]
  const uint16_t* dy;   // dx, dw: [N, M]
  const uint16_t* w;    // forward, dx: [L, M, K]
  void* out;            // y [N, M], dx [N, K] or dw [L, M, K]
  const int* rows;      // permuted_rows, or NULL: row n of x
  const int* off;
  int L, T, k, N, K, M;
  uint32_t div_m, div_s;  // division by k (set by divide_by)
};

// e / k for 0 <= e < 2^31 as e m >> (31 + s): with s = ceil(log2 k) and
// m = ceil(2^(31 + s) / k), m k - 2^(31 + s) < k <= 2^s, so the product is off
// the true quotient by less than e / 2^31 / k < 1 / k.
inline void divide_by(int k, uint32_t* m, uint32_t* s) {
  uint32_t l = 0;
  while ((1u << l) < (uint32_t)k) ++l;
  *s = l;
  *m = (uint32_t)((((uint64_t)1 << (31 + l)) + k - 1) / k);
}

// The row of x that a selection e = permuted_rows[n] stands for, or -1 (a zero
// row) when e is out of [0, T k).
template <class Args>
__device__ __forceinline__ int token_of(const Args& a, int e) {
  const int t = (int)((uint64_t)(uint32_t)e * a.div_m >> (31 + a.div_s));
  return (uint32_t)e < (uint32_t)(a.T * a.k) ? t : -1;
}

// The row of x behind row n.
template <class Args>
__device__ __forceinline__ int source_row(const Args& a, int n) {
  return a.rows ? token_of(a, a.rows[n]) : n;
}

template <typename Out>
__device__ __forceinline__ Out out_value(float v);
template <>
__device__ __forceinline__ float out_value<float>(float v) { return v; }
template <>
__device__ __forceinline__ uint16_t out_value<uint16_t>(float v) { return f32_to_bf16_bits(v); }

// Stores the accumulators of two neighbouring 16 x 16 tiles (r 0..15 and
// 16..31 from `o` on, 16 output rows of `ld` elements), lane l holding r = 4
// (l / 16) + q of row l % 16 in each. The lanes exchange their values first, so
// that 4 neighbours store 64 consecutive bytes of a row: with a row's 64 bytes
// in lanes 16 apart, as the matrix instruction leaves them, a CU stores 31 GB/s,
// and 93 like this (all CUs together reach 5.6 TB/s, 22 GB/s each, either way,
// but the loads of a CU wait behind its stores: dW of 85 rows an expert, K
// 7168, M 2048, 690 against 607 us).
// r_left: r in the matrix from `o` on, a multiple of 8 in bf16 and of 4 in fp32;
// rows: rows from `o` on. Every lane of the wave calls it.
__device__ __forceinline__ u32x4 neighbours(const u32x4& v, int from) {
  u32x4 r;
#pragma unroll
  for (int i = 0; i < 4; ++i) r[i] = (uint32_t)__builtin_amdgcn_ds_bpermute(from * 4, (int)v[i]);
  return r;
}
__device__ __forceinline__ void store_two(float* o, size_t ld, const f32x4& a, const f32x4& b,
                                          int lane, int rows, int r_left) {
  const int from = (lane & 3) * 16 + (lane >> 2), n = lane >> 2, r = (lane & 3) * 4;
  const u32x4 va = neighbours(__builtin_bit_cast(u32x4, a), from), vb = neighbours(__builtin_bit_cast(u32x4, b), from);
  float* at = o + n * ld + r;
  if (n < rows && r < r_left) *reinterpret_cast<u32x4*>(at) = va;
  if (n < rows && r + 16 < r_left) *reinterpret_cast<u32x4*>(at + 16) = vb;
}
__device__ __forceinline__ void store_two(uint16_t* o, size_t ld, const f32x4& a, const f32x4& b,
                                          int lane, int rows, int r_left) {
#if defined(__HIP_DEVICE_COMPILE__)
  // g = l / 16 holds, after the exchange of a tile with g + 1 (g even), 8
  // consecutive r: 16 (g & 1) + 8 (g / 2) on
  const auto lo = __builtin_amdgcn_permlane16_swap(pack_bf16(a[0], a[1]), pack_bf16(b[0], b[1]), false, false);
  const auto hi = __builtin_amdgcn_permlane16_swap(pack_bf16(a[2], a[3]), pack_bf16(b[2], b[3]), false, false);
  const int p = lane & 3, n = lane >> 2, r = p * 8;
  const u32x4 v = neighbours(u32x4{lo[0], hi[0], lo[1], hi[1]}, ((p >> 1) | (p & 1) << 1) * 16 + n);
  if (n < rows && r < r_left) *reinterpret_cast<u32x4*>(o + n * ld + r) = v;
#endif
}
// To be called behind a tile's stores: the exchanges are done (each store waits
// for its own, but one whose lanes are all out of the matrix is jumped over, and
// the compiler would wait in the loop that follows).
__device__ __forceinline__ void stores_end() { __builtin_amdgcn_s_waitcnt(0xC07F); }

// Store instructions of a whole 256 x 256 tile in each of eight waves.
template <typename Out>
constexpr int kTileStores = sizeof(Out) == 4 ? 32 : 16;

}  // namespace moe
