// Products over rows grouped by expert, 16-byte path: 256 x 256 output tiles,
// both operands staged in LDS.
//
// D[r, c] = sum over kk of A[r, kk] B[c, kk] (grouped.h says what r, c and kk
// are in each product). An operand is "rows" when kk is contiguous in memory
// (W and x in the forward, dy in dx) and "columns" when r or c is (W in dx, x
// and dy in dw). Both go to LDS as they lie in memory, 32 or 64 of kk a stage, by
// loads that write LDS directly; the fragments of a column operand are read
// with the transposing LDS read (ds_read_b64_tr_b16), so no product needs a
// transposed copy of anything.
//
// What bounds it. Many rows an expert (8 experts of 2048 rows, K 4096, M 14336):
// forward 1.54, dx 1.53, dw 1.79 ms (1.25, 1.26, 1.08 PFLOP/s; torch's single
// products of one expert's size reach 1.42, 1.14, 1.02). Of the forward the matrix
// instructions alone take 1.43 ms and the loads alone 1.44 ms: a tile edge of 256
// asks for 16 GB from the L2s, a fifth of it missing there, and they deliver 11 TB/s
// of such a stream whatever the number of loads in flight; the clock is 1.9 GHz
// under this load. Routed counts end experts in parts of tiles: dx takes 1.79 ms
// with 69 tiles of rows for 64 (five rounds of tiles for 4.3). dw has the same
// stream, but ends a tile after 64 stages instead of 128, 4 to 5 us each time with
// its next loads behind the stores (1.65 ms for experts of 4096 rows and M 7168,
// 1.72 at 2048 and 14336, 1.85 at 1024 and 28672, all without selections), and its
// selections take 0.08 ms. The three one after the other take 5.5 ms, 0.4 more than
// by themselves, most of it in dw (2.0). Tens of rows (77 experts of 85, K 7168, M
// 2048): forward 0.44, dx 0.45 ms, 5.1 TB/s of weights; dw 0.61 ms, its 2.26 GB of
// stores alone 0.41 ms and its loads 0.31.
#include "grouped.h"
#include "lds_dma.h"
#include "operators.h"

#include <algorithm>

namespace moe {

namespace {

constexpr int D_T = 256;            // r extent of a tile, and c where c is M
constexpr int D_K = 32;  // contraction of a matrix instruction
constexpr int D_EXPERTS = 4096;  // most local experts
constexpr int D_SEL = 256;  // dw: bytes of a wave's place for a stage's selections
constexpr int D_THREADS = 512;

typedef short s16x4 __attribute__((ext_vector_type(4)));

// ---- the two LDS layouts of an operand's stage (written in pieces of 1 KB by the
// direct loads: lane i of piece b fills bytes 1024 b + 16 i)
//
// rows:    256 rows (128 of B in the narrow tiles) of a stage's K values: 64 bytes,
//          the 16 bytes q of row r at slot q ^ ((r >> 1) & 3), or 128 bytes, at
//          q ^ (r & 7), so a fragment read (16 rows, one 16-byte piece each) meets
//          no bank twice.
// columns: the stage's K rows (kk) of 512 bytes; in units of 32 bytes, unit u of
//          row kk sits at u ^ f(kk), f(kk) = (kk & 3) | ((kk >> 3) & 1) << 2, so
//          the 8 rows that half a wave reads together lie in 8 different units.

// Place of 16-byte piece q of row r in the rows layout, or the piece at place q.
template <int K>
__device__ __forceinline__ int piece(int q, int r) {
  return K == 32 ? q ^ ((r >> 1) & 3) : q ^ (r & 7);
}
// Byte offset, within the stage, of lane's part of a fragment of 16 rows and the
// first 32 of kk (the next 32 at ^ 64).
template <int K>
__device__ __forceinline__ uint32_t rows_lane(int lane) {
  return (uint32_t)((lane & 15) * 2 * K + piece<K>(lane >> 4, lane & 15) * 16);
}
// The same for 16 columns from unit 0; unit u is at ^ (32 (u & 7)) + 256 (u >> 3),
// half h (kk + 4) at + 2048 h.
__device__ __forceinline__ uint32_t cols_lane(int lane) {
  const int g = lane >> 4, j = (lane & 15) >> 2;
  const int f = j | ((g & 1) << 2);
  return (uint32_t)((8 * g + j) * 512 + f * 32 + (lane & 3) * 8);
}

__device__ __forceinline__ bf16x8 read_rows(uint32_t at) {
  return *reinterpret_cast<const __attribute__((address_space(3))) bf16x8*>(at);
}
__device__ __forceinline__ bf16x8 read_cols(uint32_t at) {
#if defined(__HIP_DEVICE_COMPILE__)
  typedef __attribute__((address_space(3))) s16x4* P;
  const s16x4 a = __builtin_amdgcn_ds_read_tr16_b64_v4i16((P)(at));
  const s16x4 b = __builtin_amdgcn_ds_read_tr16_b64_v4i16((P)(at + 2048));
  return __builtin_bit_cast(bf16x8, __builtin_shufflevector(a, b, 0, 1, 2, 3, 4, 5, 6, 7));
#else
  (void)at;
  return bf16x8{};
#endif
}

// A tile of the block's work.
struct Tile {
  int expert, beg, rows, r0, c0;
};

// Shape of a kernel: TC columns to a tile. 256 for experts with many rows,
// which the matrix cores bound; 128 for the others, which the stream of their
// weights bounds: their stages are 64 of the contraction, whole 128-byte lines
// of rows operands (85 rows an expert, K 7168, M 2048: forward 526 -> 463 us, dx
// 469 -> 461 against stages of 32 in six slots).
template <int TC>
struct Shape {
  static constexpr int K = TC == 256 ? 32 : 64;    // contraction of a stage
  static constexpr int A = D_T * K * 2;            // bytes of operand A's stage
  static constexpr int SLOT = A + TC * K * 2;      // bytes of a stage
  static constexpr int SLOTS = TC == 256 ? 4 : 3;
  static constexpr int AN = A / 8192;              // pieces of A that a wave loads per stage
  static constexpr int BN = TC * K * 2 / 8192;     // and of B
  static constexpr int LOADS = AN + BN;
  // Whether a stage's loads are issued in front of the wait for the next stage,
  // and the stages of loads that may then be in flight.
  static constexpr bool EARLY = TC == 128;
  static constexpr int AHEAD = EARLY ? SLOTS - 2 : SLOTS - 3;
  static constexpr int CG = TC / 64;   // groups of 16 columns of a wave
};

template <Product P, int TC>
struct Work {
  GroupWalk walk;  // forward, dx
  int RT, CT, R;
  uint32_t off;           // dw: the experts' offsets in LDS
  Divisor by_expert, by_band;  // dw: tiles of an expert, and of four of its c

  __device__ __forceinline__ void start(const GroupedArgs& a, int lo, int hi, const Divisor& expert,
                                        const Divisor& band) {
    by_expert = expert;
    by_band = band;
    R = P == Product::kForward ? a.M : a.K;
    RT = (R + D_T - 1) / D_T;
    CT = (a.M + D_T - 1) / D_T;
    if (P != Product::kDw) walk.start(a.off, a.L, a.N, RT, TC, lo, hi);
  }
  // Tiles of one expert are numbered r tile by r tile, its passes of TC rows
  // side by side (dw: in blocks of 8 r by 4 c): the 32 blocks that run together
  // on an XCD share operand lines in its L2, 12 tile edges' worth a stage for
  // 32 tiles (dw numbered row by row: 18, and a third of the loads from memory).
  __device__ __forceinline__ bool find(const GroupedArgs& a, GroupWalk::Place& place, int t, Tile* o) {
    if (P == Product::kDw) {
      const int per = RT * CT;
      if (t >= a.L * per) return false;
      o->expert = divide(t, by_expert);
      const int i = t - o->expert * per;
      const int band = divide(i, by_band), wide = min(4, CT - 4 * band);
      const int in_band = i - band * 4 * RT;
      // (shifts but in the last band: a division is some forty instructions)
      const int part = wide == 4 ? in_band >> 5 : in_band / (8 * wide);
      const int at = in_band - part * 8 * wide;
      const int r = wide == 4 ? at >> 2 : at / wide;
      o->c0 = (4 * band + at - r * wide) * D_T;
      o->r0 = (8 * part + r) * D_T;
      typedef const __attribute__((address_space(3))) int* Lds;
      const int b = *reinterpret_cast<Lds>(off + 4 * o->expert);
      const int e = *reinterpret_cast<Lds>(off + 4 * o->expert + 4);
      o->beg = __builtin_amdgcn_readfirstlane(max(0, min(b, a.N)));
      o->rows = __builtin_amdgcn_readfirstlane(max(o->beg, min(e, a.N)) - o->beg);
      return true;
    }
    GroupTile g;
    if (!walk.find(place, t, &g)) return false;
    const int passes = (g.rows + TC - 1) / TC;
    o->expert = g.expert;
    o->beg = g.beg;
    o->rows = g.rows;
    o->r0 = (g.tile / passes) * D_T;
    o->c0 = (g.tile % passes) * TC;
    return true;
  }
};

// A stage of the block's work: Shape<TC>::K of the contraction of a tile.
template <Product P, int TC>
struct Cursor {
  Work<P, TC>& work;
  GroupWalk::Place place;
  Tile tile;
  int t, kc, nk;  // tile number, stage within the tile, stages of the tile

  __device__ __forceinline__ int contraction(const GroupedArgs& a) const {
    return P == Product::kForward ? a.K : P == Product::kDx ? a.M : tile.rows;
  }
  // False past the block's last tile. An expert without rows has one stage in
  // dw, of zeros.
  __device__ __forceinline__ bool at(const GroupedArgs& a, int tile_number) {
    t = tile_number;
    kc = 0;
    if (!work.find(a, place, t, &tile)) return false;
    nk = max(1, (contraction(a) + Shape<TC>::K - 1) / Shape<TC>::K);
    return true;
  }
};

// The wave's loads: AN pieces of A's stage, from AN w on, and BN of B's.
// PICKS: dw whose x rows go by selections.
template <Product P, bool PICKS, int TC>
struct Loads {
  static constexpr int AN = Shape<TC>::AN, BN = Shape<TC>::BN, K = Shape<TC>::K;
  static constexpr int LPR = K / 8;  // lanes (16-byte pieces) to a row of the rows layout
  static constexpr bool A_ROWS = P == Product::kForward;
  static constexpr bool B_ROWS = P != Product::kDw;
  u32x4 ra, rb;
  uint32_t va[AN], vb[BN];
  uint32_t src[AN];  // dw: the next stage's rows of x
  int pick[AN];      // and their selections

  __device__ __forceinline__ void tile(const GroupedArgs& a, const Tile& t, int wave, int lane) {
    const int R = P == Product::kForward ? a.M : a.K;
    const int C = P == Product::kDw ? a.M : t.rows;
    const size_t wsize = (size_t)a.M * a.K;
    ra = P == Product::kDw ? buffer_over(a.x, (uint32_t)((size_t)a.T * a.K * 2))
                           : buffer_over(a.w + (size_t)t.expert * wsize, (uint32_t)(wsize * 2));
    rb = P == Product::kForward ? buffer_over(a.x, (uint32_t)((size_t)a.T * a.K * 2))
                                : buffer_over(a.dy, (uint32_t)((size_t)a.N * a.M * 2));
#pragma unroll
    for (int j = 0; j < AN; ++j) {
      const int b = AN * wave + j;
      const int r16 = 64 / LPR * b + lane / LPR, q = piece<K>(lane % LPR, lane / LPR);  // rows layout
      const int kk = 2 * b + (lane >> 5);                                       // columns layout
      const int c8 = ((lane & 31) ^ (((kk & 3) | (((kk >> 3) & 1) << 2)) << 1)) * 8;
      if (A_ROWS) {
        const int r = t.r0 + r16;
        va[j] = r < R ? ((uint32_t)r * a.K + q * 8) * 2u : kPastEnd;
      } else {
        const int r = t.r0 + c8;
        va[j] = r < R ? ((P == Product::kDx ? (uint32_t)kk * a.K : 0u) + r) * 2u : kPastEnd;
      }
    }
#pragma unroll
    for (int j = 0; j < BN; ++j) {
      const int b = BN * wave + j;
      if (B_ROWS) {
        const int c = t.c0 + 64 / LPR * b + lane / LPR, q = piece<K>(lane % LPR, lane / LPR);
        int s = -1;
        if (c < C) s = P == Product::kForward ? source_row(a, t.beg + c) : t.beg + c;
        vb[j] = s >= 0 ? ((uint32_t)s * (P == Product::kForward ? a.K : a.M) + q * 8) * 2u : kPastEnd;
      } else {
        const int kk = 2 * b + (lane >> 5);
        const int c = t.c0 + ((lane & 31) ^ (((kk & 3) | (((kk >> 3) & 1) << 2)) << 1)) * 8;
        vb[j] = c < C ? ((uint32_t)(t.beg + kk) * a.M + c) * 2u : kPastEnd;
      }
    }
  }
  // The selections behind this lane's rows of a dw stage; sel: LDS place of the
  // stage's selections.
  __device__ __forceinline__ void picks(uint32_t sel, int wave, int lane) {
#pragma unroll
    for (int j = 0; j < AN; ++j) {
      const int kk = 2 * (AN * wave + j) + (lane >> 5);
      pick[j] = *reinterpret_cast<const __attribute__((address_space(3))) int*>(sel + 4 * kk);
    }
  }
  // Byte offsets of the rows of x behind those rows, past the end for a zero row.
  __device__ __forceinline__ void sources(const GroupedArgs& a, const Cursor<P, TC>& c, int wave,
                                          int lane) {
#pragma unroll
    for (int j = 0; j < AN; ++j) {
      const int n = c.kc * K + 2 * (AN * wave + j) + (lane >> 5);
      const int s = PICKS ? token_of(a, pick[j]) : c.tile.beg + n;
      src[j] = n < c.tile.rows && s >= 0 ? (uint32_t)s * (uint32_t)a.K * 2u : kPastEnd;
    }
  }
  // Starts the stage's loads into `slot`.
  __device__ __forceinline__ void issue(const GroupedArgs& a, const Cursor<P, TC>& c, uint32_t slot,
                                        int wave, int lane) {
    const int k0 = c.kc * K, KK = c.contraction(a);
    const bool q_in = k0 + piece<K>(lane % LPR, lane / LPR) * 8 < KK;  // rows layout
    uint32_t at_a[AN], at_b[BN];
#pragma unroll
    for (int j = 0; j < AN; ++j) {
      const int kk = 2 * (AN * wave + j) + (lane >> 5);  // columns layout
      const uint32_t v = va[j];
      if (A_ROWS)
        at_a[j] = q_in ? v : kPastEnd;
      else if (P == Product::kDx)
        at_a[j] = k0 + kk < KK ? v : kPastEnd;
      else
        at_a[j] = src[j] == kPastEnd || v == kPastEnd ? kPastEnd : src[j] + v;
    }
    dma16_run<false>(ra, slot + AN * wave * 1024u, at_a,
                     A_ROWS ? (uint32_t)k0 * 2u : P == Product::kDx ? (uint32_t)k0 * (uint32_t)a.K * 2u : 0u);
#pragma unroll
    for (int j = 0; j < BN; ++j) {
      const bool in = B_ROWS ? q_in : k0 + 2 * (BN * wave + j) + (lane >> 5) < KK;
      at_b[j] = in ? vb[j] : kPastEnd;
    }
    dma16_run<false>(rb, slot + Shape<TC>::A + BN * wave * 1024u, at_b,
                     (uint32_t)k0 * 2u * (B_ROWS ? 1u : (uint32_t)a.M));
  }
};

// Eight waves: 128 of r x CG groups of 16 of c each (every fourth group of the
// tile's, so that the waves share a partly filled tile evenly). A stage is two
// parts with a block barrier after each: reading its fragments from LDS (and
// starting the loads of the stage S - 1 ahead, S the number of slots), and its
// matrix instructions. Waves 4-7 run one part behind waves 0-3 (they meet one
// barrier more at the start), and waves w and w + 4 share a SIMD: while one of
// them multiplies the other reads.
//
// Stage i + S goes into the slot of stage i. Count the parts by the barriers
// that end them: waves 0-3 read stage i in part 2 i, waves 4-7 in part 2 i + 1,
// and wait for what they read before the barrier. The first load into the slot is
// issued in the reading part of stage i + 1, by waves 0-3 in part 2 i + 2. It is
// waited for in the reading part of stage i + S - 1, part 2 (i + S) - 2 or one
// later, and first read in part 2 (i + S). Behind the stage waited for, loads of
// AHEAD stages are then in flight: S - 3 where that part's own loads are issued
// behind the wait (256 columns: stages i + S + 1 .. i + 2 S - 3), S - 2 where they
// are issued in front of it (EARLY, 128 columns: one stage more).
//
// dw's x rows go by selections, which have to be there when the loads are
// issued: they are loaded three stages further ahead, each wave its own copy,
// the wait that publishes a stage covers them, and the rows' offsets are worked
// out among the matrix instructions of the stage before they are used.
//
// The stages between two changes of tile run in a loop of straight code: a
// taken branch costs the wave a refill of its instruction buffer, and with the
// tile changes inside the loop (ten branches a stage) a part took 400 cycles
// before it did any work.
template <Product P, bool PICKS, int TC>
constexpr int lds_bytes() {
  return Shape<TC>::SLOTS * Shape<TC>::SLOT + (PICKS ? 8 * 4 * D_SEL : 0) +
         (P == Product::kDw ? (D_EXPERTS + 1) * 4 : 0);
}

// Tiles t, t + gridDim.x, .. of the experts with more than lo and at most hi
// rows; lds: lds_bytes of it. Returns by how much the next of these numbers is
// past the last tile.
template <Product P, bool PICKS, int TC, typename Out>
__device__ __forceinline__ int dense_tiles(const GroupedArgs& a, uint8_t* lds, int lo, int hi, int t,
                                           Divisor by_expert, Divisor by_band) {
  constexpr bool DW = P == Product::kDw;
  static_assert(!DW || TC == D_T, "dw's columns are M");
  using S = Shape<TC>;
  constexpr int CG = S::CG, H = S::K / D_K;
  constexpr int SEL = S::SLOTS * S::SLOT, OFF = SEL + (PICKS ? 8 * 4 * D_SEL : 0);
  using LD = Loads<P, PICKS, TC>;
  const int lane = threadIdx.x % kWave;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
  const int wr = wave & 1, wc = wave >> 1;
  const bool behind = wave >= 4;
  const uint32_t lds0 = lds_address(lds);
  const uint32_t sel0 = lds0 + SEL + wave * 4 * D_SEL;
  const int step = gridDim.x;

  // the stages being multiplied, loaded, and (PICKS) having their selections loaded
  Work<P, TC> work;
  work.start(a, lo, hi, by_expert, by_band);
  if (DW) {
    // from LDS, a change of expert does not wait for the loads and stores in
    // flight, as reading the offsets from memory would
    work.off = lds0 + OFF;
    for (int i = threadIdx.x; i <= a.L; i += D_THREADS) reinterpret_cast<int*>(lds + OFF)[i] = a.off[i];
    __syncthreads();
  }
  Cursor<P, TC> cm{work};
  auto past = [&]() { return DW ? 0 : cm.t - (cm.place.before + work.walk.total); };
  if (!cm.at(a, t)) return past();
  Cursor<P, TC> cl = cm, cs = cm;
  const int R = work.R;
  const u32x4 rr = buffer_over(a.rows, (uint32_t)a.N * 4u);
  bool more = true, more_sel = PICKS;  // stages left to load, to select for
  int nl = 0, ns = 0;  // stages loaded, and with selections loaded
  auto select = [&]() {  // always one load, so that the waits can count on it
    const uint32_t at = (uint32_t)(cs.tile.beg + cs.kc * S::K + lane) * 4u;
    dma4(rr, sel0 + (ns & 3) * D_SEL, more_sel ? at : kPastEnd);
    if (more_sel) {
      ++ns;
      ++cs.kc;
    }
  };
  LD ld;
  ld.tile(a, cl.tile, wave, lane);
  uint32_t into = lds0;  // slot of the next load
  auto load = [&]() {
    ld.issue(a, cl, into, wave, lane);
    into = into == lds0 + (S::SLOTS - 1) * S::SLOT ? lds0 : into + S::SLOT;
    ++nl;
    ++cl.kc;
  };
  auto picks = [&](int stage) {  // of the stage of that number
    if (PICKS) ld.picks(sel0 + (stage & 3) * D_SEL, wave, lane);
  };
  auto sources = [&]() {  // for the next load, from its selections
    if (DW) ld.sources(a, cl, wave, lane);
  };
  auto next_load = [&]() {  // to the next tile where the last one is loaded
    if (more && cl.kc == cl.nk) {
      more = cl.at(a, cl.t + step);
      if (more) {
        ld.tile(a, cl.tile, wave, lane);
        picks(nl);
        sources();
      }
    }
    if (PICKS && more_sel && cs.kc == cs.nk) more_sel = cs.at(a, cs.t + step);
  };

  auto groups = [&]() {  // this wave's 16-column groups that hold columns
    const int C = DW ? a.M : cm.tile.rows;
    const int ng = (min(TC, C - cm.tile.c0) + 15) >> 4;
    return __builtin_amdgcn_readfirstlane(min(CG, max(0, (ng - wc + 3) >> 2)));
  };
  int nv = groups();

  // fragment addresses within a stage
  const uint32_t la = LD::A_ROWS ? rows_lane<S::K>(lane) + wr * (256 * S::K) : cols_lane(lane) + wr * 256;
  const uint32_t lb = S::A + (LD::B_ROWS ? rows_lane<S::K>(lane) + wc * (32 * S::K) : cols_lane(lane));
  f32x4 acc[8][CG];
  auto clear = [&]() {
#pragma unroll
    for (int i = 0; i < 8; ++i)
#pragma unroll
      for (int j = 0; j < CG; ++j) acc[i][j] = f32x4{0.f, 0.f, 0.f, 0.f};
  };
  clear();
  uint32_t from = lds0;  // slot of the stage being multiplied
  // A whole tile's stores are STORES instructions. Stage t behind them waits for
  // stage t + 1, whose loads were issued S - 1 stages before that: for t up to S - 2
  // in front of the stores, which may then still be in flight, as the AHEAD stages
  // of loads behind those waited for may.
  constexpr int STORES = kTileStores<Out> * CG / 4;
  constexpr int FLIGHT = S::AHEAD * (S::LOADS + (PICKS ? 1 : 0));
  int after_stores = 0;

  if (PICKS) {
    for (int i = 0; i < 4; ++i) {
      select();
      next_load();
    }
    wait_loads<0>();
  }
  picks(nl);
  sources();
  for (int i = 0; i < S::SLOTS - 1 && more; ++i) {
    load();
    picks(nl);
    sources();
    next_load();
  }
  if (PICKS) {
    for (int i = 0; i < 2; ++i) {
      select();
      next_load();
    }
  }
  wait_loads<0>();
  picks(nl);
  sources();
  meet();
  if (behind) meet();

  for (;;) {
    int run = cm.nk - cm.kc;
    if (more) run = min(run, cl.nk - cl.kc);
    if (PICKS && more_sel) run = min(run, cs.nk - cs.kc);
    const bool soft = after_stores > 0;
    if (soft) {
      run = min(run, after_stores);
      after_stores -= run;
    }
    cm.kc += run;
    for (int i = 0; i < run; ++i) {
      bf16x8 fa[H][8], fb[H][CG];
      // (in this order, an address right before its reads: with the additions
      // gathered in front of the reads dx and dw took 3% longer)
#pragma unroll
      for (int h = 0; h < H; ++h) {
#pragma unroll
        for (int r = 0; r < 8; ++r) {
          fa[h][r] = LD::A_ROWS ? read_rows(from + (la ^ (h * 64)) + r * (32 * S::K))
                                : read_cols(from + (la ^ (r * 32)) + h * (D_K * 512));
          __builtin_amdgcn_sched_barrier(0);
        }
#pragma unroll
        for (int c = 0; c < CG; ++c) {
          const int u = c * 4 + wc;  // group of 16 columns
          fb[h][c] = LD::B_ROWS ? read_rows(from + (lb ^ (h * 64)) + c * (128 * S::K))
                                : read_cols(from + (lb ^ ((u & 7) * 32)) + (u >> 3) * 256);
          __builtin_amdgcn_sched_barrier(0);
        }
      }
      // the next stage's loads are the oldest in flight
      if (__builtin_expect(more, 1)) {
        if (S::EARLY) load();
        if (__builtin_expect(soft, 0)) wait_loads<STORES + FLIGHT>();
        else wait_loads<FLIGHT>();
        picks(nl + 1);
        if (!S::EARLY) load();
        if (PICKS) select();
      } else {
        wait_loads<0>();
      }
      wait_lds();
      meet();
      __builtin_amdgcn_sched_barrier(0);
      __builtin_amdgcn_s_setprio(1);
#pragma unroll
      for (int c = 0; c < CG; ++c) {
        if (__builtin_expect(c < nv, 1)) {
#pragma unroll
          for (int h = 0; h < H; ++h)
#pragma unroll
            for (int r = 0; r < 8; ++r)
              acc[r][c] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(fa[h][r], fb[h][c], acc[r][c], 0, 0, 0);
        }
        if (c == 2) sources();  // next to the matrix instructions
      }
      __builtin_amdgcn_s_setprio(0);
      __builtin_amdgcn_sched_barrier(0);
      meet();
      from = from == lds0 + (S::SLOTS - 1) * S::SLOT ? lds0 : from + S::SLOT;
    }
    next_load();
    if (cm.kc == cm.nk) {
      const Tile& cur = cm.tile;
      const int C = DW ? a.M : cur.rows;
      Out* out = static_cast<Out*>(a.out) +
                 (DW ? (size_t)cur.expert * a.M * a.K : (size_t)cur.beg * R);
#pragma unroll
      for (int j = 0; j < CG; ++j) {
        const int c = cur.c0 + (j * 4 + wc) * 16;
        Out* o = out + (size_t)c * R + cur.r0 + wr * 128;
#pragma unroll
        for (int i = 0; i < 8; i += 2)
          store_two(o + i * 16, R, acc[i][j], acc[i + 1][j], lane, C - c, R - (cur.r0 + wr * 128 + i * 16));
      }
      stores_end();
      after_stores = cur.c0 + TC <= C && cur.r0 + D_T <= R ? S::SLOTS - 2 : 0;
      clear();
      if (!cm.at(a, cm.t + step)) break;
      nv = groups();
    }
  }
  if (!behind) meet();
  return past();
}

// dw of all experts.
template <bool PICKS, typename Out>
__global__ __launch_bounds__(D_THREADS, 1) void grouped_dw_kernel(GroupedArgs a, Divisor by_expert,
                                                                  Divisor by_band) {
  __shared__ __align__(1024) uint8_t lds[lds_bytes<Product::kDw, PICKS, 256>()];
  dense_tiles<Product::kDw, PICKS, 256, Out>(a, lds, 0, kAnyRows, xcd_block(blockIdx.x, gridDim.x),
                                             by_expert, by_band);
}

// Forward or dx of the experts with more than lo rows. Experts with at most
// kNarrowRows rows go to the narrow tiles. (77 experts, K 7168, M 2048, skewed
// counts, forward at 50, 85, 125, 167 rows an expert on average, us: limit 64: 465,
// 569, 588, 608; 128: 480, 537, 505, 567; 256: 431, 536, 550, 620.) Those are
// numbered on behind the wide ones, so that the blocks share all tiles evenly.
template <Product P, typename Out>
__global__ __launch_bounds__(D_THREADS, 1) void grouped_dense_kernel(GroupedArgs a, int lo) {
  constexpr int WIDE = lds_bytes<P, false, 256>(), NARROW = lds_bytes<P, false, 128>();
  __shared__ __align__(1024) uint8_t lds[WIDE > NARROW ? WIDE : NARROW];
  if (lo > 0) {  // the experts with fewer rows, if the kernel for them left them
    GroupWalk walk;
    walk.start(a.off, a.L, a.N, 1, 1, 0, lo);
    if (walk.rounds_hold(lo, (a.M + 255) / 256, gridDim.x)) lo = 0;
  }
  int t = xcd_block(blockIdx.x, gridDim.x);
  if (a.N > kNarrowRows) t = dense_tiles<P, false, 256, Out>(a, lds, kNarrowRows, kAnyRows, t, {}, {});
  dense_tiles<P, false, 128, Out>(a, lds, lo, kNarrowRows, t, {}, {});
}

template <Product P>
void launch_rows(const GroupedArgs& a, bool f32, int lo, int blocks, hipStream_t s) {
  const dim3 g(blocks), b(D_THREADS);
  if (f32) hipLaunchKernelGGL((grouped_dense_kernel<P, float>), g, b, 0, s, a, lo);
  else hipLaunchKernelGGL((grouped_dense_kernel<P, uint16_t>), g, b, 0, s, a, lo);
}

template <bool PICKS>
void launch_dw(const GroupedArgs& a, bool f32, int blocks, hipStream_t s) {
  const dim3 g(blocks), b(D_THREADS);
  const int RT = (a.K + D_T - 1) / D_T, CT = (a.M + D_T - 1) / D_T;
  const Divisor expert = divisor(RT * CT), band = divisor(4 * RT);
  if (f32) hipLaunchKernelGGL((grouped_dw_kernel<PICKS, float>), g, b, 0, s, a, expert, band);
  else hipLaunchKernelGGL((grouped_dw_kernel<PICKS, uint16_t>), g, b, 0, s, a, expert, band);
}

}  // namespace

// Forward and dx of the experts with more than `lo` rows, or dw of all.
hipError_t launch_grouped_dense(Product p, const GroupedArgs& a, bool out_fp32, int lo, int blocks,
                                hipStream_t stream) {
  if (p == Product::kForward) launch_rows<Product::kForward>(a, out_fp32, lo, blocks, stream);
  if (p == Product::kDx) launch_rows<Product::kDx>(a, out_fp32, lo, blocks, stream);
  if (p == Product::kDw && a.rows) launch_dw<true>(a, out_fp32, blocks, stream);
  if (p == Product::kDw && !a.rows) launch_dw<false>(a, out_fp32, blocks, stream);
  return hipGetLastError();
}

}  // namespace moe
