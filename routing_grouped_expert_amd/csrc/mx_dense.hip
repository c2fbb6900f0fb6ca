// Grouped product on microscaled operands for experts with many rows: 256 x
// 256 output tiles, both operands and their scales staged in LDS.
//
// The schedule is that of the bf16 products (grouped_dense.hip): eight waves
// of 128 weight rows x 64 tokens, a stage in two parts (reading, and 32 matrix
// instructions), waves 4-7 one part behind waves 0-3 on the same SIMDs. A
// stage is 128 of the contraction, one scaled matrix instruction deep: 64
// bytes of a weight row and 128 (E4M3) or 64 (E2M1) of a token's, in three to
// five LDS slots, all but one of them loading while one is multiplied; for experts
// with few rows 256 of it. Scales are loaded 16 codes of a row at a time, for runs
// of two to four stages: four at a time they were 40% of the load requests (share
// of 77 experts at 32768 tokens, K 7168, M 4096: 1408 against 1289 us).
//
// With E4M3 rows that case is bound by the matrix cores, which multiply each
// fragment in two parts (mx_matmul.h): 1.89 ms, 1.65 PFLOP/s of useful products and
// 3.3 of the instruction's (torch's fp8 product of 8192^3 reaches 2.7), 2.1 to 2.2 ms
// for routed counts; one part took 1.2 and 1.3. E2M1 rows: 1.06 ms, 2.9 PFLOP/s,
// bound by the stages' LDS traffic beside them. At 85 and 50 rows an expert, E4M3:
// 390 us, matrix instructions and the weights' stream (3.1 TB/s) alike, and 270, 4.5
// TB/s; E2M1: 300 and 238.
#include "lds_dma.h"
#include "mx_matmul.h"
#include "operators.h"

namespace moe {

namespace {

constexpr int X_T = 256;  // weight rows of a tile
constexpr int X_THREADS = 512;
constexpr int X_FEW = 64;  // rows of an expert that goes to the narrowest tiles
constexpr int X_S = X_T * 16;  // bytes of the weights' scales for a run

// Shape of a kind of tile: TC tokens. 256 for experts with many rows; 128 and 64
// for the others, which the stream of their weights bounds: 128 leaves room for
// more stages in flight, 64 for stages of 256 of the contraction, whole 128-byte
// lines of the weights (77 experts, K 7168, M 4096, E4M3 rows, us with 64 / 128
// tokens: 50 rows an expert 282 / 382, 64 282 / 380, 85 in two passes 457 / 399).
template <int XBITS, int TC>
struct Shape {
  static constexpr int K = TC == 64 ? 256 : 128;   // contraction of a stage
  static constexpr int KB = K / kMxBlock;          // its scales of a row
  static constexpr int H = K / 128;                // its matrix instructions' depths
  static constexpr int WROW = K / 2, XROW = K / 8 * XBITS;  // bytes of a stage's rows
  static constexpr int W = X_T * WROW, X = TC * XROW;
  static constexpr int SLOT = W + X, SLOTS = TC != 128 ? 3 : XBITS == kMxFp8 ? 4 : 5;
  static constexpr int RUN = X_S + TC * 16;  // bytes of a run's scales
  static constexpr int RUNS = TC == 256 ? 2 : 3;
  static constexpr int CG = TC / 64;  // groups of 16 tokens of a wave
  static constexpr int BYTES = SLOTS * SLOT + RUNS * RUN;  // of LDS
};

// ---- LDS layouts. Piece q (16 bytes) of row r sits at place q ^ ((r >> 1) & 3) in
// rows of 64 bytes, at q ^ (r & 7) in rows of 128 and at q ^ (r & 15) in rows of
// 256, so that a fragment read (16 rows, one piece each) meets no bank twice.
// Scales: the sixteen codes of row r at 16 r of the run's place, weights first.
template <int ROW>
__device__ __forceinline__ int piece_of(int place, int r) {
  return place ^ (ROW == 64 ? (r >> 1) & 3 : r & (ROW / 16 - 1));
}

typedef const __attribute__((address_space(3))) i32x4* LdsVec;
typedef const __attribute__((address_space(3))) uint8_t* LdsByte;

// This wave's loads of an operand of R rows with ROW bytes a stage: pieces of 1 KB.
template <int ROW, int R>
struct Rows {
  static constexpr int N = R * ROW / 8192;  // pieces a wave loads per stage
  static constexpr int LPR = ROW / 16;      // lanes to a row of a piece
  u32x4 rs;
  uint32_t v[N];

  // row(i): the memory row behind tile row i, or -1.
  template <class Row>
  __device__ __forceinline__ void tile(const uint8_t* base, size_t bytes, int row_bytes, int wave,
                                       int lane, Row row) {
    rs = buffer_over(base, (uint32_t)min(bytes, kMostBytes));
#pragma unroll
    for (int j = 0; j < N; ++j) {
      const int i = (N * wave + j) * (64 / LPR) + lane / LPR;
      const int m = row(i);
      v[j] = m >= 0 ? (uint32_t)m * row_bytes + piece_of<ROW>(lane % LPR, i) * 16 : kPastEnd;
    }
  }
  // The pieces of stage kc into LDS at `to`; pieces past the row's end as zeros.
  __device__ __forceinline__ void issue(int kc, int row_bytes, uint32_t to, int wave, int lane) {
    const int at = kc * ROW;
    uint32_t from[N];
#pragma unroll
    for (int j = 0; j < N; ++j) {
      const int i = (N * wave + j) * (64 / LPR) + lane / LPR;
      const bool in = at + piece_of<ROW>(lane % LPR, i) * 16 < row_bytes;
      from[j] = in ? v[j] : kPastEnd;
    }
    dma16_run<false>(rs, to + N * wave * 1024u, from, (uint32_t)at);
  }
};

// TIMES times in the compiler's order: MATRIX matrix instructions, VECTOR others.
// An E4M3 fragment has 16 and 40 (8 for its small part, 32 for the next one's large
// part), for which the matrix cores would stand still if they came together (683
// rows an expert 1979 us in the compiler's own order; 1964 one by one; 1929 with the
// first four by themselves. Narrower tiles, 50 rows: 271 one by one, 279).
template <int MATRIX, int VECTOR, int TIMES>
__device__ __forceinline__ void mx_order() {
#pragma unroll
  for (int r = 0; r < TIMES; ++r) {
    __builtin_amdgcn_sched_group_barrier(8, MATRIX, 0);
    __builtin_amdgcn_sched_group_barrier(2, VECTOR, 0);
  }
}

// Tiles tm, tm + gridDim.x, .. of the experts with more than lo and at most hi
// rows. Returns by how much the next of these numbers is past the last tile.
template <int XBITS, int TC, typename Out>
__device__ __forceinline__ int mx_dense_tiles(const MxArgs& a, uint8_t* lds, int lo, int hi, int tm) {
  using S = Shape<XBITS, TC>;
  constexpr int SLOT = S::SLOT, CG = S::CG, H = S::H;
  constexpr int LOADS = Rows<S::WROW, X_T>::N + Rows<S::XROW, TC>::N;  // a wave's per stage
  constexpr int SCALES = S::SLOTS * SLOT;
  const int lane = threadIdx.x % kWave;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
  const int wr = wave & 1, wc = wave >> 1;
  const bool behind = wave >= 4;
  const uint32_t lds0 = lds_address(lds);
  const int step = gridDim.x;
  const int KB = a.K / kMxBlock;
  // Stages of a tile, and the runs that share a load of scales. 64 tokens: two
  // stages (or one at the end), so that three slots reach into three runs. 256 and
  // 128: from kc = 0, 4, 8, .., but where the last would be a single stage the last
  // five are three and two. No run is one stage (K <= 128 takes a second one of
  // zeros), so the stages of the slots reach into two runs (three slots) or three.
  const int nk = TC > 64 ? max(2, (KB + 3) / 4) : (KB + S::KB - 1) / S::KB;
  auto next_run = [&](int kc) { return kc + (TC == 64 ? 2 : kc + 4 == nk - 1 ? 3 : 4); };
  const int RT = (a.M + X_T - 1) / X_T;
  const int wbytes = a.K / 2, xbytes = a.K / 8 * XBITS;

  GroupWalk walk;
  GroupWalk::Place wl, wm;  // of the tiles being loaded, and multiplied
  walk.start(a.off, a.L, a.N, RT, TC, lo, hi);
  struct Tile {
    int expert, beg, rows, r0, c0, kc;
  };
  auto find = [&](GroupWalk::Place& w, int t, Tile* o) {
    GroupTile g;
    if (!walk.find(w, t, &g)) return false;
    const int passes = (g.rows + TC - 1) / TC;
    *o = Tile{g.expert, g.beg, g.rows, (g.tile / passes) * X_T, (g.tile % passes) * TC, 0};
    return true;
  };
  int tl = tm;
  Tile cl, cm;
  auto past = [&]() { return tm - (wm.before + walk.total); };
  if (!find(wm, tm, &cm)) return past();
  find(wl, tl, &cl);

  Rows<S::WROW, X_T> lw;
  Rows<S::XROW, TC> lx;
  const bool scaler = wave < 4 + TC / 64;
  u32x4 rscale;      // waves 0-3: scales of 64 weight rows each, from 4 on of 64 tokens
  uint32_t vscale;   // this lane's row's first scale
  uint32_t scale_end;  // bytes behind rscale's base
  bool edge;           // a lane's scales may end the array
  auto tile_loads = [&]() {
    // (a copy that hides its value: what is computed from it is not kept in
    // registers, which the stage loop has none left of; with E4M3 rows one or two
    // values are still stored to memory and read back here)
    int lane = threadIdx.x % kWave;
    asm volatile("" : "+v"(lane));
    const size_t left = (size_t)(a.L - cl.expert) * a.M;  // weight rows to the end
    const uint8_t* wq = a.wq + (size_t)cl.expert * a.M * wbytes;
    lw.tile(wq, left * wbytes, wbytes, wave, lane, [&](int i) {
      return cl.r0 + i < a.M ? cl.r0 + i : -1;
    });
    auto token = [&](int i) {
      return cl.c0 + i < cl.rows ? source_row(a, cl.beg + cl.c0 + i) : -1;
    };
    lx.tile(a.xq, (size_t)a.T * xbytes, xbytes, wave, lane, token);
    if (!scaler) return;
    const int i = (wave & 3) * 64 + lane;
    int m;
    if (wave < 4) {
      m = cl.r0 + i < a.M ? cl.r0 + i : -1;
      scale_end = (uint32_t)min(left * KB, kMostBytes);
      rscale = buffer_over(a.ws + (size_t)cl.expert * a.M * KB, scale_end);
    } else {
      m = token(i);
      scale_end = (uint32_t)((size_t)a.T * KB);
      rscale = buffer_over(a.xs, scale_end);
    }
    vscale = m >= 0 ? (uint32_t)m * (uint32_t)KB : kPastEnd;
    edge = at_edge(vscale, KB, scale_end);
  };
  tile_loads();
  bool more = true;
  uint32_t into = lds0;                // slot of the next load
  int run_l = 0;                       // where the next run starts
  uint32_t to_scales = lds0 + SCALES;  // and its place
  bool fresh = false;                  // the last load() loaded scales
  auto next_place = [&](uint32_t at) {
    return at == lds0 + SCALES + (S::RUNS - 1) * S::RUN ? lds0 + SCALES : at + S::RUN;
  };
  auto load = [&]() {
    lw.issue(cl.kc, wbytes, into, wave, lane);
    lx.issue(cl.kc, xbytes, into + S::W, wave, lane);
    fresh = cl.kc == run_l;
    if (fresh) {
      if (scaler)
        dma16_bytes(rscale, wave < 4 ? a.ws + (size_t)cl.expert * a.M * KB : a.xs, scale_end,
                    to_scales + wave * 1024u, vscale == kPastEnd ? kPastEnd : vscale + cl.kc * (uint32_t)S::KB,
                    lane, edge);
      else
        fresh = false;
      to_scales = next_place(to_scales);
      run_l = next_run(run_l);
    }
    into = into == lds0 + (S::SLOTS - 1) * SLOT ? lds0 : into + SLOT;
    ++cl.kc;
  };
  auto next_load = [&]() {
    if (more && cl.kc == nk) {
      tl += step;
      run_l = 0;
      more = find(wl, tl, &cl);
      if (more) tile_loads();
    }
  };
  auto groups = [&]() {
    const int ng = (min(TC, cm.rows - cm.c0) + 15) >> 4;
    return __builtin_amdgcn_readfirstlane(min(CG, max(0, (ng - wc + 3) >> 2)));
  };
  int nv = groups();

  const int g = lane >> 4;
  const uint32_t la = (uint32_t)((wr * 128 + (lane & 15)) * S::WROW + piece_of<S::WROW>(g, lane & 15) * 16);
  const uint32_t lb = S::W + (uint32_t)((wc * 16 + (lane & 15)) * S::XROW +
                                        piece_of<S::XROW>(g, lane & 15) * 16);
  const uint32_t sa = (wr * 128 + (lane & 15)) * 16 + g;
  const uint32_t sb = X_S + (wc * 16 + (lane & 15)) * 16 + g;
  f32x4 acc[8][CG];
  auto clear = [&]() {
#pragma unroll
    for (int i = 0; i < 8; ++i)
#pragma unroll
      for (int j = 0; j < CG; ++j) acc[i][j] = f32x4{0.f, 0.f, 0.f, 0.f};
  };
  clear();

  for (int i = 0; i < S::SLOTS - 1 && more; ++i) {
    load();
    next_load();
  }
  wait_loads<0>();
  wait_lds();
  meet();
  if (behind) meet();

  uint32_t from = lds0;
  uint32_t at_scales = 0, run_at = lds0 + SCALES + (S::RUNS - 1) * S::RUN;  // the stage's codes, and its run's place
  int run_m = 0;  // where the next run starts
  for (;;) {
    int run = nk - cm.kc;
    if (more) run = min(run, nk - cl.kc);
    for (int i = 0; i < run; ++i) {
      i32x8 fa[H][8], fb[H][CG];
      int qa[H][8], qb[H][CG];
      if (cm.kc == run_m) {
        run_at = next_place(run_at);
        at_scales = run_at;
        run_m = next_run(run_m);
      }
#pragma unroll
      for (int h = 0; h < H; ++h) {
#pragma unroll
        for (int r = 0; r < 8; ++r) {
          const i32x4 v = *reinterpret_cast<LdsVec>(from + (la ^ (h * 64)) + r * (16 * S::WROW));
          fa[h][r] = i32x8{v[0], v[1], v[2], v[3], 0, 0, 0, 0};
          qa[h][r] = *reinterpret_cast<LdsByte>(at_scales + sa + r * 256 + h * 4);
        }
#pragma unroll
        for (int c = 0; c < CG; ++c) {
          const uint32_t at = from + (lb ^ (h * 8 * XBITS * 2)) + c * (64 * S::XROW);
          const i32x4 u = *reinterpret_cast<LdsVec>(at);
          i32x4 v = {0, 0, 0, 0};
          if (XBITS == kMxFp8) v = *reinterpret_cast<LdsVec>(at ^ 64);
          fb[h][c] = i32x8{u[0], u[1], u[2], u[3], v[0], v[1], v[2], v[3]};
          qb[h][c] = *reinterpret_cast<LdsByte>(at_scales + sb + c * 1024 + h * 4);
        }
      }
      // the next stage's loads are the oldest in flight
      if (__builtin_expect(more, 1)) {
        load();
        if (fresh) wait_loads<(S::SLOTS - 2) * LOADS + 1>();
        else wait_loads<(S::SLOTS - 2) * LOADS>();
      } else {
        wait_loads<0>();
      }
      wait_lds();
      // (the codes as whole registers from here on)
#pragma unroll
      for (int h = 0; h < H; ++h) {
#pragma unroll
        for (int r = 0; r < 8; ++r) asm volatile("" : "+v"(qa[h][r]));
#pragma unroll
        for (int c = 0; c < CG; ++c) asm volatile("" : "+v"(qb[h][c]));
      }
      if (__builtin_expect(cm.kc * S::KB + S::KB > KB, 0)) {
        // behind the row's last block the values are zeros, the scales whatever
        // follows: one, so that no NaN code meets a zero
#pragma unroll
        for (int h = 0; h < H; ++h) {
          const bool out = cm.kc * S::KB + 4 * h + g >= KB;
#pragma unroll
          for (int r = 0; r < 8; ++r) qa[h][r] = out ? 127 : qa[h][r];
#pragma unroll
          for (int c = 0; c < CG; ++c) qb[h][c] = out ? 127 : qb[h][c];
        }
      }
      // the large part of an E4M3 fragment; the small one is made where the fragment
      // was while the large one is multiplied, the next large one while the small one is
      i32x8 x = XBITS == kMxFp8 ? large_e4m3(fb[0][0]) : fb[0][0];
      meet();
      __builtin_amdgcn_sched_barrier(0);
      __builtin_amdgcn_s_setprio(1);
#pragma unroll
      for (int c = 0; c < CG; ++c) {
        if (__builtin_expect(c < nv, 1)) {
#pragma unroll
          for (int h = 0; h < H; ++h) {
            constexpr int LAST = CG * H - 1;
            const int n = min(c * H + h + 1, LAST);
#pragma unroll
            for (int r = 0; r < 8; ++r)
              acc[r][c] = mx_mfma<XBITS>(fa[h][r], x, acc[r][c], qa[h][r], qb[h][c]);
            if (XBITS == kMxFp8) {
              fb[h][c] ^= x;
              if (c * H + h < LAST) x = large_e4m3(fb[n % H][n / H]);
#pragma unroll
              for (int r = 0; r < 8; ++r)
                acc[r][c] = mx_mfma<XBITS>(fa[h][r], fb[h][c], acc[r][c], qa[h][r], qb[h][c]);
              if (TC == 256) {
                mx_order<5, 2, 1>();
                mx_order<1, 2, 3>();
              } else {
                mx_order<1, 1, 8>();
              }
              mx_order<1, 4, 8>();
            } else {
              x = fb[n % H][n / H];
            }
          }
        }
      }
      __builtin_amdgcn_s_setprio(0);
      __builtin_amdgcn_sched_barrier(0);
      meet();
      at_scales += S::KB;
      from = from == lds0 + (S::SLOTS - 1) * SLOT ? lds0 : from + SLOT;
      ++cm.kc;
    }
    next_load();
    if (cm.kc == nk) {
      const bool vec = a.M % 8 == 0 && (reinterpret_cast<uintptr_t>(a.y) & 15u) == 0;
      Out* out = static_cast<Out*>(a.y) + (size_t)cm.beg * a.M;
      const int r0 = cm.r0 + wr * 128;
#pragma unroll
      for (int c = 0; c < CG; ++c) {
        const int n0 = cm.c0 + (c * 4 + wc) * 16, n = n0 + (lane & 15);
        Out* to = out + (size_t)n0 * a.M + r0;
        Out* o = to + (size_t)(lane & 15) * a.M;
#pragma unroll
        for (int i = 0; i < 8; i += 2) {
          if (vec) {
            store_two(to + i * 16, a.M, acc[i][c], acc[i + 1][c], lane, cm.rows - n0, a.M - (r0 + i * 16));
          } else if (n < cm.rows) {
#pragma unroll
            for (int q = 0; q < 4; ++q) {
              const int r = i * 16 + g * 4 + q;
              if (r0 + r < a.M) o[r] = out_value<Out>(acc[i][c][q]);
              if (r0 + r + 16 < a.M) o[r + 16] = out_value<Out>(acc[i + 1][c][q]);
            }
          }
        }
      }
      stores_end();
      clear();
      run_m = 0;
      tm += step;
      if (!find(wm, tm, &cm)) break;
      nv = groups();
    }
  }
  if (!behind) meet();
  return past();
}

// The experts with more than lo rows. Those with at most kNarrowRows go to the
// narrow tiles (77 experts, K 7168, M 4096, E4M3 rows, skewed counts, 50, 85, 125,
// 167 rows an expert on average, us: limit 64: 372, 427, 610, 688; 128: 362, 379,
// 483, 657; 256: 333, 434, 564, 697), numbered on behind the wide ones, so that the
// blocks share all tiles evenly.
template <int XBITS, typename Out>
__global__ __launch_bounds__(X_THREADS, 1) void mx_dense_kernel(MxArgs a, int lo) {
  constexpr int B0 = Shape<XBITS, 256>::BYTES, B1 = Shape<XBITS, 128>::BYTES, B2 = Shape<XBITS, 64>::BYTES;
  constexpr int B = B0 > B1 ? B0 : B1;
  __shared__ __align__(1024) uint8_t lds[B > B2 ? B : B2];
  if (lo > 0) {  // the experts with fewer rows, if the kernel for them left them
    GroupWalk walk;
    walk.start(a.off, a.L, a.N, 1, 1, 0, lo);
    if (walk.rounds_hold(lo, (a.M + 255) / 256, gridDim.x)) lo = 0;
  }
  int t = xcd_block(blockIdx.x, gridDim.x);
  if (a.N > kNarrowRows) t = mx_dense_tiles<XBITS, 256, Out>(a, lds, kNarrowRows, kAnyRows, t);
  if (a.N > X_FEW) t = mx_dense_tiles<XBITS, 128, Out>(a, lds, X_FEW, kNarrowRows, t);
  mx_dense_tiles<XBITS, 64, Out>(a, lds, lo, X_FEW, t);
}

template <int XBITS, typename Out>
void launch(const MxArgs& a, int lo, int blocks, hipStream_t s) {
  hipLaunchKernelGGL((mx_dense_kernel<XBITS, Out>), dim3(blocks), dim3(X_THREADS), 0, s, a, lo);
}

}  // namespace

// The experts with more than `lo` rows.
hipError_t launch_mx_dense(const MxArgs& a, int x_bits, bool y_fp32, int lo, int blocks,
                           hipStream_t s) {
  if (x_bits == kMxFp8) {
    if (y_fp32) launch<8, float>(a, lo, blocks, s);
    else launch<8, uint16_t>(a, lo, blocks, s);
  } else {
    if (y_fp32) launch<4, float>(a, lo, blocks, s);
    else launch<4, uint16_t>(a, lo, blocks, s);
  }
  return hipGetLastError();
}

}  // namespace moe
