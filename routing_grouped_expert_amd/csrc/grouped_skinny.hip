// Grouped products for experts with few rows (at most 32): y[n] = W[e] x[n] is
// then a stream of the expert's weights, each used for a handful of rows, and
// bound by how fast they arrive.
//
// A tile is 32 weight rows a wave by at most 32 rows of x. Every stage is 128
// bytes of each weight row (whole cache lines): 64 of the contraction in bf16,
// 256 in E2M1. Weights, rows of x and scales go straight to LDS, four stages
// ahead in a ring of five, so that a CU has about 64 KB of weights in flight
// (four waves a block), twice what the memory's latency asks for at its full
// rate. Scales are loaded for four stages at a time (a stage at a time they
// were half of the requests: 103 against 86 us in the case below). A wave loads
// the weights it multiplies; the rows of x are loaded once a block. The stages
// run on across the block's tiles.
//
// Measured: bf16, 64 rows on 8 experts (K 4096, M 28672) 319 us, 5.9 TB/s (347
// without the read-once policy on the weights); E2M1 weights, the same shape, 84
// us with E2M1 rows, 6.0 TB/s, and 100 with E4M3 rows: 80 instructions more a
// stage to split their fragments, and twice the matrix instructions (88 us without
// either, mx_matmul.h says why they are there); one token on 8 of 256 experts (K
// 7168, M 4096) 22 and 27 us. Above 32 rows the wide tiles are faster: an expert
// of 33 to 64 rows in two passes of 32 took 741 us in bf16 (50 rows an expert; the
// wide tiles 480).
#include "lds_dma.h"
#include "mx_matmul.h"
#include "operators.h"

#include <algorithm>

namespace moe {

namespace {

constexpr int S_ROWS = 32;  // weight rows of a wave
constexpr int S_TOK = 32;   // rows of x of a tile
constexpr int S_RING = 5;
constexpr int S_RUN = 4;   // stages that share a load of scales
constexpr int S_RUNS = 3;  // places for them: five stages reach into three runs

typedef const __attribute__((address_space(3))) i32x4* LdsVec;
typedef const __attribute__((address_space(3))) uint8_t* LdsByte;

// Operand formats: XB bits of a value of x; the weights' values of a 128-byte
// line.
template <int XB>
struct Format {
  static constexpr bool MX = XB != 16;
  static constexpr int K = MX ? 256 : 64;      // contraction of a stage
  static constexpr int XROW = K * XB / 8;      // bytes of a stage's row of x
  static constexpr int XP = XROW / 16;         // its 16-byte pieces
};

// LDS place of 16-byte piece q of row r, in a row of P pieces: spread so that
// a fragment read (16 rows, one piece each) meets no bank twice.
template <int P>
__device__ __forceinline__ int place(int q, int r) {
  return q ^ (r & (P - 1));
}

// (Launch bounds of 512 threads: with the 512 registers that fewer would leave a
// lane, the compiler moves the accumulators to the other half of them and back in
// every stage, 103 against 101 us.)
template <int XB, int WAVES, typename Out>
__global__ __launch_bounds__(512) void skinny_kernel(MxArgs a, int most, int others) {
  using F = Format<XB>;
  constexpr bool MX = F::MX;
  constexpr int XPIECES = S_TOK * F::XROW / 1024;       // 1 KB pieces of a stage's x
  constexpr int XN = XPIECES / WAVES;                   // loaded by each wave
  constexpr int XROWS = 64 / F::XP;                     // rows of x in a piece
  constexpr int WAVE_BYTES = S_ROWS * 128;
  constexpr int SLOT = WAVES * WAVE_BYTES + S_TOK * F::XROW;
  constexpr int LOADS = 4 + XN;                         // a wave's per stage, without scales
  constexpr int SCALES = S_RING * SLOT;  // a wave's: S_RUNS places of 32 + 32 rows' codes
  static_assert(LOADS * (S_RING - 2) < 64, "the wait counts to 63");
  __shared__ __align__(1024) uint8_t lds[SCALES + (MX ? WAVES * S_RUNS * 2048 : 0)];
  const int lane = threadIdx.x % kWave;
  const int wave = WAVES == 1 ? 0 : __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
  const uint32_t lds0 = lds_address(lds);
  const int step = gridDim.x;
  const int KB = a.K / kMxBlock;
  // (with scales at least two stages, the second one of zeros where it has to
  // be: two neighbouring runs are then four stages or more together, and the
  // ring's five stages reach into three at most)
  const int nk = max(MX ? 2 : 1, (a.K + F::K - 1) / F::K);
  const int whole = a.K / F::K;  // stages without a row's end
  const int per = (a.M + WAVES * S_ROWS - 1) / (WAVES * S_ROWS);
  const int wbytes = MX ? a.K / 2 : a.K * 2, xbytes = a.K * XB / 8;

  struct Tile {
    int expert, beg, rows, m0, kc;
  };
  GroupWalk walk;
  GroupWalk::Place wl, wm;  // of the tiles being loaded, and multiplied
  walk.start(a.off, a.L, a.N, per, S_TOK, 0, most);
  if (others > 0 && walk.rounds_hold(most, (a.M + 255) / 256, others)) return;
  auto find = [&](GroupWalk::Place& w, int t, Tile* o) {
    GroupTile g;
    if (!walk.find(w, t, &g)) return false;
    *o = Tile{g.expert, g.beg, g.rows, (g.tile * WAVES + wave) * S_ROWS, 0};
    return true;
  };
  int tl = xcd_block(blockIdx.x, step), tm = tl;
  Tile cl, cm;
  if (!find(wl, tl, &cl)) return;
  find(wm, tm, &cm);

  u32x4 rw, rx, rws, rxs;
  uint32_t vw[4], vx[XN], vws, vxs;
  uint32_t ws_end = 0;
  const uint32_t xs_end = (uint32_t)((size_t)a.T * KB);
  bool w_edge = false, x_edge = false;  // a lane's scales may end the array
  int x_of = -1;  // expert whose rows vx and vxs name
  auto tile_loads = [&]() {
    const size_t left = (size_t)(a.L - cl.expert) * a.M;  // weight rows to the end
    rw = buffer_over(a.wq + (size_t)cl.expert * a.M * wbytes, (uint32_t)min(left * wbytes, kMostBytes));
    rx = buffer_over(a.xq, (uint32_t)((size_t)a.T * xbytes));
#pragma unroll
    for (int j = 0; j < 4; ++j) {  // 8 rows a piece
      const int i = 8 * j + (lane >> 3), m = cl.m0 + i;
      vw[j] = m < a.M ? (uint32_t)m * wbytes + place<8>(lane & 7, i) * 16 : kPastEnd;
    }
    if (MX) {  // 32 codes of a row a run: 16 a lane
      const int m = cl.m0 + (lane >> 1);
      ws_end = (uint32_t)min(left * KB, kMostBytes);
      rws = buffer_over(a.ws + (size_t)cl.expert * a.M * KB, ws_end);
      vws = m < a.M ? (uint32_t)m * (uint32_t)KB + (lane & 1) * 16 : kPastEnd;
      w_edge = at_edge(vws, KB, ws_end);
    }
    // The rows of x change with the expert only: reading permuted_rows waits
    // for every load in flight.
    if (cl.expert == x_of) return;
    x_of = cl.expert;
    auto token = [&](int i) { return i < cl.rows ? source_row(a, cl.beg + i) : -1; };
#pragma unroll
    for (int j = 0; j < XN; ++j) {
      const int i = (XN * wave + j) * XROWS + lane / F::XP;
      const int s = token(i);
      vx[j] = s >= 0 ? (uint32_t)s * xbytes + place<F::XP>(lane % F::XP, i) * 16 : kPastEnd;
    }
    if (MX) {
      const int s = token(lane >> 1);
      rxs = buffer_over(a.xs, xs_end);
      vxs = s >= 0 ? (uint32_t)s * (uint32_t)KB + (lane & 1) * 16 : kPastEnd;
      x_edge = at_edge(vxs, KB, xs_end);
    }
  };
  bool more = true;
  int sl = 0, run_l = 0;  // slot being loaded, and place of the next run's scales
  const uint32_t scales0 = lds0 + SCALES + wave * (S_RUNS * 2048);
  auto load = [&]() {
    const uint32_t mine = lds0 + sl * SLOT + wave * WAVE_BYTES, xto = lds0 + sl * SLOT + WAVES * WAVE_BYTES;
    const uint32_t aw = cl.kc * 128u, ax = cl.kc * (uint32_t)F::XROW;
    if (__builtin_expect(cl.kc < whole, 1)) {
      dma16_run<true>(rw, mine, vw, aw);
      dma16_run<false>(rx, xto + XN * wave * 1024u, vx, ax);
    } else {  // pieces behind the rows' ends as zeros
      uint32_t w_at[4], x_at[XN];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int i = 8 * j + (lane >> 3);
        w_at[j] = (int)aw + place<8>(lane & 7, i) * 16 < wbytes ? vw[j] : kPastEnd;
      }
      dma16_run<true>(rw, mine, w_at, aw);
#pragma unroll
      for (int j = 0; j < XN; ++j) {
        const int i = (XN * wave + j) * XROWS + lane / F::XP;
        x_at[j] = (int)ax + place<F::XP>(lane % F::XP, i) * 16 < xbytes ? vx[j] : kPastEnd;
      }
      dma16_run<false>(rx, xto + XN * wave * 1024u, x_at, ax);
    }
    if (MX && cl.kc % S_RUN == 0) {
      const uint32_t to = scales0 + run_l * 2048;
      dma16_bytes(rws, a.ws + (size_t)cl.expert * a.M * KB, ws_end, to,
                  vws == kPastEnd ? kPastEnd : vws + cl.kc * 8u, lane, w_edge);
      dma16_bytes(rxs, a.xs, xs_end, to + 1024, vxs == kPastEnd ? kPastEnd : vxs + cl.kc * 8u, lane,
                  x_edge);
      run_l = run_l == S_RUNS - 1 ? 0 : run_l + 1;
    }
    sl = sl == S_RING - 1 ? 0 : sl + 1;
    if (++cl.kc == nk) {
      tl += step;
      more = find(wl, tl, &cl);
      if (more) tile_loads();
    }
  };
  tile_loads();
  for (int i = 0; i < S_RING - 1 && more; ++i) load();

  const int g = lane >> 4, row = lane & 15;
  f32x4 acc[2][2] = {};
  int slot = 0, run_m = S_RUNS - 1;
  for (;;) {
    if (more) wait_loads<LOADS * (S_RING - 2)>();
    else wait_loads<0>();
    if (WAVES > 1) meet();  // the stage is there, and the one before it is read
    if (more) load();
    const uint32_t mine = lds0 + slot * SLOT + wave * WAVE_BYTES, xat = lds0 + slot * SLOT + WAVES * WAVE_BYTES;
    if (MX && cm.kc % S_RUN == 0) run_m = run_m == S_RUNS - 1 ? 0 : run_m + 1;
    const uint32_t qat = scales0 + run_m * 2048 + (cm.kc % S_RUN) * 8 + g;
    const bool two = cm.rows > 16;
    i32x4 fw[2][2], fx[2][2][XB == 8 ? 2 : 1];
    int qw[2][2], qx[2][2];
#pragma unroll
    for (int s = 0; s < 2; ++s) {
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int r = i * 16 + row;
        fw[i][s] = *reinterpret_cast<LdsVec>(mine + r * 128 + place<8>(4 * s + g, r) * 16);
        if (XB == 8) {
          fx[i][s][0] = *reinterpret_cast<LdsVec>(xat + r * F::XROW + place<F::XP>(8 * s + g, r) * 16);
          fx[i][s][XB == 8 ? 1 : 0] =
              *reinterpret_cast<LdsVec>(xat + r * F::XROW + place<F::XP>(8 * s + 4 + g, r) * 16);
        } else {
          fx[i][s][0] = *reinterpret_cast<LdsVec>(xat + r * F::XROW + place<F::XP>(4 * s + g, r) * 16);
        }
        if (MX) {
          // behind the row's last block the values are zeros, the scales
          // whatever follows: one, so that no NaN code meets a zero
          const bool in = cm.kc * 8 + 4 * s + g < KB;
          const int w = *reinterpret_cast<LdsByte>(qat + r * 32 + 4 * s);
          const int x = *reinterpret_cast<LdsByte>(qat + 1024 + r * 32 + 4 * s);
          qw[i][s] = in ? w : 127;
          qx[i][s] = in ? x : 127;
        }
      }
    }
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      if (j == 0 || two) {
#pragma unroll
        for (int s = 0; s < 2; ++s) {
          if (MX) {
            const i32x4 u = fx[j][s][0], v = fx[j][s][XB == 8 ? 1 : 0];
            i32x8 x = {u[0], u[1], u[2], u[3], 0, 0, 0, 0}, small = x;
            if (XB == 8) {
              small = i32x8{u[0], u[1], u[2], u[3], v[0], v[1], v[2], v[3]};
              x = large_e4m3(small);
              small ^= x;
            }
            i32x8 w[2];
#pragma unroll
            for (int i = 0; i < 2; ++i) {
              const i32x4 f = fw[i][s];
              w[i] = i32x8{f[0], f[1], f[2], f[3], 0, 0, 0, 0};
              acc[i][j] = mx_mfma<XB == 8 ? 8 : 4>(w[i], x, acc[i][j], qw[i][s], qx[j][s]);
            }
            if (XB == 8)
#pragma unroll
              for (int i = 0; i < 2; ++i)
                acc[i][j] = mx_mfma<8>(w[i], small, acc[i][j], qw[i][s], qx[j][s]);
          } else {
#pragma unroll
            for (int i = 0; i < 2; ++i)
              acc[i][j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(
                  __builtin_bit_cast(bf16x8, fw[i][s]), __builtin_bit_cast(bf16x8, fx[j][s][0]),
                  acc[i][j], 0, 0, 0);
          }
        }
      }
    }
    wait_lds();  // read before the block's next meeting
    slot = slot == S_RING - 1 ? 0 : slot + 1;
    if (++cm.kc == nk) {
      // (bf16 operands come here with whole 16-byte pieces of y only)
      const bool vec = !MX || (a.M % 8 == 0 && (reinterpret_cast<uintptr_t>(a.y) & 15u) == 0);
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        if (j == 1 && !two) break;
        const int n = j * 16 + row;
        Out* to = static_cast<Out*>(a.y) + (size_t)(cm.beg + j * 16) * a.M + cm.m0;
        Out* o = to + (size_t)row * a.M;
        if (vec) {
          store_two(to, a.M, acc[0][j], acc[1][j], lane, cm.rows - j * 16, a.M - cm.m0);
        } else if (n < cm.rows) {
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            const int r = g * 4 + q;
            if (cm.m0 + r < a.M) o[r] = out_value<Out>(acc[0][j][q]);
            if (cm.m0 + r + 16 < a.M) o[r + 16] = out_value<Out>(acc[1][j][q]);
          }
        }
      }
      stores_end();
#pragma unroll
      for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int j = 0; j < 2; ++j) acc[i][j] = f32x4{0.f, 0.f, 0.f, 0.f};
      tm += step;
      if (!find(wm, tm, &cm)) return;
    }
  }
}

template <int XB, int WAVES, typename Out>
void launch(const MxArgs& a, int most, int others, int blocks, hipStream_t s) {
  hipLaunchKernelGGL((skinny_kernel<XB, WAVES, Out>), dim3(blocks), dim3(WAVES * kWave), 0, s, a, most, others);
}

template <int XB>
void launch_format(const MxArgs& a, bool y_fp32, int others, hipStream_t s) {
  const int cus = compute_units();
  // At most so many tiles of four waves; where they would not reach every CU,
  // one wave a block. (K 7168, 128 / 256 tiles of four waves, us: one wave bf16 42
  // / 78, E4M3 rows 25 / 45, E2M1 17 / 30; four waves 62 / 71, 26 / 27, 21 / 23.)
  const long tiles = ((long)a.N / S_TOK + std::min(a.L, a.N)) * ((a.M + 127) / 128);
  const bool wide = tiles >= cus;
  if (wide) {
    if (y_fp32) launch<XB, 4, float>(a, S_TOK, others, cus, s);
    else launch<XB, 4, uint16_t>(a, S_TOK, others, cus, s);
  } else {
    if (y_fp32) launch<XB, 1, float>(a, S_TOK, others, 2 * cus, s);
    else launch<XB, 1, uint16_t>(a, S_TOK, others, 2 * cus, s);
  }
}

}  // namespace

// Experts with at most this many rows are the kernel's; it passes over others.
int skinny_rows() { return S_TOK; }

// x_bits 4, 8: microscaled operands; 16: bf16 (wq and xq then hold bf16). others:
// blocks of the launch that follows, for the experts with more rows, or 0; where
// it can take these experts along in its last round of tiles, it does, and this
// one ends. (77 experts of 85 rows, one with 20, K 7168, M 2048: bf16 491 -> 445 us,
// E4M3 rows 250 -> 223; 3 of 8 with 20 rows, 5 with 300, K 4096, M 14336: 355 -> 300,
// 246 -> 213. Where they make a further round, 26 of 77: taken along 434 and 189, as
// here 430 and 214.)
hipError_t launch_skinny(const MxArgs& a, int x_bits, bool y_fp32, int others, hipStream_t s) {
  if (x_bits == 4) launch_format<4>(a, y_fp32, others, s);
  if (x_bits == 8) launch_format<8>(a, y_fp32, others, s);
  if (x_bits == 16) launch_format<16>(a, y_fp32, others, s);
  return hipGetLastError();
}

}  // namespace moe
