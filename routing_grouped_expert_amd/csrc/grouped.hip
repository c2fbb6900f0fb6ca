// Products over rows grouped by expert, element by element: the path of every
// shape and alignment that the 16-byte kernels do not take.
//
// y[n] = W[e] x[n], dx[n] = W[e]^T dy[n], dW[e] = sum over the expert's rows
// of dy[n] x[n]^T, for the rows n in [offsets[e], offsets[e + 1]).
//
// A block of four waves makes 64 x 64 outputs (32 x 32 a wave, bf16 MFMA,
// fp32 accumulators). Both operands are staged in LDS as [64][32 of the
// contraction] whatever their order in memory, loaded element by element with
// the memory's contiguous index across the lanes and zeros outside the
// matrix; a stage's elements are on their way to registers while the one before
// it is multiplied (a training step at K 243, M 558 and 180 rows: 34 us, 96
// without). Bound by the loads' latency and number: K 777, M 951, 4000 rows of 16
// experts take 53 us forward, 66 dx, 63 dw, and 133 dw by selections, which are
// read and divided for every element of x (the bytes of each take 8 us).
#include "mx_matmul.h"
#include "lds_dma.h"
#include "operators.h"

#include <algorithm>
#include <atomic>

namespace moe {

namespace {

constexpr int G_T = 64;       // rows and columns of a block's outputs
constexpr int G_K = 32;       // contraction per stage
constexpr int G_LD = G_K + 8;  // LDS row of 80 bytes: 16-byte aligned, spread over the banks

template <Product P, typename Out>
__global__ __launch_bounds__(256) void grouped_any_kernel(GroupedArgs a) {
  __shared__ __align__(16) uint16_t sa[G_T][G_LD], sb[G_T][G_LD];
  __shared__ int src[G_T];
  const int tid = threadIdx.x, lane = tid % kWave, wave = tid / kWave;
  const int R = P == Product::kForward ? a.M : a.K;  // extent of r
  const int RT = (R + G_T - 1) / G_T;
  const int CT = (a.M + G_T - 1) / G_T;  // dw: tiles of c
  const size_t wsize = (size_t)a.M * a.K;
  GroupWalk walk;
  GroupWalk::Place place;
  if (P != Product::kDw) walk.start(a.off, a.L, a.N, RT, G_T, 0, kAnyRows);
  const long dw_tiles = (long)a.L * RT * CT;

  for (long t = blockIdx.x;; t += gridDim.x) {
    int expert, beg, rows, r0, c0, C, KK;
    if (P == Product::kDw) {
      if (t >= dw_tiles) return;
      expert = (int)(t / ((long)RT * CT));
      const int i = (int)(t - (long)expert * RT * CT);
      r0 = (i % RT) * G_T;
      c0 = (i / RT) * G_T;
      beg = max(0, min(a.off[expert], a.N));
      rows = max(beg, min(a.off[expert + 1], a.N)) - beg;
      C = a.M;
      KK = rows;
    } else {
      GroupTile g;
      if (!walk.find(place, (int)t, &g)) return;
      expert = g.expert;
      beg = g.beg;
      rows = g.rows;
      r0 = (g.tile % RT) * G_T;
      c0 = (g.tile / RT) * G_T;
      C = rows;
      KK = P == Product::kForward ? a.K : a.M;
    }
    const uint16_t* w = P == Product::kDw ? nullptr : a.w + (size_t)expert * wsize;
    if (P == Product::kForward) {
      if (tid < G_T) src[tid] = c0 + tid < C ? source_row(a, beg + c0 + tid) : -1;
      __syncthreads();
    }
    f32x4 acc[2][2] = {};
    const int wr = (wave & 1) * 32, wc = (wave >> 1) * 32;
    constexpr int E = G_T * G_K / 256;  // elements of each operand a thread loads
    uint16_t va[E], vb[E];
    // Row and contraction index of element i of this thread: A's contiguous
    // along kk (forward) or along r, B's along kk, or along c (dw).
    auto a_at = [&](int i, int* r, int* kk) {
      const int e = tid + i * 256;
      *r = P == Product::kForward ? e / G_K : e % G_T;
      *kk = P == Product::kForward ? e % G_K : e / G_T;
    };
    auto b_at = [&](int i, int* c, int* kk) {
      const int e = tid + i * 256;
      *c = P == Product::kDw ? e % G_T : e / G_K;
      *kk = P == Product::kDw ? e / G_T : e % G_K;
    };
    auto fetch = [&](int k0) {
#pragma unroll
      for (int i = 0; i < E; ++i) {
        int r, c, kk;
        a_at(i, &r, &kk);
        va[i] = 0;
        if (r0 + r < R && k0 + kk < KK) {
          if (P == Product::kForward) va[i] = w[(size_t)(r0 + r) * a.K + k0 + kk];
          if (P == Product::kDx) va[i] = w[(size_t)(k0 + kk) * a.K + r0 + r];
          if (P == Product::kDw) {
            const int s = source_row(a, beg + k0 + kk);
            if (s >= 0) va[i] = a.x[(size_t)s * a.K + r0 + r];
          }
        }
        b_at(i, &c, &kk);
        vb[i] = 0;
        if (c0 + c < C && k0 + kk < KK) {
          if (P == Product::kForward) {
            const int s = src[c];
            if (s >= 0) vb[i] = a.x[(size_t)s * a.K + k0 + kk];
          }
          if (P == Product::kDx) vb[i] = a.dy[(size_t)(beg + c0 + c) * a.M + k0 + kk];
          if (P == Product::kDw) vb[i] = a.dy[(size_t)(beg + k0 + kk) * a.M + c0 + c];
        }
      }
    };
    if (KK > 0) fetch(0);
    for (int k0 = 0; k0 < KK; k0 += G_K) {
#pragma unroll
      for (int i = 0; i < E; ++i) {
        int r, kk;
        a_at(i, &r, &kk);
        sa[r][kk] = va[i];
        b_at(i, &r, &kk);
        sb[r][kk] = vb[i];
      }
      __syncthreads();
      if (k0 + G_K < KK) fetch(k0 + G_K);  // on its way while this stage is multiplied
      bf16x8 fa[2], fb[2];
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        fa[i] = *reinterpret_cast<const bf16x8*>(&sa[wr + i * 16 + lane % 16][lane / 16 * 8]);
        fb[i] = *reinterpret_cast<const bf16x8*>(&sb[wc + i * 16 + lane % 16][lane / 16 * 8]);
      }
#pragma unroll
      for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int j = 0; j < 2; ++j)
          acc[i][j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(fa[i], fb[j], acc[i][j], 0, 0, 0);
      __syncthreads();
    }
    Out* out = static_cast<Out*>(a.out) + (P == Product::kDw ? (size_t)expert * wsize : (size_t)beg * R);
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const int c = c0 + wc + j * 16 + lane % 16;
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          const int r = r0 + wr + i * 16 + lane / 16 * 4 + q;
          if (c < C && r < R) out[(size_t)c * R + r] = out_value<Out>(acc[i][j][q]);
        }
      }
    if (P == Product::kForward) __syncthreads();  // src is rewritten for the next tile
  }
}

template <Product P>
void launch_any(const GroupedArgs& a, bool f32, int blocks, hipStream_t s) {
  if (f32)
    hipLaunchKernelGGL((grouped_any_kernel<P, float>), dim3(blocks), dim3(256), 0, s, a);
  else
    hipLaunchKernelGGL((grouped_any_kernel<P, uint16_t>), dim3(blocks), dim3(256), 0, s, a);
}

bool a16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

// Whether the 16-byte kernels take the call: whole 16-byte pieces along both
// widths, and 32-bit byte offsets within each operand.
bool fast_ok(const GroupedArgs& a) {
  const size_t x = (size_t)a.T * a.K * 2, n = (size_t)a.N * std::max(a.M, a.K) * 2,
               w = (size_t)a.M * a.K * 2;
  return a.K % 8 == 0 && a.M % 8 == 0 && std::max(x, std::max(n, w)) <= kMostBytes && a16(a.x) &&
         a16(a.dy) && a16(a.w) && a16(a.out);
}

}  // namespace

int compute_units() {
  static std::atomic<int> cached[64];
  int dev = 0;
  if (hipGetDevice(&dev) != hipSuccess || dev < 0 || dev >= 64) dev = 0;
  int n = cached[dev].load(std::memory_order_relaxed);
  if (n == 0) {
    if (hipDeviceGetAttribute(&n, hipDeviceAttributeMultiprocessorCount, dev) != hipSuccess || n <= 0)
      n = 256;
    cached[dev].store(n, std::memory_order_relaxed);
  }
  return n;
}

hipError_t launch_grouped(Product p, const GroupedArgs& args, bool out_fp32, hipStream_t stream) {
  GroupedArgs a = args;
  divide_by(a.k, &a.div_m, &a.div_s);
  if (fast_ok(a)) {
    // Only the device knows how many rows an expert has: in the forward both
    // kernels run, and each passes over the other's experts.
    int lo = 0;
    if (p == Product::kForward) {
      const MxArgs s{reinterpret_cast<const uint8_t*>(a.x), nullptr,
                     reinterpret_cast<const uint8_t*>(a.w), nullptr, a.out, a.rows, a.off, a.L, a.T,
                     a.k, a.N, a.K, a.M, a.div_m, a.div_s};
      lo = skinny_rows();
      const hipError_t e = launch_skinny(s, 16, out_fp32, a.N > lo ? compute_units() : 0, stream);
      if (e != hipSuccess || a.N <= lo) return e;
    }
    return launch_grouped_dense(p, a, out_fp32, lo, compute_units(), stream);
  }
  const long RT = ((p == Product::kForward ? a.M : a.K) + G_T - 1) / G_T;
  long tiles;
  if (p == Product::kDw)
    tiles = (long)a.L * RT * ((a.M + G_T - 1) / G_T);
  else  // at most: every expert may end in a part of a tile
    tiles = ((long)a.N / G_T + std::min(a.L, a.N)) * RT;
  const int blocks = (int)std::min<long>(tiles, 2048);
  if (p == Product::kForward) launch_any<Product::kForward>(a, out_fp32, blocks, stream);
  if (p == Product::kDx) launch_any<Product::kDx>(a, out_fp32, blocks, stream);
  if (p == Product::kDw) launch_any<Product::kDw>(a, out_fp32, blocks, stream);
  return hipGetLastError();
}

}  // namespace moe
