// Root-mean-square norm with the residual's addition, bf16 and MXFP8 outputs,
// and its backward.
//
//   h = bf16(x + residual)      s = 1 / sqrt(mean(h^2) + eps)     y = h s g
//   dh = s (g dy - h s^2 mean(g dy h)) + dresidual    dg = sum over rows dy h s
//
// The statistics are those of the rounded h, which is what the next block's
// residual and the backward read; sums, s and y are fp32, y is rounded once
// (to bf16, and from fp32 again to MXFP8). Bound by memory: a row is read
// once and kept in registers (8 values a lane and chunk) between its
// reduction and its outputs.
//
// Measured: 4096 rows of 7168 with residual, bf16 and MXFP8 outputs 44 us (6.0
// TB/s); 4095 rows of 4096: forward 24 us, backward 25 + 4 us (5.3 TB/s). One row
// of 7168: 2.7 us, the latency of its loads and its reduction. Rows up to 512
// take a wave each, longer ones 8 values a thread where a block can (rows of
// 4096: 26.5 us with 512 threads, 27.7 with 256 of two pieces).
#include "mx.h"
#include "operators.h"

#include <algorithm>

namespace moe {

namespace {

// Eight fp32 to bf16.
__device__ __forceinline__ u16x8 pack8(const float (&v)[8]) {
  return __builtin_bit_cast(u16x8, u32x4{pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3]),
                                         pack_bf16(v[4], v[5]), pack_bf16(v[6], v[7])});
}

// Sum over a block of NT threads, the same bits in every thread; `buf` holds
// NT / 64 floats and is free again after the caller's next barrier.
template <int NT>
__device__ __forceinline__ float block_sum(float v, float* buf) {
  v = wave_sum_f32(v);
  if (NT == kWave) return v;
  const int tid = threadIdx.x;
  if (tid % kWave == 0) buf[tid / kWave] = v;
  __syncthreads();
  float s = 0.f;
#pragma unroll
  for (int i = 0; i < NT / kWave; ++i) s += buf[i];
  return s;
}

// 1 / sqrt(sum / H + eps), rounded once: the instruction's value s (off by a
// step or two), then s + s / 2 (1 - a s^2) with 1 - a s^2 from the exact a s.
// (A root and a division, each rounded, were up to 0.97 of a step off, against
// 0.5, in the same time. The sum's own rounding is larger: of 88 million MXFP8
// codes 59 differ from those of 64 bits, 57 before.) Zero, infinite and NaN sums
// give the instruction's infinity, 0 and NaN.
__device__ __forceinline__ float rstd_of(float sum, int H, float eps) {
  const float a = sum / (float)H + eps, s = rsqrtf(a);
  const float as = a * s, low = fmaf(a, s, -as);
  const float e = fmaf(-low, s, fmaf(-as, s, 1.0f));
  return a > 0.0f && s > 0.0f ? fmaf(0.5f * s, e, s) : s;
}

// One row per NT threads (NT 64: four rows a block). H <= NT * 8 * CH, a
// multiple of 8, rows 16-byte aligned.
template <int NT, int CH>
__global__ __launch_bounds__(NT == 64 ? 256 : NT) void rms_norm_rows_kernel(
    const uint16_t* x, const uint16_t* res, const float* __restrict__ weight, float eps, int T,
    int H, uint16_t* h_out, uint16_t* y, uint8_t* yq, uint8_t* ys) {
  __shared__ float buf[NT / kWave];
  const int tid = threadIdx.x % NT;
  const int t = NT == 64 ? blockIdx.x * 4 + threadIdx.x / kWave : blockIdx.x;
  if (NT == 64 && t >= T) return;
  const size_t row = (size_t)t * H;
  float h[CH][8];
  float sum = 0.f;
#pragma unroll
  for (int i = 0; i < CH; ++i) {
    const int c = (tid + i * NT) * 8;
#pragma unroll
    for (int j = 0; j < 8; ++j) h[i][j] = 0.f;
    if (c < H) {
      const u16x8 a = *reinterpret_cast<const u16x8*>(x + row + c);
      u16x8 o = a;
      if (res) {
        const u16x8 b = *reinterpret_cast<const u16x8*>(res + row + c);
        float v[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] = bf16_bits_to_f32(a[j]) + bf16_bits_to_f32(b[j]);
        o = pack8(v);
      }
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        h[i][j] = bf16_bits_to_f32(o[j]);
        sum = fmaf(h[i][j], h[i][j], sum);
      }
      if (h_out) *reinterpret_cast<u16x8*>(h_out + row + c) = o;
    }
  }
  const float s = rstd_of(block_sum<NT>(sum, buf), H, eps);
#pragma unroll
  for (int i = 0; i < CH; ++i) {
    const int c = (tid + i * NT) * 8;
    if (c < H) {
      const f32x4 w0 = *reinterpret_cast<const f32x4*>(weight + c);
      const f32x4 w1 = *reinterpret_cast<const f32x4*>(weight + c + 4);
      float v[8];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        v[j] = h[i][j] * s * w0[j];
        v[j + 4] = h[i][j + 4] * s * w1[j];
      }
      if (y) *reinterpret_cast<u16x8*>(y + row + c) = pack8(v);
      if (yq) {  // H a multiple of 32: the four lanes of a block are in or out together
        uint32_t sc;
        const uint64_t q = mx_quantize8<kMxFp8>(v, &sc);
        *reinterpret_cast<u32x2*>(yq + row + c) = u32x2{(uint32_t)q, (uint32_t)(q >> 32)};
        if ((tid & 3) == 0) ys[(row + c) / 32] = (uint8_t)sc;
      }
    }
  }
}

// Any length and alignment: a block walks the row twice. A thread reads back
// only what it wrote or read itself, so the outputs may lie on the inputs.
__global__ __launch_bounds__(256) void rms_norm_any_kernel(
    const uint16_t* x, const uint16_t* res, const float* __restrict__ weight, float eps, int H,
    uint16_t* h_out, uint16_t* y, uint8_t* yq, uint8_t* ys) {
  __shared__ float buf[4];
  const size_t row = (size_t)blockIdx.x * H;
  auto at = [&](int c) {
    uint16_t b = x[row + c];
    if (res) b = f32_to_bf16_bits(bf16_bits_to_f32(b) + bf16_bits_to_f32(res[row + c]));
    return b;
  };
  float sum = 0.f;
  for (int c = threadIdx.x; c < H; c += 256) {
    const uint16_t b = at(c);
    const float v = bf16_bits_to_f32(b);
    sum = fmaf(v, v, sum);
    if (h_out) h_out[row + c] = b;
  }
  const float s = rstd_of(block_sum<256>(sum, buf), H, eps);
  for (int c = threadIdx.x; c < H; c += 256) {
    const float v = bf16_bits_to_f32(h_out ? h_out[row + c] : at(c)) * s * weight[c];
    if (y) y[row + c] = f32_to_bf16_bits(v);
    if (yq) {  // H a multiple of 32: 32 lanes hold a block
      uint32_t a = __float_as_uint(v) & 0x7FFFFFFFu;
#pragma unroll
      for (int m = 16; m >= 1; m >>= 1) a = max(a, (uint32_t)__shfl_xor((int)a, m, 32));
      const uint32_t code = mx_scale_code<kMxFp8>(a);
      const float u[8] = {code == kMxNan ? 0.f : mx_scaled<kMxFp8>(v, code)};
      yq[row + c] = (uint8_t)mx_pack8<kMxFp8>(u);
      if (c % 32 == 0) ys[(row + c) / 32] = (uint8_t)code;
    }
  }
}

// Backward. A block takes rows b, b + NB, ..; it keeps its part of dg for the
// columns it owns in registers and leaves it in part[b][H]. A row's loads are
// issued before the row in front of it is worked on.
template <int NT, int CH>
__global__ __launch_bounds__(NT) void rms_norm_bwd_rows_kernel(
    const uint16_t* dy, const uint16_t* h, const float* __restrict__ weight, float eps, int T,
    int H, const uint16_t* dres, uint16_t* dx, float* __restrict__ part) {
  __shared__ float buf[2][2][NT / kWave];
  const int tid = threadIdx.x;
  float dg[CH][8] = {}, w[CH][8];
  u16x8 hn[CH], dn[CH], rn[CH];
  auto fetch = [&](int t) {
    const size_t row = (size_t)t * H;
#pragma unroll
    for (int i = 0; i < CH; ++i) {
      const int c = (tid + i * NT) * 8;
      hn[i] = dn[i] = rn[i] = u16x8{};
      if (c < H) {
        hn[i] = *reinterpret_cast<const u16x8*>(h + row + c);
        dn[i] = *reinterpret_cast<const u16x8*>(dy + row + c);
        if (dres) rn[i] = *reinterpret_cast<const u16x8*>(dres + row + c);
      }
    }
  };
#pragma unroll
  for (int i = 0; i < CH; ++i) {
    const int c = (tid + i * NT) * 8;
#pragma unroll
    for (int j = 0; j < 8; ++j) w[i][j] = c < H ? weight[c + j] : 0.f;
  }
  int flip = 0;
  int t = blockIdx.x;
  if (t < T) fetch(t);
  for (; t < T; t += gridDim.x, flip ^= 1) {
    const size_t row = (size_t)t * H;
    u16x8 hv[CH], dv[CH], rv[CH];
    float ss = 0.f, sd = 0.f;
#pragma unroll
    for (int i = 0; i < CH; ++i) {
      hv[i] = hn[i];
      dv[i] = dn[i];
      rv[i] = rn[i];
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const float a = bf16_bits_to_f32(hv[i][j]);
        ss = fmaf(a, a, ss);
        sd = fmaf(w[i][j] * bf16_bits_to_f32(dv[i][j]), a, sd);
      }
    }
    if (t + (int)gridDim.x < T) fetch(t + gridDim.x);
    // two buffers in turn: a wave can be one row ahead of the slowest
    ss = wave_sum_f32(ss);
    sd = wave_sum_f32(sd);
    if (tid % kWave == 0) {
      buf[flip][0][tid / kWave] = ss;
      buf[flip][1][tid / kWave] = sd;
    }
    __syncthreads();
    ss = sd = 0.f;
#pragma unroll
    for (int i = 0; i < NT / kWave; ++i) {
      ss += buf[flip][0][i];
      sd += buf[flip][1][i];
    }
    const float s = rstd_of(ss, H, eps);
    const float m = s * s * (sd / (float)H);
#pragma unroll
    for (int i = 0; i < CH; ++i) {
      const int c = (tid + i * NT) * 8;
      float v[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const float a = bf16_bits_to_f32(hv[i][j]), d = bf16_bits_to_f32(dv[i][j]);
        v[j] = s * (w[i][j] * d - a * m);
        if (dres) v[j] += bf16_bits_to_f32(rv[i][j]);
        dg[i][j] = fmaf(d, a * s, dg[i][j]);
      }
      if (c < H) *reinterpret_cast<u16x8*>(dx + row + c) = pack8(v);
    }
  }
#pragma unroll
  for (int i = 0; i < CH; ++i) {
    const int c = (tid + i * NT) * 8;
    if (c < H) {
      float* p = part + (size_t)blockIdx.x * H + c;
      reinterpret_cast<f32x4*>(p)[0] = f32x4{dg[i][0], dg[i][1], dg[i][2], dg[i][3]};
      reinterpret_cast<f32x4*>(p)[1] = f32x4{dg[i][4], dg[i][5], dg[i][6], dg[i][7]};
    }
  }
}

// Any length and alignment; the block's part of dg lives in its row of part.
__global__ __launch_bounds__(256) void rms_norm_bwd_any_kernel(
    const uint16_t* dy, const uint16_t* h, const float* __restrict__ weight, float eps, int T,
    int H, const uint16_t* dres, uint16_t* dx, float* part) {
  __shared__ float b0[4], b1[4];
  float* p = part + (size_t)blockIdx.x * H;
  for (int c = threadIdx.x; c < H; c += 256) p[c] = 0.f;
  for (int t = blockIdx.x; t < T; t += gridDim.x) {
    const size_t row = (size_t)t * H;
    float ss = 0.f, sd = 0.f;
    for (int c = threadIdx.x; c < H; c += 256) {
      const float a = bf16_bits_to_f32(h[row + c]), d = bf16_bits_to_f32(dy[row + c]);
      ss = fmaf(a, a, ss);
      sd = fmaf(weight[c] * d, a, sd);
    }
    ss = block_sum<256>(ss, b0);
    sd = block_sum<256>(sd, b1);
    const float s = rstd_of(ss, H, eps);
    const float m = s * s * (sd / (float)H);
    for (int c = threadIdx.x; c < H; c += 256) {
      const float a = bf16_bits_to_f32(h[row + c]), d = bf16_bits_to_f32(dy[row + c]);
      float v = s * (weight[c] * d - a * m);
      if (dres) v += bf16_bits_to_f32(dres[row + c]);
      p[c] = fmaf(d, a * s, p[c]);
      dx[row + c] = f32_to_bf16_bits(v);
    }
    __syncthreads();  // b0, b1 are rewritten for the next row
  }
}

// dg[c] = sum of part[b][c] over the nb blocks: 16 columns a block, 64 slices
// of the blocks' parts, joined in slice order. (Few columns a block: at H 1024,
// 64 of them left 16 blocks to read 2 MB.)
__global__ __launch_bounds__(1024) void rms_norm_dweight_kernel(const float* __restrict__ part,
                                                                int nb, int H,
                                                                float* __restrict__ dg) {
  __shared__ float buf[64][17];
  const int col = threadIdx.x % 16, sl = threadIdx.x / 16;
  const int c = blockIdx.x * 16 + col;
  float s = 0.f;
  if (c < H) {
#pragma unroll 4
    for (int b = sl; b < nb; b += 64) s += part[(size_t)b * H + c];
  }
  buf[sl][col] = s;
  __syncthreads();
  if (sl == 0 && c < H) {
    float v = 0.f;
#pragma unroll
    for (int i = 0; i < 64; ++i) v += buf[i][col];
    dg[c] = v;
  }
}

bool a16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

int bwd_blocks(int T) { return std::min(T, 512); }

}  // namespace

hipError_t launch_rms_norm(const uint16_t* x, const uint16_t* res, const float* weight, float eps,
                           int T, int H, uint16_t* h_out, uint16_t* y, uint8_t* yq, uint8_t* ys,
                           hipStream_t s) {
  const bool vec = H % 8 == 0 && H <= 16384 && a16(x) && a16(res) && a16(weight) && a16(h_out) &&
                   a16(y) && (reinterpret_cast<uintptr_t>(yq) & 7u) == 0;
  // A launch has less than 2^32 threads: rows beyond 2^22 (short ones, up to 64
  // threads a row, or 256 off the 16-byte path) go in further launches.
  constexpr int MOST = 1 << 22;
  for (int t0 = 0; t0 < T; t0 += std::min(MOST, T - t0)) {
    const int n = std::min(MOST, T - t0);
    const size_t at = (size_t)t0 * H;
    const uint16_t* xn = x + at;
    const uint16_t* rn = res ? res + at : nullptr;
    uint16_t* hn = h_out ? h_out + at : nullptr;
    uint16_t* yn = y ? y + at : nullptr;
    uint8_t* qn = yq ? yq + at : nullptr;
    uint8_t* sn = ys ? ys + at / kMxBlock : nullptr;
#define MOE_NORM(NT, CH, BLOCKS, THREADS)                                                        \
  hipLaunchKernelGGL((rms_norm_rows_kernel<NT, CH>), dim3(BLOCKS), dim3(THREADS), 0, s, xn, rn, \
                     weight, eps, n, H, hn, yn, qn, sn)
    if (!vec)
      hipLaunchKernelGGL(rms_norm_any_kernel, dim3(n), dim3(256), 0, s, xn, rn, weight, eps, H, hn,
                         yn, qn, sn);
    else if (H <= 512) MOE_NORM(64, 1, (n + 3) / 4, 256);
    else if (H <= 2048) MOE_NORM(256, 1, n, 256);
    else if (H <= 4096) MOE_NORM(512, 1, n, 512);
    else if (H <= 8192) MOE_NORM(1024, 1, n, 1024);
    else MOE_NORM(1024, 2, n, 1024);
#undef MOE_NORM
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

size_t rms_norm_backward_workspace_bytes(int T, int H) { return (size_t)bwd_blocks(T) * H * 4; }

hipError_t launch_rms_norm_backward(const uint16_t* dy, const uint16_t* h, const float* weight,
                                    float eps, int T, int H, const uint16_t* dres, uint16_t* dx,
                                    float* dweight, float* part, hipStream_t s) {
  const int nb = bwd_blocks(T);
  const bool vec = H % 8 == 0 && H <= 16384 && a16(dy) && a16(h) && a16(weight) && a16(dres) &&
                   a16(dx);
#define MOE_NORM_BWD(NT, CH)                                                                   \
  hipLaunchKernelGGL((rms_norm_bwd_rows_kernel<NT, CH>), dim3(nb), dim3(NT), 0, s, dy, h,      \
                     weight, eps, T, H, dres, dx, part)
  if (T > 0) {
    if (!vec)
      hipLaunchKernelGGL(rms_norm_bwd_any_kernel, dim3(nb), dim3(256), 0, s, dy, h, weight, eps,
                         T, H, dres, dx, part);
    else if (H <= 512) MOE_NORM_BWD(64, 1);
    else if (H <= 2048) MOE_NORM_BWD(256, 1);
    else if (H <= 4096) MOE_NORM_BWD(512, 1);
    else if (H <= 8192) MOE_NORM_BWD(1024, 1);
    else MOE_NORM_BWD(1024, 2);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
#undef MOE_NORM_BWD
  hipLaunchKernelGGL(rms_norm_dweight_kernel, dim3((H + 15) / 16), dim3(1024), 0, s, part, nb, H,
                     dweight);
  return hipGetLastError();
}

}  // namespace moe
