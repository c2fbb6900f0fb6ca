// Quantisation to and from the microscaled formats (mx.h), and SwiGLU with a
// quantised output.
//
// One pass over the data: a lane loads eight consecutive values (16 bytes of
// bf16), four lanes share a block's largest magnitude by two lane exchanges,
// and the codes leave as 4 or 8 bytes a lane. Bound by memory: 470 million bf16
// values to 4 bits in 236 us, 5.0 TB/s (four pieces a lane at once and 8 blocks a
// CU; 16 blocks 251 us), back in 250 us.
#include "mx.h"
#include "operators.h"

#include <algorithm>

namespace moe {

namespace {

__device__ __forceinline__ void load8(const uint16_t* p, float (&v)[8]) {
  const u16x8 u = *reinterpret_cast<const u16x8*>(p);
#pragma unroll
  for (int i = 0; i < 8; ++i) v[i] = bf16_bits_to_f32(u[i]);
}
__device__ __forceinline__ void load8(const float* p, float (&v)[8]) {
  const f32x4 a = reinterpret_cast<const f32x4*>(p)[0], b = reinterpret_cast<const f32x4*>(p)[1];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    v[i] = a[i];
    v[i + 4] = b[i];
  }
}
__device__ __forceinline__ void store8(uint16_t* p, const float (&v)[8]) {
  *reinterpret_cast<u32x4*>(p) = u32x4{pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3]),
                                       pack_bf16(v[4], v[5]), pack_bf16(v[6], v[7])};
}
__device__ __forceinline__ void store8(float* p, const float (&v)[8]) {
  reinterpret_cast<f32x4*>(p)[0] = f32x4{v[0], v[1], v[2], v[3]};
  reinterpret_cast<f32x4*>(p)[1] = f32x4{v[4], v[5], v[6], v[7]};
}

// Piece p: values 8 p .. 8 p + 7. The grid covers whole blocks, so the four
// lanes of a block are in or out together.
template <int BITS>
__device__ __forceinline__ void put8(uint8_t* codes, uint8_t* scales, size_t p, uint64_t c,
                                     uint32_t s) {
  if (BITS == kMxFp4)
    reinterpret_cast<uint32_t*>(codes)[p] = (uint32_t)c;
  else
    reinterpret_cast<u32x2*>(codes)[p] = u32x2{(uint32_t)c, (uint32_t)(c >> 32)};
  if ((p & 3) == 0) scales[p >> 2] = (uint8_t)s;
}

// Pieces a lane works on at a time: their loads are in flight together.
constexpr int AT_ONCE = 4;

template <int BITS, typename In>
__global__ __launch_bounds__(256) void mx_quantize_kernel(const In* __restrict__ x, size_t pieces,
                                                          uint8_t* __restrict__ codes,
                                                          uint8_t* __restrict__ scales) {
  const size_t step = (size_t)gridDim.x * 256;
  for (size_t p0 = (size_t)blockIdx.x * 256 + threadIdx.x; p0 < pieces; p0 += AT_ONCE * step) {
    float v[AT_ONCE][8];
#pragma unroll
    for (int i = 0; i < AT_ONCE; ++i)
      if (p0 + i * step < pieces) load8(x + (p0 + i * step) * 8, v[i]);
#pragma unroll
    for (int i = 0; i < AT_ONCE; ++i) {
      const size_t p = p0 + i * step;
      if (p < pieces) {
        uint32_t s;
        const uint64_t c = mx_quantize8<BITS>(v[i], &s);
        put8<BITS>(codes, scales, p, c, s);
      }
    }
  }
}

template <int BITS, typename In>
__global__ __launch_bounds__(256) void swiglu_mx_kernel(const In* __restrict__ gu, int N, int I,
                                                        const int* __restrict__ rows,
                                                        uint8_t* __restrict__ codes,
                                                        uint8_t* __restrict__ scales) {
  const int n = rows ? max(0, min(rows[0], N)) : N;
  const int per = I / 8;
  const size_t pieces = (size_t)n * per;
  const size_t step = (size_t)gridDim.x * 256;
  for (size_t p0 = (size_t)blockIdx.x * 256 + threadIdx.x; p0 < pieces; p0 += 2 * step) {
    float g[2][8], u[2][8];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const size_t p = p0 + i * step;
      if (p < pieces) {
        // (32 bits wherever they do: a 64-bit division is a few hundred instructions)
        const size_t r = pieces <= 0xFFFFFFFFu ? (uint32_t)p / (uint32_t)per : p / per;
        const In* at = gu + r * 2 * I + (p - r * per) * 8;
        load8(at, g[i]);
        load8(at + I, u[i]);
      }
    }
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const size_t p = p0 + i * step;
      if (p < pieces) {
#pragma unroll
        for (int j = 0; j < 8; ++j) u[i][j] = g[i][j] / (1.0f + expf(-g[i][j])) * u[i][j];
        uint32_t s;
        const uint64_t q = mx_quantize8<BITS>(u[i], &s);
        put8<BITS>(codes, scales, p, q, s);
      }
    }
  }
}

__device__ __forceinline__ float e2m1_value(uint32_t c) {
  // magnitudes 0, 1/2, 1, 3/2, 2, 3, 4, 6 as eight nibbles of twice the value
  const float m = 0.5f * (float)((0xC8643210u >> ((c & 7) * 4)) & 15u);
  return c & 8 ? -m : m;
}
__device__ __forceinline__ float e4m3_value(uint32_t c) {
  const uint32_t e = (c >> 3) & 15, m = c & 7;
  if ((c & 127) == 127) return __uint_as_float(0x7FC00000u);
  const float v = e ? ldexpf((float)(8 + m), (int)e - 10) : ldexpf((float)m, -9);
  return c & 128 ? -v : v;
}

template <int BITS, typename Out>
__global__ __launch_bounds__(256) void mx_dequantize_kernel(const uint8_t* __restrict__ codes,
                                                            const uint8_t* __restrict__ scales,
                                                            size_t pieces, Out* __restrict__ out) {
  const size_t step = (size_t)gridDim.x * 256;
  for (size_t p0 = (size_t)blockIdx.x * 256 + threadIdx.x; p0 < pieces; p0 += AT_ONCE * step) {
    uint32_t s[AT_ONCE];
    uint64_t c[AT_ONCE];
#pragma unroll
    for (int i = 0; i < AT_ONCE; ++i) {
      const size_t p = p0 + i * step;
      if (p < pieces) {
        s[i] = scales[p >> 2];
        if (BITS == kMxFp4) {
          c[i] = reinterpret_cast<const uint32_t*>(codes)[p];
        } else {
          const u32x2 q = reinterpret_cast<const u32x2*>(codes)[p];
          c[i] = (uint64_t)q[1] << 32 | q[0];
        }
      }
    }
#pragma unroll
    for (int i = 0; i < AT_ONCE; ++i) {
      const size_t p = p0 + i * step;
      if (p < pieces) {
        float v[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const uint32_t q = (uint32_t)(c[i] >> (j * BITS)) & ((1u << BITS) - 1);
          v[j] = s[i] == kMxNan ? __uint_as_float(0x7FC00000u)
                                : ldexpf(BITS == kMxFp4 ? e2m1_value(q) : e4m3_value(q), (int)s[i] - 127);
        }
        store8(out + p * 8, v);
      }
    }
  }
}

int blocks_for(size_t pieces) { return (int)std::min<size_t>((pieces + 255) / 256, 256 * 8); }

}  // namespace

hipError_t launch_quantize_mx(const void* x, bool x_fp32, size_t n, int bits, uint8_t* codes,
                              uint8_t* scales, hipStream_t s) {
  const size_t p = n / 8;
  const dim3 g(blocks_for(p)), b(256);
  const float* xf = static_cast<const float*>(x);
  const uint16_t* xh = static_cast<const uint16_t*>(x);
  if (bits == kMxFp4) {
    if (x_fp32) hipLaunchKernelGGL((mx_quantize_kernel<4, float>), g, b, 0, s, xf, p, codes, scales);
    else hipLaunchKernelGGL((mx_quantize_kernel<4, uint16_t>), g, b, 0, s, xh, p, codes, scales);
  } else {
    if (x_fp32) hipLaunchKernelGGL((mx_quantize_kernel<8, float>), g, b, 0, s, xf, p, codes, scales);
    else hipLaunchKernelGGL((mx_quantize_kernel<8, uint16_t>), g, b, 0, s, xh, p, codes, scales);
  }
  return hipGetLastError();
}

hipError_t launch_swiglu_quantize_mx(const void* gu, bool gu_fp32, int N, int I, const int* rows,
                                     int bits, uint8_t* codes, uint8_t* scales, hipStream_t s) {
  const dim3 g(blocks_for((size_t)N * I / 8)), b(256);
  const float* xf = static_cast<const float*>(gu);
  const uint16_t* xh = static_cast<const uint16_t*>(gu);
  if (bits == kMxFp4) {
    if (gu_fp32) hipLaunchKernelGGL((swiglu_mx_kernel<4, float>), g, b, 0, s, xf, N, I, rows, codes, scales);
    else hipLaunchKernelGGL((swiglu_mx_kernel<4, uint16_t>), g, b, 0, s, xh, N, I, rows, codes, scales);
  } else {
    if (gu_fp32) hipLaunchKernelGGL((swiglu_mx_kernel<8, float>), g, b, 0, s, xf, N, I, rows, codes, scales);
    else hipLaunchKernelGGL((swiglu_mx_kernel<8, uint16_t>), g, b, 0, s, xh, N, I, rows, codes, scales);
  }
  return hipGetLastError();
}

hipError_t launch_dequantize_mx(const uint8_t* codes, const uint8_t* scales, size_t n, int bits,
                                void* out, bool out_fp32, hipStream_t s) {
  const size_t p = n / 8;
  const dim3 g(blocks_for(p)), b(256);
  float* of = static_cast<float*>(out);
  uint16_t* oh = static_cast<uint16_t*>(out);
  if (bits == kMxFp4) {
    if (out_fp32) hipLaunchKernelGGL((mx_dequantize_kernel<4, float>), g, b, 0, s, codes, scales, p, of);
    else hipLaunchKernelGGL((mx_dequantize_kernel<4, uint16_t>), g, b, 0, s, codes, scales, p, oh);
  } else {
    if (out_fp32) hipLaunchKernelGGL((mx_dequantize_kernel<8, float>), g, b, 0, s, codes, scales, p, of);
    else hipLaunchKernelGGL((mx_dequantize_kernel<8, uint16_t>), g, b, 0, s, codes, scales, p, oh);
  }
  return hipGetLastError();
}

}  // namespace moe
