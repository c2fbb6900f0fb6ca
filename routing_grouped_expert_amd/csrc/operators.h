// What the files of the operators around the layer call of one another.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace moe {

enum class Product;   // grouped.h
struct GroupedArgs;   // grouped.h
struct MxArgs;        // mx_matmul.h

// Compute units of the current device.
int compute_units();

// ---- grouped products
hipError_t launch_grouped(Product p, const GroupedArgs& a, bool out_fp32, hipStream_t stream);
hipError_t launch_grouped_matmul_mx(const uint8_t* xq, const uint8_t* xs, int x_bits,
                                    const int* rows, const int* off, int L, int T, int k, int N,
                                    int K, int M, const uint8_t* wq, const uint8_t* ws, void* y,
                                    bool y_fp32, hipStream_t s);

// Experts with at most skinny_rows() rows. x_bits 4, 8: microscaled operands; 16:
// bf16. others: blocks of the launch that follows, or 0.
int skinny_rows();
hipError_t launch_skinny(const MxArgs& a, int x_bits, bool y_fp32, int others, hipStream_t s);
// The experts with more than `lo` rows; Product::kDw: all.
hipError_t launch_grouped_dense(Product p, const GroupedArgs& a, bool out_fp32, int lo, int blocks,
                                hipStream_t stream);
hipError_t launch_mx_dense(const MxArgs& a, int x_bits, bool y_fp32, int lo, int blocks,
                           hipStream_t s);

// ---- norm
hipError_t launch_rms_norm(const uint16_t* x, const uint16_t* res, const float* weight, float eps,
                           int T, int H, uint16_t* h_out, uint16_t* y, uint8_t* yq, uint8_t* ys,
                           hipStream_t s);
size_t rms_norm_backward_workspace_bytes(int T, int H);
hipError_t launch_rms_norm_backward(const uint16_t* dy, const uint16_t* h, const float* weight,
                                    float eps, int T, int H, const uint16_t* dres, uint16_t* dx,
                                    float* dweight, float* part, hipStream_t s);

// ---- microscaled formats
hipError_t launch_quantize_mx(const void* x, bool x_fp32, size_t n, int bits, uint8_t* codes,
                              uint8_t* scales, hipStream_t s);
hipError_t launch_swiglu_quantize_mx(const void* gu, bool gu_fp32, int N, int I, const int* rows,
                                     int bits, uint8_t* codes, uint8_t* scales, hipStream_t s);
hipError_t launch_dequantize_mx(const uint8_t* codes, const uint8_t* scales, size_t n, int bits,
                                void* out, bool out_fp32, hipStream_t s);

}  // namespace moe
