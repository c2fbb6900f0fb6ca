// Grouped product on microscaled operands: y[n] = W[e] x[n] with MXFP4 weights
// and MXFP8 or MXFP4 rows, on the scaled matrix instruction
// v_mfma_scale_f32_16x16x128_f8f6f4 (one scale per 32 of the contraction and row
// applied by the instruction; exact products, fp32 sums, for which E4M3 rows go in
// two parts: mx_matmul.h).
//
// Only the device knows how many rows an expert has, so the kernel for experts
// with few rows and the one for the others both run, and each passes over the
// other's experts; the second is left out where no expert can have more.
#include "mx_matmul.h"
#include "operators.h"

namespace moe {

hipError_t launch_grouped_matmul_mx(const uint8_t* xq, const uint8_t* xs, int x_bits,
                                    const int* rows, const int* off, int L, int T, int k, int N,
                                    int K, int M, const uint8_t* wq, const uint8_t* ws, void* y,
                                    bool y_fp32, hipStream_t s) {
  MxArgs a{xq, xs, wq, ws, y, rows, off, L, T, k, N, K, M, 0, 0};
  divide_by(k, &a.div_m, &a.div_s);
  const bool more = N > skinny_rows();
  const int blocks = compute_units();
  hipError_t e = launch_skinny(a, x_bits, y_fp32, more ? blocks : 0, s);
  if (e == hipSuccess && more)
    e = launch_mx_dense(a, x_bits, y_fp32, skinny_rows(), blocks, s);
  return e;
}

}  // namespace moe
