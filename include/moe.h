/*
 * moe.h -- C ABI of libmoe.so, a single-GPU Mixture-of-Experts layer forward
 * pass for AMD Instinct MI355X (gfx950).
 *
 * The layer: router logits -> softmax / top-k / renormalise -> per-expert
 * histogram, prefix scan and stable token permutation -> gather of each
 * expert's activation rows -> grouped expert FFN (W1 gate/up, SwiGLU, W2 down)
 * -> routing-weighted combine back to token order. One GPU runs either all
 * experts or one contiguous share of them.
 *
 * Pages cited (analyses of merged flashinfer pull requests):
 *  [P-ACT]   "FlashInfer MoE optimisation: overlapping grouped activation
 *            staging on Ampere and Hopper" (PR #7368).
 *  [P-ROUTE] "TRTLLM-Gen MoE routing optimisation in FlashInfer: relieving
 *            register pressure" (PR #3751).
 *  [P-A2A]   "FlashInfer MoE all-to-all optimisation: TRT-LLM's one-sided A2A"
 *            (PR #3697).
 *  [P-FP4]   "Beyond the limits of NVFP4 GEMM: pipeline optimisation with L2
 *            weight prefetch" (PR #7424).
 *  [P-VSA]   "Attention optimisation for Hopper (SM90): FlashInfer 'Cake'
 *            backend" (PR #5586).
 *
 * Conventions shared by every call:
 *  - Pointers are caller-owned DEVICE pointers unless a parameter says
 *    "host". The library never allocates, frees or keeps memory, and keeps
 *    no state between calls ([P-FP4] section 2: workspace and outputs are
 *    handed in by the caller).
 *  - bf16 tensors are passed as uint16_t bit patterns. All tensors are dense
 *    row-major with the shapes written next to each parameter.
 *  - `stream` is a hipStream_t passed as void*; NULL is the null stream.
 *    Calls enqueue work and return; nothing waits for the GPU, and no call
 *    copies data to the host.
 *  - Errors: every argument the host can see is checked before anything is
 *    launched; on any error nothing is launched and no output is written
 *    (checked launches that report failure, [P-A2A] section 2). A failed
 *    launch returns MOE_ERROR_LAUNCH. Nothing throws across the ABI.
 *  - T = 0 is valid and launches nothing.
 *  - Limits: 1 <= E <= 4096, 1 <= k <= min(E, 32), H >= 1, I >= 1,
 *    T * k < 2^31, T * k * max(H, I) < 2^31 elements.
 *  - Fast path: 16-byte aligned x / w1 / w2 / expert_out / workspace and H, I
 *    multiples of 128. Any other shape or alignment runs a correct
 *    element-wise path instead of failing ([P-ACT] section 1: the 128-bit
 *    vector gather keeps a scalar fallback for unaligned inputs).
 */
#ifndef MOE_H
#define MOE_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum moe_status {
  MOE_SUCCESS = 0,
  MOE_ERROR_INVALID_VALUE = 1, /* bad size, null pointer, share out of range */
  MOE_ERROR_UNSUPPORTED = 2,   /* outside the limits above */
  MOE_ERROR_WORKSPACE = 3,     /* workspace missing, too small or misaligned */
  MOE_ERROR_LAUNCH = 4         /* a kernel launch failed */
} moe_status;

/* Human-readable name of a status code (static storage, never NULL). */
const char* moe_status_string(moe_status status);

/* Name of the HIP error behind the last MOE_ERROR_LAUNCH returned on the
 * calling host thread ("hipSuccess" if there was none). Diagnostic only. */
const char* moe_last_launch_error(void);

/*
 * moe_partition -- contiguous ceil/floor split of E experts over S shares.
 * [P-A2A] section 1, "Flexible expert-to-rank mapping": base = E / S,
 * rem = E % S; shares 0 .. rem-1 hold base + 1 experts, the others base, in
 * expert order. Pure host function; first_expert and num_local are HOST
 * pointers. E < S is allowed (the last shares are then empty).
 * Errors: E < 1, S < 1, share outside [0, S), null output pointer.
 */
moe_status moe_partition(int32_t num_experts, int32_t num_shares, int32_t share,
                         int32_t* first_expert, int32_t* num_local);

/*
 * moe_workspace_size -- bytes of device workspace that moe_forward needs
 * (*bytes, HOST pointer); the caller allocates it and passes it in ([P-FP4]
 * section 2: the caller provides the workspace and output buffers).
 * moe_router_logits, moe_permute, moe_route_permute and moe_grouped_ffn need
 * no more than this for the same sizes, so one workspace serves every call.
 * The workspace must be 256-byte aligned. Its contents need no
 * initialisation and are scratch after the call.
 */
moe_status moe_workspace_size(int32_t T, int32_t H, int32_t I, int32_t E, int32_t k,
                              int32_t num_local, size_t* bytes);

/*
 * moe_router_logits -- logits[t, e] = x[t, :] . w_gate[e, :] + bias[e].
 * The pages leave the router unstated; the logit is the fp32 value of the
 * exact affine map: the products (bf16 x fp32) are exact in fp64, the sum is
 * carried in fp64 and rounded once to fp32.
 *   x       [T, H] bf16;  w_gate [E, H] fp32;  bias [E] fp32 or NULL
 *   logits  [T, E] fp32 (output)
 *   ws / ws_bytes  workspace (moe_workspace_size with the same T, H, E; it
 *                  holds fp64 partial sums when T > 64, unused otherwise)
 */
moe_status moe_router_logits(const uint16_t* x, const float* w_gate, const float* bias, int32_t T,
                             int32_t H, int32_t E, float* logits, void* ws, size_t ws_bytes,
                             void* stream);

/*
 * moe_route -- softmax over the E logits, top-k, renormalise over the k.
 * [P-ROUTE] (routing kernel emitting routing indices; "softmax_sum" method).
 * Selection on the fp32 logits, larger first, equal logits to the lower
 * expert id (-0 equals +0); slot j holds the j-th selection. Weights:
 * w_j = exp(l_j - l_0) / sum_i exp(l_i - l_0) over the k selected logits,
 * which equals the full softmax renormalised over the selection.
 *   logits       [T, E] fp32, finite (NaN / inf give unspecified ids/weights)
 *   topk_ids     [T, k] int32 (output), distinct within a token
 *   topk_weights [T, k] fp32 (output), sum to 1 per token
 */
moe_status moe_route(const float* logits, int32_t T, int32_t E, int32_t k, int32_t* topk_ids,
                     float* topk_weights, void* stream);

/*
 * moe_permute -- per-expert histogram, prefix scan and stable permutation.
 * Entries are expanded indices r = t * k + j. The local share is experts
 * [first_expert, first_expert + num_local).
 *   topk_ids             [T, k] int32 in [0, E), distinct within a token.
 *                        Ids outside [0, E) are skipped (not counted,
 *                        expanded_to_permuted = -1); repeated ids within a
 *                        token give an unspecified permutation but never an
 *                        out-of-range write.
 *   expert_counts        [E] int32 (output): entries per expert, all E.
 *   expert_offsets       [num_local + 1] int32 (output): exclusive scan of
 *                        the local counts; offsets[num_local] = N_L.
 *   permuted_rows        [T * k] int32 (output): permuted_rows[p] = r of the
 *                        p-th local entry, experts in order and ascending r
 *                        within an expert; positions >= N_L are not written.
 *   expanded_to_permuted [T * k] int32 (output): p of entry r, or -1 when
 *                        r's expert is outside the share ([P-ACT] section 1
 *                        marks absent group members with a negative index).
 *   ws / ws_bytes        workspace (moe_workspace_size).
 */
moe_status moe_permute(const int32_t* topk_ids, int32_t T, int32_t k, int32_t E,
                       int32_t first_expert, int32_t num_local, int32_t* expert_counts,
                       int32_t* expert_offsets, int32_t* permuted_rows,
                       int32_t* expanded_to_permuted, void* ws, size_t ws_bytes, void* stream);

/*
 * moe_route_permute -- moe_route, then moe_permute on its topk_ids: the
 * routing steps of the layer in one call (the routing kernel of [P-ROUTE]
 * emits the routing indices that the permutation consumes), in the variant
 * moe_routing_plan names for these sizes. Arguments, outputs and errors are
 * those of moe_route and moe_permute; the workspace is moe_permute's
 * (moe_workspace_size covers it). Every variant gives identical outputs.
 */
moe_status moe_route_permute(const float* logits, int32_t T, int32_t E, int32_t k,
                             int32_t first_expert, int32_t num_local, int32_t* topk_ids,
                             float* topk_weights, int32_t* expert_counts, int32_t* expert_offsets,
                             int32_t* permuted_rows, int32_t* expanded_to_permuted, void* ws,
                             size_t ws_bytes, void* stream);

/*
 * Routing variants: how the selection and the permutation are split into
 * kernels ([P-ROUTE] section 1: the launch shape follows the token count;
 * section 2: the valid shapes are fixed ahead of time).
 *   MOE_ROUTING_ONE_BLOCK   T <= 64: one single-block kernel selects and
 *                           permutes in on-chip memory (one launch; the
 *                           selection runs on one compute unit).
 *   MOE_ROUTING_TWO_KERNELS a selection kernel (one wave per token), then a
 *                           single-block permutation; while every 64-token
 *                           tile's masks and bases fit in one block's LDS.
 *   MOE_ROUTING_TILED       the selection kernel also writes per-tile token
 *                           masks, then a scan kernel and a scatter kernel;
 *                           any T.
 */
typedef enum moe_routing_variant {
  MOE_ROUTING_AUTO = 0,
  MOE_ROUTING_ONE_BLOCK = 1,
  MOE_ROUTING_TWO_KERNELS = 2,
  MOE_ROUTING_TILED = 3
} moe_routing_variant;

/*
 * moe_routing_plan -- the variant moe_route_permute and moe_forward run for
 * T tokens, E experts, top-k and a share of num_local experts (*variant,
 * HOST pointer): the applicable variant with the smallest time predicted by
 * a cost model fitted to the variants' measured times ([P-VSA]'s planner
 * likewise picks a kernel configuration from a cost estimate). Pure host
 * function. Errors as moe_route.
 */
moe_status moe_routing_plan(int32_t T, int32_t E, int32_t k, int32_t num_local,
                            int32_t* variant);

/*
 * moe_route_permute_variant -- moe_route_permute in a given variant (a
 * moe_routing_variant; MOE_ROUTING_AUTO = the plan), for measurement and
 * testing. MOE_ERROR_UNSUPPORTED when the variant does not apply to these
 * sizes; otherwise as moe_route_permute.
 */
moe_status moe_route_permute_variant(const float* logits, int32_t T, int32_t E, int32_t k,
                                     int32_t first_expert, int32_t num_local, int32_t* topk_ids,
                                     float* topk_weights, int32_t* expert_counts,
                                     int32_t* expert_offsets, int32_t* permuted_rows,
                                     int32_t* expanded_to_permuted, void* ws, size_t ws_bytes,
                                     int32_t variant, void* stream);

/*
 * moe_grouped_ffn -- for every local entry p of local expert i:
 *   x_g   = x[permuted_rows[p] / k]   (gather; [P-ACT] section 1 divides the
 *                                      route index by the route divisor)
 *   g, u  = W1[i][0:I] . x_g, W1[i][I:2I] . x_g   (gate rows first, then up;
 *                                      the gate/up split of [P-ACT] section 2)
 *   a     = silu(g) * u                (kept in fp32, never rounded to bf16)
 *   out_p = W2[i] . a
 * bf16 MFMA with fp32 accumulation; a enters W2's product as the exact sum of
 * two bf16 parts (hi + lo), so only the final output is ever rounded.
 *   x              [T, H] bf16
 *   permuted_rows  [T * k] int32, entries of [0, N_L) read; values outside
 *                  [0, T * k) gather a zero row
 *   expert_offsets [num_local + 1] int32, non-decreasing from 0, last <= T*k
 *   w1             [num_local, 2I, H] bf16 (local experts only)
 *   w2             [num_local, H, I] bf16
 *   expert_out     [T * k, H] fp32 (output): rows [0, N_L) written
 *   ws / ws_bytes  workspace (moe_workspace_size)
 */
moe_status moe_grouped_ffn(const uint16_t* x, const int32_t* permuted_rows,
                           const int32_t* expert_offsets, int32_t num_local, int32_t T, int32_t k,
                           int32_t H, int32_t I, const uint16_t* w1, const uint16_t* w2,
                           float* expert_out, void* ws, size_t ws_bytes, void* stream);

/*
 * moe_grouped_ffn_fp8 -- moe_grouped_ffn with FP8 expert weights: the same
 * gather, gate/up split, SwiGLU and down projection, with each weight row
 * stored as FP8 E4M3 codes and one fp32 scale ([P-ACT] section 2 runs the
 * grouped projection on FP8 E4M3 operands beside bf16 / fp16). Reading: the
 * OCP "e4m3fn" encoding (bias 7, no infinities, 0x7F / 0xFF NaN), weights
 * only (x stays bf16), W[r, c] = scale[r] * value(code[r, c]). Codes are
 * widened to bf16 exactly, multiplied on bf16 MFMA with fp32 accumulation,
 * and each finished row sum is multiplied by its row's scale.
 *   w1q  [num_local, 2I, H] uint8 codes     w1s  [num_local, 2I] fp32 scales
 *   w2q  [num_local, H, I] uint8 codes      w2s  [num_local, H] fp32 scales
 * Every other argument, the workspace and the errors are as for
 * moe_grouped_ffn; w1s and w2s must not be NULL.
 */
moe_status moe_grouped_ffn_fp8(const uint16_t* x, const int32_t* permuted_rows,
                               const int32_t* expert_offsets, int32_t num_local, int32_t T,
                               int32_t k, int32_t H, int32_t I, const uint8_t* w1q,
                               const float* w1s, const uint8_t* w2q, const float* w2s,
                               float* expert_out, void* ws, size_t ws_bytes, void* stream);

/*
 * moe_combine -- y[t, :] = sum over j ascending of topk_weights[t, j] *
 * expert_out[expanded_to_permuted[t*k + j], :], skipping -1 entries; fp32
 * accumulation and one round-to-nearest-even to bf16 ([P-VSA] section 3
 * keeps fp32 partials until the end). A token with no local entry gets 0.
 *   expert_out           [T * k, H] fp32 (rows indexed by permuted position)
 *   expanded_to_permuted [T * k] int32, values in [-1, T * k)
 *   topk_weights         [T, k] fp32
 *   y                    [T, H] bf16 (output)
 */
moe_status moe_combine(const float* expert_out, const int32_t* expanded_to_permuted,
                       const float* topk_weights, int32_t T, int32_t k, int32_t H, uint16_t* y,
                       void* stream);

/*
 * moe_forward -- the whole layer on one GPU for one expert share:
 * moe_router_logits -> moe_route_permute -> moe_grouped_ffn -> moe_combine,
 * stream-ordered, with no host synchronisation in between. The share is the
 * contiguous expert range of the ceil/floor partition ([P-A2A] section 1;
 * moe_partition); selections of experts outside it are masked after
 * renormalisation (the non-local members of [P-ACT] section 1 carry a
 * negative index), so the outputs of all shares add up to the whole layer.
 *   x [T, H] bf16; w_gate [E, H] fp32; router_bias [E] fp32 or NULL;
 *   w1 [num_local, 2I, H] bf16; w2 [num_local, H, I] bf16 (local experts)
 *   y [T, H] bf16 (output)
 *   logits_out [T, E] fp32, topk_ids_out [T, k] int32,
 *   topk_weights_out [T, k] fp32: optional outputs (NULL = kept in ws)
 *   ws / ws_bytes: workspace of at least moe_workspace_size bytes.
 */
moe_status moe_forward(const uint16_t* x, const float* w_gate, const float* router_bias,
                       const uint16_t* w1, const uint16_t* w2, int32_t T, int32_t H, int32_t I,
                       int32_t E, int32_t k, int32_t first_expert, int32_t num_local, uint16_t* y,
                       float* logits_out, int32_t* topk_ids_out, float* topk_weights_out,
                       void* ws, size_t ws_bytes, void* stream);

/*
 * moe_forward_fp8 -- moe_forward with the FP8 expert weights of
 * moe_grouped_ffn_fp8 (E4M3 codes and one fp32 scale per row, [P-ACT]
 * section 2): router, route, permute and combine as in moe_forward, the
 * grouped FFN as in moe_grouped_ffn_fp8.
 *   w1q [num_local, 2I, H] uint8, w1s [num_local, 2I] fp32,
 *   w2q [num_local, H, I] uint8, w2s [num_local, H] fp32 (local experts)
 * Every other argument, the workspace (moe_workspace_size) and the errors
 * are as for moe_forward.
 */
moe_status moe_forward_fp8(const uint16_t* x, const float* w_gate, const float* router_bias,
                           const uint8_t* w1q, const float* w1s, const uint8_t* w2q,
                           const float* w2s, int32_t T, int32_t H, int32_t I, int32_t E,
                           int32_t k, int32_t first_expert, int32_t num_local, uint16_t* y,
                           float* logits_out, int32_t* topk_ids_out, float* topk_weights_out,
                           void* ws, size_t ws_bytes, void* stream);

/* Size of the device scratch array behind moe_forward_no_alloc (bytes). */
#define MOE_NO_ALLOC_SCRATCH_BYTES ((size_t)128 << 20)

/*
 * moe_forward_no_alloc -- moe_forward without a workspace argument, for
 * callers that cannot allocate device memory (code under stream capture,
 * tight serving loops, hosts that forbid allocation). The workspace is a
 * device array of MOE_NO_ALLOC_SCRATCH_BYTES inside the library; each GPU
 * holds its own copy from the first call on it until the process ends. No
 * call allocates or frees memory.
 *   Every argument, output and error is as for moe_forward, plus:
 *   MOE_ERROR_WORKSPACE when moe_workspace_size for these sizes exceeds
 *   MOE_NO_ALLOC_SCRATCH_BYTES (128 MiB): decode-shaped layers (8.5 MiB at
 *   T 32, H 4096, I 14336, 8 experts, top-2) fit; shapes with more than
 *   about 16 entries per expert, whose FFN stages token rows in LDS and keeps
 *   ~130 MiB of cross-block partial sums, do not.
 *   MOE_ERROR_LAUNCH when the array's device address cannot be obtained.
 * Every call on one GPU uses that GPU's one array: calls that overlap on the
 * same GPU (concurrent streams or host threads) race and must be ordered by
 * the caller. The array keeps the last call's contents; every value a call
 * reads from it is written earlier in the same call.
 */
moe_status moe_forward_no_alloc(const uint16_t* x, const float* w_gate,
                                const float* router_bias, const uint16_t* w1,
                                const uint16_t* w2, int32_t T, int32_t H, int32_t I, int32_t E,
                                int32_t k, int32_t first_expert, int32_t num_local, uint16_t* y,
                                float* logits_out, int32_t* topk_ids_out,
                                float* topk_weights_out, void* stream);

/*
 * Products over rows grouped by expert: the expert projections on their own,
 * with their gradients, for training and for layers that moe_grouped_ffn does
 * not describe. Rows are in the order of moe_permute: expert i of the share
 * has rows [expert_offsets[i], expert_offsets[i + 1]), any number of them,
 * none included. Offsets are read on the device and cut to [0, N]; an end
 * below its begin is no rows; a row that two ranges name gets either expert's
 * values. bf16 MFMA, fp32 accumulation over the whole contraction in
 * a fixed order, one rounding at the output (bf16, or none for fp32).
 *
 * moe_grouped_matmul     y[n, :]  = w[i] . x_n           n in expert i's rows
 * moe_grouped_matmul_dx  dx[n, :] = w[i]^T . dy[n, :]    n in expert i's rows
 * moe_grouped_matmul_dw  dw[i]    = sum over expert i's rows of dy[n, :] x_n^T
 *
 *   x_n    x[permuted_rows[n] / k, :]; a zero row when permuted_rows[n] is
 *          outside [0, T * k). With permuted_rows NULL x_n = x[n, :], and then
 *          T = N and k = 1. (The gradient of a gathered x is the sum of a
 *          token's dx rows: moe_combine on fp32 dx with weights 1.)
 *   x      [T, K] bf16                  w    [num_local, M, K] bf16
 *   y      [N, M], dx [N, K] (output)   dy   [N, M] bf16
 *          rows outside the experts' ranges are not written
 *   dw     [num_local, M, K] (output): zeros for an expert without rows
 *   *_fp32 0: the output is bf16, otherwise fp32
 * The output must not overlap an input. N = 0 or num_local = 0 launches
 * nothing (moe_grouped_matmul_dw writes its zeros for N = 0).
 * Limits: num_local <= 4096, K and M <= 2^20, k <= 32; T * k, T * K, N * K,
 * N * M and M * K < 2^31.
 * Fast path: 16-byte aligned pointers, K and M multiples of 8; other shapes
 * run element by element.
 */
moe_status moe_grouped_matmul(const uint16_t* x, const int32_t* permuted_rows,
                              const int32_t* expert_offsets, int32_t num_local, int32_t T,
                              int32_t k, int32_t N, int32_t K, int32_t M, const uint16_t* w,
                              void* y, int32_t y_fp32, void* stream);
moe_status moe_grouped_matmul_dx(const uint16_t* dy, const int32_t* expert_offsets,
                                 int32_t num_local, int32_t N, int32_t K, int32_t M,
                                 const uint16_t* w, void* dx, int32_t dx_fp32, void* stream);
moe_status moe_grouped_matmul_dw(const uint16_t* dy, const uint16_t* x,
                                 const int32_t* permuted_rows, const int32_t* expert_offsets,
                                 int32_t num_local, int32_t T, int32_t k, int32_t N, int32_t K,
                                 int32_t M, void* dw, int32_t dw_fp32, void* stream);

/*
 * moe_rms_norm -- the step in front of the layer: residual addition, root-
 * mean-square norm, and the normed rows in bf16 (for the router and bf16
 * experts) and / or in 8 bits (for moe_grouped_matmul_mx).
 *   h = bf16(x + residual)  (x without a residual)
 *   y = h / sqrt(mean(h^2) + eps) * weight
 * The mean is that of the rounded h, which the backward reads. fp32 sums; y
 * is rounded once to each output's type.
 *   x, residual   [T, H] bf16; residual may be NULL
 *   weight        [H] fp32
 *   residual_out  [T, H] bf16 h (output) or NULL
 *   y             [T, H] bf16 (output) or NULL
 *   yq, ys        [T, H] E4M3 codes and [T, H / 32] E8M0 scales (outputs, as
 *                 moe_quantize_mx of the unrounded y), both or neither; then
 *                 H must be a multiple of 32
 * residual_out and y may be x or residual themselves (in place); outputs must
 * not overlap otherwise. eps >= 0. The squares are summed in fp32: a row whose
 * squares add up to more than 3.4e38 (values of 1e19, or of 1e17 in long rows) has
 * an infinite mean and zeros in y. Limits: H <= 2^20, T * H < 2^31.
 */
moe_status moe_rms_norm(const uint16_t* x, const uint16_t* residual, const float* weight,
                        float eps, int32_t T, int32_t H, uint16_t* residual_out, uint16_t* y,
                        uint8_t* yq, uint8_t* ys, void* stream);

/*
 * moe_rms_norm_backward -- gradients of moe_rms_norm's bf16 y, with s the
 * row's 1 / sqrt(mean(h^2) + eps):
 *   dx = s (weight dy - h s^2 mean(weight dy h)) + dresidual
 *   dweight = sum over rows of dy h s   (a fixed order)
 * dx is the gradient of x and of residual alike. A row whose mean is infinite
 * has s = 0: dx = dresidual and nothing in dweight, NaN where the mean of
 * weight dy h is not finite either.
 *   dy, h       [T, H] bf16: the gradient of y, and moe_rms_norm's h
 *   dresidual   [T, H] bf16, the gradient arriving at residual_out, or NULL
 *   dx          [T, H] bf16 (output); may be dy or dresidual itself
 *   dweight     [H] fp32 (output); zeros for T = 0
 *   ws          workspace of moe_rms_norm_backward_workspace_size bytes,
 *               256-byte aligned; NULL allowed when that is 0. Calls that may
 *               run at the same time need one each.
 */
moe_status moe_rms_norm_backward_workspace_size(int32_t T, int32_t H, size_t* bytes);
moe_status moe_rms_norm_backward(const uint16_t* dy, const uint16_t* h, const float* weight,
                                 float eps, int32_t T, int32_t H, const uint16_t* dresidual,
                                 uint16_t* dx, float* dweight, void* ws, size_t ws_bytes,
                                 void* stream);

/*
 * Microscaled formats (OCP MX): 32 consecutive values of a row share an E8M0
 * scale 2^(code - 127); values are E2M1 (bits = 4: MXFP4, two codes to a byte,
 * the first in the low half) or E4M3 (bits = 8: MXFP8).
 *
 * moe_quantize_mx -- per block: scale exponent floor(log2 max|v|) minus the
 * exponent of the format's largest power of two (2 for E2M1, 8 for E4M3), cut
 * to [-127, 127], -127 for a block of zeros; values divided by the scale, cut
 * to the format's largest (6, 448), rounded to nearest, ties to even. A block
 * that holds an infinity or a NaN gets scale code 255 (NaN) and zero codes.
 *   x       [R, K] bf16, or fp32 when x_fp32 is not 0; K a multiple of 32
 *   codes   [R, K / 2] (bits 4) or [R, K] (bits 8) (output)
 *   scales  [R, K / 32] (output)
 * moe_swiglu_quantize_mx -- the same of a = silu(gu[r, 0:I]) * gu[r, I:2I]
 * (a in fp32; gates below -88.7, whose exponential overflows, give -0), the step
 * between an expert's two products.
 *   gu      [N, 2I] bf16 or fp32; I a multiple of 32
 *   num_rows  DEVICE pointer to the number of rows to take (cut to [0, N];
 *           rows behind are neither read nor written), for instance
 *           expert_offsets + num_local; NULL: N
 *   codes, scales  as above with R = N, K = I
 * moe_dequantize_mx -- out[r, c] = value(code) * 2^(scale code - 127), exact
 * in fp32 (infinity past its largest value, which E4M3 reaches under scale codes
 * from 247 on and E2M1 from 253 on) and rounded once in bf16; NaN for scale code
 * 255.
 *
 * Limits: R * K, N * 2I < 2^34. Pointers must be 16-byte aligned except
 * scales. Outputs must not overlap inputs. R = 0 or N = 0 launches nothing.
 */
moe_status moe_quantize_mx(const void* x, int32_t x_fp32, int32_t R, int32_t K, int32_t bits,
                           uint8_t* codes, uint8_t* scales, void* stream);
moe_status moe_swiglu_quantize_mx(const void* gu, int32_t gu_fp32, int32_t N, int32_t I,
                                  const int32_t* num_rows, int32_t bits, uint8_t* codes,
                                  uint8_t* scales, void* stream);
moe_status moe_dequantize_mx(const uint8_t* codes, const uint8_t* scales, int32_t R, int32_t K,
                             int32_t bits, void* out, int32_t out_fp32, void* stream);

/*
 * moe_grouped_matmul_mx -- moe_grouped_matmul on microscaled operands: MXFP4
 * weights, MXFP8 or MXFP4 rows, multiplied on the scaled matrix instruction.
 * Products are exact and summed in fp32 over the whole contraction: MXFP8 rows
 * in two parts by magnitude, because the instruction drops what lies far below
 * the largest of 8 products. That doubles its work: MXFP4 rows, which need one
 * part, are faster where experts have many rows.
 *   xq  [T, K] E4M3 (x_bits = 8) or [T, K / 2] E2M1 (x_bits = 4)
 *   xs  [T, K / 32] scales
 *   wq  [num_local, M, K / 2] E2M1;  ws  [num_local, M, K / 32] scales
 *   K a multiple of 32; xq and wq 16-byte aligned
 * A NaN code or scale makes the outputs it enters NaN. Every other argument,
 * the untouched rows, the limits and the errors are as for moe_grouped_matmul.
 */
moe_status moe_grouped_matmul_mx(const uint8_t* xq, const uint8_t* xs, int32_t x_bits,
                                 const int32_t* permuted_rows, const int32_t* expert_offsets,
                                 int32_t num_local, int32_t T, int32_t k, int32_t N, int32_t K,
                                 int32_t M, const uint8_t* wq, const uint8_t* ws, void* y,
                                 int32_t y_fp32, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* MOE_H */
