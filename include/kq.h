/*
 * kq.h — k-quant weight matmul on NVIDIA GB300 (sm_103a): C ABI of libkq.
 *
 *   Y[M, N] = dequant(W)[M, K] . X[K, N]
 *
 * W holds 4-bit Q4_K, 5-bit Q5_K or 6-bit Q6_K super-blocks; X is fp32 and is
 * quantised to
 * Q8_1 (int8 codes with an fp16 scale per 32 values) inside every call. The
 * decode matvec also takes TQ4_1S weights (WHT-rotated 4-bit Lloyd-Max codes),
 * which it multiplies with the fp32 activations directly.
 *
 * Sources (page title, section):
 *  [MMVQ]  "06 · 8e/8e② — decode MMVQ: dp4a integer dot products + the llama.cpp
 *          launch table": §2 Principle (Q4_K value d*sc*nib - dmin*m, the min-term
 *          identity, the q8 activation quantiser), §3.2 Key code (Q4_K byte
 *          offsets, quantize_pad40_block), §3.3 Pitfalls (Q6_K layout, d at 208).
 *  [MMQv2] "ZINC MMQ v2 — Fused Q4_K×Q8_1 Tensor-Core GEMM (beat llama.cpp)": What
 *          they do right (Q8_1 activations, fused dequant), Kernel architecture,
 *          Persistent kernel + atomic work queue, MoE routing (fused gather).
 *  [GAP]   "Prefill Gap Closure Plan — ZINC CUDA vs llama.cpp": T1 (fused dequant
 *          tensor-core GEMM), T2 (grouped MoE expert GEMM: histogram, prefix sum,
 *          scatter, per-expert GEMM).
 *  [TQ]    "TQ4_1S Weight Kernel Optimization": Architecture Overview (rotated
 *          4-bit weights, dequant = centroid[index] * half-block scale, inverse
 *          WHT, pre-rotated activation), Block Layout, Centroid Table.
 *
 * Conventions for every entry point
 *  - Pointers are device pointers owned by the caller (cudaMalloc / a framework
 *    allocator) unless stated otherwise. The library allocates no memory, keeps
 *    no pointer after the call returns, and does not synchronise the stream
 *    (except kq_get_device_error).
 *  - Layouts (row-major everywhere):
 *      W : M rows x (K/256) super-blocks; a Q4_K block is 144 bytes
 *          [fp16 d][fp16 dmin][12 B packed 6-bit scales/mins][128 B nibbles],
 *          a Q6_K block is 210 bytes [ql 128][qh 64][int8 scales 16][fp16 d].
 *          Q5_K (the GGUF layout; the pages give none): 176 bytes [fp16 d][fp16 dmin]
 *          [12 B scales/mins packed as Q4_K][qh 32][128 B nibbles], weight r of
 *          sub-block j taking its fifth bit from bit j of qh[r].
 *          TQ4_1S: M rows x (K/32) blocks of 20 bytes [fp16 d0][fp16 d1][qs 16],
 *          element j's centroid index in qs[j/2], low nibble for even j.
 *          For MoE the experts' matrices are concatenated, expert-major.
 *      X : fp32, token-major: token n occupies X[n*K .. n*K+K-1].
 *      Y : fp32, token-major: Y[n*M + m].
 *      Xq: N x (K/32) Q8_1 blocks of 36 bytes [fp16 d][fp16 s][int8 q[32]].
 *  - Alignment: W, X, Y, Xq and ws must be 16-byte aligned.
 *  - Sizes: K must be a multiple of 256 (32 for kq_quantize_q8_1 and for TQ4_1S);
 *    M, N, T >= 1; all sizes below 2^31.
 *  - Work is queued on `stream` (a cudaStream_t; NULL = legacy default stream).
 *    A status other than KQ_OK means nothing was queued, except KQ_ERR_CUDA
 *    after a failed launch.
 *  - Results are deterministic: the same inputs give bit-identical outputs.
 *  - Per-device state: the library looks up, once per device, the device
 *    addresses of its error word (and of kq_gemm_noalloc's scratch) and sets
 *    its kernels' shared-memory limits. That state belongs to the device's
 *    primary context: do not call the library after cudaDeviceReset in the
 *    same process.
 *  - Accuracy: Q8_1 codes and block sums are bit-exact against the IEEE fp32
 *    definition. Y satisfies |Y - Y_ref| <= 1e-3 * Sum_k |w_k x_k| + 1e-5 per
 *    element, Y_ref being the exact product of the dequantised operands. The
 *    tensor-core paths (kq_gemm, kq_moe_grouped_gemm) round dequantised
 *    weights and activations to fp16, so they need |w|, |x| < 65504.
 */
#ifndef KQ_H
#define KQ_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

#if defined(__GNUC__)
#define KQ_API __attribute__((visibility("default")))
#else
#define KQ_API
#endif

/* Same type as cudaStream_t. */
typedef struct CUstream_st* kq_stream_t;

typedef enum kq_status {
  KQ_OK = 0,
  KQ_ERR_NULL = 1,      /* a required pointer is NULL */
  KQ_ERR_SHAPE = 2,     /* a size is out of range or not a multiple of its block */
  KQ_ERR_ALIGN = 3,     /* a pointer is not 16-byte aligned */
  KQ_ERR_TYPE = 4,      /* unknown weight type */
  KQ_ERR_WORKSPACE = 5, /* ws_bytes is smaller than kq_workspace_bytes() */
  KQ_ERR_CUDA = 6,      /* a CUDA runtime call failed (no device, launch failure) */
  KQ_ERR_DEVICE = 7     /* a kernel recorded an error; see kq_get_device_error */
} kq_status;

/* KQ_Q5_K is taken wherever Q4_K is; KQ_TQ4_1S by kq_matvec only (the other
 * entry points return KQ_ERR_TYPE for it). */
typedef enum kq_wtype { KQ_Q4_K = 1, KQ_Q6_K = 2, KQ_TQ4_1S = 3, KQ_Q5_K = 4 } kq_wtype;

/* Element types of the row operators' inputs and of the group scales. */
typedef enum kq_dtype { KQ_F32 = 1, KQ_F16 = 2, KQ_BF16 = 3 } kq_dtype;

/* Score function of kq_moe_route. */
typedef enum kq_score { KQ_SCORE_SOFTMAX = 1, KQ_SCORE_SIGMOID = 2 } kq_score;

/* Which elements of a head the position rotation turns together. */
typedef enum kq_rope {
  KQ_ROPE_HALF = 1, /* i and i + rot_dim / 2 */
  KQ_ROPE_PAIRS = 2 /* 2i and 2i + 1 */
} kq_rope;

typedef enum kq_op { KQ_OP_MATVEC = 1, KQ_OP_GEMM = 2, KQ_OP_MOE = 3 } kq_op;

/* Device error codes reported by kq_get_device_error. */
#define KQ_DEVERR_NONE 0
#define KQ_DEVERR_WAIT_TIMEOUT 1 /* a pipeline wait gave up (the kernel returned early) */
#define KQ_DEVERR_EXPERT_ID 2    /* an expert id was outside [0, n_experts) */
#define KQ_DEVERR_POSITION 3     /* a position was not below n_positions */
#define KQ_DEVERR_PAGE 4         /* a place's sequence, table entry or page was out of range */

/*
 * kq_quantize_q8_1 — fp32 activations to Q8_1 blocks ([MMVQ] §2 and §3.2
 * quantize_pad40_block; the Q8_1 block sum of [MMQv2] "What they do right").
 * For every 32 consecutive values x of a token:
 *   d = max|x| / 127, q = clamp(rint(x * (d != 0 ? 1/d : 0)), -128, 127),
 *   stored d_h = fp16(d), s_h = fp16(d_h * Sum q), all in IEEE fp32 with
 *   round-half-even.
 * X: fp32 [N][K]; Xq: N*(K/32)*36 bytes, written. K % 32 == 0.
 */
KQ_API kq_status kq_quantize_q8_1(const float* X, void* Xq, int64_t K, int64_t N, kq_stream_t stream);

/*
 * kq_matvec — decode matvec y = dequant(W) . x for one token ([MMVQ] §2, §3.2:
 * integer dot products of the 4/6-bit codes with the Q8_1 codes of x, the
 * min term from the Q8_1 block sum, warp-shuffle row reductions). x is
 * quantised to Q8_1 inside the call. Needs no workspace.
 * wtype: KQ_Q4_K, KQ_Q6_K or KQ_Q5_K (the Q4_K value d*sc*q - dmin*m with a
 * 5-bit q; the pages ship it as a sibling decode kernel). W: M rows of K/256
 * blocks; x: fp32 [K];
 * y: fp32 [M], written.
 * Weight streaming starts before the kernel waits for the previous kernel on
 * the stream: W must not be written by a kernel that is still running when this
 * call starts, i.e. by a preceding kernel that allows programmatic dependent
 * launch. (A preceding ordinary kernel, copy or event is always complete.)
 * A Q6_K row whose byte length is not a multiple of 16 must have K <= 15360.
 * The k-quant decode kernels hold the whole Q8_1 activation in shared memory:
 * K <= 121600 is always taken; a larger K only when a CTA's rows fit the staged
 * kernel (few rows), else KQ_ERR_SHAPE with nothing queued. TQ4_1S has no such
 * limit (its fallback rotates x in segments).
 *
 * wtype KQ_TQ4_1S ([TQ]): W holds rotated weights r_b[j] = c[idx_j] * d_h(j)
 * per 32-block b (c the page's 16-entry centroid table, d0 for j < 16, d1
 * otherwise), and y[m] = Sum_b w_b . x_b with w_b = H^-1 r_b, H the orthonormal
 * 32-point Walsh-Hadamard transform in natural order (H[i][j] =
 * (-1)^popcount(i & j) / sqrt(32), its own inverse). The call rotates x once
 * (x_r = H x_b, fp32) and computes Sum_b r_b . x_r in fp32; no Q8_1 step.
 * K must be a multiple of 32 (multiples of 128 take the TMA-staged kernel).
 * Accuracy: |y - y_ref| <= 1e-3 * Sum_b Sum_j Sum_k |r_b[j] H[j][k] x_b[k]| + 1e-5,
 * y_ref the exact product. Weight streaming starts before the dependency wait,
 * as above.
 */
KQ_API kq_status kq_matvec(int wtype, const void* W, const float* x, float* y, int64_t M, int64_t K,
                           kq_stream_t stream);

/*
 * kq_matvec_prefetch — kq_matvec, and while it runs each CTA also asks L2 to
 * fetch its share of W_next[0, W_next_bytes) (rounded down to a multiple of 16):
 * the weights of the call that follows on the stream, e.g. the next layer's
 * matrix in a decode step. That call's weight stream then starts from L2 while
 * this one computes (the staged lane-row forms and the item kernel of Q6_K
 * ask for it once their activations are in, so that it does not delay them;
 * the lane-row ring form once its ring is primed). y is bit-identical to
 * kq_matvec's; the prefetch is a hint (nothing waits for it). An addition of
 * this library (the pages launch one matrix per call without it). Every decode
 * kernel form takes it except the TQ4_1S fallback for K % 128 != 0.
 * W_next: NULL (no prefetch) or 16-byte aligned device memory readable for
 * W_next_bytes bytes (KQ_ERR_ALIGN otherwise). Other arguments as kq_matvec.
 */
KQ_API kq_status kq_matvec_prefetch(int wtype, const void* W, const float* x, float* y, int64_t M, int64_t K,
                                    const void* W_next, size_t W_next_bytes, kq_stream_t stream);

/*
 * kq_matvec_swiglu, kq_matvec_rmsnorm — kq_matvec with the producer of its
 * activations fused into the Q8_1 quantiser ([MMVQ] §3.2 Key code: the
 * quantisation body moved into the RMSNorm and SwiGLU producers), so the
 * produced activations never go to memory:
 *   swiglu:  x[k] = silu(gate[k]) * up[k],  silu(g) = g / (1 + exp(-g));
 *   rmsnorm: x[k] = x_in[k] * r * gamma[k], r = 1 / sqrt(Sum_k x_in[k]^2 / K + eps)
 *            (eps >= 0; the sum of squares is taken in a fixed order).
 * gate, up, x_in, gamma: fp32 [K], 16-byte aligned. The producers compute in
 * fp32; the Q8_1 codes are then made from those fp32 values exactly as in
 * kq_matvec, and Y meets the accuracy bound against the exact product of the
 * dequantised weights with the Q8_1 codes of the produced activations.
 * Otherwise as kq_matvec (wtype, layouts, W streamed before the dependency wait);
 * KQ_TQ4_1S is not taken here (KQ_ERR_TYPE).
 */
KQ_API kq_status kq_matvec_swiglu(int wtype, const void* W, const float* gate, const float* up, float* y, int64_t M,
                                  int64_t K, kq_stream_t stream);
KQ_API kq_status kq_matvec_rmsnorm(int wtype, const void* W, const float* x, const float* gamma, float eps, float* y,
                                   int64_t M, int64_t K, kq_stream_t stream);

/*
 * kq_gemm — prefill GEMM Y = dequant(W) . X for N tokens ([MMQv2] Kernel
 * architecture; [GAP] T1). X is quantised to Q8_1 (as x_hat = fp16(d_h * q))
 * into the workspace once per call; weight super-blocks are staged by TMA and
 * unpacked to fp16 into tensor memory; tcgen05 MMAs accumulate in tensor memory.
 * A few tokens are a decode rather than a GEMM: Q4_K and Q5_K with 2 <= N <= 7 run on
 * the decode matvec path instead ([MMVQ] §2: dp4a on the Q8_1 codes, the min
 * term from the block sums; the tokens' codes are made once into the
 * workspace, the weights are read once for all tokens). Both paths meet the
 * accuracy bound above; a token's result may differ in the last bits with the
 * number of tokens in the call (the partial sums are grouped differently).
 * W: M x K weights; X: fp32 [N][K]; Y: fp32 [N][M], written.
 * ws: device workspace of at least kq_workspace_bytes(KQ_OP_GEMM, ...) bytes.
 * Q6_K needs K % 2048 == 0 (rows whose byte length is a multiple of 16).
 * As in kq_matvec, W is streamed before the GEMM waits for the previous kernel
 * on the stream: W must not be written by a still-running predecessor that
 * allows programmatic dependent launch.
 */
KQ_API kq_status kq_gemm(int wtype, const void* W, const float* X, float* Y, int64_t M, int64_t K, int64_t N, void* ws,
                  size_t ws_bytes, kq_stream_t stream);

/*
 * kq_gemm_noalloc — kq_gemm without a workspace argument. This entry point is
 * an addition of this library; the source pages have no counterpart to it.
 * Same operation, arguments (minus ws/ws_bytes), layouts, accuracy and
 * determinism as kq_gemm; it runs the same kernels.
 *
 * Who needs it: callers that cannot hand the library device memory per call,
 * e.g. plain C hosts with no device allocator of their own, or runtimes that
 * plan all device memory ahead and forbid allocation on the per-token path
 * (cudaMalloc may synchronise the device, which such a loop cannot afford).
 * The library itself allocates nothing here: the scratch (fp16 x_hat and
 * split-K partials) is a fixed array of KQ_GEMM_STATIC_WS_BYTES per device,
 * part of the library's device image, which no caller has to clear. With
 * CUDA's default lazy module loading the array takes device memory only once
 * this entry point is first called on a device; with eager loading
 * (CUDA_MODULE_LOADING=EAGER) every context that loads the library reserves it.
 *
 * Limit: returns KQ_ERR_WORKSPACE, with nothing queued, when the call would
 * need more scratch than KQ_GEMM_STATIC_WS_BYTES, i.e. when
 * kq_workspace_bytes(KQ_OP_GEMM, wtype, M, K, N, 0, 0) > KQ_GEMM_STATIC_WS_BYTES
 * (for instance N = 2048 tokens with K = 14336). Use kq_gemm there.
 *
 * Set-up: the first call on each device (with that device current) looks up
 * the array's device address, which loads the array's module; make that first
 * call before any stream capture.
 *
 * Concurrency: all calls on one device share the one array. Two calls whose
 * kernels may overlap (on different streams, or from several host threads
 * without ordering) race on it and give wrong results; order them on one
 * stream (or with events).
 */
#define KQ_GEMM_STATIC_WS_BYTES ((size_t)32 << 20)

KQ_API kq_status kq_gemm_noalloc(int wtype, const void* W, const float* X, float* Y, int64_t M, int64_t K,
                                 int64_t N, kq_stream_t stream);

/*
 * kq_moe_grouped_gemm — MoE expert matmul ([MMQv2] MoE routing; [GAP] T2).
 * For every token t and slot j < top_k: Y[t][j][:] = dequant(W_e) . x_t with
 * e = expert_ids[t*top_k + j]. The (token, slot) pairs are grouped by expert
 * (histogram, prefix sum, scatter), the activations are gathered per expert,
 * and each expert's weight tile is read once for all of its tokens.
 * W_experts: n_experts * M rows of K/256 blocks (expert-major);
 * expert_ids: int32 [T][top_k]; X: fp32 [T][K]; Y: fp32 [T][top_k][M], written.
 * No router weighting and no sum over slots. An out-of-range expert id records
 * KQ_DEVERR_EXPERT_ID and that slot's output row is written as zeros.
 * ws: at least kq_workspace_bytes(KQ_OP_MOE, ...) bytes.
 */
KQ_API kq_status kq_moe_grouped_gemm(int wtype, const void* W_experts, int32_t n_experts, const int32_t* expert_ids,
                              int32_t top_k, const float* X, float* Y, int64_t M, int64_t K, int64_t T, void* ws,
                              size_t ws_bytes, kq_stream_t stream);

/*
 * kq_moe_combine — the step after kq_moe_grouped_gemm: each token's slot rows
 * go back to the token, weighted by the router probabilities ([GAP] T2,
 * "scatter back"; read as the usual weighted MoE combine):
 *   out[t][m] = Sum_{j < top_k} probs[t][j] * Y[t][j][m],
 * summed in fp32 in slot order with one fused multiply-add per slot
 * (deterministic). Y: fp32 [T][top_k][M] (as kq_moe_grouped_gemm writes it);
 * probs: fp32 [T][top_k]; out: fp32 [T][M], written. 1 <= top_k <= 512.
 * Needs no workspace; out must not overlap Y or probs.
 */
KQ_API kq_status kq_moe_combine(const float* Y, const float* probs, float* out, int64_t M, int64_t T, int32_t top_k,
                                kq_stream_t stream);

/*
 * The operators of a decode step around 4-bit experts with group scales. They
 * hand Q8_1 rows to one another: kq_add_rmsnorm_q8_1 makes the layer's
 * activations, kq_moe_route chooses the experts, kq_moe_matvec_g4 multiplies
 * with the chosen experts' matrices (gate and up, then, after kq_swiglu_q8_1,
 * down), kq_moe_combine sums the slots. They are additions of this library; the
 * source pages have no counterpart to them. None needs a workspace. The Q8_1 rows are
 * operands of the group-scaled products only: kq_matvec, kq_gemm and
 * kq_moe_grouped_gemm take fp32 activations and quantise them themselves.
 *
 * Rows of floating-point operands are `ld` elements apart and contiguous within
 * a row; dtype is a kq_dtype (KQ_ERR_TYPE otherwise). For inputs ld is 0 (one
 * row read for all) or at least the row's length, for outputs at least the
 * row's length. Base pointers are 16-byte aligned; any ld is taken (rows that
 * are not 16-byte aligned are read and written by pairs of elements).
 *
 * kq_add_rmsnorm_q8_1 — residual addition, RMSNorm and quantisation of N rows:
 *   h = x + r (R NULL: h = x),  y[k] = h[k] * (1 / sqrt(Sum_k h[k]^2 / K + eps)) * gamma[k],
 *   H = h, Y = y, each rounded once to dtype; Xq = Q8_1(y) from the unrounded y.
 * All arithmetic is fp32 (the norm is that of the unrounded h, the sum of
 * squares in a fixed order). Each operand is X, R, H, Y: dtype [N][K]; gamma:
 * fp32 [K]; Xq: N * (K/32) * 36 bytes, written. R, H and Y may be NULL. H may be
 * X or R itself (the same pointer and ld); outputs overlap nothing else.
 * K % 32 == 0, eps >= 0.
 * y is within 64 * 2^-24 of its exact value, relative, or within fp32's least value, for
 * every row of finite h (its squares may pass fp32's range or fall below it; a row of
 * zeros with eps = 0 gives NaN).
 * A block of y with an infinity or a NaN gets an infinite or NaN scale d_h (the
 * block stands for non-finite values); so does one whose maximum is above
 * 127 * 65504.
 */
KQ_API kq_status kq_add_rmsnorm_q8_1(int dtype, const void* X, int64_t ldx, const void* R, int64_t ldr,
                                     const float* gamma, float eps, void* H, int64_t ldh, void* Y, int64_t ldy,
                                     void* Xq, int64_t K, int64_t N, kq_stream_t stream);

/*
 * kq_swiglu_q8_1 — v[k] = silu(gate[k]) * up[k], silu(g) = g / (1 + exp(-g)), in
 * fp32, quantised to Q8_1 as above. gate, up: dtype [N][K] (for instance the
 * halves of one [N][2K] buffer, ld = 2K); Xq: N * (K/32) * 36 bytes, written.
 * K % 32 == 0. v is within 10 * 2^-24 of its exact value, relative (a silu
 * below 2^-119 in magnitude may become 0).
 */
KQ_API kq_status kq_swiglu_q8_1(int dtype, const void* gate, int64_t ldg, const void* up, int64_t ldu, void* Xq,
                                int64_t K, int64_t N, kq_stream_t stream);

/*
 * kq_moe_route — routing of T tokens to top_k of n_experts experts.
 *   s = softmax(l) over the token's experts, or 1 / (1 + exp(-l));
 *   key = s + bias (bias NULL: s); the bias decides the selection only;
 *   with topk_groups < n_groups: the experts form n_groups equal runs; a group's
 *   score is the sum of its group_top (1 or 2) largest keys (fewer if it has
 *   fewer available experts); only experts of the topk_groups best groups stay;
 *   the top_k largest keys are chosen, in descending order; w_j = s_j; with
 *   renormalise w_j /= Sum_j w_j (0 where the sum is 0); w_j *= scale.
 * Ties go to the lowest index (of groups, of experts). The choice is that of
 * the definition evaluated in 64 bits: keys that 32 bits cannot tell apart are
 * computed again in fp64 (without a bias the experts are ordered by their
 * logits, whose order is that of the scores). The weights are computed in fp32.
 * An expert whose logit is -inf or NaN is not available: score 0, chosen by no
 * token; so is one whose bias is -inf or NaN, but it keeps its share of the
 * softmax sum. A logit of +inf counts as the largest finite fp32. A token with
 * fewer available experts than slots gets the lowest-numbered experts not yet
 * chosen for the others, with weight 0 (ids are always valid and distinct).
 * Each weight is within 120 * 2^-24 of its exact value, relative: a renormalised one for
 * logits within 60 of the token's largest chosen logit (however far those lie below the
 * largest of all, or below zero), another for logits within 60 of the token's largest
 * and weights of at least 2^-126. A score that is 0 in 64 bits (a softmax logit some
 * 745 below the largest, a sigmoid logit below -709.8) has weight 0.
 * logits: dtype [T][n_experts], rows ld apart; bias: fp32 [n_experts] or NULL;
 * ids: int32 [T][top_k], probs: fp32 [T][top_k], written. 1 <= n_experts <= 512,
 * n_experts % n_groups == 0, 1 <= topk_groups <= n_groups,
 * 1 <= top_k <= topk_groups * n_experts / n_groups.
 */
KQ_API kq_status kq_moe_route(int dtype, const void* logits, int64_t ld, const float* bias, int score, int32_t n_groups,
                              int32_t topk_groups, int32_t group_top, int32_t top_k, int renormalise, float scale,
                              int32_t* ids, float* probs, int32_t n_experts, int64_t T, kq_stream_t stream);

/*
 * kq_matvec_g4 — Y[n][m] = Sum_k w[m][k] x_n[k] for Q8_1 rows x and 4-bit weights
 * with group scales, w[m][k] = s[m][k / group] * (c[m][k] - z[m][k / group]).
 * W: M rows of K/2 bytes, byte i of a row holding the code of k = 2i in its low
 * half and of k = 2i + 1 in its high half; scales: scale_dtype (KQ_F16 or
 * KQ_BF16) [M][ceil(K/group)]; zeros: uint8 [M][ceil(K/group)], any value, or
 * NULL (8 everywhere). group: a power of two >= 32, not necessarily dividing K
 * (a group >= K is one scale per row). Xq: N * (K/32) * 36 bytes as
 * kq_quantize_q8_1, kq_add_rmsnorm_q8_1 and kq_swiglu_q8_1 write them (the
 * stored block sums are not read). Y: fp32 [N][M], written. K % 32 == 0; W,
 * scales, zeros, Xq and Y are 16-byte aligned.
 * A decode operator: made for up to a few dozen rows of Xq; any N is taken.
 * Accuracy: the dot products of 32-element blocks are exact integers and are
 * multiplied with the scales and summed in fp32; |Y - Y_ref| is at most
 * (K/32 + 12) * 2^-24 times the sum of the blocks' absolute contributions, Y_ref
 * the exact product of the dequantised operands. Results do not depend on
 * scheduling; a row's result may differ in the last bits with the number of
 * rows in the call (the sums are grouped differently). The bound is for products of
 * scales in fp32's normal range.
 * As in kq_matvec, W, scales and zeros are streamed before the call waits for the
 * previous kernel on the stream: they must not be written by a still-running
 * predecessor that allows programmatic dependent launch, and none of Xq (or expert
 * ids) that such a predecessor writes may lie in the same 32-byte sector as their
 * ends (separate allocations never do).
 */
KQ_API kq_status kq_matvec_g4(const void* W, const void* scales, int scale_dtype, const void* zeros, int64_t group,
                              const void* Xq, float* Y, int64_t M, int64_t K, int64_t N, kq_stream_t stream);

/*
 * kq_moe_matvec_g4 — kq_matvec_g4 with the matrices that a router chose:
 * Y[t][j][:] = W_e . x with e = expert_ids[t*top_k + j] and x row t of Xq, or row
 * t*top_k + j where x_per_slot is non-zero. W, scales, zeros: the experts'
 * matrices one after the other (n_experts * M rows); expert_ids: int32
 * [T][top_k]; Y: fp32 [T][top_k][M], written. n_experts <= 512,
 * top_k <= n_experts. An out-of-range expert id records KQ_DEVERR_EXPERT_ID and
 * that slot's output row is written as zeros; ids may repeat within a token.
 * W, scales and zeros may be streamed early as above when T * top_k >= n_experts.
 */
KQ_API kq_status kq_moe_matvec_g4(const void* W, const void* scales, int scale_dtype, const void* zeros, int64_t group,
                                  int32_t n_experts, const int32_t* expert_ids, int32_t top_k, int x_per_slot,
                                  const void* Xq, float* Y, int64_t M, int64_t K, int64_t T, kq_stream_t stream);

/*
 * The operators of a decode step's attention, and the choice of its tokens. They are
 * additions of this library; the source pages have no counterpart to them. A row of
 * queries, keys or values holds its heads one after the other, head_dim elements each;
 * dtypes, rows and ld are as above (base pointers of rows, tables of cosines, gammas,
 * caches, workspaces and Xq are 16-byte aligned; index and parameter arrays 4-byte).
 *
 * kq_qk_norm_rope — the norm of every head of N rows of queries and keys, then the
 * position rotation:
 *   y[i] = x[i] * (1 / sqrt(Sum_i x[i]^2 / head_dim + eps)) * gamma[i]   (gamma NULL: y = x),
 *   (a, b) -> (a cos - b sin, b cos + a sin) for the pairs that `pairing` (kq_rope) makes
 *   of the first rot_dim elements; the others stay. cos_sin NULL: no rotation.
 * cos_sin: fp32 [n_positions][rot_dim], a position's rot_dim / 2 cosines, then their sines.
 * positions: int32 [N], or NULL (row n is at position n). A row with a negative position
 * is passed over: nothing is written for it. So is one whose position is not in the
 * table, and KQ_DEVERR_POSITION is recorded.
 * Q: dtype [N][n_q_heads * head_dim]; K likewise with n_k_heads, NULL where that is 0;
 * Qo, Ko: out_dtype, written; out_dtype is dtype, or any for fp32 inputs. Qo may be Q and
 * Ko K (the same pointer, ld and type); outputs overlap nothing else. q_gamma, k_gamma:
 * fp32 [head_dim] or NULL. head_dim: a multiple of 16 from 16 to 256; rot_dim: a multiple of 16
 * up to head_dim; eps >= 0; N * (n_q_heads + n_k_heads) <= 2^30. All arithmetic is fp32, rounded once to out_dtype; an
 * unrounded result is within 16 * 2^-24 * (|a cos| + |b sin|) of its exact value (16 * 2^-24 * |y| where
 * nothing is turned), for every head of finite x (a head of zeros with eps = 0 gives NaN).
 */
KQ_API kq_status kq_qk_norm_rope(int dtype, const void* Q, int64_t ldq, int32_t n_q_heads, const void* K, int64_t ldk,
                                 int32_t n_k_heads, int32_t head_dim, const float* q_gamma, const float* k_gamma,
                                 float eps, const float* cos_sin, int32_t rot_dim, int64_t n_positions, int pairing,
                                 const int32_t* positions, int out_dtype, void* Qo, int64_t ldqo, void* Ko, int64_t ldko,
                                 int64_t N, kq_stream_t stream);

/*
 * The 4-bit paged cache. Place p of sequence s is place p % page_size of page
 * block_table[s * ldt + p / page_size]; page_size is a power of two from 16 to 65536.
 * A head's 32-element blocks are stored as fp16 s and m and 4-bit codes c, standing for
 * m + s * c:
 *   m = fp16(min v), s = fp16((max v - min v) * (1 / 15 as fp32)),
 *   c = clamp(rint((v - m) / s), 0, 15) (0 where s is 0), all in IEEE fp32.
 * A block with an infinity or a NaN, or whose m or s would not be finite in fp16, has s = NaN and
 * m = 0 and stands for NaN.
 * cache: bytes [n_pages][n_heads][page_size / 16][20 * head_dim]: granules of 16 places of
 * one head, in each, with G = head_dim / 32,
 *   [16][head_dim / 2] key codes: element r of block g in byte 4G * (r / 8) + 4g + (r % 8) / 2,
 *   [16][2][G] fp16 key parameters: the blocks' s, then their m,
 *   [16][head_dim / 2] value codes: element r of block g in byte 2G * (r / 4) + 2g + (r % 4) / 2,
 *   [16][2][G] fp16 value parameters;
 *   an even r has the low half of its byte. 5 bits a value; head_dim is 64, 128 or 256.
 * Memory that no token was written to may hold anything: no operator uses it.
 *
 * kq_kv_append_q4 — writes N tokens' keys and values to their places, the keys turned by
 * their positions on the way (cos_sin NULL: as they are; the table and pairing as in
 * kq_qk_norm_rope, each product and each sum rounded to fp32).
 * K, V: dtype [N][n_heads * head_dim]. positions: int32 [N], a token's place in its
 * sequence and the row of cos_sin; seq_ids: int32 [N], its sequence, or NULL (token n
 * belongs to sequence n). block_table: int32 [n_seqs][ldt]. A token with a negative position
 * is passed over; so is one whose sequence, place or page is out of range (KQ_DEVERR_PAGE
 * is recorded) or whose position is not in the table of cosines (KQ_DEVERR_POSITION). No
 * two tokens of a call have the same place (the bytes there would be of either). 2 * N * n_heads <= 2^30.
 */
KQ_API kq_status kq_kv_append_q4(int dtype, const void* K, int64_t ldk, const void* V, int64_t ldv, int32_t n_heads,
                                 int32_t head_dim, const float* cos_sin, int32_t rot_dim, int64_t n_positions,
                                 int pairing, const int32_t* positions, const int32_t* seq_ids,
                                 const int32_t* block_table, int64_t ldt, int64_t n_seqs, void* cache, int64_t n_pages,
                                 int32_t page_size, int64_t N, kq_stream_t stream);

/*
 * kq_kv_gather_q4 — reads places of the cache back as rows: K, V: dtype
 * [N][n_heads * head_dim], written with m + s * c, computed in fp32 and rounded once. The
 * other arguments are those of kq_kv_append_q4; rows that it would pass over are left as they were.
 */
KQ_API kq_status kq_kv_gather_q4(const void* cache, int64_t n_pages, int32_t page_size, int32_t n_heads,
                                 int32_t head_dim, const int32_t* block_table, int64_t ldt, int64_t n_seqs,
                                 const int32_t* positions, const int32_t* seq_ids, int dtype, void* K, int64_t ldk,
                                 void* V, int64_t ldv, int64_t N, kq_stream_t stream);

/*
 * kq_attn_q4 — attention of N rows of queries over the cache. Query head i attends to key
 * head i / (n_q_heads / n_kv_heads). Sequence b has the rows q_start[b] to q_start[b + 1] - 1
 * of Q (q_start: int32 [n_seqs + 1], ascending, or NULL: row b, with N = n_seqs) and
 * kv_len[b] places in the cache, the rows' own among them. Row i of n sees the places below
 * kv_len[b] - n + 1 + i and, with window > 0, only the last `window` of those:
 *   o = Sum_t p_t v_t, p = softmax_t(scale * q . k_t); a row that sees no place gives zeros.
 * Q: dtype; O: dtype [N][n_q_heads * head_dim], or NULL; Xq: N * (n_q_heads * head_dim / 32) * 36
 * bytes, the Q8_1 blocks of the unrounded o, or NULL; one of the two is given. Rows of Q that belong
 * to no sequence are not read, and theirs of O and Xq left as they were. O, Xq and ws overlap neither the inputs nor one another.
 * A place whose page is out of range counts as one that no row sees, and KQ_DEVERR_PAGE is recorded; table entries of places that no
 * row sees are not looked at (those before a window may be anything).
 * A query head with an infinity, a NaN or a value of 2^118 or more gives NaN, and so does one with a score (times log2 e) above
 * fp32's range, or with none that is not below it. N * n_q_heads <= 2^30.
 * A NaN among a place's keys makes the rows that see it NaN, one among its values their elements of that block (one whose place has less
 * than 2^-34 of a row's largest weight may not).
 * ws: at least kq_attn_q4_workspace_bytes(...) bytes, whatever they hold; calls that may
 * overlap need one each.
 * Scores, softmax statistics and sums are fp32; a score is a sum of exact products of q and the codes (fp32 q: of its first 22 bits) by
 * the tensor cores, whose additions cut off: it is within 2^-18 of scale * Sum (s c + |m|) |q| over the head. The softmax's
 * weights, their products with s, and m + 8 s are rounded for the tensor cores: to fp16 (relative 2^-11 each; the rows o are then
 * rounded to 16 bits themselves; what the sums cut off is below 2^-16 of Sum_t p_t (s c + |m|)), or, for fp32 rows and wherever Xq is
 * asked for, to two fp16 halves (2^-22). Below fp16's range errors are absolute: 2^-35 of the largest weight; (1 + s) S 2^-35
 * of it for products with s, S the power of two not below the largest s gone over (at least 1); 2^-23 for m + 8 s, 2^-20 where
 * an s of 2 or more has been gone over.
 * Made for the rows of decode steps: any number of new rows is taken, in tiles that each read the cache again.
 */
KQ_API size_t kq_attn_q4_workspace_bytes(int32_t n_q_heads, int32_t n_kv_heads, int32_t head_dim, int64_t N,
                                         int64_t n_seqs);
KQ_API kq_status kq_attn_q4(int dtype, const void* Q, int64_t ldq, int32_t n_q_heads, const void* cache, int64_t n_pages,
                            int32_t page_size, int32_t n_kv_heads, int32_t head_dim, const int32_t* block_table,
                            int64_t ldt, int64_t n_seqs, const int32_t* kv_len, const int32_t* q_start, float scale,
                            int64_t window, void* O, int64_t ldo, void* Xq, int64_t N, void* ws, size_t ws_bytes,
                            kq_stream_t stream);

/*
 * kq_sample — the next token of each of N rows of logits, for given random numbers u in [0, 1).
 * With a row's tokens in descending order of their logits (ties to the lower index) and
 * weights w = exp((l - max l) / T), three prefixes of that order limit the choice: the
 * first top_k tokens (top_k <= 0: all); the shortest prefix with at least top_p of the
 * weight of those (top_p not below 1: all); the tokens with w >= min_p (1 for larger ones). The
 * shortest is kept; at least one token always is. The token chosen is the first, by index, at
 * which the sum of the kept weights passes u times their total; its probability is its share of
 * that total. T not above 0: the first token with the largest logit, with probability 1.
 * A logit of -inf or NaN is never chosen; +inf counts as the largest finite fp32. A row without
 * any other gives token 0 with probability 0.
 * logits: dtype [N][V], rows ld apart, V <= 524288. temperature, top_p, min_p: fp32 [N], or NULL
 * (1, 1, 0); top_k: int32 [N] or NULL; u: fp32 [N]; ids: int32 [N], probs: fp32 [N] or NULL, written.
 * Weights are within 2^-30 of theirs, relative (with 2^-43 of the largest), for T from 2^-126 to 2^110; the sums that are
 * compared are exact sums of them, so the choice is that of the definition unless two sums
 * that it compares are that close. Logits further apart than fp32's largest number count as infinitely far.
 * N * V <= 2^40.
 */
KQ_API kq_status kq_sample(int dtype, const void* logits, int64_t ld, const float* temperature, const int32_t* top_k,
                           const float* top_p, const float* min_p, const float* u, int32_t* ids, float* probs, int64_t V,
                           int64_t N, kq_stream_t stream);

/*
 * kq_workspace_bytes — device workspace needed by an operation (0 for
 * KQ_OP_MATVEC). N_or_T is N for KQ_OP_GEMM and T for KQ_OP_MOE; n_experts
 * and top_k are read for KQ_OP_MOE only. The size depends on the SM count of
 * the current device. Returns 0 for invalid arguments.
 */
KQ_API size_t kq_workspace_bytes(int op, int wtype, int64_t M, int64_t K, int64_t N_or_T, int32_t n_experts,
                          int32_t top_k);

/*
 * kq_get_device_error — waits for `stream`, then returns in *code the first
 * device error recorded on the current device since the previous call
 * (KQ_DEVERR_*), and clears it. Returns KQ_ERR_DEVICE when *code != 0.
 * There is one error word per device, shared by every stream and every call
 * on it (not one per workspace): with kernels in flight on other streams, a
 * code may come from one of those, and only `stream` is waited for.
 */
KQ_API kq_status kq_get_device_error(int32_t* code, kq_stream_t stream);

/*
 * kq_test_hold_copies — a test hook for the library's failure detection; the
 * source pages have no counterpart to it. While `hold` is non-zero, launches
 * made afterwards by kq_matvec, kq_matvec_prefetch and the fused matvecs (Q4_K,
 * Q5_K, Q6_K), by kq_gemm's tensor-core kernel and by kq_moe_grouped_gemm run
 * with their weight producer issuing no copy (and, on the tensor-core paths,
 * handing out no tile). Their consumers' pipeline waits then run out after
 * their limit (2 s), the kernel records KQ_DEVERR_WAIT_TIMEOUT, leaves its
 * loops, frees its tensor memory and returns: the path a wait that gives up
 * takes, with no copy in flight. Outputs of such calls are undefined. The
 * flag is per process and is read when a call queues its launch (a call
 * captured in a CUDA graph keeps the value it saw). Not for production use:
 * hold = 0 (the default) restores normal calls. Always returns KQ_OK.
 * Calls that take other kernels (TQ4_1S, the small-N decode of kq_gemm, the
 * group-scaled products) are not affected.
 */
KQ_API kq_status kq_test_hold_copies(int hold);

/* Name of a status code (static string). */
KQ_API const char* kq_status_str(int status);

#ifdef __cplusplus
}
#endif

#endif /* KQ_H */
