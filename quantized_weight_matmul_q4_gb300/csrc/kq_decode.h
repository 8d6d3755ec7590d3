// Internal interface of the decode-step operators (Q8_1 row producers, expert routing, products with
// group-scaled 4-bit weights): their checks and entry points are in kq_decode_api.cu, their
// kernels in kq_rows.cu, kq_route.cu and kq_g4.cu.
#pragma once

#include "kq_internal.h"

namespace kq {

// Row producers with a Q8_1 output (kq_rows.cu); dtype: kq_dtype, ld*: elements
// from row to row.
cudaError_t launch_add_rmsnorm_q8_1(int dtype, const void* X, int64_t ldx, const void* R, int64_t ldr,
                                    const float* gamma, float eps, void* H, int64_t ldh, void* Y, int64_t ldy,
                                    void* Xq, int64_t K, int64_t N, int num_sms, cudaStream_t s);
cudaError_t launch_swiglu_q8_1(int dtype, const void* G, int64_t ldg, const void* U, int64_t ldu, void* Xq, int64_t K,
                               int64_t N, int num_sms, cudaStream_t s);

cudaError_t launch_moe_route(int dtype, const void* logits, int64_t ld, const float* bias, int score, int n_groups,
                             int topk_groups, int group_top, int top_k, bool renorm, float scale, int* ids, float* probs,
                             int E, int64_t T, cudaStream_t s);

// 4-bit weights with group scales (kq_g4.cu). group = 1 << group_shift 32-element
// blocks; groups per row: `groups`; zeros may be null (8 everywhere).
struct G4Weights {
  const uint8_t* codes;
  const void* scales;
  int scale_dtype;
  const uint8_t* zeros;
  int group_shift;
  int64_t groups;
};
// One matrix: Y[N][M] for N rows of Xq.
cudaError_t launch_matvec_g4(const G4Weights& w, const uint8_t* Xq, float* Y, int64_t M, int64_t K, int64_t N,
                             int num_sms, cudaStream_t s);
// Y[t][j][M] with the matrix of expert ids[t][j].
cudaError_t launch_moe_matvec_g4(const G4Weights& w, int n_experts, const int32_t* ids, int top_k, bool x_per_slot,
                                 const uint8_t* Xq, float* Y, int64_t M, int64_t K, int64_t T, int* err, int num_sms,
                                 cudaStream_t s);

}  // namespace kq
