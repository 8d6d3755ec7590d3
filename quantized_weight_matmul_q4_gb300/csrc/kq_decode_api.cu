// C ABI of the decode-step operators: argument checks and dispatch to the kernels. Declarations
// and contracts: include/kq.h. (Apart from kq_api.cu, whose counters are recorded against its text.)
#include "kq_common.cuh"
#include "kq_decode.h"

namespace kq {
namespace {

inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
constexpr int64_t kMaxDim = (int64_t(1) << 31) - 1;

kq_status finish(cudaError_t e) { return e == cudaSuccess ? KQ_OK : KQ_ERR_CUDA; }

bool valid_dtype(int t) { return t == KQ_F32 || t == KQ_F16 || t == KQ_BF16; }
// Row strides in elements: an output's rows do not overlap; an input's may be one row (0).
bool valid_ld_out(int64_t ld, int64_t K) { return ld >= K && ld <= kMaxDim; }
bool valid_ld_in(int64_t ld, int64_t K) { return ld == 0 || valid_ld_out(ld, K); }

// The checks that both group-scaled products share; fills *w.
kq_status g4_weights(const void* W, const void* scales, int scale_dtype, const void* zeros, int64_t group,
                     const void* Xq, const float* Y, int64_t M, int64_t K, int64_t N, G4Weights* w) {
  if (scale_dtype != KQ_F16 && scale_dtype != KQ_BF16) return KQ_ERR_TYPE;
  if (!W || !scales || !Xq || !Y) return KQ_ERR_NULL;
  if (M <= 0 || K <= 0 || N <= 0 || K % QK8_1 != 0 || M > kMaxDim || K > kMaxDim || N > kMaxDim ||
      M * N > (int64_t(1) << 40) || N * K > (int64_t(1) << 40) || group < 32 || (group & (group - 1)) != 0)
    return KQ_ERR_SHAPE;
  if (!aligned16(W) || !aligned16(scales) || !aligned16(zeros) || !aligned16(Xq) || !aligned16(Y)) return KQ_ERR_ALIGN;
  int shift = 0;
  while (shift < 30 && (int64_t(32) << shift) < group) ++shift;
  w->codes = static_cast<const uint8_t*>(W);
  w->scales = scales;
  w->scale_dtype = scale_dtype;
  w->zeros = static_cast<const uint8_t*>(zeros);
  w->group_shift = shift;
  w->groups = (K - 1) / group + 1;
  return KQ_OK;
}

}  // namespace
}  // namespace kq

using namespace kq;

extern "C" {

kq_status kq_add_rmsnorm_q8_1(int dtype, const void* X, int64_t ldx, const void* R, int64_t ldr, const float* gamma,
                              float eps, void* H, int64_t ldh, void* Y, int64_t ldy, void* Xq, int64_t K, int64_t N,
                              kq_stream_t stream) {
  if (!valid_dtype(dtype)) return KQ_ERR_TYPE;
  if (!X || !gamma || !Xq) return KQ_ERR_NULL;
  if (K <= 0 || N <= 0 || K % QK8_1 != 0 || K > kMaxDim || N > kMaxDim || K * N > (int64_t(1) << 40) ||
      !valid_ld_in(ldx, K) || (R && !valid_ld_in(ldr, K)) || (H && !valid_ld_out(ldh, K)) ||
      (Y && !valid_ld_out(ldy, K)) || !(eps >= 0.f && eps < 1e30f))  // also rejects NaN
    return KQ_ERR_SHAPE;
  if (!aligned16(X) || !aligned16(R) || !aligned16(gamma) || !aligned16(H) || !aligned16(Y) || !aligned16(Xq))
    return KQ_ERR_ALIGN;
  int dev, sms;
  int* err;
  cudaError_t e = device_context(&dev, &sms, &err);
  if (e != cudaSuccess) return KQ_ERR_CUDA;
  return finish(launch_add_rmsnorm_q8_1(dtype, X, ldx, R, ldr, gamma, eps, H, ldh, Y, ldy, Xq, K, N, sms,
                                        reinterpret_cast<cudaStream_t>(stream)));
}

kq_status kq_swiglu_q8_1(int dtype, const void* gate, int64_t ldg, const void* up, int64_t ldu, void* Xq, int64_t K,
                         int64_t N, kq_stream_t stream) {
  if (!valid_dtype(dtype)) return KQ_ERR_TYPE;
  if (!gate || !up || !Xq) return KQ_ERR_NULL;
  if (K <= 0 || N <= 0 || K % QK8_1 != 0 || K > kMaxDim || N > kMaxDim || K * N > (int64_t(1) << 40) ||
      !valid_ld_in(ldg, K) || !valid_ld_in(ldu, K))
    return KQ_ERR_SHAPE;
  if (!aligned16(gate) || !aligned16(up) || !aligned16(Xq)) return KQ_ERR_ALIGN;
  int dev, sms;
  int* err;
  cudaError_t e = device_context(&dev, &sms, &err);
  if (e != cudaSuccess) return KQ_ERR_CUDA;
  return finish(launch_swiglu_q8_1(dtype, gate, ldg, up, ldu, Xq, K, N, sms, reinterpret_cast<cudaStream_t>(stream)));
}

kq_status kq_moe_route(int dtype, const void* logits, int64_t ld, const float* bias, int score, int32_t n_groups,
                       int32_t topk_groups, int32_t group_top, int32_t top_k, int renormalise, float scale, int32_t* ids,
                       float* probs, int32_t n_experts, int64_t T, kq_stream_t stream) {
  if (!valid_dtype(dtype) || (score != KQ_SCORE_SOFTMAX && score != KQ_SCORE_SIGMOID)) return KQ_ERR_TYPE;
  if (!logits || !ids || !probs) return KQ_ERR_NULL;
  if (n_experts <= 0 || n_experts > 512 || T <= 0 || T > kMaxDim || n_groups <= 0 || n_groups > n_experts ||
      n_experts % n_groups != 0 || topk_groups <= 0 || topk_groups > n_groups || (group_top != 1 && group_top != 2) ||
      top_k <= 0 || top_k > topk_groups * (n_experts / n_groups) || !valid_ld_in(ld, n_experts) ||
      !(scale >= -1e30f && scale <= 1e30f))
    return KQ_ERR_SHAPE;
  if (!aligned16(logits) || !aligned16(bias) || !aligned16(ids) || !aligned16(probs)) return KQ_ERR_ALIGN;
  int dev, sms;
  int* err;
  cudaError_t e = device_context(&dev, &sms, &err);
  if (e != cudaSuccess) return KQ_ERR_CUDA;
  return finish(launch_moe_route(dtype, logits, ld, bias, score, n_groups, topk_groups, group_top, top_k,
                                 renormalise != 0, scale, ids, probs, n_experts, T,
                                 reinterpret_cast<cudaStream_t>(stream)));
}

kq_status kq_matvec_g4(const void* W, const void* scales, int scale_dtype, const void* zeros, int64_t group,
                       const void* Xq, float* Y, int64_t M, int64_t K, int64_t N, kq_stream_t stream) {
  G4Weights w;
  const kq_status st = g4_weights(W, scales, scale_dtype, zeros, group, Xq, Y, M, K, N, &w);
  if (st != KQ_OK) return st;
  int dev, sms;
  int* err;
  cudaError_t e = device_context(&dev, &sms, &err);
  if (e != cudaSuccess) return KQ_ERR_CUDA;
  return finish(launch_matvec_g4(w, static_cast<const uint8_t*>(Xq), Y, M, K, N, sms,
                                 reinterpret_cast<cudaStream_t>(stream)));
}

kq_status kq_moe_matvec_g4(const void* W, const void* scales, int scale_dtype, const void* zeros, int64_t group,
                           int32_t n_experts, const int32_t* expert_ids, int32_t top_k, int x_per_slot, const void* Xq,
                           float* Y, int64_t M, int64_t K, int64_t T, kq_stream_t stream) {
  G4Weights w;
  if (scale_dtype == KQ_F16 || scale_dtype == KQ_BF16) {
    if (!expert_ids) return KQ_ERR_NULL;
    if (n_experts <= 0 || n_experts > 512 || top_k <= 0 || top_k > n_experts || T <= 0 || T > kMaxDim ||
        T * top_k > kMaxDim || M > kMaxDim || n_experts * M > kMaxDim)
      return KQ_ERR_SHAPE;
  }
  const kq_status st = g4_weights(W, scales, scale_dtype, zeros, group, Xq, Y, M, K, T * top_k, &w);
  if (st != KQ_OK) return st;
  if (!aligned16(expert_ids)) return KQ_ERR_ALIGN;
  int dev, sms;
  int* err;
  cudaError_t e = device_context(&dev, &sms, &err);
  if (e != cudaSuccess) return KQ_ERR_CUDA;
  return finish(launch_moe_matvec_g4(w, n_experts, expert_ids, top_k, x_per_slot != 0, static_cast<const uint8_t*>(Xq),
                                     Y, M, K, T, err, sms, reinterpret_cast<cudaStream_t>(stream)));
}

}  // extern "C"
