// Products of Q8_1 activations with 4-bit weights that carry group scales:
//
//   y[m] = Sum_b d_b * s(m, b) * ( Sum_k c[m][k] q[k] - z(m, b) * Sum_k q[k] )
//
// over the 32-element blocks b, c the 4-bit codes, s and z the scale and zero
// point of the block's group, d and q the block's Q8_1 scale and codes. The two
// sums over a block are exact in 32-bit integers (dp4a); the products with the
// scales and the sum over the blocks are fp32.
#include <cuda_bf16.h>

#include <algorithm>

#include "kq_internal.h"
#include "kq_types.cuh"

namespace kq {
namespace {

constexpr int G4_WARPS = 8;

template <typename S>
__device__ __forceinline__ float scale_at(const void* scales, int64_t i) {
  return to_f32(static_cast<const S*>(scales)[i]);
}

// One warp per output row and activation row; lane l takes the blocks l, l + 32, ...
template <typename S, bool MOE>
__global__ void __launch_bounds__(G4_WARPS * 32) g4_simple_kernel(G4Weights w, const int32_t* __restrict__ ids,
                                                                  int n_experts, int top_k, bool x_per_slot,
                                                                  const uint8_t* __restrict__ Xq, float* __restrict__ Y,
                                                                  int64_t M, int blocks, int64_t rows, int* err) {
  pdl_enter();
  const int lane = threadIdx.x & 31;
  const int64_t m = static_cast<int64_t>(blockIdx.x) * G4_WARPS + (threadIdx.x >> 5);
  if (m >= M) return;
  for (int64_t p = blockIdx.y; p < rows; p += gridDim.y) {
    int64_t r = m, xr = p;
    if (MOE) {
      const int e = ids[p];
      if (e < 0 || e >= n_experts) {
        if (lane == 0) {
          if (m == 0) report_error(err, ERR_EXPERT_ID);
          Y[p * M + m] = 0.f;
        }
        continue;
      }
      r = static_cast<int64_t>(e) * M + m;
      xr = x_per_slot ? p : p / top_k;
    }
    const uint4* codes = reinterpret_cast<const uint4*>(w.codes) + r * blocks;
    const uint8_t* xrow = Xq + xr * blocks * Q8_1_BYTES;
    float acc = 0.f;
    for (int b = lane; b < blocks; b += 32) {
      const uint4 c = codes[b];
      const int64_t gi = r * w.groups + (b >> w.group_shift);
      const float s = scale_at<S>(w.scales, gi);
      const int z = w.zeros ? w.zeros[gi] : 8;
      const uint32_t* xb = reinterpret_cast<const uint32_t*>(xrow + static_cast<int64_t>(b) * Q8_1_BYTES);
      const float d = __low2float(bits_half2(xb[0]));
      const uint32_t cw[4] = {c.x, c.y, c.z, c.w};
      int dot = 0, sum = 0;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const uint32_t x0 = xb[1 + 2 * i], x1 = xb[2 + 2 * i];  // elements 8i..8i+3, 8i+4..8i+7
        dot = dp4a_us(cw[i] & 0x0f0f0f0fu, static_cast<int>(__byte_perm(x0, x1, 0x6420)), dot);
        dot = dp4a_us((cw[i] >> 4) & 0x0f0f0f0fu, static_cast<int>(__byte_perm(x0, x1, 0x7531)), dot);
        sum = __dp4a(static_cast<int>(x0), 0x01010101, sum);
        sum = __dp4a(static_cast<int>(x1), 0x01010101, sum);
      }
      acc = fmaf(s * d, static_cast<float>(dot - z * sum), acc);
    }
    acc = warp_sum_f(acc);
    if (lane == 0) Y[p * M + m] = acc;
  }
}

template <bool MOE>
cudaError_t launch_simple(const G4Weights& w, const int32_t* ids, int n_experts, int top_k, bool x_per_slot,
                          const uint8_t* Xq, float* Y, int64_t M, int64_t K, int64_t rows, int* err, cudaStream_t s) {
  const dim3 grid(static_cast<unsigned>((M + G4_WARPS - 1) / G4_WARPS),
                  static_cast<unsigned>(std::min<int64_t>(rows, 65535)));
  auto k = w.scale_dtype == KQ_F16 ? g4_simple_kernel<__half, MOE> : g4_simple_kernel<__nv_bfloat16, MOE>;
  return launch_pdl(k, grid, dim3(G4_WARPS * 32), 0, s, w, ids, n_experts, top_k, x_per_slot, Xq, Y, M,
                    static_cast<int>(K / 32), rows, err);
}

}  // namespace

cudaError_t launch_matvec_g4(const G4Weights& w, const uint8_t* Xq, float* Y, int64_t M, int64_t K, int64_t N,
                             int num_sms, cudaStream_t s) {
  return launch_simple<false>(w, nullptr, 0, 1, false, Xq, Y, M, K, N, nullptr, s);
}

cudaError_t launch_moe_matvec_g4(const G4Weights& w, int n_experts, const int32_t* ids, int top_k, bool x_per_slot,
                                 const uint8_t* Xq, float* Y, int64_t M, int64_t K, int64_t T, int* err, int num_sms,
                                 cudaStream_t s) {
  return launch_simple<true>(w, ids, n_experts, top_k, x_per_slot, Xq, Y, M, K, T * top_k, err, s);
}

}  // namespace kq
