// Row producers with a Q8_1 output: the residual addition with RMSNorm, and
// SwiGLU. Each reads its rows once, computes in fp32 and quantises the produced
// fp32 values, so that the activations of the next weight product go to memory
// as 36 bytes per 32 values. Inputs are read by ordinary loads: the previous kernel may have
// written them after this one began, which the read-only path does not allow.
//
//   add + RMSNorm:  h = x + r,  y = (h * 1 / sqrt(Sum h^2 / K + eps)) * gamma
//   SwiGLU:         v = gate / (1 + exp(-gate)) * up
#include <cuda_bf16.h>

#include <algorithm>

#include "kq_decode.h"
#include "kq_q8_rows.cuh"
#include "kq_types.cuh"

namespace kq {
namespace {

// Sum of v over the CTA, in a fixed order (part: one float per warp).
__device__ __forceinline__ float block_sum(float v, float* part) {
  v = warp_sum_f(v);
  if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = v;
  __syncthreads();
  v = 0.f;
  for (int i = 0; i < static_cast<int>(blockDim.x >> 5); ++i) v += part[i];
  return v;
}

// A sum of many terms in fp32 with the part that its additions round away (by Knuth's two-sum).
struct LongSum {
  float hi = 0.f, lo = 0.f;
  __device__ __forceinline__ void add(float v) {
    const float t = __fadd_rn(hi, v), b = __fsub_rn(t, hi);
    lo = __fadd_rn(lo, __fadd_rn(__fsub_rn(hi, __fsub_rn(t, b)), __fsub_rn(v, b)));
    hi = t;
  }
  __device__ __forceinline__ float value() const { return hi < INFINITY ? hi + lo : hi; }
};

// Largest v over the CTA (part: one float per warp); a NaN counts for nothing.
__device__ __forceinline__ float block_max(float v, float* part) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, o));
  if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = v;
  __syncthreads();
  v = 0.f;
  for (int i = 0; i < static_cast<int>(blockDim.x >> 5); ++i) v = fmaxf(v, part[i]);
  return v;
}

// 1 / sqrt(Sum h^2 / K + eps) and whether it may be taken from the fp32 sum: no square and no sum has
// passed the range, and what fell below it (2^-150 a square at most) is far below the mean.
__device__ __forceinline__ bool rms_scale(float ss, int K, float eps, float& rr) {
  const float m = __fdiv_rn(ss, static_cast<float>(K)) + eps;
  rr = __fdiv_rn(1.0f, sqrtf(m));
  return ss < INFINITY && m >= 0x1p-100f;
}

// Where it may not, h is taken times s = s1 * s2, a power of two (two factors: it can be beyond
// 2^127) that brings the larger of max |h| and sqrt(eps) to 2^40 (subnormal ones to 2^18 at least):
// then the sum of 2^31 squares stays below 2^128, and a product below 2^-126 is under 2^-166 of the
// largest and gives a y below fp32's least. The result, 1 / sqrt(Sum (s h)^2 / K + s^2 eps), is the
// factor of s h.
struct Pow2 {
  float s1, s2;
  __device__ __forceinline__ Pow2(float hmax, float eps) {
    const int e = 40 + 127 - static_cast<int>(__float_as_uint(fmaxf(hmax, sqrtf(eps))) >> 23), e1 = e >> 1;
    s1 = __uint_as_float(static_cast<uint32_t>(127 + e1) << 23);
    s2 = __uint_as_float(static_cast<uint32_t>(127 + e - e1) << 23);
  }
  __device__ __forceinline__ float operator()(float h) const { return h * s1 * s2; }
  __device__ __forceinline__ float square(float eps) const { return eps * s1 * s1 * s2 * s2; }
};

// One row per CTA, held in registers: thread t has the row's runs of eight values
// t, t + blockDim, ... (CH of them). Read once, all loads of a row in flight
// together; H may be X or R themselves (an element is read and written by the
// same thread, the read first).
//
// Bound by HBM for many rows: 4099 x 4096 bf16 with residual, H and Y 29.1 us, 153 MB,
// 5.3 TB/s = 0.78 of the measured copy (issue slots 60 % busy, most of it the
// quantiser). One fp32 row: 2.4 us, a launch, a row's load, the CTA's sum and the quantiser's chain.
template <typename T, bool VEC, int CH>
__global__ void __launch_bounds__(CH == 2 ? 512 : 1024) add_rmsnorm_reg_kernel(const T* X, int64_t ldx, const T* R, int64_t ldr,
                                                              const float* gamma, float eps, T* H,
                                                              int64_t ldh, T* Y, int64_t ldy, uint8_t* __restrict__ Xq,
                                                              int K) {
  __shared__ float part[32], far_max[32], far_sum[32];
  pdl_enter();
  const int64_t n = blockIdx.x;
  const T* x = X + n * ldx;
  const int runs = K >> 3;
  float v[CH][8];
#pragma unroll
  for (int c = 0; c < CH; ++c) {
    const int i = threadIdx.x + c * blockDim.x;
#pragma unroll
    for (int k = 0; k < 8; ++k) v[c][k] = 0.f;
    if (i < runs) load8<T, VEC>(x + 8 * i, v[c]);
  }
  if (R) {
    const T* r = R + n * ldr;
#pragma unroll
    for (int c = 0; c < CH; ++c) {
      const int i = threadIdx.x + c * blockDim.x;
      float w[8];
      if (i < runs) {
        load8<T, VEC>(r + 8 * i, w);
#pragma unroll
        for (int k = 0; k < 8; ++k) v[c][k] += w[k];
      }
    }
  }
  float ss = 0.f;
#pragma unroll
  for (int c = 0; c < CH; ++c) {
    const int i = threadIdx.x + c * blockDim.x;
    if (H && i < runs) store8<T, VEC>(H + n * ldh + 8 * i, v[c]);
#pragma unroll
    for (int k = 0; k < 8; ++k) ss = fmaf(v[c][k], v[c][k], ss);
  }
  ss = block_sum(ss, part);
  float rr;
  if (!rms_scale(ss, K, eps, rr)) {   // the same for all threads
    float m = 0.f;
#pragma unroll
    for (int c = 0; c < CH; ++c)
#pragma unroll
      for (int k = 0; k < 8; ++k) m = fmaxf(m, fabsf(v[c][k]));
    const Pow2 scaled(block_max(m, far_max), eps);
    ss = 0.f;
#pragma unroll
    for (int c = 0; c < CH; ++c)
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        v[c][k] = scaled(v[c][k]);
        ss = fmaf(v[c][k], v[c][k], ss);
      }
    rms_scale(block_sum(ss, far_sum), K, scaled.square(eps), rr);
  }
  uint8_t* xq = Xq + n * (K >> 5) * Q8_1_BYTES;
#pragma unroll
  for (int c = 0; c < CH; ++c) {
    const int i = threadIdx.x + c * blockDim.x;
    if (i < runs) {
      float w[8];
      load8<float, true>(gamma + 8 * i, w);
#pragma unroll
      for (int k = 0; k < 8; ++k) v[c][k] = v[c][k] * rr * w[k];
      if (Y) store8<T, VEC>(Y + n * ldy + 8 * i, v[c]);
    }
  }
#pragma unroll
  for (int c = 0; c < CH; ++c) {
    const int i = threadIdx.x + c * blockDim.x;
    store_q8_block(v[c], xq + (i >> 2) * Q8_1_BYTES, i < runs);
  }
}

// The same for rows too long for registers. The row is read twice (the second time
// from L2): once for the sum of squares and once for the outputs. A thread has K / 512
// squares: the runs' sums are added with what each addition rounds away, as one fp32 sum of
// them all would be off by as many roundings. H may be X or R
// themselves: an element is read and written by the same thread, the read first.
template <typename T, bool VEC>
__global__ void __launch_bounds__(512) add_rmsnorm_kernel(const T* X, int64_t ldx, const T* R, int64_t ldr,
                                                          const float* gamma, float eps, T* H, int64_t ldh,
                                                          T* Y, int64_t ldy, uint8_t* __restrict__ Xq, int K) {
  __shared__ float part[16], far_max[16], far_sum[16];
  pdl_enter();
  const int64_t n = blockIdx.x;
  const T* x = X + n * ldx;
  const T* r = R ? R + n * ldr : nullptr;
  const int runs = K >> 3;
  LongSum ss;
  for (int i = threadIdx.x; i < runs; i += blockDim.x) {
    float v[8], w[8], s8 = 0.f;
    load8<T, VEC>(x + 8 * i, v);
    if (r) {
      load8<T, VEC>(r + 8 * i, w);
#pragma unroll
      for (int k = 0; k < 8; ++k) v[k] += w[k];
    }
#pragma unroll
    for (int k = 0; k < 8; ++k) s8 = fmaf(v[k], v[k], s8);
    ss.add(s8);
  }
  float rr;
  const bool far = !rms_scale(block_sum(ss.value(), part), K, eps, rr);   // the same for all threads
  Pow2 scaled(0x1p40f, 0.f);   // by 1
  if (far) {
    // Two passes: the largest, then the sum.
    float m = 0.f;
    for (int pass = 0; pass < 2; ++pass) {
      ss = LongSum();
      for (int i = threadIdx.x; i < runs; i += blockDim.x) {
        float v[8], w[8], s8 = 0.f;
        load8<T, VEC>(x + 8 * i, v);
        if (r) {
          load8<T, VEC>(r + 8 * i, w);
#pragma unroll
          for (int k = 0; k < 8; ++k) v[k] += w[k];
        }
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          m = fmaxf(m, fabsf(v[k]));
          s8 = fmaf(scaled(v[k]), scaled(v[k]), s8);
        }
        ss.add(s8);
      }
      if (pass == 0) scaled = Pow2(block_max(m, far_max), eps);
    }
    rms_scale(block_sum(ss.value(), far_sum), K, scaled.square(eps), rr);
  }
  uint8_t* xq = Xq + n * (K >> 5) * Q8_1_BYTES;
  for (int i0 = 0; i0 < runs; i0 += blockDim.x) {
    const int i = i0 + threadIdx.x;
    const bool in = i < runs;
    float v[8] = {}, w[8];
    if (in) {
      load8<T, VEC>(x + 8 * i, v);
      if (r) {
        load8<T, VEC>(r + 8 * i, w);
#pragma unroll
        for (int k = 0; k < 8; ++k) v[k] += w[k];
      }
      load8<float, true>(gamma + 8 * i, w);   // before the stores, behind which it would wait
      if (H) store8<T, VEC>(H + n * ldh + 8 * i, v);
      if (far) {
#pragma unroll
        for (int k = 0; k < 8; ++k) v[k] = scaled(v[k]);
      }
#pragma unroll
      for (int k = 0; k < 8; ++k) v[k] = v[k] * rr * w[k];
      if (Y) store8<T, VEC>(Y + n * ldy + 8 * i, v);
    }
    store_q8_block(v, xq + (i >> 2) * Q8_1_BYTES, in);
  }
}

// silu(g) * u. The division is a product with the reciprocal (rcp.approx, at most
// 2^-23 off): with expf's 2 ulp, the sum and the two products at most 9 * 2^-24.
__device__ __forceinline__ float swiglu(float g, float u) {
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(1.0f + expf(-g)));
  return g * r * u;
}

// A thread takes runs of eight values, a grid's threads apart; the next run's
// loads are in flight while one is computed. Row and place in the row are
// carried along (no division per run): a step is `rows` rows and `places` places. (Four
// runs a thread, a lane of each quad making one block's scale for all: 35.6 us instead
// of 32.5 for 2048 x 14336 in bf16, and 2.4 instead of 1.5 for eight rows of 768.)
//
// Bound by issue: 33 instructions per value (exp, reciprocal, products, rounding
// to codes), 80 % of the slots busy. 2048 x 14336 bf16 32.3 us, 150 MB, 4.7 TB/s = 0.69 of
// the measured copy; eight rows of 768 1.5 us, the launch.
template <typename T>
constexpr int swiglu_ctas() { return sizeof(T) == 4 ? 5 : 6; }   // per SM: what the registers allow
template <typename T, bool VEC>
__global__ void __launch_bounds__(256, swiglu_ctas<T>()) swiglu_kernel(const T* G, int64_t ldg, const T* U,
                                                     int64_t ldu, uint8_t* __restrict__ Xq, int runs, int64_t total,
                                                     int64_t rows, int places) {
  pdl_enter();
  int64_t t = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x;
  int64_t n = t / runs;
  int i = static_cast<int>(t - n * runs);
  const int64_t stride = static_cast<int64_t>(gridDim.x) * 256;
  Raw8<T> g = {}, u = {};
  if (t < total) {
    g.template load<VEC>(G + n * ldg + 8 * i);
    u.template load<VEC>(U + n * ldu + 8 * i);
  }
  while (t - static_cast<int>(threadIdx.x & 31) < total) {   // warp-uniform
    Raw8<T> gn = {}, un = {};
    n += rows;
    i += places;
    if (i >= runs) {
      i -= runs;
      ++n;
    }
    if (t + stride < total) {
      gn.template load<VEC>(G + n * ldg + 8 * i);
      un.template load<VEC>(U + n * ldu + 8 * i);
    }
    float v[8];
#pragma unroll
    for (int k = 0; k < 8; ++k) v[k] = swiglu(g[k], u[k]);
    store_q8_block(v, Xq + (t >> 2) * Q8_1_BYTES, t < total);
    t += stride;
    g = gn;
    u = un;
  }
}

// Sixteen-byte accesses are taken where every row starts on such a boundary.
bool rows16(int64_t ld, int size) { return (ld * size) % 16 == 0; }

template <typename T>
cudaError_t launch_norm_t(const void* X, int64_t ldx, const void* R, int64_t ldr, const float* gamma, float eps, void* H,
                          int64_t ldh, void* Y, int64_t ldy, void* Xq, int64_t K, int64_t N, int num_sms, cudaStream_t s) {
  const int sz = sizeof(T);
  const bool vec = rows16(ldx, sz) && (!R || rows16(ldr, sz)) && (!H || rows16(ldh, sz)) && (!Y || rows16(ldy, sz));
  auto go = [&](auto k, int64_t threads) {
    return launch_pdl(k, dim3(static_cast<unsigned>(N)), dim3(static_cast<unsigned>((threads + 31) / 32 * 32)), 0, s,
                      static_cast<const T*>(X), ldx, static_cast<const T*>(R), ldr, gamma, eps, static_cast<T*>(H), ldh,
                      static_cast<T*>(Y), ldy, static_cast<uint8_t*>(Xq), static_cast<int>(K));
  };
  // As many threads as a row has runs, for the latency of a row; two runs a thread where
  // there are many rows, so that more rows share an SM (bf16, K = 4096: 1024 rows 9.7 us
  // against 10.9, 2048 rows 17.2 against 16.9, 4099 rows 30.5 against 28.9); four where the row is long.
  const int64_t runs = K / 8;
  if (N <= 10 * num_sms && runs <= 1024)
    return go(vec ? add_rmsnorm_reg_kernel<T, true, 1> : add_rmsnorm_reg_kernel<T, false, 1>, runs);
  if (runs <= 1024)
    return go(vec ? add_rmsnorm_reg_kernel<T, true, 2> : add_rmsnorm_reg_kernel<T, false, 2>, (runs + 1) / 2);
  if (runs <= 4096)
    return go(vec ? add_rmsnorm_reg_kernel<T, true, 4> : add_rmsnorm_reg_kernel<T, false, 4>, (runs + 3) / 4);
  return go(vec ? add_rmsnorm_kernel<T, true> : add_rmsnorm_kernel<T, false>, 512);
}

template <typename T>
cudaError_t launch_swiglu_t(const void* G, int64_t ldg, const void* U, int64_t ldu, void* Xq, int64_t K, int64_t N,
                            int num_sms, cudaStream_t s) {
  const bool vec = rows16(ldg, sizeof(T)) && rows16(ldu, sizeof(T));
  const int64_t runs = K / 8, total = N * runs;
  const int64_t blocks = std::min<int64_t>((total + 255) / 256, static_cast<int64_t>(num_sms) * swiglu_ctas<T>());
  const int64_t stride = blocks * 256;
  auto k = vec ? swiglu_kernel<T, true> : swiglu_kernel<T, false>;
  return launch_pdl(k, dim3(static_cast<unsigned>(blocks)), dim3(256), 0, s, static_cast<const T*>(G), ldg,
                    static_cast<const T*>(U), ldu, static_cast<uint8_t*>(Xq), static_cast<int>(runs), total, stride / runs,
                    static_cast<int>(stride % runs));
}

}  // namespace

cudaError_t launch_add_rmsnorm_q8_1(int dtype, const void* X, int64_t ldx, const void* R, int64_t ldr,
                                    const float* gamma, float eps, void* H, int64_t ldh, void* Y, int64_t ldy,
                                    void* Xq, int64_t K, int64_t N, int num_sms, cudaStream_t s) {
  if (dtype == KQ_F32) return launch_norm_t<float>(X, ldx, R, ldr, gamma, eps, H, ldh, Y, ldy, Xq, K, N, num_sms, s);
  if (dtype == KQ_F16) return launch_norm_t<__half>(X, ldx, R, ldr, gamma, eps, H, ldh, Y, ldy, Xq, K, N, num_sms, s);
  return launch_norm_t<__nv_bfloat16>(X, ldx, R, ldr, gamma, eps, H, ldh, Y, ldy, Xq, K, N, num_sms, s);
}

cudaError_t launch_swiglu_q8_1(int dtype, const void* G, int64_t ldg, const void* U, int64_t ldu, void* Xq, int64_t K,
                               int64_t N, int num_sms, cudaStream_t s) {
  if (dtype == KQ_F32) return launch_swiglu_t<float>(G, ldg, U, ldu, Xq, K, N, num_sms, s);
  if (dtype == KQ_F16) return launch_swiglu_t<__half>(G, ldg, U, ldu, Xq, K, N, num_sms, s);
  return launch_swiglu_t<__nv_bfloat16>(G, ldg, U, ldu, Xq, K, N, num_sms, s);
}

}  // namespace kq
