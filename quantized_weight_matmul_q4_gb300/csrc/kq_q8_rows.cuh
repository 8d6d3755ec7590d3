// Q8_1 blocks of produced values, written by the operators whose outputs are such rows.
#pragma once

#include "kq_quant.cuh"

namespace kq {

__device__ __forceinline__ float max_nan(float a, float b) {   // a NaN stays
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}

__device__ __forceinline__ float min_nan(float a, float b) {
  float r;
  asm("min.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}

// The Q8_1 block of 32 values held by the four lanes of an aligned lane quad,
// eight each (v), written to block `dst`. All 32 lanes of the warp call it;
// lanes without `store` take part in the shuffles only.
//
// Same codes and scales as quantize_oct for finite values. Here a NaN or an
// infinity reaches the scale, so that such a block stands for non-finite values
// instead of hiding them.
__device__ __forceinline__ void store_q8_block(const float (&v)[8], uint8_t* dst, bool store) {
  float a = fabsf(v[0]);
#pragma unroll
  for (int i = 1; i < 8; ++i) a = max_nan(a, fabsf(v[i]));
  a = max_nan(a, __shfl_xor_sync(0xffffffffu, a, 1));
  a = max_nan(a, __shfl_xor_sync(0xffffffffu, a, 2));
  const float d = __fdiv_rn(a, 127.0f);
  const float di = q8_inv_scale(d);
  uint32_t q[2];
  int s = 0;
#pragma unroll
  for (int w = 0; w < 2; ++w) {
    uint32_t u[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) u[k] = __float_as_uint(__fadd_rn(__fmul_rn(v[4 * w + k], di), 12582912.0f));
    q[w] = __byte_perm(__byte_perm(u[0], u[1], 0x0040), __byte_perm(u[2], u[3], 0x0040), 0x5410);
    s = __dp4a(static_cast<int>(q[w]), 0x01010101, s);
  }
  s += __shfl_xor_sync(0xffffffffu, s, 1);
  s += __shfl_xor_sync(0xffffffffu, s, 2);
  if (!store) return;
  const int j = threadIdx.x & 3;
  // Blocks are 36 bytes apart: 4-byte stores.
  uint32_t* p = reinterpret_cast<uint32_t*>(dst + 4 + 8 * j);
  p[0] = q[0];
  p[1] = q[1];
  if (j == 0) {
    const __half dh = __float2half_rn(d);
    const __half sh = __float2half_rn(__fmul_rn(__half2float(dh), static_cast<float>(s)));
    *reinterpret_cast<uint32_t*>(dst) =
        static_cast<uint32_t>(__half_as_ushort(dh)) | (static_cast<uint32_t>(__half_as_ushort(sh)) << 16);
  }
}

}  // namespace kq
