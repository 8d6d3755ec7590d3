// Reads and writes of eight consecutive elements of a row in fp32, fp16 or bf16.
#pragma once

#include <cuda_bf16.h>

#include "kq_common.cuh"

namespace kq {

__device__ __forceinline__ float to_f32(float v) { return v; }
__device__ __forceinline__ float to_f32(__half v) { return __half2float(v); }
__device__ __forceinline__ float to_f32(__nv_bfloat16 v) { return __bfloat162float(v); }
template <typename T>
__device__ __forceinline__ T from_f32(float v);
template <>
__device__ __forceinline__ float from_f32<float>(float v) { return v; }
template <>
__device__ __forceinline__ __half from_f32<__half>(float v) { return __float2half_rn(v); }
template <>
__device__ __forceinline__ __nv_bfloat16 from_f32<__nv_bfloat16>(float v) { return __float2bfloat16_rn(v); }

// Eight elements at any address, by the pairs that lie on a boundary of theirs, and the first and the
// last by themselves where pairs begin with the second (2048 rows of 4736, with residual, h
// and y, one element between rows: bf16 24.9 us against 44.2 element by element, fp32 40.5 against 55.6).
template <typename T>
__device__ __forceinline__ void load8_any(const T* p, T (&e)[8]) {
  if constexpr (sizeof(T) == 2) {
    uint32_t* w = reinterpret_cast<uint32_t*>(e);
    if ((reinterpret_cast<uintptr_t>(p) & 3) == 0) {
#pragma unroll
      for (int i = 0; i < 4; ++i) w[i] = reinterpret_cast<const uint32_t*>(p)[i];
    } else {
      const uint32_t a = reinterpret_cast<const uint16_t*>(p)[0], b = reinterpret_cast<const uint16_t*>(p)[7];
      uint32_t m[3];
#pragma unroll
      for (int i = 0; i < 3; ++i) m[i] = reinterpret_cast<const uint32_t*>(p + 1)[i];
      w[0] = __byte_perm(a, m[0], 0x5410);
      w[1] = __byte_perm(m[0], m[1], 0x5432);
      w[2] = __byte_perm(m[1], m[2], 0x5432);
      w[3] = __byte_perm(m[2], b, 0x5432);
    }
  } else {
    if ((reinterpret_cast<uintptr_t>(p) & 7) == 0) {
#pragma unroll
      for (int i = 0; i < 4; ++i) reinterpret_cast<float2*>(e)[i] = reinterpret_cast<const float2*>(p)[i];
    } else {
      e[0] = p[0];
      e[7] = p[7];
#pragma unroll
      for (int i = 0; i < 3; ++i) {
        const float2 v = reinterpret_cast<const float2*>(p + 1)[i];
        e[2 * i + 1] = v.x;
        e[2 * i + 2] = v.y;
      }
    }
  }
}
template <typename T>
__device__ __forceinline__ void store8_any(T* p, const T (&e)[8]) {
  if constexpr (sizeof(T) == 2) {
    const uint32_t* w = reinterpret_cast<const uint32_t*>(e);
    if ((reinterpret_cast<uintptr_t>(p) & 3) == 0) {
#pragma unroll
      for (int i = 0; i < 4; ++i) reinterpret_cast<uint32_t*>(p)[i] = w[i];
    } else {
      reinterpret_cast<uint16_t*>(p)[0] = static_cast<uint16_t>(w[0]);
#pragma unroll
      for (int i = 0; i < 3; ++i) reinterpret_cast<uint32_t*>(p + 1)[i] = __byte_perm(w[i], w[i + 1], 0x5432);
      reinterpret_cast<uint16_t*>(p)[7] = static_cast<uint16_t>(w[3] >> 16);
    }
  } else {
    if ((reinterpret_cast<uintptr_t>(p) & 7) == 0) {
#pragma unroll
      for (int i = 0; i < 4; ++i) reinterpret_cast<float2*>(p)[i] = reinterpret_cast<const float2*>(e)[i];
    } else {
      p[0] = e[0];
      p[7] = e[7];
#pragma unroll
      for (int i = 0; i < 3; ++i) reinterpret_cast<float2*>(p + 1)[i] = make_float2(e[2 * i + 1], e[2 * i + 2]);
    }
  }
}

// VEC: p is 16-byte aligned (one or two 16-byte accesses). Plain loads, not the
// read-only path: an output may be the input.
template <typename T, bool VEC>
__device__ __forceinline__ void load8(const T* p, float (&v)[8]) {
  if constexpr (VEC) {
    constexpr int W = sizeof(T) * 8 / 16;
    alignas(16) uint4 raw[W];
#pragma unroll
    for (int i = 0; i < W; ++i) raw[i] = reinterpret_cast<const uint4*>(p)[i];
    const T* e = reinterpret_cast<const T*>(raw);
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = to_f32(e[i]);
  } else {
    alignas(16) T e[8];
    load8_any(p, e);
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = to_f32(e[i]);
  }
}

// Eight elements as loaded, to be converted where they are used.
template <typename T>
struct Raw8 {
  alignas(16) T e[8];
  template <bool VEC>
  __device__ __forceinline__ void load(const T* p) {
    if constexpr (VEC) {
#pragma unroll
      for (int i = 0; i < static_cast<int>(sizeof(T)) / 2; ++i)
        reinterpret_cast<uint4*>(e)[i] = reinterpret_cast<const uint4*>(p)[i];
    } else {
      load8_any(p, e);
    }
  }
  __device__ __forceinline__ float operator[](int i) const { return to_f32(e[i]); }
};

template <typename T, bool VEC>
__device__ __forceinline__ void store8(T* p, const float (&v)[8]) {
  alignas(16) T e[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) e[i] = from_f32<T>(v[i]);
  if constexpr (VEC) {
    constexpr int W = sizeof(T) * 8 / 16;
#pragma unroll
    for (int i = 0; i < W; ++i) reinterpret_cast<uint4*>(p)[i] = reinterpret_cast<const uint4*>(e)[i];
  } else {
    store8_any(p, e);
  }
}

}  // namespace kq
