// Routing of tokens to experts: scores, the balance bias, group limits, top-k
// and the renormalised weights.
//
//   s_e = exp(l_e - max l) / Sum exp(l - max l)   or   1 / (1 + exp(-l_e))
//   key_e = s_e + bias_e (selection only)
//   group score = sum of the group's `group_top` largest keys; the topk_groups
//   best groups stay; the top_k largest keys in them are chosen, in order, ties
//   to the lowest index; weight_j = s_j [/ Sum_j s_j] * scale.
//
// One warp per token. The keys are computed in fp32 first. A key's fp32 error
// is bounded (below), so the order of two keys further apart than twice that is
// the order of the exact keys. Where a decision is closer than that, the warp
// computes the row's keys again in fp64 and selects again from those: the
// chosen experts are those of the 64-bit definition, at the fp32 path's cost
// for all but about one row in a thousand.
#include <algorithm>

#include <cuda_bf16.h>

#include "kq_internal.h"
#include "kq_types.cuh"

namespace kq {
namespace {

constexpr unsigned FULL = 0xffffffffu;
constexpr int RT_WARPS = 4;

// Order-preserving maps of keys to unsigned integers; -inf (not available, or
// already taken) maps to 0, below every other key.
__device__ __forceinline__ uint32_t ord(float v) {
  const uint32_t b = __float_as_uint(v == 0.f ? 0.f : v);
  if (b == 0xff800000u) return 0;
  return (b & 0x80000000u) ? ~b : (b | 0x80000000u);
}
__device__ __forceinline__ uint64_t ord(double v) {
  const uint64_t b = static_cast<uint64_t>(__double_as_longlong(v == 0. ? 0. : v));
  if (b == 0xfff0000000000000ull) return 0;
  return (b >> 63) ? ~b : (b | 0x8000000000000000ull);
}
__device__ __forceinline__ uint32_t warp_max(uint32_t v) { return __reduce_max_sync(FULL, v); }
__device__ __forceinline__ uint64_t warp_max(uint64_t v) {
  const uint32_t hi = __reduce_max_sync(FULL, static_cast<uint32_t>(v >> 32));
  const uint32_t lo = __reduce_max_sync(FULL, static_cast<uint32_t>(v >> 32) == hi ? static_cast<uint32_t>(v) : 0u);
  return (static_cast<uint64_t>(hi) << 32) | lo;
}

template <typename KT>
struct Ord;
template <>
struct Ord<float> { using U = uint32_t; };
template <>
struct Ord<double> { using U = uint64_t; };

template <typename KT>
__device__ __forceinline__ KT minus_inf() { return static_cast<KT>(-INFINITY); }

__device__ __forceinline__ float warp_max_f(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(FULL, v, o));
  return v;
}

// The lowest index of the largest of key[0, n) (shared memory), or -1 when all
// are -inf. All lanes get the answer.
template <typename KT>
__device__ __forceinline__ int warp_argmax(const KT* key, int n, int lane, KT* best) {
  typename Ord<KT>::U m = 0;
  int at = 0x7fffffff;
  for (int i = lane; i < n; i += 32) {
    const typename Ord<KT>::U o = ord(key[i]);
    if (o > m) {
      m = o;
      at = i;
    }
  }
  const typename Ord<KT>::U w = warp_max(m);
  if (w == 0) return -1;
  const int e = static_cast<int>(__reduce_min_sync(FULL, m == w ? static_cast<unsigned>(at) : 0x7fffffffu));
  *best = key[e];
  return e;
}

struct RouteArgs {
  const void* logits;
  int64_t ld;
  const float* bias;
  int score, n_groups, topk_groups, group_top, top_k, renorm;
  float scale;
  int* ids;
  float* probs;
  int E;
  int64_t T;
};

// The selection of one token from key (destroyed). Writes the chosen experts to
// ids[0, top_k) (shared), -1 for a slot without one. Returns whether every
// decision was further than `tol` from going the other way.
template <typename KT>
__device__ bool select_experts(const RouteArgs& a, KT* key, KT* gkey, const float* l, int* ids, int lane, KT tol) {
  bool clear = true;
  const int per = a.E / a.n_groups;
  if (a.topk_groups < a.n_groups) {
    for (int g = lane; g < a.n_groups; g += 32) {
      KT m1 = minus_inf<KT>(), m2 = minus_inf<KT>();
      for (int i = 0; i < per; ++i) {
        const KT v = key[g * per + i];
        m2 = v > m1 ? m1 : (v > m2 ? v : m2);
        m1 = v > m1 ? v : m1;
      }
      gkey[g] = (a.group_top == 2 && m2 != minus_inf<KT>()) ? m1 + m2 : m1;
    }
    __syncwarp();
    KT last = 0, best = 0;
    for (int r = 0; r < a.topk_groups; ++r) {
      const int g = warp_argmax(gkey, a.n_groups, lane, &best);
      if (g < 0) break;
      last = best;
      __syncwarp();
      if (lane == 0) gkey[g] = minus_inf<KT>();
      __syncwarp();
    }
    // The keys of the groups that are left go out.
    // A group's score is the sum of two keys: twice a key's error, and a rounding.
    if (warp_argmax(gkey, a.n_groups, lane, &best) >= 0) clear = !(last - best <= 4 * tol);
    for (int i = lane; i < a.E; i += 32)
      if (gkey[i / per] != minus_inf<KT>()) key[i] = minus_inf<KT>();
    __syncwarp();
  }
  if (!a.bias) {
    // The scores have the logits' order: chosen by the logits, nothing is close.
    for (int i = lane; i < a.E; i += 32)
      if (key[i] != minus_inf<KT>()) key[i] = l[i];
    __syncwarp();
    tol = -1;
  }
  KT prev = 0;
  int prev_e = -1;
  for (int j = 0; j <= a.top_k; ++j) {
    KT best = 0;
    const int e = warp_argmax(key, a.E, lane, &best);
    if (e >= 0 && prev_e >= 0 && prev - best <= tol) {
      // Two experts with the same logit and the same bias have the same key in
      // any precision: the lower index is first, as it should be.
      if (!(l[e] == l[prev_e] && a.bias[e] == a.bias[prev_e])) clear = false;
    }
    if (j == a.top_k) break;
    if (lane == 0) ids[j] = e;
    prev = best;
    prev_e = e;
    __syncwarp();
    if (e >= 0 && lane == 0) key[e] = minus_inf<KT>();
    __syncwarp();
  }
  return clear;
}

template <typename T>
__global__ void __launch_bounds__(RT_WARPS * 32) route_kernel(RouteArgs a, int warp_bytes) {
  extern __shared__ __align__(16) uint8_t smem[];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  uint8_t* base = smem + warp * warp_bytes;
  double* kd = reinterpret_cast<double*>(base);  // keys, fp64 (the fp32 ones first)
  double* gd = kd + a.E;                         // group scores
  float* l = reinterpret_cast<float*>(gd + a.n_groups);
  float* s = l + a.E;
  int* ids = reinterpret_cast<int*>(s + a.E);
  pdl_enter();
  const int64_t t = static_cast<int64_t>(blockIdx.x) * RT_WARPS + warp;
  if (t >= a.T) return;  // no block-wide barrier below

  const T* row = static_cast<const T*>(a.logits) + t * a.ld;
  float mx = -INFINITY;
  for (int e = lane; e < a.E; e += 32) {
    float v = to_f32(row[e]);
    // Out of service: -inf or NaN. Above the largest finite fp32: taken as that.
    v = (v != v) ? -INFINITY : fminf(v, 3.402823466e38f);
    l[e] = v;
    mx = fmaxf(mx, v);
  }
  mx = warp_max_f(mx);
  float sum = 0.f;
  const bool softmax = a.score == KQ_SCORE_SOFTMAX;
  for (int e = lane; e < a.E; e += 32) {
    const float v = l[e];
    const float x = v == -INFINITY ? 0.f : softmax ? expf(v - mx) : __fdiv_rn(1.0f, 1.0f + expf(-v));
    s[e] = x;
    sum += x;
  }
  sum = warp_sum_f(sum);
  const float inv = softmax && sum > 0.f ? __fdiv_rn(1.0f, sum) : 1.0f;
  const bool groups = a.topk_groups < a.n_groups;
  const bool by_logit = !a.bias && !(groups && a.group_top == 2);  // scores have the logits' order
  float bmax = 0.f;
  float* kf = reinterpret_cast<float*>(kd);
  for (int e = lane; e < a.E; e += 32) {
    const float x = s[e] * inv;
    s[e] = x;
    float k = l[e];
    if (!by_logit && k != -INFINITY) {
      const float b = a.bias ? a.bias[e] : 0.f;
      k = x + b;
      k = (k != k) ? -INFINITY : k;
      if (fabsf(b) < INFINITY) bmax = fmaxf(bmax, fabsf(b));
    }
    kf[e] = k;
  }
  __syncwarp();
  // What two fp32 keys can be apart and still be in the wrong order. A softmax
  // score is off by at most 2 ulp of expf, the rounding of l - max (for a score
  // of e^-x it is x * 2^-24 relative, at most 2^-24 * 0.37 of the largest), the
  // sum's E / 32 + 5 roundings and two more: under 2^-18 of the largest score,
  // which is 1 / Sum. A sigmoid is off by under 2^-21 of 1. Adding the bias
  // rounds once more, by 2^-24 of the key.
  const float smax = softmax ? inv : 1.0f;
  const float tol = by_logit ? -1.0f : 2.f * (smax * (softmax ? 3.8147e-6f : 4.7684e-7f) + 5.9605e-8f * (smax + warp_max_f(bmax)));
  bool clear = select_experts<float>(a, kf, reinterpret_cast<float*>(gd), l, ids, lane, tol);
  if (!clear) {  // warp-uniform
    double dsum = 0.;
    for (int e = lane; e < a.E; e += 32) {
      const double v = l[e];
      const double x = l[e] == -INFINITY ? 0. : softmax ? exp(v - static_cast<double>(mx)) : 1. / (1. + exp(-v));
      kd[e] = x;
      dsum += x;
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) dsum += __shfl_xor_sync(FULL, dsum, o);
    for (int e = lane; e < a.E; e += 32) {
      double k = -INFINITY;
      if (l[e] != -INFINITY) {
        k = (softmax ? kd[e] / dsum : kd[e]) + (a.bias ? static_cast<double>(a.bias[e]) : 0.);
        k = (k != k) ? -INFINITY : k;
      }
      kd[e] = k;
    }
    __syncwarp();
    select_experts<double>(a, kd, gd, l, ids, lane, -1.0);
  }
  __syncwarp();
  // Weights, in slot order; slots without an available expert take the
  // lowest-numbered experts not chosen, with weight 0.
  float tot = 0.f;
  for (int j = lane; j < a.top_k; j += 32) tot += ids[j] >= 0 ? s[ids[j]] : 0.f;
  tot = warp_sum_f(tot);
  const float f = a.renorm ? (tot > 0.f ? __fdiv_rn(1.0f, tot) : 0.f) : 1.0f;
  for (int j = lane; j < a.top_k; j += 32) {
    a.probs[t * a.top_k + j] = ids[j] >= 0 ? s[ids[j]] * f * a.scale : 0.f;
    if (ids[j] >= 0) a.ids[t * a.top_k + j] = ids[j];
  }
  const bool empty = ids[a.top_k - 1] < 0;
  __syncwarp();
  if (empty) {  // rare: fewer experts than slots
    if (lane == 0) {
      int e = 0;
      for (int j = 0; j < a.top_k; ++j) {
        if (ids[j] >= 0) continue;
        for (;; ++e) {
          bool used = false;
          for (int i = 0; i < j; ++i) used |= ids[i] == e;
          if (!used) break;
        }
        ids[j] = e;
        a.ids[t * a.top_k + j] = e;
      }
    }
  }
}

}  // namespace

cudaError_t launch_moe_route(int dtype, const void* logits, int64_t ld, const float* bias, int score, int n_groups,
                             int topk_groups, int group_top, int top_k, bool renorm, float scale, int* ids, float* probs,
                             int E, int64_t T, cudaStream_t s) {
  RouteArgs a{logits, ld, bias, score, n_groups, topk_groups, group_top, top_k, renorm, scale, ids, probs, E, T};
  const int warp_bytes = (8 * E + 8 * n_groups + 8 * E + 4 * top_k + 15) / 16 * 16;
  const size_t smem = static_cast<size_t>(RT_WARPS) * warp_bytes;
  auto k = dtype == KQ_F32 ? route_kernel<float> : dtype == KQ_F16 ? route_kernel<__half> : route_kernel<__nv_bfloat16>;
  if (smem > 48 * 1024) {
    const cudaError_t e = allow_max_smem(reinterpret_cast<const void*>(k), kSmemRoute + dtype - 1);
    if (e != cudaSuccess) return e;
  }
  return launch_pdl(k, dim3(static_cast<unsigned>((T + RT_WARPS - 1) / RT_WARPS)), dim3(RT_WARPS * 32), smem, s, a,
                    warp_bytes);
}

}  // namespace kq
