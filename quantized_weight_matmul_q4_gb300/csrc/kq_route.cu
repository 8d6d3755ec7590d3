// Routing of tokens to experts: scores, the balance bias, group limits, top-k
// and the renormalised weights.
//
//   s_e = exp(l_e - max l) / Sum exp(l - max l)   or   1 / (1 + exp(-l_e))
//   key_e = s_e + bias_e (selection only)
//   group score = sum of the group's `group_top` largest keys; the topk_groups
//   best groups stay; the top_k largest keys in them are chosen, in order, ties
//   to the lowest index; weight_j = s_j [/ Sum_j s_j] * scale.
//
// One warp per token, its experts in registers (expert e in lane e % 32). The
// keys are computed in fp32 first. A key's fp32 error is bounded (below), so the
// order of two keys further apart than twice that is the order of the exact
// keys. Where a decision is closer than that (about one row in a thousand), the
// few experts that it is between get their keys in fp64, one in each lane, and
// are ordered by those: the chosen experts are those of the 64-bit definition.
// (All of a row's keys in fp64, chosen one after the other, kept the whole call
// waiting for such a row: 8192 x 384 in 12 groups took 58 us.)
//
// A lane keeps its two best experts, so that a round costs two warp reductions and
// a rescan is rare. Bound by the latency of one token's chain of decisions (one
// token of 128 experts, top 8: 2.4 us; 1024 tokens: 3.9) and by issue for many tokens: 8192 x 384 in
// 12 groups, top 6, sigmoid with bias, bf16 17.7 us, some 1670 instructions per token,
// 73 % of the slots busy, against 1 us for its 6.7 MB.
#include <algorithm>

#include <cuda_bf16.h>

#include "kq_decode.h"
#include "kq_types.cuh"

namespace kq {
namespace {

constexpr unsigned FULL = 0xffffffffu;
constexpr int RT_WARPS = 4;

__device__ __forceinline__ float warp_max(float v) {   // no NaN
  float r;
  asm volatile("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(r) : "f"(v));
  return r;
}
__device__ __forceinline__ float warp_min(float v) { return -warp_max(-v); }
// e^x as 2^(x log2 e): relative error at most 2^-22 (ex2.approx) and 1.5 |x| 2^-24 (the
// product and its constant).
__device__ __forceinline__ float fast_exp(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x * 1.4426950408889634f));
  return r;
}
__device__ __forceinline__ float fast_rcp(float x) {   // relative error at most 2^-23
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}

// Order-preserving map of fp64 keys to integers; -inf (not available, or already
// taken) maps to 0, below every other key.
__device__ __forceinline__ uint64_t ord(double v) {
  const uint64_t b = static_cast<uint64_t>(__double_as_longlong(v + 0.));
  if (b == 0xfff0000000000000ull) return 0;
  return (b >> 63) ? ~b : (b | 0x8000000000000000ull);
}
__device__ __forceinline__ uint64_t warp_max(uint64_t v) {
  const uint32_t hi = __reduce_max_sync(FULL, static_cast<uint32_t>(v >> 32));
  const uint32_t lo = __reduce_max_sync(FULL, static_cast<uint32_t>(v >> 32) == hi ? static_cast<uint32_t>(v) : 0u);
  return (static_cast<uint64_t>(hi) << 32) | lo;
}

struct RouteArgs {
  uint32_t per, recip;   // experts of a group; e / per = e * recip >> 20 for e < 512
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

// A logit as the definition takes it: NaN is -inf (not available), anything
// above the largest finite fp32 is that.
template <typename T>
__device__ __forceinline__ float logit(const T* row, int e) {
  return fminf(fmaxf(to_f32(row[e]), -INFINITY), 3.402823466e38f);   // fmaxf(NaN, x) is x
}

// The lowest index of the largest of key[0, n) (shared memory), or -1 when all are -inf.
__device__ __forceinline__ int warp_argmax(const double* key, int n, int lane) {
  uint64_t m = 0;
  unsigned at = 0x7fffffffu;
  for (int i = lane; i < n; i += 32) {
    const uint64_t o = ord(key[i]);
    if (o > m) {
      m = o;
      at = static_cast<unsigned>(i);
    }
  }
  const uint64_t w = warp_max(m);
  if (w == 0) return -1;
  return static_cast<int>(__reduce_min_sync(FULL, m == w ? at : 0x7fffffffu));
}

// The selection of one token in fp64, step by step from the definition: ids[0, top_k)
// (shared), -1 for a slot without an expert. key, gkey: shared, E and n_groups.
template <typename T>
__device__ __noinline__ void select_exact(const RouteArgs& a, const T* row, float mx, double* key, double* gkey, int* ids, int lane) {
  const bool softmax = a.score == KQ_SCORE_SOFTMAX;
  double sum = 0.;
  for (int e = lane; e < a.E; e += 32) {
    const float l = logit(row, e);
    const double x = l == -INFINITY ? 0. : softmax ? exp(static_cast<double>(l) - static_cast<double>(mx)) : 1. / (1. + exp(-static_cast<double>(l)));
    key[e] = x;
    sum += x;
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(FULL, sum, o);
  for (int e = lane; e < a.E; e += 32) {
    double k = -INFINITY;
    if (logit(row, e) != -INFINITY) {
      k = (softmax ? key[e] / sum : key[e]) + (a.bias ? static_cast<double>(a.bias[e]) : 0.);
      k = (k != k) ? -INFINITY : k;
    }
    key[e] = k;
  }
  __syncwarp();
  if (a.topk_groups < a.n_groups) {
    const int per = static_cast<int>(a.per);
    for (int g = lane; g < a.n_groups; g += 32) {
      double m1 = -INFINITY, m2 = -INFINITY;
      for (int i = 0; i < per; ++i) {
        const double v = key[g * per + i];
        m2 = v > m1 ? m1 : (v > m2 ? v : m2);
        m1 = v > m1 ? v : m1;
      }
      gkey[g] = (a.group_top == 2 && m2 != -INFINITY) ? m1 + m2 : m1;
    }
    __syncwarp();
    for (int r = 0; r < a.topk_groups; ++r) {
      const int g = warp_argmax(gkey, a.n_groups, lane);
      if (g < 0) break;
      __syncwarp();
      if (lane == 0) gkey[g] = -INFINITY;
      __syncwarp();
    }
    // The experts of the groups that are left go out.
    for (int e = lane; e < a.E; e += 32)
      if (gkey[e / per] != -INFINITY) key[e] = -INFINITY;
    __syncwarp();
  }
  if (!a.bias) {   // the scores have the logits' order, and the logits are exact
    for (int e = lane; e < a.E; e += 32)
      if (key[e] != -INFINITY) key[e] = logit(row, e);
    __syncwarp();
  }
  for (int j = 0; j < a.top_k; ++j) {
    const int e = warp_argmax(key, a.E, lane);
    __syncwarp();
    if (lane == 0) {
      ids[j] = e;
      if (e >= 0) key[e] = -INFINITY;
    }
    __syncwarp();
  }
}

// Experts marked by `in` (of those in this lane's registers) into list[0, 32), in
// ascending order; how many there are.
template <int PER, typename F>
__device__ __forceinline__ int compact(F in, int* list, int lane) {
  int n = 0;
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    const unsigned b = __ballot_sync(FULL, in(i));
    const int at = n + __popc(b & ((1u << lane) - 1));
    if ((b >> lane & 1) && at < 32) list[at] = lane + 32 * i;
    n += __popc(b);
  }
  __syncwarp();
  return n;
}

// The fp64 softmax sum of a row (all lanes).
template <typename T>
__device__ __noinline__ double exact_sum(const T* row, int E, float mx, int lane) {
  double sum = 0.;
#pragma unroll 4
  for (int e = lane; e < E; e += 32) sum += exp(static_cast<double>(logit(row, e)) - static_cast<double>(mx));   // exp(-inf) = 0
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(FULL, sum, o);
  return sum;
}

// The fp64 key of one expert that is available.
template <typename T>
__device__ __noinline__ double exact_key(const RouteArgs& a, const T* row, int e, float mx, double sum) {
  const double l = logit(row, e);
  const double s = a.score == KQ_SCORE_SOFTMAX ? exp(l - static_cast<double>(mx)) / sum : 1. / (1. + exp(-l));
  return s + (a.bias ? static_cast<double>(a.bias[e]) : 0.);
}

// The renormalised weights of a token whose chosen scores are all tiny. Weights are ratios, and only
// the chosen experts' distances from `top`, the largest chosen logit, count: a softmax score is taken
// as e^(l - top) (its factor e^(top - mx) / Sum cancels), a sigmoid score as e^(l - top) / (1 + e^l)
// (top < 0). The largest of them is at least a half, however far the chosen experts lie below mx or
// below zero. A score that is zero in the 64-bit definition has weight zero.
template <typename T>
__device__ __noinline__ void weights_of_tiny_scores(const RouteArgs& a, int64_t t, const int* ids) {
  const int lane = threadIdx.x & 31;
  const T* row = static_cast<const T*>(a.logits) + t * a.ld;
  float* probs = a.probs + t * a.top_k;
  const bool softmax = a.score == KQ_SCORE_SOFTMAX;
  float mx = -INFINITY, top = -INFINITY;
  for (int e = lane; e < a.E; e += 32) mx = fmaxf(mx, logit(row, e));
  mx = warp_max(mx);
  for (int j = lane; j < a.top_k; j += 32)
    if (ids[j] >= 0) top = fmaxf(top, logit(row, ids[j]));
  top = warp_max(top);
  float tot = 0.f;
  for (int j = lane; j < a.top_k; j += 32) {
    float w = 0.f;
    if (ids[j] >= 0) {
      const float v = logit(row, ids[j]);
      if (softmax ? v - mx >= -745.14f : v >= -709.79f)   // else e^(v - mx) is 0 in fp64, e^-v infinite
        w = softmax ? expf(v - top) : __fdiv_rn(expf(v - top), 1.0f + expf(v));
    }
    tot += w;
    probs[j] = w;
  }
  tot = warp_sum_f(tot);
  const float f = tot > 0.f ? __fdiv_rn(1.0f, tot) : 0.f;
  for (int j = lane; j < a.top_k; j += 32) probs[j] = probs[j] * f * a.scale;   // this lane's own
}

// PER: experts per lane (E <= 32 * PER).
template <typename T, int PER>
__global__ void __launch_bounds__(RT_WARPS * 32, 8) route_kernel(const __grid_constant__ RouteArgs a, int warp_bytes) {
  extern __shared__ __align__(16) uint8_t smem[];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  uint8_t* base = smem + warp * warp_bytes;
  double* kd = reinterpret_cast<double*>(base);    // keys (fp64 only if needed; fp32 ones for the groups)
  double* gd = kd + a.E;                           // group scores
  int* ids = reinterpret_cast<int*>(gd + a.n_groups);
  int* list = ids + a.top_k;                       // of 32: experts between which a decision is close
  pdl_enter();
  const int64_t t = static_cast<int64_t>(blockIdx.x) * RT_WARPS + warp;
  if (t >= a.T) return;  // no block-wide barrier below

  const T* row = static_cast<const T*>(a.logits) + t * a.ld;
  const bool softmax = a.score == KQ_SCORE_SOFTMAX, groups = a.topk_groups < a.n_groups;
  const bool by_score = a.bias || (groups && a.group_top == 2);   // else by the logits, in the scores' order
  float key[PER];   // the logits at first
#pragma unroll
  for (int i = 0; i < PER; ++i) key[i] = lane + 32 * i < a.E ? logit(row, lane + 32 * i) : -INFINITY;
  float mx = 0.f, inv = 1.f;
  if (softmax) {
    mx = key[0];
#pragma unroll
    for (int i = 1; i < PER; ++i) mx = fmaxf(mx, key[i]);
    mx = warp_max(mx);
    if (mx == -INFINITY) mx = 0.f;   // no expert is available
    if (a.bias || !a.renorm) {   // without a bias the common factor 1 / Sum changes no order
      float sum = 0.f;
#pragma unroll
      for (int i = 0; i < PER; ++i) sum += fast_exp(key[i] - mx);
      sum = warp_sum_f(sum);
      inv = sum > 0.f ? __fdiv_rn(1.0f, sum) : 1.f;
    }
  }
  const float kinv = a.bias ? inv : 1.f;
  if (by_score) {
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      const float b = a.bias && lane + 32 * i < a.E ? a.bias[lane + 32 * i] : 0.f;
      const float k = (softmax ? fast_exp(key[i] - mx) * kinv : fast_rcp(1.0f + fast_exp(-key[i]))) + b;
      key[i] = key[i] == -INFINITY ? -INFINITY : fmaxf(k, -INFINITY);   // a NaN is -inf
    }
  }
  // What two fp32 keys can be apart and still be in the wrong order: tol + 2^-22 of the
  // key. An e^-x <= 1 is off by 2^-22 + 0.37 * 1.5 * 2^-24. A softmax score is off by that,
  // by the sum's own error (2^-22 and, as the scores' mean x is at most ln 512, 9.4 * 2^-24;
  // E / 32 + 5 roundings of 2^-24) and by three roundings: under 2^-18 of the largest
  // score, which is 1 / Sum (without a bias the scores are compared as e^-x: 2^-21). A sigmoid
  // s is off by s (1 - s) times its exponential's error and by two roundings of 2^-23: under
  // 2^-21 of 1. Adding the bias rounds by 2^-24 of the key.
  const bool near = by_score && a.bias;   // else the experts go by the exact logits
  const float tol = 2.f * (softmax && a.bias ? inv * 3.8147e-6f : 4.7684e-7f);

  bool clear = true;
  if (groups) {
    // Keys by group, the groups an odd number of words apart: lanes that read the same
    // place of different groups meet different banks.
    float* kf = reinterpret_cast<float*>(kd);
    float* gf = reinterpret_cast<float*>(gd);
    float* in = gf + a.n_groups;
    const int per = static_cast<int>(a.per), pitch = per | 1;
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      const int e = lane + 32 * i;
      if (e < a.E) kf[e + static_cast<int>((e * a.recip) >> 20) * (pitch - per)] = key[i];
    }
    __syncwarp();
    // 2^sl lanes share a group, each with every 2^sl-th expert of it.
    int sl = 0;
    while (sl < 5 && (a.n_groups << (sl + 1)) <= 32) ++sl;
    const int step = 1 << sl, sub = lane & (step - 1);
    // Scores of two keys are held halved: their sum can pass fp32's range (keys next to its end by
    // their bias).
    const float half = a.group_top == 2 ? 0.5f : 1.f;
    float mag = 0.f;   // of the keys in the scores
    for (int g0 = 0; g0 < a.n_groups; g0 += 32 >> sl) {
      const int g = g0 + (lane >> sl);
      float m1 = -INFINITY, m2 = -INFINITY;
      if (g < a.n_groups) {
        const float* k = kf + g * pitch;
#pragma unroll 4
        for (int j = sub; j < per; j += step) {
          const float v = k[j];
          m2 = fmaxf(m2, fminf(m1, v));
          m1 = fmaxf(m1, v);
        }
      }
      for (int o = 1; o < step; o <<= 1) {
        const float x1 = __shfl_xor_sync(FULL, m1, o), x2 = __shfl_xor_sync(FULL, m2, o);
        m2 = fmaxf(fmaxf(m2, x2), fminf(m1, x1));
        m1 = fmaxf(m1, x1);
      }
      if (g < a.n_groups && sub == 0) {
        const bool two = a.group_top == 2 && m2 != -INFINITY;
        gf[g] = two ? half * m1 + half * m2 : half * m1;
        const float x = half * fabsf(m1) + (two ? half * fabsf(m2) : 0.f);
        if (x < INFINITY) mag = fmaxf(mag, x);
      }
    }
    __syncwarp();
    // A group stays if fewer than topk_groups others are before it.
    float cut_in = INFINITY, cut_out = -INFINITY;
    for (int g = lane; g < a.n_groups; g += 32) {
      const float v = gf[g];
      int before = 0;
      for (int h = 0; h < a.n_groups; ++h) {
        const float w = gf[h];
        before += (w > v || (w == v && h < g)) ? 1 : 0;
      }
      const bool stays = before < a.topk_groups;
      if (stays && v != -INFINITY) cut_in = fminf(cut_in, v);
      if (!stays) cut_out = fmaxf(cut_out, v);
      in[g] = stays ? 1.f : 0.f;
    }
    __syncwarp();
    cut_out = warp_max(cut_out);
    if (cut_out != -INFINITY && by_score) {
      // A group's score is the sum of two keys: twice a key's error, and a rounding.
      const float gtol = 2.f * half * tol + 4.7684e-7f * warp_max(mag);
      cut_in = warp_min(cut_in);
      if (cut_in - cut_out <= gtol) {
        // The groups that could be on either side, and of their experts those that could
        // be among the best group_top.
        float least[PER];
#pragma unroll
        for (int i = 0; i < PER; ++i) least[i] = INFINITY;
        for (int g = 0; g < a.n_groups; ++g) {
          const float v = gf[g];
          if (v == -INFINITY || (in[g] != 0.f ? v > cut_out + gtol : v < cut_in - gtol)) continue;
          float m = -INFINITY;
#pragma unroll
          for (int i = 0; i < PER; ++i) {
            const int e = lane + 32 * i;
            if (e < a.E && static_cast<int>((e * a.recip) >> 20) == g) m = fmaxf(m, key[i]);
          }
          // With group_top 2 the least key that counts is the score (2 v) less the largest key.
          const float top = warp_max(m);
          const float low = a.group_top == 2 ? fminf(v + (v - top), top) - 2.f * gtol : top - gtol;
#pragma unroll
          for (int i = 0; i < PER; ++i) {
            const int e = lane + 32 * i;
            if (e < a.E && static_cast<int>((e * a.recip) >> 20) == g) least[i] = low;
          }
        }
        const int n = compact<PER>([&](int i) { return key[i] != -INFINITY && key[i] >= least[i]; }, list, lane);
        if (n <= 32) {
          const double sum = softmax && a.bias ? exact_sum(row, a.E, mx, lane) : 1.;
          const int e = lane < n ? list[lane] : -1;
          const int g = e >= 0 ? static_cast<int>((e * a.recip) >> 20) : -1;
          const double k = e >= 0 ? exact_key(a, row, e, mx, sum) : 0.;
          double m1 = -INFINITY, m2 = -INFINITY;   // of this lane's group
          for (int c = 0; c < n; ++c) {
            const double v = __shfl_sync(FULL, k, c);
            if (__shfl_sync(FULL, g, c) == g) {
              m2 = v > m1 ? m1 : (v > m2 ? v : m2);
              m1 = v > m1 ? v : m1;
            }
          }
          const double score = (a.group_top == 2 && m2 != -INFINITY) ? m1 + m2 : m1;
          const int g_left = __shfl_up_sync(FULL, g, 1);
          const bool head = e >= 0 && (lane == 0 || g_left != g);   // the list is in order: one lane per group
          const unsigned heads = __ballot_sync(FULL, head);
          // Places for them: all but those of the groups that are surely in.
          unsigned sure = 0;
          for (int h = lane; h < a.n_groups; h += 32) sure += in[h] != 0.f && gf[h] > cut_out + gtol ? 1 : 0;
          sure = __reduce_add_sync(FULL, sure);
          int before = 0;
          for (int c = 0; c < n; ++c) {
            const double v = __shfl_sync(FULL, score, c);
            if ((heads >> c & 1) && (v > score || (v == score && c < lane))) ++before;
          }
          if (head) in[g] = static_cast<int>(sure) + before < a.topk_groups ? 1.f : 0.f;
          __syncwarp();
        } else {
          clear = false;
        }
      }
    }
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      const int e = lane + 32 * i;
      if (e < a.E && in[(e * a.recip) >> 20] == 0.f) key[i] = -INFINITY;
    }
    if (by_score && !a.bias) {
#pragma unroll
      for (int i = 0; i < PER; ++i)
        if (key[i] != -INFINITY) key[i] = logit(row, lane + 32 * i);
    }
  }

  // Top k: each lane keeps its two best keys of those not taken.
  uint32_t taken = 0;
  float b1, b2;
  int e1, e2;
  b1 = b2 = -INFINITY;
  e1 = e2 = 0x7fffffff;
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    const float k = key[i];
    const bool p = k > b1, q = k > b2;
    b2 = p ? b1 : q ? k : b2;
    e2 = p ? e1 : q ? lane + 32 * i : e2;
    b1 = p ? k : b1;
    e1 = p ? lane + 32 * i : e1;
  }
  int held = 2;   // of this lane's best two, not taken yet
  float prev = 0.f;
  int prev_e = -1, found = 0;
  bool close = false;
  const int rounds = near ? a.top_k + 1 : a.top_k;   // the last one only to see how close it is
  for (int j = 0; j < rounds; ++j) {
    const float best = warp_max(b1);
    if (best == -INFINITY) {   // no expert is left
      for (int i = j + lane; i < a.top_k; i += 32) ids[i] = -1;
      break;
    }
    const unsigned mine = b1 == best ? static_cast<unsigned>(e1) : 0x7fffffffu;
    const unsigned e = __reduce_min_sync(FULL, mine);
    if (near) {
      // Two experts with the same logit and the same bias have the same key in
      // any precision: the lower index is first, as it should be.
      if (prev_e >= 0 && prev - best <= fmaf(2.3842e-7f, fabsf(best), tol) &&
          !(logit(row, e) == logit(row, prev_e) && a.bias[e] == a.bias[prev_e]))
        close = true;
      prev_e = static_cast<int>(e);
    }
    if (j == a.top_k) break;
    prev = best;
    ++found;
    if (mine == e) {
      ids[j] = static_cast<int>(e);
      taken |= 1u << (e1 >> 5);
      b1 = b2;
      e1 = e2;
      b2 = -INFINITY;
      --held;
    }
    if (PER > 2 && j + 1 < rounds && __any_sync(FULL, held == 0)) {
      if (held == 0) {   // the best of what is left
        held = 1;
#pragma unroll
        for (int i = 0; i < PER; ++i) {
          const bool p = key[i] > b1 && !(taken >> i & 1);
          b1 = p ? key[i] : b1;
          e1 = p ? lane + 32 * i : e1;
        }
      }
    }
  }
  __syncwarp();
  if (close && clear) {   // warp-uniform
    // The experts that could be among the top k, in the order of their fp64 keys.
    const float low = found == a.top_k ? prev - fmaf(2.3842e-7f, fabsf(prev), tol) : -INFINITY;
    const int n = compact<PER>([&](int i) { return key[i] != -INFINITY && key[i] >= low; }, list, lane);
    if (n <= 32) {
      const double sum = softmax && a.bias ? exact_sum(row, a.E, mx, lane) : 1.;
      const int e = lane < n ? list[lane] : 0;
      const double k = lane < n ? exact_key(a, row, e, mx, sum) : 0.;
      int before = 0;
      for (int c = 0; c < n; ++c) {
        const double v = __shfl_sync(FULL, k, c);
        before += (v > k || (v == k && c < lane)) ? 1 : 0;   // the list is in the order of the indices
      }
      if (lane < n && before < a.top_k) ids[before] = e;
    } else {
      clear = false;
    }
  }
  if (!clear) select_exact(a, row, mx, kd, gd, ids, lane);   // warp-uniform: more than 32 of them
  __syncwarp();
  // Weights, in slot order; slots without an available expert take the
  // lowest-numbered experts not chosen, with weight 0.
  float w = 0.f, tot = 0.f;
  for (int j = lane; j < a.top_k; j += 32) {
    const int e = ids[j];
    w = 0.f;
    if (e >= 0) {
      const float v = logit(row, e);
      w = softmax ? expf(v - mx) * inv : __fdiv_rn(1.0f, 1.0f + expf(-v));
      a.ids[t * a.top_k + j] = e;
    }
    tot += w;
    if (a.top_k > 32 || !a.renorm) a.probs[t * a.top_k + j] = w * (a.renorm ? 1.f : a.scale);
  }
  if (a.renorm) {
    tot = warp_sum_f(tot);
    // The largest of 512 scores that sum to 2^-30 is at least 2^-39, and a score e^-60 = 2^-87 of
    // that still a normal number.
    if (tot >= 0x1p-30f) {
      const float f = __fdiv_rn(1.0f, tot);
      for (int j = lane; j < a.top_k; j += 32) {
        if (a.top_k > 32) w = a.probs[t * a.top_k + j];   // this lane's own
        a.probs[t * a.top_k + j] = w * f * a.scale;
      }
    } else {
      weights_of_tiny_scores<T>(a, t, ids);
    }
  }
  const bool empty = ids[a.top_k - 1] < 0;
  __syncwarp();
  if (empty && lane == 0) {  // rare: fewer experts than slots
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

template <typename T>
void (*route_for(int E))(RouteArgs, int) {
  return E <= 32    ? route_kernel<T, 1>
         : E <= 128 ? route_kernel<T, 4>
         : E <= 256 ? route_kernel<T, 8>
         : E <= 384 ? route_kernel<T, 12>
                    : route_kernel<T, 16>;
}

}  // namespace

cudaError_t launch_moe_route(int dtype, const void* logits, int64_t ld, const float* bias, int score, int n_groups,
                             int topk_groups, int group_top, int top_k, bool renorm, float scale, int* ids, float* probs,
                             int E, int64_t T, cudaStream_t s) {
  const uint32_t per = static_cast<uint32_t>(E / n_groups);
  RouteArgs a{per, ((1u << 20) + per - 1) / per, logits, ld, bias, score, n_groups, topk_groups, group_top, top_k, renorm, scale, ids, probs, E, T};
  const int warp_bytes = (8 * E + 8 * n_groups + 4 * top_k + 128 + 15) / 16 * 16;
  const size_t smem = static_cast<size_t>(RT_WARPS) * warp_bytes;   // at most 40 KB
  auto k = dtype == KQ_F32 ? route_for<float>(E) : dtype == KQ_F16 ? route_for<__half>(E) : route_for<__nv_bfloat16>(E);
  return launch_pdl(k, dim3(static_cast<unsigned>((T + RT_WARPS - 1) / RT_WARPS)), dim3(RT_WARPS * 32), smem, s, a,
                    warp_bytes);
}

}  // namespace kq
