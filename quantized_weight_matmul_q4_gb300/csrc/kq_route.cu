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
// waiting for such a row: 8192 x 384 in 12 groups took 58 us.) Bound by the latency of one token's chain of decisions, and by issue
// for many tokens: a lane keeps its two best experts, so that a round costs two
// warp reductions and a rescan is rare.
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
  const uint32_t b = __float_as_uint(v + 0.f);   // -0 and 0 are one key
  if (b == 0xff800000u) return 0;
  return (b & 0x80000000u) ? ~b : (b | 0x80000000u);
}
__device__ __forceinline__ float from_ord(uint32_t o) {
  return __uint_as_float(o == 0 ? 0xff800000u : (o & 0x80000000u) ? (o & 0x7fffffffu) : ~o);
}
__device__ __forceinline__ uint64_t ord(double v) {
  const uint64_t b = static_cast<uint64_t>(__double_as_longlong(v + 0.));
  if (b == 0xfff0000000000000ull) return 0;
  return (b >> 63) ? ~b : (b | 0x8000000000000000ull);
}
__device__ __forceinline__ uint32_t warp_max(uint32_t v) { return __reduce_max_sync(FULL, v); }
__device__ __forceinline__ uint64_t warp_max(uint64_t v) {
  const uint32_t hi = __reduce_max_sync(FULL, static_cast<uint32_t>(v >> 32));
  const uint32_t lo = __reduce_max_sync(FULL, static_cast<uint32_t>(v >> 32) == hi ? static_cast<uint32_t>(v) : 0u);
  return (static_cast<uint64_t>(hi) << 32) | lo;
}
__device__ __forceinline__ float warp_max_f(float v) { return from_ord(warp_max(ord(v))); }

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
    const int per = a.E / a.n_groups;
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
  for (int e = lane; e < E; e += 32) {
    const float l = logit(row, e);
    if (l != -INFINITY) sum += exp(static_cast<double>(l) - static_cast<double>(mx));
  }
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
    mx = warp_max_f(mx);
    if (by_score || !a.renorm) {
      float sum = 0.f;
#pragma unroll
      for (int i = 0; i < PER; ++i) sum += key[i] == -INFINITY ? 0.f : __expf(key[i] - mx);
      sum = warp_sum_f(sum);
      inv = sum > 0.f ? __fdiv_rn(1.0f, sum) : 1.f;
    }
  }
  float bmax = 0.f;
  if (by_score) {
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      const float b = a.bias && lane + 32 * i < a.E ? __ldg(a.bias + lane + 32 * i) : 0.f;
      const float k = (softmax ? __expf(key[i] - mx) * inv : __fdividef(1.0f, 1.0f + __expf(-key[i]))) + b;
      key[i] = (key[i] == -INFINITY || k != k) ? -INFINITY : k;
      if (fabsf(b) < INFINITY) bmax = fmaxf(bmax, fabsf(b));
    }
  }
  // What two fp32 keys can be apart and still be in the wrong order. __expf(-x) is
  // off by (2 + 1.173 x) ulp, so e^-x by 2.5 ulp of 1 at most. A softmax score is off
  // by that, by the sum's own error (the scores' mean x is at most ln 512: 9.4 ulp, and
  // E / 32 + 5 roundings) and by three roundings: under 2^-18 of the largest score,
  // which is 1 / Sum. A sigmoid is off by a quarter of 2 + 1.173 ulp and a division of
  // 2 ulp: under 2^-20 of 1. Adding the bias rounds once more, by 2^-24 of the key.
  float tol = -1.f;
  if (by_score) {
    const float smax = softmax ? inv : 1.0f;
    tol = 2.f * (smax * (softmax ? 3.8147e-6f : 9.5368e-7f) + 5.9605e-8f * (smax + warp_max_f(bmax)));
  }

  bool clear = true;
  if (groups) {
    float* kf = reinterpret_cast<float*>(kd);
    float* gf = reinterpret_cast<float*>(gd);
    const int per = a.E / a.n_groups;
#pragma unroll
    for (int i = 0; i < PER; ++i)
      if (lane + 32 * i < a.E) kf[lane + 32 * i] = key[i];
    __syncwarp();
    // 2^sl lanes share a group, each with every 2^sl-th expert of it; a lane starts where
    // its group's number says, so that groups of 32 do not meet in one bank.
    int sl = 0;
    while (sl < 5 && (a.n_groups << (sl + 1)) <= 32) ++sl;
    const int step = 1 << sl, sub = lane & (step - 1);
    for (int g0 = 0; g0 < a.n_groups; g0 += 32 >> sl) {
      const int g = g0 + (lane >> sl);
      float m1 = -INFINITY, m2 = -INFINITY;
      if (g < a.n_groups) {
        const int n = (per - sub + step - 1) >> sl;   // this lane's experts
        int j = n > 0 ? g % n : 0;
        for (int i = 0; i < n; ++i) {
          const float v = kf[g * per + sub + (j << sl)];
          j = j + 1 == n ? 0 : j + 1;
          m2 = fmaxf(m2, fminf(m1, v));
          m1 = fmaxf(m1, v);
        }
      }
      for (int o = 1; o < step; o <<= 1) {
        const float x1 = __shfl_xor_sync(FULL, m1, o), x2 = __shfl_xor_sync(FULL, m2, o);
        m2 = fmaxf(fmaxf(m2, x2), fminf(m1, x1));
        m1 = fmaxf(m1, x1);
      }
      if (g < a.n_groups && sub == 0) gf[g] = (a.group_top == 2 && m2 != -INFINITY) ? m1 + m2 : m1;
    }
    __syncwarp();
    // A group stays if fewer than topk_groups others are before it.
    uint32_t worst_in = 0xffffffffu, best_out = 0;
    for (int g = lane; g < a.n_groups; g += 32) {
      const float v = gf[g];
      int before = 0;
      for (int h = 0; h < a.n_groups; ++h) {
        const float w = gf[h];
        before += (w > v || (w == v && h < g)) ? 1 : 0;
      }
      const bool in = before < a.topk_groups;
      const uint32_t o = ord(v);
      if (o != 0) {
        if (in) worst_in = min(worst_in, o); else best_out = max(best_out, o);
      }
      kf[g] = in ? 1.f : 0.f;   // the keys are in registers: their place is free
    }
    __syncwarp();
    best_out = warp_max(best_out);
    const uint32_t recip = ((1u << 20) + per - 1) / per;   // e / per = e * recip >> 20, as e * per < 2^20
    if (best_out != 0 && by_score) {
      // A group's score is the sum of two keys: twice a key's error, and a rounding.
      const float cut_in = from_ord(__reduce_min_sync(FULL, worst_in)), cut_out = from_ord(best_out);
      if (cut_in - cut_out <= 4 * tol) {
        // The groups that could be on either side, and of their experts those that could
        // be among the best group_top.
        float least[PER];
#pragma unroll
        for (int i = 0; i < PER; ++i) least[i] = INFINITY;
        for (int g = 0; g < a.n_groups; ++g) {
          const float v = gf[g];
          if (v == -INFINITY || (kf[g] != 0.f ? v > cut_out + 4 * tol : v < cut_in - 4 * tol)) continue;
          uint32_t m = 0;
#pragma unroll
          for (int i = 0; i < PER; ++i) {
            const int e = lane + 32 * i;
            if (e < a.E && static_cast<int>((e * recip) >> 20) == g) m = max(m, ord(key[i]));
          }
          // With group_top 2 the least key that counts is the score less the largest key.
          const float top = from_ord(warp_max(m));
          const float low = (a.group_top == 2 ? fminf(v - top, top) : top) - 2 * tol;
#pragma unroll
          for (int i = 0; i < PER; ++i) {
            const int e = lane + 32 * i;
            if (e < a.E && static_cast<int>((e * recip) >> 20) == g) least[i] = low;
          }
        }
        const int n = compact<PER>([&](int i) { return key[i] != -INFINITY && key[i] >= least[i]; }, list, lane);
        if (n <= 32) {
          const double sum = softmax ? exact_sum(row, a.E, mx, lane) : 1.;
          const int e = lane < n ? list[lane] : -1;
          const int g = e >= 0 ? e / per : -1;
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
          const bool head = e >= 0 && (lane == 0 || list[lane - 1] / per != g);   // the list is in order: one lane per group
          const unsigned heads = __ballot_sync(FULL, head);
          // Places for them: all but those of the groups that are surely in.
          int sure = 0;
          for (int h = lane; h < a.n_groups; h += 32) sure += kf[h] != 0.f && gf[h] > cut_out + 4 * tol ? 1 : 0;
          sure = static_cast<int>(__reduce_add_sync(FULL, static_cast<unsigned>(sure)));
          int before = 0;
          for (int c = 0; c < n; ++c) {
            const double v = __shfl_sync(FULL, score, c);
            if ((heads >> c & 1) && (v > score || (v == score && c < lane))) ++before;
          }
          if (head) kf[g] = sure + before < a.topk_groups ? 1.f : 0.f;
          __syncwarp();
        } else {
          clear = false;
        }
      }
    }
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      const int e = lane + 32 * i;
      if (e < a.E && kf[(e * recip) >> 20] == 0.f) key[i] = -INFINITY;
    }
    if (!a.bias) {
      // Chosen by the logits: nothing is close.
#pragma unroll
      for (int i = 0; i < PER; ++i)
        if (key[i] != -INFINITY) key[i] = logit(row, lane + 32 * i);
      tol = -1.f;
    }
  }

  // Top k: each lane keeps its two best keys of those not taken.
  uint32_t taken = 0, b1, b2;
  int i1, i2;
  auto scan = [&] {
    b1 = b2 = 0;
    i1 = i2 = 0;
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      const uint32_t o = (taken >> i) & 1 ? 0 : ord(key[i]);
      if (o > b1) {
        b2 = b1;
        i2 = i1;
        b1 = o;
        i1 = i;
      } else if (o > b2) {
        b2 = o;
        i2 = i;
      }
    }
  };
  scan();
  int held = 2;   // of this lane's best two, not taken yet
  float prev = 0.f;
  int prev_e = -1, found = 0;
  bool close = false;
  const int rounds = tol >= 0.f ? a.top_k + 1 : a.top_k;   // the last one only to see how close it is
  for (int j = 0; j < rounds; ++j) {
    const uint32_t m = warp_max(b1);
    if (m == 0) {   // no expert is left
      for (int i = j + lane; i < a.top_k; i += 32) ids[i] = -1;
      break;
    }
    const unsigned mine = b1 == m ? static_cast<unsigned>(lane + 32 * i1) : 0x7fffffffu;
    const unsigned e = __reduce_min_sync(FULL, mine);
    const float best = from_ord(m);
    if (prev_e >= 0 && prev - best <= tol) {
      // Two experts with the same logit and the same bias have the same key in
      // any precision: the lower index is first, as it should be.
      if (!(logit(row, e) == logit(row, prev_e) && a.bias[e] == a.bias[prev_e])) close = true;
    }
    if (j == a.top_k) break;
    prev = best;
    prev_e = static_cast<int>(e);
    ++found;
    if (mine == e) {
      ids[j] = static_cast<int>(e);
      taken |= 1u << i1;
      b1 = b2;
      i1 = i2;
      b2 = 0;
      --held;
    }
    if (PER > 1 && __any_sync(FULL, held == 0)) {
      if (held == 0) scan();
      held = held == 0 ? 2 : held;
    }
  }
  __syncwarp();
  if (close && clear) {   // warp-uniform
    // The experts that could be among the top k, in the order of their fp64 keys.
    const float low = found == a.top_k ? prev - tol : -INFINITY;
    const int n = compact<PER>([&](int i) { return key[i] != -INFINITY && key[i] >= low; }, list, lane);
    if (n <= 32) {
      const double sum = softmax ? exact_sum(row, a.E, mx, lane) : 1.;
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
    const float f = tot > 0.f ? __fdiv_rn(1.0f, tot) : 0.f;
    for (int j = lane; j < a.top_k; j += 32) {
      if (a.top_k > 32) w = a.probs[t * a.top_k + j];   // this lane's own
      a.probs[t * a.top_k + j] = w * f * a.scale;
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
  RouteArgs a{logits, ld, bias, score, n_groups, topk_groups, group_top, top_k, renorm, scale, ids, probs, E, T};
  const int warp_bytes = (8 * E + 8 * n_groups + 4 * top_k + 128 + 15) / 16 * 16;
  const size_t smem = static_cast<size_t>(RT_WARPS) * warp_bytes;   // at most 40 KB
  auto k = dtype == KQ_F32 ? route_for<float>(E) : dtype == KQ_F16 ? route_for<__half>(E) : route_for<__nv_bfloat16>(E);
  return launch_pdl(k, dim3(static_cast<unsigned>((T + RT_WARPS - 1) / RT_WARPS)), dim3(RT_WARPS * 32), smem, s, a,
                    warp_bytes);
}

}  // namespace kq
