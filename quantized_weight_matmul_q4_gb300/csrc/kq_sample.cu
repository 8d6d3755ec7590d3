// The next token of each row of logits, for given random numbers.
//
// With a row's tokens in descending order of their logits (ties to the lower index) and weights
// w = exp((l - max l) / T), three prefixes of that order limit the choice: the first top_k tokens,
// the shortest prefix with at least top_p of the weight of those, and the tokens with w >= min_p. The
// shortest of them is kept, and the token is the first, by index, at which the sum of
// the kept weights passes u times their total.
//
// Weights are whole numbers, w * 2^43 to within 2^-30 of their size: sums of them are exact in 64
// bits and the same in any order, so nothing here depends on scheduling, and two sums compare as
// those of the definition do but for that relative error.
#include <cuda_bf16.h>

#include <algorithm>

#include "kq_attn.h"
#include "kq_types.cuh"

namespace kq {
namespace {

constexpr int kThreads = 512;
constexpr int kWarps = kThreads / 32;
constexpr uint64_t kOne = uint64_t(1) << 43;     // the weight of the largest logit

// 2^(31 - j / 64), rounded.
__constant__ uint32_t kPow2[64] = {
    0x80000000u, 0x7e9f0606u, 0x7d41d96eu, 0x7be86fbau, 0x7a92be8bu, 0x7940bb9eu, 0x77f25cceu, 0x76a7980fu,
    0x75606374u, 0x741cb528u, 0x72dc8374u, 0x719fc4b9u, 0x70666f76u, 0x6f307a41u, 0x6dfddbccu, 0x6cce8ae1u,
    0x6ba27e65u, 0x6a79ad56u, 0x69540ec9u, 0x683199edu, 0x6712460bu, 0x65f60a7fu, 0x64dcdec3u, 0x63c6ba64u,
    0x62b39509u, 0x61a3666du, 0x60962665u, 0x5f8bccdbu, 0x5e8451d0u, 0x5d7fad59u, 0x5c7dd7a4u, 0x5b7ec8f2u,
    0x5a82799au, 0x5988e209u, 0x5891fac1u, 0x579dbc57u, 0x56ac1f75u, 0x55bd1cdbu, 0x54d0ad5au, 0x53e6c9dau,
    0x52ff6b55u, 0x521a8ad7u, 0x51382182u, 0x50582888u, 0x4f7a9930u, 0x4e9f6cd4u, 0x4dc69cddu, 0x4cf022cau,
    0x4c1bf829u, 0x4b4a169cu, 0x4a7a77d4u, 0x49ad1598u, 0x48e1e9bau, 0x4818ee22u, 0x47521cc6u, 0x468d6faeu,
    0x45cae0f2u, 0x450a6abbu, 0x444c0740u, 0x438fb0cbu, 0x42d561b4u, 0x421d1462u, 0x4166c34cu, 0x40b268fau};

// The logit as it is used: no NaN (such a token is not available) and no +inf (the largest finite).
__device__ __forceinline__ float usable(float l) { return l != l ? -INFINITY : fminf(l, 3.402823466e38f); }

// Whole numbers in the order of the logits; 0 is below all of them.
__device__ __forceinline__ uint32_t key_of(float l) {
  const uint32_t b = __float_as_uint(l == 0.f ? 0.f : l);      // -0 is 0
  return b ^ (static_cast<uint32_t>(static_cast<int32_t>(b) >> 31) | 0x80000000u);
}
constexpr uint32_t kNone = 0x007fffffu;                        // the key of -inf

// exp((l - M) / T) * 2^43: with x = (M - l) log2(e) / T as e + r, r in [-1/2, 1/2], and r = j / 64 + f,
// it is 2^(43 - e) 2^(-j / 64) (1 + q), q = 2^-f - 1 by its series (|f| <= 1/128: |q| < 0.0055, so that the
// rounding of q to fp32 and to 2^-31 leaves an error below 2^-30 with that of the table).
struct Weigh {
  float M, ch, cl;                 // log2(e) / T as a sum of two
  const uint32_t* table;           // kPow2 in shared memory

  __device__ __forceinline__ void set(float max, double T, const uint32_t* t) {
    M = max;
    const double c = 1.4426950408889634 / T;
    ch = static_cast<float>(c);
    cl = ch < INFINITY ? static_cast<float>(c - static_cast<double>(ch)) : 0.f;
    table = t;
  }
  __device__ __forceinline__ uint64_t operator()(float l) const {
    const float dh = __fsub_rn(M, l);                          // M - l as dh + dl, exactly
    if (dh == 0.f) return kOne;
    const float b = __fsub_rn(M, dh), dl = __fadd_rn(__fsub_rn(M, __fadd_rn(dh, b)), __fsub_rn(b, l));
    const float xh = __fmul_rn(dh, ch);
    if (!(xh < 64.f)) return 0;
    const float xl = __fmaf_rn(dl, ch, __fmaf_rn(dh, cl, __fmaf_rn(dh, ch, -xh)));
    const float e = rintf(xh), rh = __fsub_rn(xh, e), r = __fadd_rn(rh, xl), rl = __fsub_rn(xl, __fsub_rn(r, rh));
    const float j = floorf(__fmaf_rn(r, 64.f, 0.5f));
    const float f = __fadd_rn(__fmaf_rn(j, -0.015625f, r), rl);
    const float t = f * -0.69314718f;
    // f * ln 2 to the last bit of its product: the rest of -f ln 2 beyond t, then t^2 / 2 + t^3 / 6 + t^4 / 24.
    const float rest = __fmaf_rn(f, -0.69314718f, -t) + f * 1.904654e-9f;
    const float q = t + (rest + t * t * __fmaf_rn(t, __fmaf_rn(t, 0.041666667f, 0.16666667f), 0.5f));
    const int ji = static_cast<int>(j);
    const int shift = 19 + static_cast<int>(e) + (ji >> 6);     // j may be negative: 2^(-j / 64) = 2^-(j >> 6) 2^-((j & 63) / 64)
    const uint64_t p = static_cast<uint64_t>(table[ji & 63]) * static_cast<uint32_t>(0x80000000u + __float2int_rn(q * 2147483648.f));
    return shift >= 64 ? 0 : p >> shift;
  }
};

template <typename V>
__device__ __forceinline__ V block_all(V v, V* part, bool largest) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    const V w = __shfl_xor_sync(0xffffffffu, v, o);
    v = largest ? max(v, w) : v + w;
  }
  __syncthreads();
  if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = v;
  __syncthreads();
  v = part[0];
#pragma unroll
  for (int i = 1; i < kWarps; ++i) v = largest ? max(v, part[i]) : v + part[i];
  return v;
}

// A row per CTA, read again for every step: thresholds by bisection over the keys.
template <typename T>
__global__ void __launch_bounds__(kThreads) sample_rows_kernel(const SampleArgs a) {
  __shared__ uint32_t table[64];
  __shared__ uint64_t part[kWarps];
  __shared__ uint64_t sums[kThreads + 1];
  __shared__ uint32_t ties[kThreads + 1];
  pdl_enter();
  if (threadIdx.x < 64) table[threadIdx.x] = kPow2[threadIdx.x];
  const int64_t n = blockIdx.x;
  const T* x = static_cast<const T*>(a.logits) + n * a.ld;
  const int V = static_cast<int>(a.V);
  auto at = [&](int i) { return usable(to_f32(x[i])); };
  auto sum = [&](auto f) {
    uint64_t s = 0;
    for (int i = threadIdx.x; i < V; i += kThreads) s += f(at(i));
    return block_all<uint64_t>(s, part, false);
  };
  uint32_t top = kNone;
  for (int i = threadIdx.x; i < V; i += kThreads) top = max(top, key_of(at(i)));
  top = block_all<uint32_t>(top, reinterpret_cast<uint32_t*>(part), true);
  if (top == kNone) {
    if (threadIdx.x == 0) {
      a.ids[n] = 0;
      if (a.probs) a.probs[n] = 0.f;
    }
    return;
  }
  float M = -INFINITY;
  M = __uint_as_float(top & 0x80000000u ? top ^ 0x80000000u : ~top);
  const float T0 = a.temperature ? a.temperature[n] : 1.f;
  const bool greedy = !(T0 > 0.f);
  Weigh w;
  w.set(M, greedy ? 1.0 : static_cast<double>(T0), table);
  // Kept: keys above `key`, and the first `extra` tokens, by index, of those with that key.
  uint32_t key = kNone + 1, extra = 0xffffffffu;
  if (greedy) {
    key = top;
    extra = 1;
  } else {
    const int k = a.top_k ? a.top_k[n] : 0;
    if (k > 0 && k < V) {
      uint32_t lo = kNone + 1, hi = top;      // the largest key that k tokens reach
      while (lo < hi) {
        const uint32_t mid = lo + (hi - lo + 1) / 2;
        if (sum([&](float l) { return static_cast<uint64_t>(key_of(l) >= mid); }) >= static_cast<uint64_t>(k)) lo = mid;
        else hi = mid - 1;
      }
      const uint64_t above = sum([&](float l) { return static_cast<uint64_t>(key_of(l) > lo); });
      key = lo;
      extra = static_cast<uint32_t>(k - above);
    }
    const float p = a.top_p ? a.top_p[n] : 1.f;
    if (p < 1.f) {
      const uint64_t wk = w(__uint_as_float(key & 0x80000000u ? key ^ 0x80000000u : ~key));
      const uint64_t same = sum([&](float l) { return static_cast<uint64_t>(key_of(l) == key); });
      const uint64_t some = min(same, static_cast<uint64_t>(extra));
      const uint64_t all = sum([&](float l) { return key_of(l) > key ? w(l) : 0; }) + some * wk;
      const double goal = static_cast<double>(p) * static_cast<double>(all);
      uint32_t lo = key, hi = top;            // the largest key whose prefix has that weight
      while (lo < hi) {
        const uint32_t mid = lo + (hi - lo + 1) / 2;
        const uint64_t s = sum([&](float l) { return key_of(l) >= mid ? w(l) : 0; });
        if (static_cast<double>(s) >= goal) lo = mid;
        else hi = mid - 1;
      }
      const uint64_t above = sum([&](float l) { return key_of(l) > lo ? w(l) : 0; });
      const uint64_t one = w(__uint_as_float(lo & 0x80000000u ? lo ^ 0x80000000u : ~lo));
      // Of the tokens with that key: the fewest that bring the sum to the goal, one at least.
      uint64_t c = 1;
      if (one > 0) {
        const double need = (goal - static_cast<double>(above)) / static_cast<double>(one);
        c = need > 1.0 ? static_cast<uint64_t>(ceil(need)) : 1;
      }
      extra = static_cast<uint32_t>(min(c, static_cast<uint64_t>(lo == key ? extra : 0xffffffffu)));
      key = lo;
    }
  }
  const float mp = a.min_p && !greedy ? a.min_p[n] : 0.f;
  const double least = mp > 0.f ? fmin(static_cast<double>(mp), 1.0) * static_cast<double>(kOne) : 0.0;
  // The kept weights by index: a run of tokens for each thread.
  const int run = (V + kThreads - 1) / kThreads, i0 = min(V, static_cast<int>(threadIdx.x) * run), i1 = min(V, i0 + run);
  uint32_t same = 0;
  for (int i = i0; i < i1; ++i) same += key_of(at(i)) == key;
  ties[threadIdx.x + 1] = same;
  __syncthreads();
  if (threadIdx.x == 0) {
    ties[0] = 0;
    for (int i = 0; i < kThreads; ++i) ties[i + 1] += ties[i];
  }
  __syncthreads();
  auto kept = [&](float l, uint32_t& seen) -> uint64_t {
    const uint32_t k = key_of(l);
    if (k < key || (k == key && seen++ >= extra)) return 0;
    const uint64_t v = greedy ? kOne : w(l);
    return static_cast<double>(v) >= least ? v : 0;
  };
  uint64_t mine = 0;
  uint32_t seen = ties[threadIdx.x];
  for (int i = i0; i < i1; ++i) mine += kept(at(i), seen);
  sums[threadIdx.x + 1] = mine;
  __syncthreads();
  if (threadIdx.x == 0) {
    sums[0] = 0;
    for (int i = 0; i < kThreads; ++i) sums[i + 1] += sums[i];
  }
  __syncthreads();
  const uint64_t total = sums[kThreads];
  const float u = a.u[n];
  // The first sum above u * total: at least floor(u * total) + 1, and at most all of it.
  uint64_t goal = u > 0.f ? static_cast<uint64_t>(static_cast<double>(u) * static_cast<double>(total)) : 0;
  goal = min(goal, total - 1);
  if (sums[threadIdx.x] <= goal && goal < sums[threadIdx.x + 1]) {
    uint64_t c = sums[threadIdx.x];
    seen = ties[threadIdx.x];
    for (int i = i0; i < i1; ++i) {
      const uint64_t v = kept(at(i), seen);
      c += v;
      if (c > goal) {
        a.ids[n] = i;
        if (a.probs) a.probs[n] = static_cast<float>(static_cast<double>(v) / static_cast<double>(total));
        break;
      }
    }
  }
}

}  // namespace

cudaError_t launch_sample(int dtype, const SampleArgs& a, int, cudaStream_t s) {
  const dim3 grid(static_cast<unsigned>(a.N)), block(kThreads);
  if (dtype == KQ_F16) return launch_pdl(sample_rows_kernel<__half>, grid, block, 0, s, a);
  if (dtype == KQ_BF16) return launch_pdl(sample_rows_kernel<__nv_bfloat16>, grid, block, 0, s, a);
  return launch_pdl(sample_rows_kernel<float>, grid, block, 0, s, a);
}

}  // namespace kq
