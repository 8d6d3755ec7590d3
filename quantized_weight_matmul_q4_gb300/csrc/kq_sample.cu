// The next token of each row of logits, for given random numbers.
//
// With a row's tokens in descending order of their logits (ties to the lower index) and weights
// w = exp((l - max l) / T), three prefixes of that order limit the choice: the first top_k tokens,
// the shortest prefix with at least top_p of the weight of those, and the tokens with w >= min_p. The
// shortest of them is kept, and the token is the first, by index, at which the sum of
// the kept weights passes u times their total.
//
// A row is held in the shared memory of a cluster of CTAs. Where top_k or top_p limit it, a histogram over bins of (max l - l) / T
// of 1/16 of an octave finds the bin that the limit falls into; the tokens that may be kept, if they are
// few, then go to one CTA, else the cluster goes on. The limit itself is found by histograms of ever
// finer runs of the logits' bits, until one value is left; of its equals the first by index are kept.
//
// Weights are whole numbers, w * 2^43 to within 2^-30 of their size: sums of them are exact in 64
// bits and the same in any order, so nothing here depends on scheduling, and two sums compare as
// those of the definition do but for that relative error.
//
// What bounds it (one GB300, in a graph): one row (152064 logits, all limits: 23.5 us) the chain of steps between barriers of
// the cluster, about twenty of them at 0.5 to 1 us. Many rows of top_p alone (64 of 152064 of 16 bits: 119 us, 0.02 of the copy bandwidth)
// the issue of instructions on the SMs that have two CTAs: a token's weight takes 33, its bin and the histogram's addition
// about 20, and the limit's and the choice's passes take the kept tokens' weights again. With top_k (47 us) only the
// tokens of the list have weights; with min_p alone (29 us) those that it leaves.
#include <cuda_bf16.h>

#include <algorithm>
#include <atomic>
#include <type_traits>

#include "kq_attn.h"
#include "kq_types.cuh"

namespace kq {
namespace {

constexpr int kThreads = 512;
constexpr int kWarps = kThreads / 32;
constexpr int kBins = 1024, kPerThread = kBins / kThreads;      // 64 octaves: later ones weigh nothing
constexpr int kList = 2048;                      // tokens that one CTA takes over (64 rows with top-k and top-p: 47.2 us, with 1024
                                                 // 49.8, with 4096, which leave one CTA on an SM, 62.9)
constexpr int kMostCtas = 16;
constexpr int kSliceBytes = 128 * 1024;
constexpr uint64_t kOne = uint64_t(1) << 43;     // the weight of the largest logit

// 2^(31 - j / 256), rounded.
__constant__ uint32_t kPow2[256] = {
    0x80000000u, 0x7fa765adu, 0x7f4f08aeu, 0x7ef6e8dau, 0x7e9f0606u, 0x7e476009u, 0x7deff6b6u, 0x7d98c9e6u, 0x7d41d96eu, 0x7ceb2523u,
    0x7c94acdeu, 0x7c3e7073u, 0x7be86fbau, 0x7b92aa88u, 0x7b3d20b6u, 0x7ae7d21au, 0x7a92be8bu, 0x7a3de5dfu, 0x79e947efu, 0x7994e492u,
    0x7940bb9eu, 0x78ecccecu, 0x78991854u, 0x78459dacu, 0x77f25cceu, 0x779f5590u, 0x774c87ccu, 0x76f9f359u, 0x76a7980fu, 0x765575c8u,
    0x76038c5bu, 0x75b1dba2u, 0x75606374u, 0x750f23abu, 0x74be1c20u, 0x746d4cacu, 0x741cb528u, 0x73cc556du, 0x737c2d55u, 0x732c3cbau,
    0x72dc8374u, 0x728d015du, 0x723db650u, 0x71eea226u, 0x719fc4b9u, 0x71511de4u, 0x7102ad80u, 0x70b47368u, 0x70666f76u, 0x7018a185u,
    0x6fcb096fu, 0x6f7da710u, 0x6f307a41u, 0x6ee382deu, 0x6e96c0c3u, 0x6e4a33c9u, 0x6dfddbccu, 0x6db1b8a8u, 0x6d65ca38u, 0x6d1a1057u,
    0x6cce8ae1u, 0x6c8339b2u, 0x6c381ca6u, 0x6bed3399u, 0x6ba27e65u, 0x6b57fce9u, 0x6b0daeffu, 0x6ac39485u, 0x6a79ad56u, 0x6a2ff94fu,
    0x69e6784du, 0x699d2a2cu, 0x69540ec9u, 0x690b2601u, 0x68c26fb1u, 0x6879ebb6u, 0x683199edu, 0x67e97a34u, 0x67a18c68u, 0x6759d065u,
    0x6712460bu, 0x66caed35u, 0x6683c5c3u, 0x663ccf92u, 0x65f60a7fu, 0x65af766au, 0x6569132fu, 0x6522e0adu, 0x64dcdec3u, 0x64970d4fu,
    0x64516c2eu, 0x640bfb41u, 0x63c6ba64u, 0x6381a978u, 0x633cc85bu, 0x62f816ebu, 0x62b39509u, 0x626f4292u, 0x622b1f66u, 0x61e72b65u,
    0x61a3666du, 0x615fd05eu, 0x611c6919u, 0x60d9307bu, 0x60962665u, 0x60534ab7u, 0x60109d51u, 0x5fce1e12u, 0x5f8bccdbu, 0x5f49a98cu,
    0x5f07b405u, 0x5ec5ec26u, 0x5e8451d0u, 0x5e42e4e3u, 0x5e01a53fu, 0x5dc092c7u, 0x5d7fad59u, 0x5d3ef4d7u, 0x5cfe6923u, 0x5cbe0a1cu,
    0x5c7dd7a4u, 0x5c3dd19cu, 0x5bfdf7e5u, 0x5bbe4a61u, 0x5b7ec8f2u, 0x5b3f7377u, 0x5b0049d4u, 0x5ac14beau, 0x5a82799au, 0x5a43d2c6u,
    0x5a055751u, 0x59c7071cu, 0x5988e209u, 0x594ae7fbu, 0x590d18d3u, 0x58cf7474u, 0x5891fac1u, 0x5854ab9bu, 0x581786e6u, 0x57da8c83u,
    0x579dbc57u, 0x57611642u, 0x57249a29u, 0x56e847efu, 0x56ac1f75u, 0x567020a0u, 0x56344b52u, 0x55f89f70u, 0x55bd1cdbu, 0x5581c378u,
    0x55469329u, 0x550b8bd4u, 0x54d0ad5au, 0x5495f7a1u, 0x545b6a8bu, 0x542105fdu, 0x53e6c9dau, 0x53acb607u, 0x5372ca68u, 0x533906e0u,
    0x52ff6b55u, 0x52c5f7aau, 0x528cabc3u, 0x52538786u, 0x521a8ad7u, 0x51e1b59au, 0x51a907b4u, 0x5170810bu, 0x51382182u, 0x50ffe8feu,
    0x50c7d765u, 0x508fec9cu, 0x50582888u, 0x50208b0eu, 0x4fe91413u, 0x4fb1c37cu, 0x4f7a9930u, 0x4f439514u, 0x4f0cb70cu, 0x4ed5ff00u,
    0x4e9f6cd4u, 0x4e69006eu, 0x4e32b9b4u, 0x4dfc988cu, 0x4dc69cddu, 0x4d90c68bu, 0x4d5b157eu, 0x4d25899cu, 0x4cf022cau, 0x4cbae0efu,
    0x4c85c3f1u, 0x4c50cbb8u, 0x4c1bf829u, 0x4be7492bu, 0x4bb2bea5u, 0x4b7e587eu, 0x4b4a169cu, 0x4b15f8e6u, 0x4ae1ff43u, 0x4aae299bu,
    0x4a7a77d4u, 0x4a46e9d6u, 0x4a137f88u, 0x49e038d0u, 0x49ad1598u, 0x497a15c4u, 0x4947393fu, 0x49147feeu, 0x48e1e9bau, 0x48af768au,
    0x487d2646u, 0x484af8d6u, 0x4818ee22u, 0x47e70611u, 0x47b5408cu, 0x47839d7bu, 0x47521cc6u, 0x4720be55u, 0x46ef8210u, 0x46be67e0u,
    0x468d6faeu, 0x465c9961u, 0x462be4e2u, 0x45fb521au, 0x45cae0f2u, 0x459a9152u, 0x456a6323u, 0x453a564du, 0x450a6abbu, 0x44daa054u,
    0x44aaf702u, 0x447b6eadu, 0x444c0740u, 0x441cc0a3u, 0x43ed9ac0u, 0x43be957fu, 0x438fb0cbu, 0x4360ec8du, 0x433248aeu, 0x4303c518u,
    0x42d561b4u, 0x42a71e6cu, 0x4278fb2bu, 0x424af7dau, 0x421d1462u, 0x41ef50aeu, 0x41c1aca7u, 0x41942839u, 0x4166c34cu, 0x41397dccu,
    0x410c57a2u, 0x40df50b8u, 0x40b268fau, 0x4085a051u, 0x4058f6a8u, 0x402c6be9u};

// The logit as it is used: no NaN (such a token is not available: -inf in its place) and no +inf (the largest finite).
__device__ __forceinline__ float usable(float l) { return fminf(l, 3.402823466e38f); }
template <typename T>
__device__ __forceinline__ float take(T& v) {
  const float l = to_f32(v);
  if (l != l) {
    v = from_f32<T>(-INFINITY);
    return -INFINITY;
  }
  return usable(l);
}

// Whole numbers in the order of the logits; 0 is below all of them.
__device__ __forceinline__ uint32_t key_of(float l) {
  const uint32_t b = __float_as_uint(l == 0.f ? 0.f : l);      // -0 is 0
  return b ^ (static_cast<uint32_t>(static_cast<int32_t>(b) >> 31) | 0x80000000u);
}
constexpr uint32_t kNone = 0x007fffffu;                        // the key of -inf
constexpr uint32_t kAll = 0xffffffffu;

// Adding it to an fp32 below 2^22 in magnitude rounds that to a whole number, which the sum has in its low bits.
constexpr float kWhole = 12582912.f;
constexpr int kWholeBits = 0x4b400000;

// exp((l - M) / T) * 2^43: with x = (M - l) log2(e) / T as k / 256 + f, |f| little above 1/512, it is
// 2^(43 - (k >> 8)) 2^(-(k & 255) / 256) (1 + q), q = 2^-f - 1 by its series (|q| < 0.00137: fp32's rounding of f and of the series
// is below 2^-33, that of q and of the table to 2^-31 below 2^-31 of the weight: in all below 2^-30).
struct Weigh {
  float M, ch, cl;                 // log2(e) / T as a sum of two
  const uint32_t* table;           // kPow2 in shared memory

  __device__ __forceinline__ uint64_t operator()(float l) const {
    const float dh = __fsub_rn(M, l);                          // M - l as dh + dl, exactly
    const float b = __fsub_rn(M, dh), dl = __fadd_rn(__fsub_rn(M, __fadd_rn(dh, b)), __fsub_rn(b, l));
    const float xh = __fmul_rn(dh, ch);
    const float xl = __fmaf_rn(dl, ch, __fmaf_rn(dh, cl, __fmaf_rn(dh, ch, -xh)));
    const float tk = __fmaf_rn(xh, 256.f, kWhole), k = __fsub_rn(tk, kWhole);
    const float f = __fadd_rn(__fmaf_rn(k, -0.00390625f, xh), xl);            // (the difference without xl is exact)
    const float t = f * -0.69314718f, q = __fmaf_rn(t * t, __fmaf_rn(t, 0.16666667f, 0.5f), t);
    const int ki = __float_as_int(tk) - kWholeBits;
    const uint32_t u = 0x80000000u + static_cast<uint32_t>(__float_as_int(__fmaf_rn(q, 2147483648.f, kWhole)) - kWholeBits);
    const uint64_t w = static_cast<uint64_t>(table[ki & 255]) * u;
    uint64_t v;
    asm("shr.b64 %0, %1, %2;" : "=l"(v) : "l"(w), "r"(19 + (ki >> 8)));       // (0 beyond 63)
    return xh < 64.f ? v : dh == 0.f ? kOne : 0;               // (0 times an infinite 1 / T is a NaN)
  }
};

__device__ __forceinline__ float exp2_fast(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}

__device__ __forceinline__ float value_of(uint32_t key) {
  return __uint_as_float(key & 0x80000000u ? key ^ 0x80000000u : ~key);
}

__device__ __forceinline__ uint64_t load_cluster(uint32_t addr) {
  uint64_t v;
  asm volatile("ld.shared::cluster.u64 %0, [%1];" : "=l"(v) : "r"(addr) : "memory");
  return v;
}
__device__ __forceinline__ void store_cluster(uint32_t addr, uint64_t v) {
  asm volatile("st.shared::cluster.u64 [%0], %1;" ::"r"(addr), "l"(v) : "memory");
}

// What the CTAs that work on a row share: the row's cluster, or (ctas = 1) one CTA.
struct Team {
  int ctas, rank;
  uint64_t* slots;           // [2]: what this CTA tells the others, in turn; [2], [3]: and with its histogram; [4], [5]: what
                             // the others may still be reading when it tells the next
  uint64_t* part;            // [2 * kWarps]
  uint64_t* hist;            // [kBins], this CTA's
  uint64_t* all;             // [kBins], the team's
  int turn;

  __device__ __forceinline__ void sync() const {
    if (ctas > 1) cluster_sync();
    else __syncthreads();
  }

  // The value over the team (and over the CTAs before this one, for sums), from each thread's.
  template <typename Op>
  __device__ __forceinline__ uint64_t reduce(uint64_t v, Op op, uint64_t zero, uint64_t* before = nullptr) {
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v = op(v, __shfl_xor_sync(0xffffffffu, v, o));
    __syncthreads();
    if (lane == 0) part[threadIdx.x >> 5] = v;
    __syncthreads();
    if (threadIdx.x < 32) {
      v = lane < kWarps ? part[lane] : zero;
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) v = op(v, __shfl_xor_sync(0xffffffffu, v, o));
    }
    if (ctas > 1) {
      if (threadIdx.x == 0) slots[turn] = v;
      cluster_sync();
      if (threadIdx.x < 32) {
        v = lane < ctas ? load_cluster(mapa_shared(slots + turn, lane)) : zero;
        uint64_t b = lane < rank ? v : zero;
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) {
          v = op(v, __shfl_xor_sync(0xffffffffu, v, o));
          b = op(b, __shfl_xor_sync(0xffffffffu, b, o));
        }
        if (lane == 0) part[kWarps + 1] = b;
      }
      turn ^= 1;
    } else if (threadIdx.x == 0) {
      part[kWarps + 1] = zero;
    }
    if (threadIdx.x == 0) part[kWarps] = v;
    __syncthreads();
    if (before) *before = part[kWarps + 1];
    return part[kWarps];
  }
  __device__ __forceinline__ uint64_t sum(uint64_t v, uint64_t* before = nullptr) {
    return reduce(v, [](uint64_t a, uint64_t b) { return a + b; }, 0, before);
  }
  __device__ __forceinline__ uint64_t most(uint64_t v) {
    return reduce(v, [](uint64_t a, uint64_t b) { return max(a, b); }, 0);
  }

  // This CTA's sums, told to the others with its next histogram or sync, and the team's once that is done. A word is written
  // again only after a sync that follows its last reading: `to` is where they go.
  __device__ __forceinline__ void tell(uint64_t v, uint64_t w, int to = 2) const {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      v += __shfl_xor_sync(0xffffffffu, v, o);
      w += __shfl_xor_sync(0xffffffffu, w, o);
    }
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    __syncthreads();
    if (lane == 0) part[warp] = v, part[kWarps + warp] = w;
    __syncthreads();
    if (threadIdx.x < 32) {
      static_assert(2 * kWarps == 32, "two words of a lane half each");
      v = part[lane];
#pragma unroll
      for (int o = 8; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
      if ((lane & 15) == 0) slots[to + (lane >> 4)] = v;
    }
  }
  __device__ __forceinline__ uint64_t told(int word, uint64_t* before = nullptr) const {      // of slots[2 + word]
    const int lane = threadIdx.x & 31;
    uint64_t v = lane < ctas ? load_cluster(mapa_shared(slots + 2 + word, lane)) : 0, b = lane < rank ? v : 0;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      v += __shfl_xor_sync(0xffffffffu, v, o);
      b += __shfl_xor_sync(0xffffffffu, b, o);
    }
    if (before) *before = b;
    return v;
  }

  __device__ __forceinline__ void clear() const {
    for (int i = threadIdx.x; i < kBins; i += kThreads) hist[i] = 0;
    __syncthreads();
  }
  // The team's histogram: each CTA adds up its share of the bins over all, and hands it to all.
  template <typename Add>
  __device__ __forceinline__ const uint64_t* gather(Add add) const {
    sync();
    if (ctas == 1) return hist;
    const int share = kBins / ctas;
    for (int i = threadIdx.x; i < share; i += kThreads) {
      const int b = rank * share + i;
      uint64_t v = 0;
      for (int c = 0; c < ctas; ++c) v = add(v, load_cluster(mapa_shared(hist + b, c)));
      for (int c = 0; c < ctas; ++c) store_cluster(mapa_shared(all + b, c), v);
    }
    cluster_sync();
    return all;
  }
};

__device__ __forceinline__ void add_shared(void* p, uint32_t v) {
  asm volatile("red.shared::cta.add.u32 [%0], %1;" ::"r"(smem_u32(p)), "r"(v) : "memory");
}

// The least value of type T that is not below l.
template <typename T>
__device__ __forceinline__ T at_least(float l) {
  if constexpr (sizeof(T) == 4) return l;
  else if constexpr (std::is_same_v<T, __half>) return __float2half_ru(l);
  else return __float2bfloat16_ru(l);
}
// Bit j: element j of the sixteen bytes v is not below `least`.
__device__ __forceinline__ uint32_t kept_bits(const uint4& v, float least) {
  return (__uint_as_float(v.x) >= least) | (__uint_as_float(v.y) >= least) << 1 | (__uint_as_float(v.z) >= least) << 2 |
         (__uint_as_float(v.w) >= least) << 3;
}
template <typename T>
__device__ __forceinline__ uint32_t kept_bits(const uint4& v, T least) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
  uint32_t b = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    uint32_t m;
    if constexpr (std::is_same_v<T, __half>) m = __hge2_mask(*reinterpret_cast<const __half2*>(&w[i]), __half2half2(least));
    else m = __hge2_mask(*reinterpret_cast<const __nv_bfloat162*>(&w[i]), __bfloat162bfloat162(least));
    b |= (m & 0x00010002u) << (2 * i);           // bit 1 of the lower, bit 16 of the upper
  }
  // Lower elements are in bits 1, 3, 5, 7, upper ones in bits 16, 18, 20, 22: to 0, 2, 4, 6 and 1, 3, 5, 7.
  return (b & 0xffu) >> 1 | (b >> 15 & 0xffu);
}

// f * v rounded down or up, for 0 < f < 1: f is m * 2^-s with a 24-bit m.
__device__ __forceinline__ uint64_t share_of(float f, uint64_t v, bool up) {
  const uint32_t bits = __float_as_uint(f), e = bits >> 23;
  const uint64_t m = e ? (bits & 0x7fffffu) | 0x800000u : bits & 0x7fffffu;
  const int s = 150 - static_cast<int>(e ? e : 1);               // 24 at least
  uint64_t lo = m * v, hi = __umul64hi(m, v);                  // hi is below 2^24
  if (up) {                                                     // + 2^s - 1
    const uint64_t a_lo = s < 64 ? (uint64_t(1) << s) - 1 : ~uint64_t(0), a_hi = s <= 64 ? 0 : s < 128 ? (uint64_t(1) << (s - 64)) - 1 : ~uint64_t(0) >> 1;
    lo += a_lo;
    hi += a_hi + (lo < a_lo);
  }
  return s < 64 ? lo >> s | hi << (64 - s) : s < 128 ? hi >> (s - 64) : up && m != 0;
}

// The sum of v over the threads before this one.
template <typename V>
__device__ __forceinline__ V sum_before(V v, V* part) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  V x = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const V y = __shfl_up_sync(0xffffffffu, x, o);
    if (lane >= o) x += y;
  }
  __syncthreads();
  if (lane == 31) part[warp] = x;
  __syncthreads();
  V s = 0;
#pragma unroll
  for (int w = 0; w < kWarps; ++w) s += w < warp ? part[w] : 0;
  return s + x - v;
}

// The first key up to top at which `in` is true (it is at top, and at all keys from the first on), by 32 tries at a time; guess and
// around: where it most likely is. Every warp finds it for itself.
template <typename In>
__device__ __forceinline__ uint32_t first_key(uint32_t top, float guess, float around, In in) {
  const int lane = threadIdx.x & 31;
  uint32_t lo = kNone, hi = top;                 // the key is in (lo, hi]
  const uint32_t g_lo = guess > -INFINITY ? key_of(guess - around) : kNone, g_hi = guess > -INFINITY ? key_of(guess + around) : top;
  // Lane 0 tries the lower end of the guess, the others the upper.
  const uint32_t at = lane == 0 ? g_lo : g_hi;
  const uint32_t tried = __ballot_sync(0xffffffffu, at > kNone && at < top && in(at));
  if (tried & 1) hi = g_lo;
  else if (g_lo > kNone && g_lo < top) lo = g_lo;
  if (!(tried & 1) && (tried & 2)) hi = g_hi;
  else if (!(tried & 2) && g_hi > lo && g_hi < top) lo = g_hi;
  while (hi - lo > 1) {
    const uint32_t step = (hi - lo + 31) / 32;
    const int i = __ffs(__ballot_sync(0xffffffffu, in(min(lo + step * (lane + 1), hi)))) - 1;      // (hi is among the tries)
    hi = min(lo + step * (i + 1), hi);
    lo = lo + step * i;
  }
  return hi;
}

struct Row {
  uint32_t k;                // 0: no limit
  float p;                   // 1: none
  uint64_t least;            // weights below are not kept
  float u;
  Weigh w;
};

// A row of logits in the shared memory of a cluster: the largest, and (T not above 0) its first token; else the limits of top_k
// and top_p, and the choice among the tokens kept. Steps that the weights' sums decide are taken in whole numbers.
template <typename T>
__global__ void __launch_bounds__(kThreads, 2) sample_kernel(const SampleArgs a, int ctas, int per) {
  extern __shared__ __align__(16) uint8_t smem[];
  __shared__ uint32_t table[256];
  __shared__ float per_T[2];
  __shared__ uint64_t least, slots[6], part[2 * kWarps], found_above;
  __shared__ float partf[kWarps];
  __shared__ int bin_of, found;
  __shared__ float up_to, available;
  uint64_t* hist = reinterpret_cast<uint64_t*>(smem + (static_cast<size_t>(per) * sizeof(T) + 31) / 16 * 16);
  T* list = reinterpret_cast<T*>(hist + 2 * kBins);
  int* list_at = reinterpret_cast<int*>(list + kList);
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  pdl_enter();
  if (threadIdx.x < 256) table[threadIdx.x] = kPow2[threadIdx.x];
  const int64_t n = blockIdx.x / ctas;
  Team team = {ctas, static_cast<int>(cluster_ctarank()), slots, part, hist, hist + kBins, 0};
  const int first = team.rank * per;
  // This CTA's tokens, in the order of their indexes: token i is `first` + i, or index[i].
  int count = max(0, min(per, static_cast<int>(a.V) - first));
  const T* x = static_cast<const T*>(a.logits) + n * a.ld + first;
  // In shared memory the slice lies as far from a 16-byte boundary as in memory: `lead` tokens come before the first one.
  constexpr int E = 16 / sizeof(T);
  const int beyond = static_cast<int>(reinterpret_cast<uintptr_t>(x) & 15) / static_cast<int>(sizeof(T));
  int lead = min(count, beyond ? E - beyond : 0);
  int runs = (count - lead) / E;
  T* slice = reinterpret_cast<T*>(smem) + beyond;
  const T* tokens = slice;
  const int* index = nullptr;

  // The slice, and the row's largest logit.
  float top = -INFINITY;
#pragma unroll 4
  for (int i = threadIdx.x; i < runs; i += kThreads) {
    uint4 v = reinterpret_cast<const uint4*>(x + lead)[i];
    T* e = reinterpret_cast<T*>(&v);
#pragma unroll
    for (int j = 0; j < E; ++j) top = fmaxf(top, take(e[j]));
    reinterpret_cast<uint4*>(slice + lead)[i] = v;
  }
  // The tokens before the first run and after the last: fewer than 2 E.
  if (static_cast<int>(threadIdx.x) < count - runs * E) {
    const int i = static_cast<int>(threadIdx.x) < lead ? threadIdx.x : threadIdx.x + runs * E;
    T v = x[i];
    top = fmaxf(top, take(v));
    slice[i] = v;
  }
  Row row;
  const int k = a.top_k ? a.top_k[n] : 0;
  row.k = k > 0 && k < a.V ? k : 0;
  row.p = a.top_p ? a.top_p[n] : 1.f;
  if (!(row.p < 1.f)) row.p = 1.f;
  const float T0 = a.temperature ? a.temperature[n] : 1.f, min_p = a.min_p ? a.min_p[n] : 0.f;
  row.u = a.u[n];
  if (threadIdx.x == 0) {    // in 64 bits, by one thread
    const double c = 1.4426950408889634 / static_cast<double>(T0);
    per_T[0] = static_cast<float>(c);
    per_T[1] = per_T[0] < INFINITY ? static_cast<float>(c - static_cast<double>(per_T[0])) : 0.f;
    least = min_p > 0.f ? static_cast<uint64_t>(ceil(fmin(static_cast<double>(min_p), 1.0) * static_cast<double>(kOne))) : 0;
  }
  const uint32_t top_key = static_cast<uint32_t>(team.most(key_of(top)));
  auto at = [&](int i) { return usable(to_f32(tokens[i])); };
  const auto words = [&](int i) { return reinterpret_cast<const uint4*>(tokens + lead)[i]; };
  // All tokens, by sixteen bytes; those before the first sixteen and after the last, fewer than 2 E, one by one.
  auto each = [&](auto f) {
#pragma unroll 1
    for (int i = threadIdx.x; i < runs; i += kThreads) {
      uint4 v = words(i);
      const T* e = reinterpret_cast<const T*>(&v);
#pragma unroll
      for (int j = 0; j < E; ++j) f(usable(to_f32(e[j])), lead + i * E + j);
    }
    if (static_cast<int>(threadIdx.x) < count - runs * E) {
      const int i = static_cast<int>(threadIdx.x) < lead ? threadIdx.x : threadIdx.x + runs * E;
      f(at(i), i);
    }
  };
  // Those not below `from`, of the sixteens w0, w0 + by, ... up to w1 and (single) the token that has number `single` among those one
  // by one: a lane goes over its sixteen bytes' alone, so that few tokens cost few steps. Where many are expected, all of the
  // tokens i0, i0 + by, ... up to i1 (the same ones, over the warp's or the CTA's lanes), -inf in the place of those below.
  bool dense = true;
  auto each_from = [&](float from, int by, int w0, int w1, int single, int i0, int i1, auto f) {
    if (dense) {
#pragma unroll 4
      for (int i = i0; i < i1; i += by) {
        const float l = at(i);
        f(l >= from ? l : -INFINITY, i);
      }
      return;
    }
    const T least_T = at_least<T>(from);
#pragma unroll 2
    for (int i = w0; i < w1; i += by)
#pragma unroll 1
      for (uint32_t b = kept_bits(words(i), least_T); b; b &= b - 1) {
        const int k = lead + i * E + __ffs(b) - 1;
        f(at(k), k);
      }
    if (single >= 0 && single < count - runs * E) {
      const int k = single < lead ? single : single + runs * E;
      const float l = at(k);
      if (l >= from) f(l, k);
    }
  };
  auto all_from = [&](float from, auto f) { each_from(from, kThreads, threadIdx.x, runs, threadIdx.x, threadIdx.x, count, f); };
  const float M = value_of(top_key);
  if (top_key == kNone || !(T0 > 0.f)) {         // no token at all, or the first with the largest logit
    int id = 0x7fffffff;
    each([&](float l, int i) { id = min(id, l == M ? first + i : 0x7fffffff); });
    id = 0x7fffffff - static_cast<int>(team.most(static_cast<uint64_t>(0x7fffffff - id)));
    if (threadIdx.x == 0 && team.rank == 0) {
      a.ids[n] = top_key == kNone ? 0 : id;
      if (a.probs) a.probs[n] = top_key == kNone ? 0.f : 1.f;
    }
    team.sync();             // nobody leaves while its memory is read
    return;
  }
  row.w = Weigh{M, per_T[0], per_T[1], table};
  row.least = least;

  // The limit: keys above limit_key are within it, and the first `extra`, by index, of the tokens with that key.
  uint32_t limit_key = kNone + 1, extra = kAll;
  if (row.k > 0 || row.p < 1.f) {
    // Histogram by bins of (M - l) log2(e) / T of 1/16: with top_k of tokens, else of weights relative to the bin's largest possible,
    // in 2^-15 (those of the last bin are below 2^-63), and with it the exact weight of all.
    const float scale = 16.f * 1.44269504f / T0;
    auto bin_at = [&](float l, float& frac) {
      const float d = l == M ? 0.f : fminf(__fsub_rn(M, l) * scale, static_cast<float>(kBins - 1));   // (a NaN: the last)
      const float t = __fadd_rd(d, 8388608.f);                 // the whole number below d in its low bits
      frac = d - (t - 8388608.f);
      return __float_as_int(t) - 0x4b000000;
    };
    const bool by_weight = row.p < 1.f;
    uint64_t whole = 0;
    // Tokens or weights up to each bin: fp32 has these numbers of tokens exactly.
    float to_bin[kPerThread], sum_to, before;
    const auto tally = [&] {
      team.clear();
      if (row.k > 0) {
        each([&](float l, int) {
          float frac;
          if (l != -INFINITY) add_shared(hist + bin_at(l, frac), 1u);
        });
      } else {
        each([&](float l, int) {
          if (l == -INFINITY) return;
          float frac;
          uint64_t* h = hist + bin_at(l, frac);
          add_shared(h, static_cast<uint32_t>(__float_as_int(__fmaf_rn(exp2_fast(frac * -0.0625f), 32768.f, kWhole)) - kWholeBits));
          whole += row.w(l);
        });
        team.tell(whole, 0);
      }
      const uint64_t* all = team.gather([](uint64_t v, uint64_t w) { return v + w; });
      if (row.k == 0) whole = team.told(0);
      sum_to = 0.f;
#pragma unroll
      for (int i = 0; i < kPerThread; ++i) {
        const int b = kPerThread * threadIdx.x + i;
        const float h = static_cast<float>(all[b]);
        to_bin[i] = sum_to += row.k > 0 ? h : b < kBins - 1 ? h * exp2_fast(b * -0.0625f) * 0x1p-15f : 0.f;
      }
      before = sum_before<float>(sum_to, partf);
    };
    tally();
    // The first bin up to which there is so much, or the last bin if there never is. What is before it in up_to, and all in available.
    auto find = [&](float least) {
      __syncthreads();
      if (threadIdx.x == 0) bin_of = kBins - 1;
      __syncthreads();
#pragma unroll
      for (int i = kPerThread - 1; i >= 0; --i)
        if (before + to_bin[i] >= least) atomicMin(&bin_of, static_cast<int>(kPerThread * threadIdx.x + i));
      __syncthreads();
      const int b = bin_of;
#pragma unroll
      for (int i = 0; i < kPerThread; ++i)
        if (b == static_cast<int>(kPerThread * threadIdx.x) + i) up_to = before + (i > 0 ? to_bin[i > 0 ? i - 1 : 0] : 0.f);
      if (threadIdx.x == kThreads - 1) available = before + sum_to;
      __syncthreads();
      return b;
    };
    // The bins' weights are within 2^-14 of the exact ones, and fp32's sums of them: 2^-11 is beyond that on both sides.
    const float around = 0x1p-11f, in_units = 1.f / static_cast<float>(kOne);
    int last = kBins - 1;    // no token of a later bin is kept
    uint32_t k_before = 0;
    if (row.k > 0) {
      last = find(static_cast<float>(row.k));
      k_before = static_cast<uint32_t>(up_to);
      if (available <= static_cast<float>(row.k)) {          // top_k leaves all of them
        row.k = 0;
        last = kBins - 1;
        if (by_weight) tally();
      }
    }
    const bool weights = row.k == 0 && by_weight;
    if (weights) last = find(row.p * (static_cast<float>(whole) * in_units) * (1.f + around));
    // The least key whose bin is b or an earlier one: near M - (b + 1) / scale.
    auto least_key = [&](int b) {
      const float frac_at = static_cast<float>(b + 1) / scale;
      return first_key(top_key, M - frac_at, 0x1p-20f * (fabsf(M) + frac_at), [&](uint32_t k) {
        float frac;
        return bin_at(value_of(k), frac) <= b;
      });
    };
    // The k-th token is in that bin.
    uint32_t lo = least_key(last), hi = row.k > 0 && last > 0 ? least_key(last - 1) - 1 : top_key;
    uint64_t above = row.k > 0 ? k_before : 0;
    const float least_kept = value_of(lo);

    // How many are those. Tokens go by sixteen bytes, E side by side to a lane, and a warp takes a stretch of them (the first also
    // those before, the last those after).
    const int stretch = ((runs + kWarps - 1) / kWarps + 31) / 32 * 32, w0 = min(runs, warp * stretch), w1 = min(runs, w0 + stretch);
    const int tail = lead + runs * E;
    const T least_T = at_least<T>(least_kept);
    // Bit j: token j of the run is kept; lanes beyond the stretch have none.
    const auto bits_of = [&](int i) { return i < w1 ? kept_bits(words(i), least_T) : 0u; };
    const auto single = [&](int i, int end) { return i < end && at(i) >= least_kept; };
    uint32_t mine = 0;
#pragma unroll 4
    for (int i = w0 + lane; i < w1; i += 32) mine += __popc(bits_of(i));
    if (warp == 0) mine += single(lane, lead);
    if (warp == kWarps - 1) mine += single(tail + lane, count);
    mine = __reduce_add_sync(0xffffffffu, mine);
    uint64_t to;
    const uint64_t there = team.sum(lane == 0 ? mine : 0, &to);
    // (By sixteens where fewer than a sixteenth: 64 nuclei of 152064, us: never 204 and 136, below 1/4 144 and 118, below
    // 1/16 140 and 119, flat and of a spread of 2.5.)
    dense = static_cast<int64_t>(there) * 16 > a.V;
    if (there <= kList) {
      // Few: to the first CTA, in the order of their indexes.
      to += sum_before<uint64_t>(lane == 0 ? mine : 0, part);
      uint32_t place = __shfl_sync(0xffffffffu, static_cast<uint32_t>(to), 0);
      const uint32_t list0 = mapa_shared(list, 0), at0 = mapa_shared(list_at, 0);
      // Puts the tokens i + j of the bits j, after those of the lanes before.
      const auto put = [&](int i, uint32_t bits) {
        if (!__any_sync(0xffffffffu, bits != 0)) return;
        uint32_t before = __popc(bits);
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const uint32_t y = __shfl_up_sync(0xffffffffu, before, o);
          if (lane >= o) before += y;
        }
        uint32_t to_place = place + before - __popc(bits);
        place += __shfl_sync(0xffffffffu, before, 31);
        for (; bits; bits &= bits - 1, ++to_place) {
          const int k = i + __ffs(bits) - 1;
          if constexpr (sizeof(T) == 4)
            asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(list0 + 4 * to_place), "f"(slice[k]) : "memory");
          else
            asm volatile("st.shared::cluster.u16 [%0], %1;" ::"r"(list0 + 2 * to_place),
                         "h"(*reinterpret_cast<const uint16_t*>(slice + k)) : "memory");
          asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(at0 + 4 * to_place), "r"(first + k) : "memory");
        }
        __syncwarp();
      };
      if (warp == 0) put(lane, single(lane, lead));
#pragma unroll 2
      for (int i = w0; i < w1; i += 32) put(lead + (i + lane) * E, bits_of(i + lane));
      if (warp == kWarps - 1) put(tail + lane, single(tail + lane, count));
      team.sync();
      if (team.rank > 0) return;
      team = Team{1, 0, slots, part, hist, hist, 0};
      tokens = list;
      index = list_at;
      count = static_cast<int>(there);
      lead = 0;
      runs = count / E;
      dense = true;
    }                        // Many: the cluster goes on

    // The limits one after the other: the largest key at which the sum of tokens, or of weights, over the keys from the largest
    // down reaches its goal. The sum is by histograms of runs of keys in [lo, hi], `above` that of the keys beyond hi.
#pragma unroll 1
    for (int what = row.k > 0 ? 0 : 1; what < (by_weight ? 2 : 1); ++what) {
      uint64_t goal = row.k;
      bool beyond_told = false;
      if (what == 1) {
        const float edge = value_of(limit_key);
        if (row.k > 0) {
          uint64_t mine = 0;
          all_from(edge, [&](float l, int) { mine += l > edge ? row.w(l) : 0; });
          whole = team.sum(mine) + extra * row.w(edge);
        }
        goal = row.p > 0.f ? max(share_of(row.p, whole, true), static_cast<uint64_t>(1)) : 1;      // the least sum that is enough
        lo = max(least_key(last), limit_key);
        hi = top_key;
        above = 0;
        if (weights && team.ctas > 1) {
          // Between the bins in which the prefix may end; what lies beyond is added up.
          const float g = static_cast<float>(goal) * in_units;
          const int b0 = find(g * (1.f - around)), b1 = max(b0, find(g * (1.f + around)));
          lo = max(least_key(b1), limit_key);
          hi = max(lo, b0 > 0 ? least_key(b0 - 1) - 1 : top_key);
          const float beyond = value_of(hi);
          uint64_t mine = 0;
          all_from(beyond, [&](float l, int) { mine += l > beyond ? row.w(l) : 0; });
          // In words of its own: if the search ends with its first histogram, no sync follows before the choice tells.
          team.tell(mine, 0, 4);
          beyond_told = true;
        }
      }
      for (;;) {
        const uint32_t span = hi - lo;
        const int s = span < kBins ? 0 : 22 - __clz(span);
        team.clear();
        const float l_lo = value_of(lo), l_hi = value_of(hi);
        all_from(l_lo, [&](float l, int) {
          if (l >= l_lo && l <= l_hi) {
            uint64_t* h = hist + ((hi - key_of(l)) >> s);
            if (what == 0) add_shared(h, 1u);
            else atomicAdd(reinterpret_cast<unsigned long long*>(h), static_cast<unsigned long long>(row.w(l)));
          }
        });
        if (threadIdx.x == 0) found = -1;
        const uint64_t* h = team.gather([](uint64_t v, uint64_t w) { return v + w; });
        if (beyond_told) above = team.told(2), beyond_told = false;
        uint64_t bin[kPerThread], mine = 0;
#pragma unroll
        for (int i = 0; i < kPerThread; ++i) mine += bin[i] = h[kPerThread * threadIdx.x + i];
        uint64_t c = above + sum_before<uint64_t>(mine, part);
#pragma unroll
        for (int i = 0; i < kPerThread; ++i) {
          if (c < goal && c + bin[i] >= goal) {
            found = kPerThread * threadIdx.x + i;
            found_above = c;
          }
          c += bin[i];
        }
        __syncthreads();
        if (found < 0) {                         // (a goal that rounding has put above the whole sum)
          hi = lo;
          break;
        }
        above = found_above;
        hi -= static_cast<uint32_t>(found) << s;
        if (s == 0) break;
        lo = max(lo, hi - ((1u << s) - 1));
        __syncthreads();
      }
      if (what == 0) {
        limit_key = hi;
        extra = static_cast<uint32_t>(goal - above);
      } else {
        // Of the tokens with that key: the fewest that bring the sum to the goal, one at least.
        const uint64_t one = row.w(value_of(hi));
        const uint64_t c = one > 0 && goal > above ? (goal - above + one - 1) / one : 1;
        extra = static_cast<uint32_t>(min(c, static_cast<uint64_t>(hi == limit_key ? extra : kAll - 1)));
        limit_key = hi;
      }
      __syncthreads();
    }
  }

  // min_p as a least key, where it is beyond the limit.
  if (row.least > 0) {
    const float below = -logf(fminf(min_p, 1.f)) * T0;
    const uint32_t least_kept = first_key(top_key, M - below, 0x1p-20f * (fabsf(M) + below), [&](uint32_t k) { return row.w(value_of(k)) >= row.least; });
    if (limit_key == kNone + 1) dense = false;   // (alone it leaves few)
    if (least_kept > limit_key) limit_key = least_kept, extra = kAll;
  }

  // The choice. A warp has a stretch of sixteens (the first also the tokens before them, the last those after).
  const int stretch = (runs + kWarps - 1) / kWarps, w0 = min(runs, warp * stretch), w1 = min(runs, w0 + stretch);
  const int i0 = warp > 0 ? lead + w0 * E : 0, i1 = warp < kWarps - 1 ? lead + w1 * E : count;
  const float edge = value_of(limit_key);
  // This CTA's tokens with the limit's key, of which those after the first `extra` of the row are not kept, and the weight of the
  // others that are: told to the other CTAs at once. A weight with the limit's key is `one`.
  const uint64_t one = extra != kAll ? row.w(edge) : 0;
  uint32_t same = 0;
  uint64_t mine = 0;
  // Of the tokens one by one the first warp has those before, the last those after.
  const int single = warp == 0 && lane < lead ? lane : warp == kWarps - 1 ? lead + lane : -1;
  each_from(edge, 32, w0 + lane, w1, single, i0 + lane, i1, [&](float l, int) {
    if (extra != kAll && l == edge) ++same;
    else mine += row.w(l);
  });
  same = __reduce_add_sync(0xffffffffu, same);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) mine += __shfl_xor_sync(0xffffffffu, mine, o);
  team.tell(lane == 0 ? same : 0, lane == 0 ? mine : 0);
  team.sync();
  uint64_t ties, c;
  const uint64_t all_same = team.told(0, &ties), all_above = team.told(1, &c), limit = extra;
  const uint64_t total = all_above + min(all_same, limit) * one;
  c += min(ties, limit) * one;                   // of the CTAs before this one
  ties += sum_before<uint64_t>(lane == 0 ? same : 0, part);
  ties = __shfl_sync(0xffffffffu, ties, 0);
  const uint64_t kept_ties = min(ties + same, limit) - min(ties, limit), of_warp = mine + kept_ties * one;
  c += sum_before<uint64_t>(lane == 0 ? of_warp : 0, part);
  c = __shfl_sync(0xffffffffu, c, 0);
  // The weight of token i if it is kept; seen: tokens with the limit's key so far. All lanes of the warp call it.
  auto kept = [&](int i, uint64_t& seen) -> uint64_t {
    const float l = i < i1 ? at(i) : -INFINITY;
    if (extra != kAll) {
      const uint32_t equal = __ballot_sync(0xffffffffu, l == edge);
      const bool in = seen + __popc(equal & ((1u << lane) - 1)) < limit;
      seen += __popc(equal);
      if (l == edge) return in ? one : 0;
    }
    return l >= edge ? row.w(l) : 0;
  };
  // The first sum above u * total: at least floor(u * total) + 1, and at most all of it.
  const uint64_t goal = min(row.u >= 1.f ? total : row.u > 0.f ? share_of(row.u, total, false) : 0, total - 1);
  if (c <= goal && goal < c + of_warp) {
    uint64_t seen = ties;
    for (int i = i0; i < i1; i += 32) {
      if (!__any_sync(0xffffffffu, i + lane < i1 && at(i + lane) >= edge)) continue;
      const uint64_t v = kept(i + lane, seen);
      uint64_t s = v;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const uint64_t y = __shfl_up_sync(0xffffffffu, s, o);
        if (lane >= o) s += y;
      }
      const uint32_t past = __ballot_sync(0xffffffffu, c + s > goal);
      if (past) {
        if (lane == __ffs(past) - 1) {
          a.ids[n] = index ? index[i + lane] : first + i + lane;
          if (a.probs) a.probs[n] = static_cast<float>(static_cast<double>(v) / static_cast<double>(total));
        }
        break;
      }
      c += __shfl_sync(0xffffffffu, s, 31);
    }
  }
  team.sync();
}

template <typename T>
cudaError_t sample(const SampleArgs& a, int num_sms, cudaStream_t s) {
  // CTAs of a row: enough to hold it with two on an SM (80 KB of logits each; with 64 KB, and so eight CTAs for 152064 of 16
  // bits, 64 rows with top-k and top-p took 73 us against 58), and as many as leave 2048 tokens each while all
  // rows' run at once (one row of 32000: 21.1 us, with 4096 tokens each 21.7, with 1024 21.3).
  constexpr int kMost = 80 * 1024 / sizeof(T);
  int ctas = 1;
  while (ctas < kMostCtas && (a.V > static_cast<int64_t>(ctas) * kMost ||
                              (a.V >= 4096 * static_cast<int64_t>(ctas) && a.N * ctas <= num_sms)))
    ctas *= 2;
  const int per = static_cast<int>(((a.V + ctas - 1) / ctas + 7) / 8 * 8);
  const size_t smem = (static_cast<size_t>(per) * sizeof(T) + 31) / 16 * 16 + 2 * kBins * sizeof(uint64_t) + kList * 8;
  static std::atomic<uint64_t> allowed{0};
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev >= 64 || !(allowed.load(std::memory_order_acquire) >> dev & 1)) {
    e = cudaFuncSetAttribute(sample_kernel<T>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             kSliceBytes + 2 * kBins * sizeof(uint64_t) + kList * 8 + 64);
    if (e == cudaSuccess) e = cudaFuncSetAttribute(sample_kernel<T>, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
    if (e != cudaSuccess) return e;
    if (dev < 64) allowed.fetch_or(uint64_t(1) << dev, std::memory_order_release);
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(a.N * ctas));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = static_cast<unsigned>(ctas);
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, sample_kernel<T>, a, ctas, per);
}

}  // namespace

cudaError_t launch_sample(int dtype, const SampleArgs& a, int num_sms, cudaStream_t s) {
  if (dtype == KQ_F16) return sample<__half>(a, num_sms, s);
  if (dtype == KQ_BF16) return sample<__nv_bfloat16>(a, num_sms, s);
  return sample<float>(a, num_sms, s);
}

}  // namespace kq
