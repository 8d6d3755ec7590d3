// Head rows: the norm of a head with the position rotation, and the writing and reading of the
// 4-bit paged cache. A head of D elements is held by D / 8 lanes, eight elements each; a group of
// lanes takes several heads of one token, so that the token's cosines and sines are read
// once for them.
//
//   norm:      y = (x * 1 / sqrt(Sum x^2 / D + eps)) * gamma
//   rotation:  (a, b) -> (a cos - b sin, b cos + a sin), each product and each sum rounded to fp32
//   block:     m = fp16(min v), s = fp16((max v - min v) * (1 / 15)), c = clamp(rint((v - m) / s), 0, 15)
//
// What bounds it (one GB300, in a graph, inputs larger than L2): of many rows half memory, half the issue of
// instructions. 4099 rows of 32 + 8 bf16 heads of 128, normed and turned: 21.7 us (0.59 of the copy bandwidth); 8191 tokens of 8 heads
// written to the cache: 20 us, most of it the codes; read back: 13 us (0.5). One row: 2 us, the launch and three loads
// one after the other.
#include <cuda_bf16.h>

#include <algorithm>

#include "kq_kv4.cuh"
#include "kq_q8_rows.cuh"
#include "kq_types.cuh"

namespace kq {
namespace {

constexpr int kThreads = 256;

// Group `lane`'s share of a token's row of the table: for lanes of the first rot elements, the
// cosines and sines of their eight elements. With halves a lane of the first half has its
// sines negated (v cos + other * (-sin)); with pairs c[i], s[i] (i < 4) are those of pair i.
struct Turn {
  float c[8], s[8];
  int from;        // lane of the group that holds the other halves
  bool on;

  __device__ __forceinline__ void load(const float* row, int rot, bool pairs, int lane) {
    on = row != nullptr && 8 * lane < rot;
    from = lane;
    if (!on) return;
    const int half = rot >> 1;
    if (pairs) {
      *reinterpret_cast<float4*>(c) = *reinterpret_cast<const float4*>(row + 4 * lane);
      *reinterpret_cast<float4*>(s) = *reinterpret_cast<const float4*>(row + half + 4 * lane);
      return;
    }
    const bool second = 8 * lane >= half;
    const int at = 8 * lane - (second ? half : 0);
    from = second ? lane - (half >> 3) : lane + (half >> 3);
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      reinterpret_cast<float4*>(c)[i] = *reinterpret_cast<const float4*>(row + at + 4 * i);
      reinterpret_cast<float4*>(s)[i] = *reinterpret_cast<const float4*>(row + half + at + 4 * i);
    }
    if (!second) {
#pragma unroll
      for (int i = 0; i < 8; ++i) s[i] = -s[i];
    }
  }

  // All lanes of the warp call it (`base`: the first lane of the group).
  __device__ __forceinline__ void apply(float (&v)[8], bool pairs, int base) const {
    if (pairs) {
      if (!on) return;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float a = v[2 * i], b = v[2 * i + 1];
        v[2 * i] = __fsub_rn(__fmul_rn(a, c[i]), __fmul_rn(b, s[i]));
        v[2 * i + 1] = __fadd_rn(__fmul_rn(b, c[i]), __fmul_rn(a, s[i]));
      }
      return;
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float o = __shfl_sync(0xffffffffu, v[i], base + from);
      if (on) v[i] = __fadd_rn(__fmul_rn(v[i], c[i]), __fmul_rn(o, s[i]));
    }
  }
};

// A token's row of the table; null where its position is outside (recorded) or there is no table.
__device__ __forceinline__ const float* table_row(const Rope& rope, int64_t pos, bool& ok, int* err) {
  if (!rope.cos_sin || !ok) return nullptr;
  if (pos >= rope.n_positions) {
    report_error(err, ERR_POSITION);
    ok = false;
    return nullptr;
  }
  return rope.cos_sin + pos * rope.rot;
}

template <int LANES>
__device__ __forceinline__ float group_sum(float v) {
#pragma unroll
  for (int o = LANES / 2; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// A lane's eight gammas (row null: none): loaded once for several heads, or where they are used (held for one head they are
// eight registers more: 256 rows of 40 heads 4.0 us, 3.1 so).
template <bool HELD>
struct Gamma {
  const float* row;
  float held[8];
  __device__ __forceinline__ Gamma(const float* gamma, int lane, bool mine) : row(gamma ? gamma + 8 * lane : nullptr) {
    if constexpr (HELD) {
#pragma unroll
      for (int i = 0; i < 8; ++i) held[i] = 0.f;
      if (row && mine) load(held);
    }
  }
  __device__ __forceinline__ void load(float (&g)[8]) const {
#pragma unroll
    for (int i = 0; i < 2; ++i) *reinterpret_cast<float4*>(g + 4 * i) = *reinterpret_cast<const float4*>(row + 4 * i);
  }
  __device__ __forceinline__ void get(float (&g)[8]) const {
    if constexpr (HELD) {
#pragma unroll
      for (int i = 0; i < 8; ++i) g[i] = held[i];
    } else {
      load(g);
    }
  }
};

// v = (v * r) * gamma (gamma null: v), r = 1 / sqrt(Sum v^2 / D + eps). Where squares leave fp32's range, or are so small that
// their sum loses bits, the head is taken times the power of two that brings the larger of max |v| and sqrt(eps) to between 1 and
// 2 (in two factors: it can be beyond 2^127), and r is that of those values. (In 64 bits instead, and so for every
// head since the compiler ran them beside the usual path: 120 us for 4099 x 40 heads of 128, against 25 for fp32 alone at that time.)
template <int LANES, typename Gammas>
__device__ __forceinline__ void norm_head(float (&v)[8], const Gammas& gamma, bool mine, float inv_D, float eps) {
  float ss = 0.f;
#pragma unroll
  for (int i = 0; i < 8; ++i) ss = fmaf(v[i], v[i], ss);
  ss = group_sum<LANES>(ss);
  float m = fmaf(ss, inv_D, eps);
  const bool far = !(ss < INFINITY && m >= 0x1p-90f) && gamma.row;
  if (__any_sync(0xffffffffu, far)) {
    float most = sqrtf(eps), sum = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) most = fmaxf(most, fabsf(v[i]));
#pragma unroll
    for (int o = LANES / 2; o > 0; o >>= 1) most = fmaxf(most, __shfl_xor_sync(0xffffffffu, most, o));
    const int e = 127 - static_cast<int>(__float_as_uint(most) >> 23), e1 = e >> 1;
    const float s1 = __uint_as_float(static_cast<uint32_t>(127 + e1) << 23), s2 = __uint_as_float(static_cast<uint32_t>(127 + e - e1) << 23);
    float w[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      w[i] = v[i] * s1 * s2;
      sum = fmaf(w[i], w[i], sum);
    }
    sum = group_sum<LANES>(sum);
    if (far) {
      m = fmaf(sum, inv_D, eps * s1 * s1 * s2 * s2);
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] = w[i];
    }
  }
  if (!mine || !gamma.row) return;
  const float r = rsqrtf(m);
  float g[8];
  gamma.get(g);
#pragma unroll
  for (int i = 0; i < 8; ++i) v[i] = v[i] * r * g[i];
}

struct HeadRows {
  const void* Q;
  const void* K;
  void* Qo;
  void* Ko;
  int64_t ldq, ldk, ldqo, ldko;
  const float* q_gamma;
  const float* k_gamma;
  int n_q, n_k, D;
  float eps;
  Rope rope;
  const int32_t* positions;
  int64_t N;
  int* err;
};

// LANES: a power of two >= D / 8; HPI: heads of one token, of queries or of keys, that a group takes.
template <typename T, typename TO, bool VEC, int LANES, int HPI>
__global__ void __launch_bounds__(kThreads) qk_norm_rope_kernel(const HeadRows a) {
  pdl_enter();
  const int lane = threadIdx.x & (LANES - 1), base = threadIdx.x & 31 & ~(LANES - 1);
  const int q_chunks = (a.n_q + HPI - 1) / HPI, chunks = q_chunks + (a.n_k + HPI - 1) / HPI;
  const float inv_D = __fdividef(1.0f, static_cast<float>(a.D));
  const uint32_t item = blockIdx.x * (kThreads / LANES) + threadIdx.x / LANES;      // (host: below 2^31)
  const uint32_t n = item / static_cast<uint32_t>(chunks);
  const int chunk = static_cast<int>(item - n * chunks);
  const bool key = chunk >= q_chunks;
  const int h0 = (key ? chunk - q_chunks : chunk) * HPI, some = min(HPI, (key ? a.n_k : a.n_q) - h0);
  bool ok = n < a.N;
  // The heads are on their way while the position and its row of the table are looked up.
  const bool lanes = ok && 8 * lane < a.D;
  const int64_t at = static_cast<int64_t>(h0) * a.D + 8 * lane;
  const T* x = (key ? static_cast<const T*>(a.K) + n * a.ldk : static_cast<const T*>(a.Q) + n * a.ldq) + at;
  Raw8<T> raw[HPI];
#pragma unroll
  for (int i = 0; i < HPI; ++i)
    if (lanes && i < some) raw[i].template load<VEC>(x + i * a.D);
  const int64_t pos = !ok ? 0 : a.positions ? a.positions[n] : n;
  ok = ok && pos >= 0;
  Turn turn;
  turn.load(table_row(a.rope, pos, ok, a.err), a.rope.rot, a.rope.pairs, lane);
  const bool mine = ok && lanes;
  const Gamma<(HPI > 1)> gamma(key ? a.k_gamma : a.q_gamma, lane, mine);
  TO* y = (key ? static_cast<TO*>(a.Ko) + n * a.ldko : static_cast<TO*>(a.Qo) + n * a.ldqo) + at;
#pragma unroll
  for (int i = 0; i < HPI; ++i) {
    const bool here = mine && i < some;
    float v[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = here ? raw[i][j] : 0.f;
    if (a.q_gamma || a.k_gamma) norm_head<LANES>(v, gamma, here, inv_D, a.eps);
    if (a.rope.cos_sin) turn.apply(v, a.rope.pairs, base);
    if (here) store8<TO, VEC>(y + i * a.D, v);
  }
}

// The codes of the eight values v of a lane, the block being held by an aligned quad of lanes:
// code i in bits 4i. s and m are as stored. The quotient is that of IEEE division: 15 times the product
// with 1 / (15 s), held to 0 .. 1 by the multiplication itself, is within 15 * 6 * 2^-24 < 10^-5 of it held to 0 .. 15, so only
// where it is that near a half is the division made.
__device__ __forceinline__ uint32_t block_codes(const float (&v)[8], __half& sh, __half& mh) {
  float lo = v[0], hi = v[0];
#pragma unroll
  for (int i = 1; i < 8; ++i) lo = min_nan(lo, v[i]), hi = max_nan(hi, v[i]);
#pragma unroll
  for (int o = 1; o <= 2; o <<= 1) {
    lo = min_nan(lo, __shfl_xor_sync(0xffffffffu, lo, o));
    hi = max_nan(hi, __shfl_xor_sync(0xffffffffu, hi, o));
  }
  mh = __float2half_rn(lo);
  sh = __float2half_rn(__fmul_rn(__fsub_rn(hi, lo), 1.0f / 15.0f));
  const float m = __half2float(mh), s = __half2float(sh);
  const bool numbers = fabsf(m) < INFINITY && s < INFINITY, codes = numbers && s > 0.f;
  if (!numbers) {            // a value that fp16 cannot hold, an infinity or a NaN
    sh = __ushort_as_half(static_cast<unsigned short>(0x7fff));
    mh = __ushort_as_half(static_cast<unsigned short>(0));
  }
  // Without codes all are 0: a NaN held to 0 .. 1 is 0 too.
  float inv;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(inv) : "f"(s));
  inv = codes ? inv * (1.0f / 15.0f) : 0.f;
  // The whole number nearest to a quotient (the even one of two) is in the low bits of its sum with 1.5 * 2^23; the sum
  // of these words times 16^i is the codes' word and a constant.
  constexpr float kWhole = 12582912.f;
  uint32_t w = 0;
  float worst = 0.f;
#pragma unroll
  for (int i = 7; i >= 0; --i) {
    float t;
    asm("mul.rn.sat.f32 %0, %1, %2;" : "=f"(t) : "f"(__fsub_rn(v[i], m)), "f"(inv));
    const float c = __fmaf_rn(t, 15.f, kWhole);
    worst = fmaxf(worst, fabsf(__fmaf_rn(t, 15.f, -__fsub_rn(c, kWhole))));
    w = (w << 4) + __float_as_uint(c);
  }
  if (codes && worst > 0.49999f) {
    w = 0;
#pragma unroll
    for (int i = 7; i >= 0; --i) {
      const float t = fminf(fmaxf(__fdiv_rn(__fsub_rn(v[i], m), s), 0.f), 15.f);
      w = (w << 4) + __float_as_uint(__fadd_rn(t, kWhole));
    }
  }
  constexpr uint32_t kOnes = 0x11111111u * 0x4b400000u;
  return w - kOnes;
}

struct AppendArgs {
  const void* K;
  const void* V;
  int64_t ldk, ldv;
  Rope rope;
  const int32_t* positions;
  const int32_t* seq_ids;
  KvCache c;
  int64_t N;
  int* err;
};

// The token's granule of head 0, or -1 (nothing is written for it).
__device__ __forceinline__ int64_t place_of(const KvCache& c, const int32_t* positions, const int32_t* seq_ids, int64_t n,
                                            int64_t& pos, int* err) {
  pos = positions[n];
  if (pos < 0) return -1;
  const int64_t at = granule_of(c, seq_ids ? seq_ids[n] : n, pos);
  if (at < 0) report_error(err, ERR_PAGE);
  return at;
}

template <typename T, bool VEC, int D, int HPI>
__global__ void __launch_bounds__(kThreads) kv_append_q4_kernel(const AppendArgs a) {
  pdl_enter();
  using Gr = Granule<D>;
  constexpr int LANES = D / 8, G = D / 32;
  const int lane = threadIdx.x & (LANES - 1), base = threadIdx.x & 31 & ~(LANES - 1);
  const int per_kind = (a.c.heads + HPI - 1) / HPI, chunks = 2 * per_kind;      // a token's key heads, then its value heads
  const uint32_t item = blockIdx.x * (kThreads / LANES) + threadIdx.x / LANES;      // (host: below 2^31)
  const uint32_t n = item / static_cast<uint32_t>(chunks), chunk = item - n * static_cast<uint32_t>(chunks);
  const bool key = chunk < static_cast<uint32_t>(per_kind);
  const int h0 = static_cast<int>(key ? chunk : chunk - per_kind) * HPI, some = min(HPI, a.c.heads - h0);
  // The heads are on their way while the place and the row of the table are looked up.
  Raw8<T> raw[HPI];
  const T* p = (key ? static_cast<const T*>(a.K) + n * a.ldk : static_cast<const T*>(a.V) + n * a.ldv) + h0 * D + 8 * lane;
#pragma unroll
  for (int i = 0; i < HPI; ++i)
    if (n < a.N && i < some) raw[i].template load<VEC>(p + i * D);
  int64_t pos = 0, at = -1;
  if (n < a.N) at = place_of(a.c, a.positions, a.seq_ids, n, pos, a.err);
  bool ok = at >= 0;
  const float* row = table_row(a.rope, pos, ok, a.err);
  Turn turn;
  turn.load(key ? row : nullptr, a.rope.rot, a.rope.pairs, lane);
  const bool turns = a.rope.cos_sin && __any_sync(0xffffffffu, key);
  const int t = static_cast<int>(pos & 15), g = lane >> 2, j = lane & 3;
  uint8_t* gr = a.c.data + (at + (static_cast<int64_t>(h0) << (a.c.page_shift - 4))) * Gr::kBytes + (key ? 0 : Gr::kValues);
#pragma unroll
  for (int i = 0; i < HPI; ++i) {
    const bool here = ok && i < some;
    float v[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = here ? raw[i][j] : 0.f;
    if (turns) turn.apply(v, a.rope.pairs, base);
    __half s, m;
    uint32_t w = block_codes(v, s, m);
    // Of values, a lane's low four codes go beside those of the next block, or its high four beside those of the one before.
    const uint32_t other = __shfl_xor_sync(0xffffffffu, g & 1 ? w : w >> 16, 4);
    if (here) {
      uint8_t* codes = gr + t * (D / 2);
      if (key) codes += 4 * G * j + 4 * g;
      else codes += 2 * G * (2 * j + (g & 1)) + 2 * (g & ~1);
      if (!key) w = g & 1 ? __byte_perm(other, w, 0x7610) : __byte_perm(w, other, 0x5410);
      *reinterpret_cast<uint32_t*>(codes) = w;
      if (j == 0) {
        __half* par = reinterpret_cast<__half*>(gr + Gr::kCodes + t * (4 * G));
        par[g] = s;
        par[G + g] = m;
      }
    }
    gr += static_cast<int64_t>(Gr::kBytes) << (a.c.page_shift - 4);
  }
}

struct GatherArgs {
  KvCache c;
  const int32_t* positions;
  const int32_t* seq_ids;
  void* K;
  void* V;
  int64_t ldk, ldv, N;
  int* err;
};

template <typename T, bool VEC, int D, int HPI>
__global__ void __launch_bounds__(kThreads) kv_gather_q4_kernel(const GatherArgs a) {
  pdl_enter();
  using Gr = Granule<D>;
  constexpr int LANES = D / 8, G = D / 32;
  const int lane = threadIdx.x & (LANES - 1);
  const int rows = 2 * a.c.heads, chunks = (rows + HPI - 1) / HPI;
  const uint32_t item = blockIdx.x * (kThreads / LANES) + threadIdx.x / LANES;      // (host: below 2^31)
  const uint32_t n = item / static_cast<uint32_t>(chunks);
  const int r0 = static_cast<int>(item - n * chunks) * HPI;
  if (n >= a.N) return;
  int64_t pos;
  const int64_t at = place_of(a.c, a.positions, a.seq_ids, n, pos, a.err);
  if (at < 0) return;
  const int t = static_cast<int>(pos & 15), g = lane >> 2, j = lane & 3;
  uint32_t w[HPI];
  __half s[HPI], m[HPI];
#pragma unroll
  for (int i = 0; i < HPI; ++i) {
    const int r = r0 + i, h = r < a.c.heads ? r : r - a.c.heads;
    if (r >= rows) break;
    const bool key = r < a.c.heads;
    const uint8_t* gr =
        a.c.data + (at + (static_cast<int64_t>(h) << (a.c.page_shift - 4))) * Gr::kBytes + (key ? 0 : Gr::kValues);
    const uint8_t* codes = gr + t * (D / 2);
    w[i] = key ? *reinterpret_cast<const uint32_t*>(codes + 4 * G * j + 4 * g)
               : *reinterpret_cast<const uint16_t*>(codes + 2 * G * (2 * j) + 2 * g) |
                     (static_cast<uint32_t>(*reinterpret_cast<const uint16_t*>(codes + 2 * G * (2 * j + 1) + 2 * g)) << 16);
    const __half* par = reinterpret_cast<const __half*>(gr + Gr::kCodes + t * (4 * G));
    s[i] = par[g];
    m[i] = par[G + g];
  }
#pragma unroll
  for (int i = 0; i < HPI; ++i) {
    const int r = r0 + i, h = r < a.c.heads ? r : r - a.c.heads;
    if (r >= rows) break;
    float v[8];
#pragma unroll
    for (int k = 0; k < 8; ++k)
      v[k] = fmaf(static_cast<float>((w[i] >> (4 * k)) & 15u), __half2float(s[i]), __half2float(m[i]));
    T* p = (r < a.c.heads ? static_cast<T*>(a.K) + n * a.ldk : static_cast<T*>(a.V) + n * a.ldv) + static_cast<int64_t>(h) * D;
    store8<T, VEC>(p + 8 * lane, v);
  }
}

// Whether rows `ld` elements apart, of heads of D elements, keep a 16-byte boundary.
template <typename T>
bool even_rows(int64_t ld) {
  return ld * static_cast<int64_t>(sizeof(T)) % 16 == 0;
}

// Heads that a group takes: one until groups of one would fill every SM's threads. us with one, two, four and eight heads for
// 8191 tokens of 8 heads written 29.5, 24.8, 22.2, 25.8 and read 19.1, 14.7, 13.0, 17.7; with one and four for 4099 rows of 40 heads 28
// and 21.6, 512 rows 5.0 and 4.7, 256 rows 3.1 and 4.9; 2048 tokens of 8 heads written 10.7 and 8.6, 1024 tokens 5.6 and 6.7.
int heads_per_item(int64_t N, int rows, int lanes, int num_sms) {
  return N * rows * lanes >= static_cast<int64_t>(num_sms) * 2048 ? 4 : 1;
}

unsigned blocks_of(int64_t items, int lanes) {
  const int64_t per = kThreads / lanes;
  return static_cast<unsigned>((items + per - 1) / per);
}

template <typename T, typename TO, bool VEC, int LANES>
cudaError_t norm_rope(const HeadRows& a, int num_sms, cudaStream_t s) {
  const int heads = a.n_q + a.n_k;
  if (heads_per_item(a.N, heads, LANES, num_sms) == 4)
    return launch_pdl(qk_norm_rope_kernel<T, TO, VEC, LANES, 4>, dim3(blocks_of(a.N * ((a.n_q + 3) / 4 + (a.n_k + 3) / 4), LANES)),
                      dim3(kThreads), 0, s, a);
  return launch_pdl(qk_norm_rope_kernel<T, TO, VEC, LANES, 1>, dim3(blocks_of(a.N * heads, LANES)), dim3(kThreads), 0, s, a);
}

template <typename T, typename TO>
cudaError_t norm_rope(const HeadRows& a, int num_sms, cudaStream_t s) {
  const bool vec = even_rows<T>(a.ldq) && even_rows<TO>(a.ldqo) && (!a.n_k || (even_rows<T>(a.ldk) && even_rows<TO>(a.ldko)));
  if (vec) {
    if (a.D <= 64) return norm_rope<T, TO, true, 8>(a, num_sms, s);
    if (a.D <= 128) return norm_rope<T, TO, true, 16>(a, num_sms, s);
    return norm_rope<T, TO, true, 32>(a, num_sms, s);
  }
  if (a.D <= 64) return norm_rope<T, TO, false, 8>(a, num_sms, s);
  if (a.D <= 128) return norm_rope<T, TO, false, 16>(a, num_sms, s);
  return norm_rope<T, TO, false, 32>(a, num_sms, s);
}

template <typename T, int D>
cudaError_t append(const AppendArgs& a, int num_sms, cudaStream_t s) {
  const int rows = 2 * a.c.heads, lanes = D / 8;
  const bool vec = even_rows<T>(a.ldk) && even_rows<T>(a.ldv), four = heads_per_item(a.N, rows, lanes, num_sms) == 4;
  const dim3 grid(blocks_of(a.N * 2 * (four ? (a.c.heads + 3) / 4 : a.c.heads), lanes));
  if (vec) return four ? launch_pdl(kv_append_q4_kernel<T, true, D, 4>, grid, dim3(kThreads), 0, s, a)
                       : launch_pdl(kv_append_q4_kernel<T, true, D, 1>, grid, dim3(kThreads), 0, s, a);
  return four ? launch_pdl(kv_append_q4_kernel<T, false, D, 4>, grid, dim3(kThreads), 0, s, a)
              : launch_pdl(kv_append_q4_kernel<T, false, D, 1>, grid, dim3(kThreads), 0, s, a);
}

template <typename T, int D>
cudaError_t gather(const GatherArgs& a, int num_sms, cudaStream_t s) {
  const int rows = 2 * a.c.heads, lanes = D / 8;
  const bool vec = even_rows<T>(a.ldk) && even_rows<T>(a.ldv), four = heads_per_item(a.N, rows, lanes, num_sms) == 4;
  const dim3 grid(blocks_of(a.N * (four ? (rows + 3) / 4 : rows), lanes));
  if (vec) return four ? launch_pdl(kv_gather_q4_kernel<T, true, D, 4>, grid, dim3(kThreads), 0, s, a)
                       : launch_pdl(kv_gather_q4_kernel<T, true, D, 1>, grid, dim3(kThreads), 0, s, a);
  return four ? launch_pdl(kv_gather_q4_kernel<T, false, D, 4>, grid, dim3(kThreads), 0, s, a)
              : launch_pdl(kv_gather_q4_kernel<T, false, D, 1>, grid, dim3(kThreads), 0, s, a);
}

template <typename T>
cudaError_t append(const AppendArgs& a, int num_sms, cudaStream_t s) {
  return a.c.D == 64 ? append<T, 64>(a, num_sms, s) : a.c.D == 128 ? append<T, 128>(a, num_sms, s) : append<T, 256>(a, num_sms, s);
}
template <typename T>
cudaError_t gather(const GatherArgs& a, int num_sms, cudaStream_t s) {
  return a.c.D == 64 ? gather<T, 64>(a, num_sms, s) : a.c.D == 128 ? gather<T, 128>(a, num_sms, s) : gather<T, 256>(a, num_sms, s);
}

}  // namespace

cudaError_t launch_qk_norm_rope(int dtype, const void* Q, int64_t ldq, int n_q, const void* K, int64_t ldk, int n_k, int D,
                                const float* q_gamma, const float* k_gamma, float eps, const Rope& rope,
                                const int32_t* positions, int out_dtype, void* Qo, int64_t ldqo, void* Ko, int64_t ldko,
                                int64_t N, int* err, int num_sms, cudaStream_t s) {
  const HeadRows a = {Q,   K,   Qo, Ko,  ldq,  ldk,       ldqo, ldko, q_gamma, n_k ? k_gamma : nullptr,
                      n_q, n_k, D,  eps, rope, positions, N,    err};
  if (dtype == KQ_F16) return norm_rope<__half, __half>(a, num_sms, s);
  if (dtype == KQ_BF16) return norm_rope<__nv_bfloat16, __nv_bfloat16>(a, num_sms, s);
  if (out_dtype == KQ_F16) return norm_rope<float, __half>(a, num_sms, s);
  if (out_dtype == KQ_BF16) return norm_rope<float, __nv_bfloat16>(a, num_sms, s);
  return norm_rope<float, float>(a, num_sms, s);
}

cudaError_t launch_kv_append_q4(int dtype, const void* K, int64_t ldk, const void* V, int64_t ldv, const Rope& rope,
                                const int32_t* positions, const int32_t* seq_ids, const KvCache& c, int64_t N, int* err,
                                int num_sms, cudaStream_t s) {
  const AppendArgs a = {K, V, ldk, ldv, rope, positions, seq_ids, c, N, err};
  if (dtype == KQ_F16) return append<__half>(a, num_sms, s);
  if (dtype == KQ_BF16) return append<__nv_bfloat16>(a, num_sms, s);
  return append<float>(a, num_sms, s);
}

cudaError_t launch_kv_gather_q4(const KvCache& c, const int32_t* positions, const int32_t* seq_ids, int dtype, void* K,
                                int64_t ldk, void* V, int64_t ldv, int64_t N, int* err, int num_sms, cudaStream_t s) {
  const GatherArgs a = {c, positions, seq_ids, K, V, ldk, ldv, N, err};
  if (dtype == KQ_F16) return gather<__half>(a, num_sms, s);
  if (dtype == KQ_BF16) return gather<__nv_bfloat16>(a, num_sms, s);
  return gather<float>(a, num_sms, s);
}

}  // namespace kq
