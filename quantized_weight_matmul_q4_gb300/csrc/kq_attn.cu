// Attention over the 4-bit paged cache, for the new rows of a decode step.
//
//   o = Sum_t softmax_t(scale q . k_t) v_t   over the places t that a row sees
//
// Row i of a sequence's n new rows sees the places below kv_len - n + 1 + i and, with a window, the
// last `window` of those; a row that sees none gives zeros.
//
// One pass over the cache with a running maximum. The codes themselves are the operands of the tensor cores: four
// bits in the low bits of an fp16 are the exact number c * 2^-24 (c * 2^-20 four bits higher), so
// a word of eight codes becomes four operand registers by masks and one shift. With blocks g of 32 elements,
//   q . k_t = Sum_g s_tg (c_tg . q_g) + Sum_g m_tg Sum(q_g)
//   o       = Sum_g Sum_t (p_t s_tg) c_tg + Sum_t p_t m_tg
// The first sum of each is a product of codes per block, scaled after (scores) or before (weights);
// the second is one more product, of the m themselves, which also gives Sum_t p_t by a row of ones.
//
// Scores are exact products summed in fp32. Weights are rounded to fp16 as operands (a relative 2^-12, which
// 16-bit outputs do not show; fp32 rows have theirs split into two halves, as their queries are); they are
// taken relative to a power of two near the largest s so far, so that none leaves fp16's range.
//
// Work is shared out evenly whatever the sequences' lengths: the granules of 16 places of all (sequence,
// key head, tile of rows) segments stand in one line, of which each CTA takes an equal run. A segment that
// lies in several runs is joined by a second kernel from the parts that the first leaves in the workspace, in
// their order: results do not depend on scheduling.
#include <cuda_bf16.h>

#include <algorithm>
#include <atomic>
#include <type_traits>

#include "kq_kv4.cuh"
#include "kq_q8_rows.cuh"
#include "kq_types.cuh"

namespace kq {
namespace {

constexpr int kWarps = 4, kThreads = 32 * kWarps;
constexpr float kLow = -1e30f;          // the maximum before any score
constexpr float kAhead = 4.f;           // how far a score may pass the maximum (log2) before it is moved
constexpr float kTop = 11.f;            // weights are 2^(score - maximum + kTop): 2^15 at most
constexpr int kSegmentUnits = 4;        // what beginning and ending a segment costs, in granules
constexpr int kLeastUnits = 12;         // the shortest run of a CTA

struct Attn {
  AttnArgs a;
  KvCache c;
  float* parts;              // [CTAs][2]: unfinished segments, kPart floats each
  int4* meta;                // [CTAs]: what part 1 is (sequence or -1, key head, tile, parts)
  int group;                 // query heads of a key head
  bool vec;                  // rows of Q (and of O) lie on 16-byte boundaries
  int* err;
};

template <int D, int R>
constexpr int kPart = R * D + 2 * R;    // sums [R][D], then maxima [R] and totals [R]

__device__ __forceinline__ void mma_f16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                        uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
// The transpose of an 8 x 8 matrix of fp16 held two to a lane.
__device__ __forceinline__ uint32_t transpose8(uint32_t v) {
  uint32_t r;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(v));
  return r;
}
__device__ __forceinline__ uint32_t pack_half2(float lo, float hi) { return half2_bits(__floats2half2_rn(lo, hi)); }
__device__ __forceinline__ float low_part(float v) { return v - __half2float(__float2half_rn(v)); }
__device__ __forceinline__ float exp2_fast(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}
__device__ __forceinline__ float pow2(int e) { return __uint_as_float(static_cast<uint32_t>(127 + e) << 23); }
__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// A sequence's rows and the granules that any of them sees.
struct Sequence {
  int64_t n0, len;
  int rows;                  // new rows
  int tiles;                 // of R rows (row, query head of the key head)
  int first, granules;       // of 16 places
  __device__ __forceinline__ void load(const Attn& p, int64_t b, int R) {
    n0 = p.a.q_start ? p.a.q_start[b] : b;
    const int64_t n1 = p.a.q_start ? min(static_cast<int64_t>(p.a.q_start[b + 1]), p.a.N) : b + 1;
    rows = n0 < 0 || n1 <= n0 ? 0 : static_cast<int>(n1 - n0);
    len = max(0, p.a.kv_len[b]);
    tiles = (static_cast<int64_t>(rows) * p.group + R - 1) / R;
    // The first row sees the earliest places, the last row the latest.
    const int64_t begin = p.a.window > 0 ? max(int64_t(0), len - rows + 1 - p.a.window) : 0;
    first = static_cast<int>(begin >> 4);
    granules = len > begin ? static_cast<int>((len + 15) >> 4) - first : 0;
  }
  __device__ __forceinline__ int64_t units(int heads) const {
    return static_cast<int64_t>(heads) * tiles * (kSegmentUnits + granules);
  }
};

// One row's outputs, eight elements v of a lane, the row's D / 8 lanes side by side. All lanes of the warp call it.
template <typename T, int D>
__device__ __forceinline__ void store_row(const Attn& p, bool here, int64_t n, int hq, int lane8, const float (&v)[8]) {
  if (p.a.O && here) {
    T* o = static_cast<T*>(p.a.O) + n * p.a.ldo + static_cast<int64_t>(hq) * D + 8 * lane8;
    if (p.vec) store8<T, true>(o, v);
    else store8<T, false>(o, v);
  }
  if (p.a.Xq) store_q8_block(v, p.a.Xq + ((n * p.a.n_q + hq) * (D / 32) + (lane8 >> 2)) * Q8_1_BYTES, here);
}

template <typename T, int D, int NT>
struct Shape {
  static constexpr int R = 8 * NT;
  static constexpr bool kSplit = sizeof(T) == 4;
  static constexpr int kStages = D == 64 ? 5 : D == 128 ? 4 : 3;
  static constexpr int kCtas = D == 256 ? (kSplit ? 2 : 3) : NT == 2 ? (kSplit ? 2 : 3) : (kSplit ? 3 : 4);
  static constexpr int kRing = kWarps * kStages * Granule<D>::kBytes;
  static constexpr int kPitch = D + 4;                                // of the sums that the warps join
  static constexpr size_t kSmem = kRing + (R * kPitch + 2 * kWarps * R) * sizeof(float);
};

template <typename T, int D, int NT>
__global__ void __launch_bounds__(kThreads, Shape<T, D, NT>::kCtas) attn_q4_kernel(const Attn p) {
  using Gr = Granule<D>;
  using Sh = Shape<T, D, NT>;
  constexpr int G = Gr::G, R = Sh::R, S = Sh::kStages;
  constexpr bool kSplit = Sh::kSplit;
  constexpr uint32_t M0 = 0x000f000fu, M1 = 0x00f000f0u;
  extern __shared__ __align__(16) uint8_t smem[];
  __shared__ int64_t scan[kWarps + 3];
  float* joined = reinterpret_cast<float*>(smem + Sh::kRing);         // [R][kPitch]
  float* stat = joined + R * Sh::kPitch;                              // maxima [kWarps][R], totals [kWarps][R]
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, gid = lane >> 2, tig = lane & 3;
  const uint8_t* ring = smem + warp * (S * Gr::kBytes);
  const uint32_t ring_u = smem_u32(ring);
  pdl_enter();

  // This CTA's run [u, u1) of the line, and the sequence that it begins in.
  const int64_t B = p.c.n_seqs;
  int64_t total = 0, u, u1, per, seq_at = 0, b = 0;
  {
    auto block_scan = [&](int64_t v, int64_t& sum) {                  // sum of the threads before this one; of all
      int64_t x = v;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int64_t y = __shfl_up_sync(0xffffffffu, x, o);
        if (lane >= o) x += y;
      }
      __syncthreads();
      if (lane == 31) scan[warp] = x;
      __syncthreads();
      int64_t before = 0;
      sum = 0;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) {
        before += w < warp ? scan[w] : 0;
        sum += scan[w];
      }
      return before + x - v;
    };
    auto units_of = [&](int64_t i) {
      if (i >= B) return int64_t(0);
      Sequence s;
      s.load(p, i, R);
      return s.units(p.c.heads);
    };
    int64_t sum, mine = 0;
    for (int64_t i = threadIdx.x; i < B; i += kThreads) mine += units_of(i);
    block_scan(mine, total);
    per = max(static_cast<int64_t>(kLeastUnits), (total + gridDim.x - 1) / gridDim.x);
    u = blockIdx.x * per;
    u1 = min(u + per, total);
    if (threadIdx.x == 0) p.meta[blockIdx.x] = make_int4(-1, 0, 0, 0);
    if (u >= u1) return;
    for (int64_t i = 0, at = 0; i < B; i += kThreads) {
      const int64_t v = units_of(i + threadIdx.x), x = at + block_scan(v, sum);
      if (x <= u && u < x + v) {
        scan[kWarps] = i + threadIdx.x;
        scan[kWarps + 1] = x;
      }
      at += sum;
      if (at > u) break;
    }
    __syncthreads();
    b = scan[kWarps];
    seq_at = scan[kWarps + 1];
  }
  Sequence q;
  q.load(p, b, R);

  while (u < u1) {
    // The segment that u lies in: [at, end) of the line.
    const int size = kSegmentUnits + q.granules;
    const int seg = static_cast<int>((u - seq_at) / size);
    const int64_t at = seq_at + static_cast<int64_t>(seg) * size, end = at + size;
    const int h = seg / q.tiles, tile = seg - h * q.tiles;
    const bool begins = u == at, ends = end <= u1;
    int g0 = max(0, static_cast<int>(u - at) - kSegmentUnits), g1 = max(0, static_cast<int>(min(end, u1) - at) - kSegmentUnits);

    // Row r of the tile: new row i = r' / group, head r' % group, r' = tile * R + r. See [low, seen).
    const int rows = q.rows * p.group;
    auto row_of = [&](int r, int& i, int& hq) {
      const int rr = tile * R + r;
      i = rr / p.group;
      hq = h * p.group + rr - i * p.group;
      return rr < rows;
    };
    auto seen_of = [&](int i) { return static_cast<int>(q.len) - q.rows + 1 + i; };
    auto low_of = [&](int seen) { return p.a.window > 0 ? static_cast<int>(max(int64_t(0), seen - p.a.window)) : 0; };
    const int i_first = tile * R / p.group, i_last = min(tile * R + R, rows) - 1 < 0 ? 0 : (min(tile * R + R, rows) - 1) / p.group;
    const int seen_most = seen_of(i_last), seen_least = seen_of(i_first);
    const int low_least = low_of(seen_least), low_most = low_of(seen_most);
    // Granules that a row of this tile sees, of those of the run.
    g0 = max(g0 + q.first, low_least >> 4);
    g1 = min(g1 + q.first, (seen_most + 15) >> 4);
    const int mine = g1 > g0 + warp ? (g1 - g0 - warp + kWarps - 1) / kWarps : 0;

    // Copies of this warp's granules g0 + warp + k * kWarps, S - 1 ahead; the page of the next is looked up one ahead.
    const int per_page = p.c.page_shift - 4;
    const int64_t head_at = static_cast<int64_t>(h) << per_page;
    const int32_t* table = p.c.table + b * p.c.ldt;
    auto page_of = [&](int k) {
      const int64_t i = static_cast<int64_t>(g0 + warp + k * kWarps) >> per_page;
      return k < mine && i < p.c.ldt ? table[i] : -1;
    };
    int page = page_of(0);
    uint32_t missing = 0;                                             // bit k % S: granule k has no page
    auto issue = [&](int k) {
      if (k < mine) {
        const int slot = k % S;
        const bool there = page >= 0 && page < p.c.n_pages;
        missing = there ? missing & ~(1u << slot) : missing | (1u << slot);
        if (there) {
          const int64_t gr = ((static_cast<int64_t>(page) * p.c.heads) << per_page) + head_at +
                             ((g0 + warp + k * kWarps) & ((1 << per_page) - 1));
          const uint8_t* src = p.c.data + gr * Gr::kBytes + 16 * lane;
          const uint32_t dst = ring_u + slot * Gr::kBytes + 16 * lane;
#pragma unroll
          for (int i = 0; i < (Gr::kBytes + 511) / 512; ++i)
            if (Gr::kBytes % 512 == 0 || 512 * i + 16 * lane < Gr::kBytes) cp_async16(dst + 512 * i, src + 512 * i);
        } else if (lane == 0) {
          report_error(p.err, ERR_PAGE);
        }
        page = page_of(k + 1);
      }
      cp_commit();
    };
#pragma unroll
    for (int k = 0; k < S - 1; ++k) issue(k);

    // Queries as operands: lane (gid, tig) has of row gid the elements 32 g + 8 tig + 0..7, times 2^a with the
    // row's largest between 2^14 and 2^15 (so that fp16 and bf16 queries are exact), the odd ones
    // also times 2^-4 for the codes that are four bits higher.
    uint32_t qb[NT][G][2][2], ql[kSplit ? NT : 1][kSplit ? G : 1][2][2], qs[NT][(G + 3) / 4][2];
    float factor[NT][2];                                              // of the scores of columns 2 tig, 2 tig + 1
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      int i, hq;
      const bool here = row_of(8 * nt + gid, i, hq);
      const T* src = static_cast<const T*>(p.a.Q) + (q.n0 + i) * p.a.ldq + static_cast<int64_t>(hq) * D + 8 * tig;
      float v[G][8], top = 0.f, sums[G];
#pragma unroll
      for (int g = 0; g < G; ++g) {
        if (!here) {
#pragma unroll
          for (int j = 0; j < 8; ++j) v[g][j] = 0.f;
        } else if (p.vec) {
          load8<T, true>(src + 32 * g, v[g]);
        } else {
          load8<T, false>(src + 32 * g, v[g]);
        }
#pragma unroll
        for (int j = 0; j < 8; ++j) top = fmaxf(top, fabsf(v[g][j]));
      }
      top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
      top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
      // 2^e <= top < 2^(e + 1); rows below 2^-86 have scores of nothing, and those beyond 2^118 are NaN all over.
      const int e = max(-86, min(127, static_cast<int>(__float_as_uint(top) >> 23) - 127));
      const float up1 = pow2((14 - e) >> 1), up2 = pow2(14 - e - ((14 - e) >> 1));
#pragma unroll
      for (int g = 0; g < G; ++g) {
        sums[g] = 0.f;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          v[g][j] = v[g][j] * up1 * up2;
          sums[g] += v[g][j];
        }
        sums[g] += __shfl_xor_sync(0xffffffffu, sums[g], 1);
        sums[g] += __shfl_xor_sync(0xffffffffu, sums[g], 2);
        sums[g] *= 0x1p-6f;
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          const float x0 = v[g][2 * k], x4 = v[g][2 * k + 4], x1 = v[g][2 * k + 1] * 0.0625f, x5 = v[g][2 * k + 5] * 0.0625f;
          qb[nt][g][k][0] = pack_half2(x0, x4);
          qb[nt][g][k][1] = pack_half2(x1, x5);
          if constexpr (kSplit) {
            ql[nt][g][k][0] = pack_half2(low_part(x0), low_part(x4));
            ql[nt][g][k][1] = pack_half2(low_part(x1), low_part(x5));
          }
        }
        // The blocks' sums in three parts of fp16, one for each of the lanes tig = 0, 1, 2.
        float part = sums[g];
        if (tig > 0) part = low_part(part);
        if (tig > 1) part = low_part(part);
        sums[g] = tig > 2 ? 0.f : part;
      }
#pragma unroll
      for (int k = 0; k < (G + 3) / 4; ++k) {
        qs[nt][k][0] = pack_half2(sums[4 * k], sums[4 * k + 1]);
        qs[nt][k][1] = G > 2 ? pack_half2(sums[(4 * k + 2) % G], sums[(4 * k + 3) % G]) : 0u;
      }
      const float f = top < 0x1p118f ? p.a.scale * 1.44269504f * pow2(10 + min(e, 117)) : NAN;
#pragma unroll
      for (int c = 0; c < 2; ++c) factor[nt][c] = __shfl_sync(0xffffffffu, f, 4 * (2 * tig + c));
    }

    float o[NT][G][2][4], om[NT][4], top[NT][2];
    int sigma = -24;                                                  // weights are relative to 2^sigma
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      top[nt][0] = top[nt][1] = kLow;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        om[nt][j] = 0.f;
#pragma unroll
        for (int g = 0; g < G; ++g) o[nt][g][0][j] = o[nt][g][1][j] = 0.f;
      }
    }

    // Rows 0..15 of the operands are places in this order, so that the value codes of lanes side by side lie in
    // different banks: row r is place r / 2 + 4 (r % 2), of the lower or upper eight.
    const int ta = (gid >> 1) + 4 * (gid & 1);
    auto granule = [&](auto edge_tag, const uint8_t* gr, int place0) {
      constexpr bool kEdge = decltype(edge_tag)::value;
      float s[NT][4];
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int j = 0; j < 4; ++j) s[nt][j] = 0.f;
      {
        uint32_t ka[G], kb[G], pa[G], pb[G];                          // pa, pb: G / 2 words of s, then G / 2 of m
        auto words = [](uint32_t (&w)[G], const uint8_t* src) {
          if constexpr (G == 2) {
            *reinterpret_cast<uint2*>(w) = *reinterpret_cast<const uint2*>(src);
          } else {
#pragma unroll
            for (int i = 0; i < G / 4; ++i) *reinterpret_cast<uint4*>(w + 4 * i) = reinterpret_cast<const uint4*>(src)[i];
          }
        };
        words(ka, gr + ta * (D / 2) + tig * (4 * G));
        words(kb, gr + (ta + 8) * (D / 2) + tig * (4 * G));
        words(pa, gr + Gr::kCodes + ta * (4 * G));
        words(pb, gr + Gr::kCodes + (ta + 8) * (4 * G));
        float sm[NT][4];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
          for (int j = 0; j < 4; ++j) sm[nt][j] = 0.f;
          if constexpr (G == 2) {
            mma_f16(sm[nt], pa[1], pb[1], 0u, 0u, qs[nt][0][0], 0u);
          } else {
#pragma unroll
            for (int k = 0; k < G / 4; ++k)
              mma_f16(sm[nt], pa[G / 2 + 2 * k], pb[G / 2 + 2 * k], pa[G / 2 + 2 * k + 1], pb[G / 2 + 2 * k + 1], qs[nt][k][0],
                      qs[nt][k][1]);
          }
        }
#pragma unroll
        for (int g = 0; g < G; ++g) {
          const float2 sa2 = __half22float2(bits_half2(pa[g / 2])), sb2 = __half22float2(bits_half2(pb[g / 2]));
          const float sa = g & 1 ? sa2.y : sa2.x, sb = g & 1 ? sb2.y : sb2.x;
          const uint32_t a0 = ka[g] & M0, a1 = kb[g] & M0, a2 = ka[g] & M1, a3 = kb[g] & M1;
          const uint32_t c0 = (ka[g] >> 8) & M0, c1 = (kb[g] >> 8) & M0, c2 = (ka[g] >> 8) & M1, c3 = (kb[g] >> 8) & M1;
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) {
            float acc[4] = {0.f, 0.f, 0.f, 0.f};
            mma_f16(acc, a0, a1, a2, a3, qb[nt][g][0][0], qb[nt][g][0][1]);
            mma_f16(acc, c0, c1, c2, c3, qb[nt][g][1][0], qb[nt][g][1][1]);
            if constexpr (kSplit) {
              mma_f16(acc, a0, a1, a2, a3, ql[nt][g][0][0], ql[nt][g][0][1]);
              mma_f16(acc, c0, c1, c2, c3, ql[nt][g][1][0], ql[nt][g][1][1]);
            }
            s[nt][0] = fmaf(sa, acc[0], s[nt][0]);
            s[nt][1] = fmaf(sa, acc[1], s[nt][1]);
            s[nt][2] = fmaf(sb, acc[2], s[nt][2]);
            s[nt][3] = fmaf(sb, acc[3], s[nt][3]);
          }
        }
        // Sum s acc is of 2^(a - 24) q . (k - m), sm of 2^(a - 6) q . m.
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int j = 0; j < 4; ++j) s[nt][j] = fmaf(sm[nt][j], 0x1p-18f, s[nt][j]) * factor[nt][j & 1];
      }
      const bool out_a = kEdge && (place0 + ta < low_least || place0 + ta >= seen_most);
      const bool out_b = kEdge && (place0 + ta + 8 < low_least || place0 + ta + 8 >= seen_most);
      if constexpr (kEdge) {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            int i, hq;
            row_of(8 * nt + 2 * tig + (j & 1), i, hq);
            const int seen = seen_of(i), place = place0 + ta + (j < 2 ? 0 : 8);
            if (place >= seen || place < low_of(seen)) s[nt][j] = -INFINITY;
          }
      }

      // Parameters of the values: of places ta and ta + 8 the s, as halves.
      const uint8_t* vp = gr + Gr::kValues + Gr::kCodes;
      uint32_t va[G / 2], vb[G / 2];
      if constexpr (G == 2) {
        va[0] = *reinterpret_cast<const uint32_t*>(vp + ta * (4 * G));
        vb[0] = *reinterpret_cast<const uint32_t*>(vp + (ta + 8) * (4 * G));
      } else {
#pragma unroll
        for (int i = 0; i < G / 4; ++i) {
          *reinterpret_cast<uint2*>(va + 2 * i) = reinterpret_cast<const uint2*>(vp + ta * (4 * G))[i];
          *reinterpret_cast<uint2*>(vb + 2 * i) = reinterpret_cast<const uint2*>(vp + (ta + 8) * (4 * G))[i];
        }
      }
      if constexpr (kEdge) {
#pragma unroll
        for (int i = 0; i < G / 2; ++i) {
          if (out_a) va[i] = 0;
          if (out_b) vb[i] = 0;
        }
      }
      // The largest s of the granule: a NaN counts for nothing, an infinity as fp16's largest.
      __half2 big = __habs2(bits_half2(va[0]));
#pragma unroll
      for (int i = 0; i < G / 2; ++i) big = __hmax2(big, __hmax2(__habs2(bits_half2(va[i])), __habs2(bits_half2(vb[i]))));
      const float largest = fminf(fmaxf(__low2float(big), __high2float(big)), 65504.f);

      bool move = largest > pow2(sigma);
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int j = 0; j < 4; ++j) move |= s[nt][j] > top[nt][j & 1] + kAhead;
      if (__any_sync(0xffffffffu, move)) {
        const uint32_t bits = __reduce_max_sync(0xffffffffu, __float_as_uint(largest > 0.f ? largest : 0.f));
        const int want = max(sigma, static_cast<int>((bits + 0x007fffffu) >> 23) - 127);   // the power of two not below it
        const float by = pow2(max(-126, sigma - want));
        sigma = want;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            float m = fmaxf(s[nt][c], s[nt][c + 2]);
            m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 4));
            m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 8));
            m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 16));
            m = fmaxf(m, top[nt][c]);
            const float f = exp2_fast(top[nt][c] - m), fs = f * by;
            top[nt][c] = m;
            om[nt][c] *= f;
            om[nt][c + 2] *= f;
#pragma unroll
            for (int g = 0; g < G; ++g)
#pragma unroll
              for (int k = 0; k < 2; ++k) {
                o[nt][g][k][c] *= fs;
                o[nt][g][k][c + 2] *= fs;
              }
          }
      }

      // Weights: of the codes' sums relative to 2^sigma.
      const float up = pow2(sigma);
      uint32_t pb2[NT][2];
      [[maybe_unused]] uint32_t pl2[kSplit ? NT : 1][2];
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        const float b0 = top[nt][0] + (static_cast<float>(sigma) - kTop), b1 = top[nt][1] + (static_cast<float>(sigma) - kTop);
#pragma unroll
        for (int j = 0; j < 4; ++j) s[nt][j] = exp2_fast(s[nt][j] - (j & 1 ? b1 : b0));
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          const float x = s[nt][2 * k] * up, y = s[nt][2 * k + 1] * up;
          pb2[nt][k] = transpose8(pack_half2(x, y));
          if constexpr (kSplit) pl2[nt][k] = transpose8(pack_half2(low_part(x), low_part(y)));
        }
      }

      // The m of the values and a row of ones: rows g < G are the blocks' m, row 8 (or a row of the lower eight) the ones.
      {
        uint32_t m0 = 0, m1 = 0;
        if (gid < G) {
          const uint8_t* mp = vp + 2 * G + 2 * gid;
          const auto half_at = [&](int place) -> uint32_t {
            const uint32_t v = *reinterpret_cast<const uint16_t*>(mp + place * (4 * G));
            return kEdge && (place0 + place < low_least || place0 + place >= seen_most) ? 0u : v;
          };
          m0 = half_at(tig) | half_at(tig + 4) << 16;
          m1 = half_at(tig + 8) | half_at(tig + 12) << 16;
        }
        const uint32_t one = gid == 0 ? 0x3c003c00u : 0u;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          mma_f16(om[nt], m0, one, m1, one, pb2[nt][0], pb2[nt][1]);
          if constexpr (kSplit) mma_f16(om[nt], m0, one, m1, one, pl2[nt][0], pl2[nt][1]);
        }
      }

      // The values' codes: of places tig, tig + 4, tig + 8, tig + 12 four elements of each block (row gid of the operand
      // the first of them, row gid + 8 the second, and so on).
      const uint8_t* vc = gr + Gr::kValues + gid * (2 * G);
      uint32_t w[4][G / 2];
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const uint8_t* src = vc + (tig + 4 * k) * (D / 2);
        if constexpr (G == 2) {
          w[k][0] = *reinterpret_cast<const uint32_t*>(src);
        } else {
#pragma unroll
          for (int i = 0; i < G / 4; ++i) *reinterpret_cast<uint2*>(&w[k][2 * i]) = reinterpret_cast<const uint2*>(src)[i];
        }
      }
#pragma unroll
      for (int g = 0; g < G; ++g) {
        const float2 sa2 = __half22float2(bits_half2(va[g / 2])), sb2 = __half22float2(bits_half2(vb[g / 2]));
        const float sa = g & 1 ? sa2.y : sa2.x, sb = g & 1 ? sb2.y : sb2.x;
        const uint32_t pick = g & 1 ? 0x7632u : 0x5410u;
        const uint32_t x = __byte_perm(w[0][g / 2], w[1][g / 2], pick), y = __byte_perm(w[2][g / 2], w[3][g / 2], pick);
        const uint32_t a0 = x & M0, a1 = x & M1, a2 = y & M0, a3 = y & M1;
        const uint32_t c0 = (x >> 8) & M0, c1 = (x >> 8) & M1, c2 = (y >> 8) & M0, c3 = (y >> 8) & M1;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          float t[4] = {s[nt][0] * sa, s[nt][1] * sa, s[nt][2] * sb, s[nt][3] * sb};
          if constexpr (kEdge) {                                      // a NaN of a place that a row does not see
#pragma unroll
            for (int j = 0; j < 4; ++j) t[j] = s[nt][j] == 0.f ? 0.f : t[j];
          }
          const uint32_t b0 = transpose8(pack_half2(t[0], t[1])), b1 = transpose8(pack_half2(t[2], t[3]));
          mma_f16(o[nt][g][0], a0, a1, a2, a3, b0, b1);
          mma_f16(o[nt][g][1], c0, c1, c2, c3, b0, b1);
          if constexpr (kSplit) {
            const uint32_t l0 = transpose8(pack_half2(low_part(t[0]), low_part(t[1])));
            const uint32_t l1 = transpose8(pack_half2(low_part(t[2]), low_part(t[3])));
            mma_f16(o[nt][g][0], a0, a1, a2, a3, l0, l1);
            mma_f16(o[nt][g][1], c0, c1, c2, c3, l0, l1);
          }
        }
      }
    };

    for (int k = 0; k < mine; ++k) {
      cp_wait<S - 2>();
      __syncwarp();
      const bool gone = (missing >> (k % S)) & 1;
      issue(k + S - 1);
      if (gone) continue;
      const int place0 = 16 * (g0 + warp + k * kWarps);
      const uint8_t* gr = ring + (k % S) * Gr::kBytes;
      if (place0 >= low_most && place0 + 16 <= seen_least) granule(std::false_type{}, gr, place0);
      else granule(std::true_type{}, gr, place0);
    }
    cp_wait<0>();

    // The warps' sums joined, one warp after the other.
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int c = 0; c < 2; ++c)
        if (gid == 0) {
          stat[warp * R + 8 * nt + 2 * tig + c] = top[nt][c];
          stat[(kWarps + warp) * R + 8 * nt + 2 * tig + c] = om[nt][c + 2];
        }
    __syncthreads();
    const float up = 0x1p24f * pow2(sigma);
#pragma unroll 1
    for (int turn = 0; turn < kWarps; ++turn) {
      if (warp == turn) {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            const int r = 8 * nt + 2 * tig + c;
            float most = stat[r];
#pragma unroll
            for (int w = 1; w < kWarps; ++w) most = fmaxf(most, stat[w * R + r]);
            const float f = exp2_fast(top[nt][c] - most);
#pragma unroll
            for (int g = 0; g < G; ++g) {
              const float m = __shfl_sync(0xffffffffu, om[nt][c], 4 * g + tig);
              float4 v = make_float4(fmaf(o[nt][g][0][c], up, m) * f, fmaf(o[nt][g][0][c + 2], up * 0.0625f, m) * f,
                                     fmaf(o[nt][g][1][c], up, m) * f, fmaf(o[nt][g][1][c + 2], up * 0.0625f, m) * f);
              float4* dst = reinterpret_cast<float4*>(joined + r * Sh::kPitch + 32 * g + 4 * gid);
              if (turn > 0) {
                const float4 x = *dst;
                v = make_float4(x.x + v.x, x.y + v.y, x.z + v.z, x.w + v.w);
              }
              *dst = v;
            }
          }
      }
      __syncthreads();
    }

    // Outputs of a whole segment; else a part for the second kernel.
    constexpr int L = D / 8;                                          // lanes of a row
    float* part = p.parts + (2 * static_cast<int64_t>(blockIdx.x) + (begins ? 1 : 0)) * kPart<D, R>;
#pragma unroll 1
    for (int r0 = 0; r0 < R; r0 += kThreads / L) {
      const int r = r0 + threadIdx.x / L, l8 = threadIdx.x % L;
      int i = 0, hq = 0;
      const bool here = r < R && row_of(r, i, hq);
      float v[8], most = kLow, sum = 0.f;
      if (r < R) {
#pragma unroll
        for (int w = 0; w < kWarps; ++w) most = fmaxf(most, stat[w * R + r]);
#pragma unroll
        for (int w = 0; w < kWarps; ++w) sum = fmaf(stat[(kWarps + w) * R + r], exp2_fast(stat[w * R + r] - most), sum);
#pragma unroll
        for (int j = 0; j < 2; ++j)
          *reinterpret_cast<float4*>(v + 4 * j) = *reinterpret_cast<const float4*>(joined + r * Sh::kPitch + 8 * l8 + 4 * j);
      }
      if (begins && ends) {
        const float inv = sum == 0.f ? 0.f : __fdiv_rn(1.0f, sum);    // a row that sees nothing
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] = sum == 0.f ? 0.f : v[j] * inv;
        store_row<T, D>(p, here, q.n0 + i, hq, l8, v);
      } else if (r < R) {
#pragma unroll
        for (int j = 0; j < 2; ++j)
          *reinterpret_cast<float4*>(part + r * D + 8 * l8 + 4 * j) = *reinterpret_cast<const float4*>(v + 4 * j);
        if (l8 == 0) {
          part[R * D + r] = most;
          part[R * D + R + r] = sum;
        }
      }
    }
    if (begins && !ends && threadIdx.x == 0)
      p.meta[blockIdx.x] = make_int4(static_cast<int>(b), h, tile, static_cast<int>((end - 1) / per - blockIdx.x) + 1);
    __syncthreads();

    // On to the next segment, in this sequence or the next that has any.
    u = min(end, u1);
    if (u < u1) {
      int64_t n = q.units(p.c.heads);
      while (u >= seq_at + n) {
        seq_at += n;
        q.load(p, ++b, R);
        n = q.units(p.c.heads);
      }
    }
  }
}

// The segments that several CTAs had parts of: for the CTA blockIdx.x that began one, row blockIdx.y of its tile.
template <typename T, int D, int R>
__global__ void __launch_bounds__(kThreads) attn_q4_join_kernel(const Attn p) {
  constexpr int L4 = D / 4, P = kThreads / L4;                        // lanes of a row, parts read at a time
  extern __shared__ float weight[];
  __shared__ float red[kWarps], sums[P][D];
  pdl_enter();
  const int4 meta = p.meta[blockIdx.x];
  if (meta.x < 0) return;
  const int r = blockIdx.y, rr = meta.z * R + r, i = rr / p.group, hq = meta.y * p.group + rr - i * p.group;
  Sequence q;
  q.load(p, meta.x, R);
  if (rr >= q.rows * p.group) return;
  const float* base = p.parts + 2 * static_cast<int64_t>(blockIdx.x) * kPart<D, R>;
  auto part = [&](int k) { return base + (k == 0 ? 1 : 2 * static_cast<int64_t>(k)) * kPart<D, R>; };
  float most = kLow;
  for (int k = threadIdx.x; k < meta.w; k += kThreads) most = fmaxf(most, part(k)[R * D + r]);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) most = fmaxf(most, __shfl_xor_sync(0xffffffffu, most, o));
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = most;
  __syncthreads();
  most = red[0];
#pragma unroll
  for (int w = 1; w < kWarps; ++w) most = fmaxf(most, red[w]);
  float sum = 0.f;
  for (int k = threadIdx.x; k < meta.w; k += kThreads) {
    weight[k] = exp2_fast(part(k)[R * D + r] - most);
    sum = fmaf(weight[k], part(k)[R * D + R + r], sum);
  }
  sum = warp_sum_f(sum);
  __syncthreads();
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = sum;
  __syncthreads();
  sum = red[0];
#pragma unroll
  for (int w = 1; w < kWarps; ++w) sum += red[w];
  const int l4 = threadIdx.x % L4, k0 = threadIdx.x / L4;
  float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
  for (int k = k0; k < meta.w; k += P) {
    const float4 v = *reinterpret_cast<const float4*>(part(k) + r * D + 4 * l4);
    const float f = weight[k];
    acc = make_float4(fmaf(f, v.x, acc.x), fmaf(f, v.y, acc.y), fmaf(f, v.z, acc.z), fmaf(f, v.w, acc.w));
  }
  *reinterpret_cast<float4*>(&sums[k0][4 * l4]) = acc;
  __syncthreads();
  if (threadIdx.x >= 32) return;
  const int l8 = threadIdx.x;
  const bool here = l8 < D / 8;
  const float inv = sum == 0.f ? 0.f : __fdiv_rn(1.0f, sum);
  float v[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    v[j] = 0.f;
    if (here)
      for (int k = 0; k < P; ++k) v[j] += sums[k][8 * l8 + j];
    v[j] = sum == 0.f ? 0.f : v[j] * inv;
  }
  store_row<T, D>(p, here, q.n0 + i, hq, l8, v);
}

// Rows of a tile: 8 where a sequence's (row, query head) pairs are 8 or fewer on the average, else 16 (of heads of 256
// elements always 8: their sums are 128 registers for 16 rows).
int tile_rows(int group, int D, int64_t N, int64_t n_seqs) { return D == 256 || group * N <= 8 * n_seqs ? 8 : 16; }

template <typename T, int D, int NT>
cudaError_t run(const Attn& p, int num_sms, cudaStream_t s) {
  using Sh = Shape<T, D, NT>;
  static std::atomic<uint64_t> allowed{0};                            // devices on which the shared memory is set
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 64 && !(allowed.load(std::memory_order_acquire) >> dev & 1)) {
    e = cudaFuncSetAttribute(attn_q4_kernel<T, D, NT>, cudaFuncAttributeMaxDynamicSharedMemorySize, Sh::kSmem);
    if (e != cudaSuccess) return e;
    allowed.fetch_or(uint64_t(1) << dev, std::memory_order_release);
  }
  const int grid = num_sms * Sh::kCtas;
  e = launch_pdl(attn_q4_kernel<T, D, NT>, dim3(grid), dim3(kThreads), Sh::kSmem, s, p);
  if (e != cudaSuccess) return e;
  return launch_pdl(attn_q4_join_kernel<T, D, Sh::R>, dim3(grid, Sh::R), dim3(kThreads), grid * sizeof(float), s, p);
}

template <typename T>
cudaError_t run(const Attn& p, int num_sms, cudaStream_t s) {
  const bool wide = tile_rows(p.group, p.c.D, p.a.N, p.c.n_seqs) == 16;
  if (p.c.D == 64) return wide ? run<T, 64, 2>(p, num_sms, s) : run<T, 64, 1>(p, num_sms, s);
  if (p.c.D == 128) return wide ? run<T, 128, 2>(p, num_sms, s) : run<T, 128, 1>(p, num_sms, s);
  return run<T, 256, 1>(p, num_sms, s);
}

constexpr int kMostCtas = 4;            // of an SM, of any form

}  // namespace

size_t attn_q4_workspace(int n_q, int n_kv, int D, int64_t N, int64_t n_seqs, int num_sms) {
  const int R = tile_rows(n_q / n_kv, D, N, n_seqs);
  const size_t ctas = static_cast<size_t>(num_sms) * kMostCtas;
  return ctas * (sizeof(int4) + 2 * sizeof(float) * (static_cast<size_t>(R) * D + 2 * R));
}

cudaError_t launch_attn_q4(int dtype, const AttnArgs& a, const KvCache& c, void* ws, int* err, int num_sms, cudaStream_t s) {
  const int64_t size = dtype == KQ_F32 ? 4 : 2;
  Attn p = {a, c, nullptr, static_cast<int4*>(ws), a.n_q / c.heads,
            a.ldq * size % 16 == 0 && (!a.O || a.ldo * size % 16 == 0), err};
  p.parts = reinterpret_cast<float*>(p.meta + static_cast<size_t>(num_sms) * kMostCtas);
  if (dtype == KQ_F16) return run<__half>(p, num_sms, s);
  if (dtype == KQ_BF16) return run<__nv_bfloat16>(p, num_sms, s);
  return run<float>(p, num_sms, s);
}

}  // namespace kq
