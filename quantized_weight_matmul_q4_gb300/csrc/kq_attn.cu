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
//   o       = Sum_g Sum_t (p_t s_tg) (c_tg - 8) + Sum_t p_t (m_tg + 8 s_tg)
// The first sum of each is a product of codes per block, scaled after (scores) or before (weights). Without the 8 both sums of
// o are many times as large as their difference where many tokens count, and the tensor cores' additions, which cut
// off, would show (8192 tokens: 1.8e-3 of o); it is one more product, with a constant operand. The second
// sum is a product of the m + 8 s, which also gives Sum_t p_t by a row of ones; it is taken for each step by itself and
// added in fp32.
//
// Scores are exact products summed in fp32. Weights are rounded to fp16 as operands (a relative 2^-11 at most each time,
// twice for those of the codes, which 16-bit outputs show in their last bit). For fp32 rows, and where Q8_1 rows are asked for (a code
// that a rounding moves is a whole step), weights are split into two halves, the codes are operands less 8, and sums of a granule
// are added in fp32; fp32 queries are split as well. A weight's products with s are relative to a power of two not below the largest
// s so far, so that none leaves fp16's range; the total and the sum of the m + 8 s take weights that are not.
//
// Work is shared out evenly whatever the sequences' lengths: all (sequence, key head, tile of rows) segments stand
// in one line, of which each warp takes an equal run. Where segments are few and short, the line is of pieces of so many steps of
// 32 places that there is at most one for each warp; else of steps, and a warp may have the end of a segment, others whole,
// and the beginning of one. The pieces of a segment in a CTA's warps are joined there; what lies in several CTAs is
// joined by a second kernel from the parts that the first leaves in the workspace. Both go by the
// order of the line: results do not depend on scheduling.
//
// What bounds it (one GB300, calls in a graph over caches larger than L2, both kernels): at many places the issue of instructions. A
// granule of 16 places of a head of 128 costs a warp 355 for up to 8 rows,
// nearly twice that where weights are split: 32 sequences of up to 32768 places, 64 query heads on 8 of 128, 72 us (0.67 of
// the copy bandwidth), one of 131072 with 32 heads on 8, 43 us (0.58). Below some 4000 places a sequence the ends bound it:
// finding the runs, pages and queries 3 to 4 us before the first step, 3 us for outputs and the second kernel. One sequence of
// 1000 places 14 us, 256 of up to 900 38 us (0.28). Tensor cores are a third busy, with mma.sync: the codes are
// operands as they lie in the cache's bytes, in registers; tcgen05 would take them from shared memory as 16-bit numbers, four times
// what was loaded to write and to read again, for tiles of which 8 of 128 rows are used.
#include <cuda_bf16.h>

#include <algorithm>
#include <atomic>
#include <type_traits>

#include "kq_kv4.cuh"
#include "kq_q8_rows.cuh"
#include "kq_types.cuh"

namespace kq {
namespace {

constexpr float kLow = -3.402823466e38f;           // the maximum before any score: no finite score is below it
constexpr float kAhead = 4.f;           // how far a score may pass the maximum (log2) before it is moved
constexpr float kTop = 10.f;            // weights are 2^(score - maximum + kTop): 2^14 at most
constexpr int kSegmentUnits = 3;        // what beginning and ending a segment costs, in steps of 32 places
constexpr int kLongPiece = 10;          // longer pieces' rounding costs more than runs that have parts of two segments (drafts of
                                        // 5 rows for 32 heads of 64: 23.6 us, with 5 steps 24.8; 64 sequences with 20: 34.3 for 32.3)
constexpr int kRound = 2;               // steps that a segment is cut by, and the fewest of a piece

struct Attn {
  AttnArgs a;
  KvCache c;
  float* parts;              // [CTAs][2]: pieces of segments that another CTA began, or ends; kPart floats each
  int4* meta;                // [CTAs][2]: what part 1 is (key head or -1, tile, parts; the sequence's first row, its pairs)
  int group;                 // query heads of a key head
  bool vec;                  // rows of Q (and of O) lie on 16-byte boundaries
  int* err;
};

template <int D, int R>
constexpr int kPart = R * D + 2 * R;    // sums [R][D], then maxima [R] and totals [R]

__device__ __forceinline__ void mma_f16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                        uint32_t b1) {
  asm(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
// The same beginning from zero.
__device__ __forceinline__ void mma_f16_zero(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                             uint32_t b1) {
  asm(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%10,%10,%10};"
      : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.f));
}
// The transpose of an 8 x 8 matrix of fp16 held two to a lane.
__device__ __forceinline__ uint32_t transpose8(uint32_t v) {
  uint32_t r;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(v));
  return r;
}
// The codes in bits AT to AT + 3 of both halves less 8, as fp16: in the low bits of 1024 or of 64 they add their value.
template <int AT>
__device__ __forceinline__ uint32_t codes_less_8(uint32_t w) {
  const uint32_t x = AT ? (w & 0x00f000f0u) | 0x54005400u : (w & 0x000f000fu) | 0x64006400u;
  return half2_bits(__hsub2(bits_half2(x), __float2half2_rn(AT ? 72.f : 1032.f)));
}
// Two 8 x 8 matrices of fp16 from shared memory, transposed: lanes 0..7 give the rows of the first, 8..15 of the second.
__device__ __forceinline__ void load_transposed(uint32_t& x, uint32_t& y, const void* row) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x2.trans.shared.b16 {%0,%1}, [%2];" : "=r"(x), "=r"(y) : "r"(smem_u32(row)));
}
__device__ __forceinline__ uint32_t pack_half2(float lo, float hi) { return half2_bits(__floats2half2_rn(lo, hi)); }
__device__ __forceinline__ float low_part(float v) { return v - __half2float(__float2half_rn(v)); }
__device__ __forceinline__ float exp2_fast(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}
__device__ __forceinline__ float pow2(int e) { return __uint_as_float(static_cast<uint32_t>(127 + e) << 23); }
// a / b of whole numbers that are seldom beyond 32 bits.
__device__ __forceinline__ int64_t quotient(int64_t a, int64_t b) {
  return (a | b) >> 32 == 0 ? static_cast<uint32_t>(a) / static_cast<uint32_t>(b) : a / b;
}

// a / b for 0 <= a, exactly: (a + 1/2) / b is at least 1 / (2 b) from a whole number, and the quotient, of 2 ulp at most, within
// 2^-22 of itself: 1 / (4 b) for a < 2^20, half of that distance.
__device__ __forceinline__ int divide(int a, int b) {
  return a < (1 << 20) ? static_cast<int>(__fdividef(static_cast<float>(a) + 0.5f, static_cast<float>(b))) : a / b;
}

// A sequence's rows and the steps of 32 places that any of them sees.
struct Sequence {
  int64_t n0;
  int len, rows;             // places; new rows
  int tiles;                 // of R rows (row, query head of the key head)
  int first, steps;
  __device__ __forceinline__ void load(const Attn& p, int64_t b, int R) {
    n0 = p.a.q_start ? p.a.q_start[b] : b;
    const int64_t n1 = p.a.q_start ? min(static_cast<int64_t>(p.a.q_start[b + 1]), p.a.N) : b + 1;
    rows = n0 < 0 || n1 <= n0 ? 0 : static_cast<int>(n1 - n0);
    len = max(0, p.a.kv_len[b]);
    tiles = (rows * p.group + R - 1) / R;
    // The first row sees the earliest places, the last row the latest.
    const int64_t begin = p.a.window > 0 ? max(int64_t(0), static_cast<int64_t>(len) - rows + 1 - p.a.window) : 0;
    first = static_cast<int>(begin >> 5);
    steps = len > begin ? ((len - 1) >> 5) + 1 - first : 0;
  }
};

// The line's units: pieces of `piece` steps, or (piece 0) steps, and kSegmentUnits for each segment.
struct Line {
  int piece;
  int64_t per;               // units of a run
  __device__ __forceinline__ int size(const Sequence& s) const {
    return piece ? max(1, (s.steps + piece - 1) / piece) : kSegmentUnits + s.steps;
  }
  __device__ __forceinline__ int64_t units(const Sequence& s, int heads) const {
    return static_cast<int64_t>(heads) * s.tiles * size(s);
  }
  // Where a cut `off` units into a segment of `size` is made: before it, after it, or after a whole number of rounds.
  __device__ __forceinline__ int64_t cut_at(int64_t off, int size) const {
    if (piece) return off;
    const int w = static_cast<int>(off) - kSegmentUnits;
    if (w <= 0) return 0;
    const int to = kSegmentUnits + (w + kRound - 1) / kRound * kRound;
    return to + kRound / 2 >= size ? size : to;
  }
  // The segment's steps before its unit `off`.
  __device__ __forceinline__ int steps_before(int64_t off, const Sequence& s) const {
    return piece ? static_cast<int>(min(off * piece, static_cast<int64_t>(s.steps))) : max(0, static_cast<int>(off) - kSegmentUnits);
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

template <typename T, int D, int NT, bool FINE>
struct Shape {
  static constexpr int R = 8 * NT;
  static constexpr bool kSplitQ = sizeof(T) == 4;                     // queries in two halves
  // Of a CTA, one to an SM: as many as have the registers that they need (8 heads of 128, 32 sequences of up to 32768
  // places: 12 warps 68 us at that time, 10 warps 75, 14 warps of 144 registers 87).
  static constexpr int kWarps = D == 256 ? 7 : NT == 2 || kSplitQ ? 8 : 12;
  static constexpr int kThreads = 32 * kWarps;
  static constexpr int kStep = 2 * Granule<D>::kBytes;
  static constexpr int kPitch = D + 4;                                // of the rows of a piece's sums
  static constexpr int kHeld = (R * kPitch * 4 + kStep - 1) / kStep;  // stages that a piece takes
  static constexpr int kStages = kHeld + (D == 64 ? 3 : 2);
  static constexpr int kRing = kStages * kStep;
  static constexpr size_t kSmem = static_cast<size_t>(kWarps) * kRing;
};

// What a warp leaves for its CTA: the piece of a segment that was begun before its run (it may end there), and of
// one that its run begins and does not end.
struct Piece {
  int64_t n0;                // the sequence's first row
  int h, tile, parts;        // key head, tile of rows; parts, where it begins a segment
  int rows;                  // (row, query head) pairs of the sequence and the key head
  bool begins, ends;
};

template <typename T, int D, int NT, bool FINE>
__global__ void __launch_bounds__(Shape<T, D, NT, FINE>::kThreads) attn_q4_kernel(const Attn p) {
  using Gr = Granule<D>;
  using Sh = Shape<T, D, NT, FINE>;
  constexpr int G = Gr::G, R = Sh::R, S = Sh::kStages, kWarps = Sh::kWarps, kThreads = Sh::kThreads, L = D / 8;
  constexpr bool kSplitQ = Sh::kSplitQ, kSplit = FINE;                // weights in two halves
  constexpr uint32_t M0 = 0x000f000fu, M1 = 0x00f000f0u;
  constexpr uint32_t kEven = 0x80088008u, kOdd = 0x80808080u;         // -8 as the codes are: times 2^-24, times 2^-20
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ int64_t scan[kWarps], cut_b[kWarps + 1], cut_seq[kWarps + 1], cut_u[kWarps + 1], first_unit[kThreads];
  __shared__ int segment_size[kThreads];
  __shared__ uint64_t full[kWarps][S];
  __shared__ int2 range[kWarps][R];                                   // what the rows of a tile see: [x, y)
  __shared__ Piece piece[kWarps][2];
  __shared__ float stat[kWarps][2][2][R];                             // maxima and totals of the pieces
  __shared__ uint32_t there;                                          // bit 2 w, 2 w + 1: warp w's pieces
  __shared__ int abort;                                               // a wait gave up
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, gid = lane >> 2, tig = lane & 3;
  uint8_t* ring = smem + warp * Sh::kRing;
  if (lane == 0) {
#pragma unroll
    for (int k = 0; k < S; ++k) mbar_init(&full[warp][k], 1);
    fence_mbar_init();
  }
  if (threadIdx.x == 0) abort = 0, there = 0;
  pdl_enter();

  // The CTA's runs: run i begins at the cut cut_u[i] of the line, in the sequence cut_b[i], whose first unit is cut_seq[i]. A
  // pass over the sequences adds up their segments and steps; another finds the cuts.
  Line line = {0, 1};
  int64_t total = 0, c0 = 0, u, u1, b, seq_at;
  if (threadIdx.x == 0) p.meta[2 * blockIdx.x] = make_int4(-1, 0, 0, 0);
  const int64_t n_seqs = p.c.n_seqs, runs = static_cast<int64_t>(gridDim.x) * kWarps;
  // The line of so many segments with so many steps in all, and this CTA's first cut; `total` is at most what it says then.
  const auto lay = [&](int64_t segments, int64_t steps) {
    // Pieces of so many steps that with one shorter piece a segment they are no more than the runs.
    const int64_t piece = 2 * segments <= runs ? quotient(steps + runs - segments - 1, runs - segments) : kLongPiece + 1;
    if (piece <= kLongPiece) {
      line.piece = max(kRound, static_cast<int>(piece));
      total = runs;
    } else {
      total = steps + kSegmentUnits * segments;
      line.per = max(static_cast<int64_t>(kSegmentUnits + kRound), quotient(total + runs - 1, runs));
    }
    c0 = static_cast<int64_t>(blockIdx.x) * kWarps * line.per;
  };
  // Up to 32 sequences whose units 32 bits hold: every warp for itself, a sequence to a lane (37 places 9.3 us at that time, one sequence
  // of 1000 13.9, where the passes below with their eight barriers took 10.7 and 15.2).
  Sequence q = {};
  bool small = n_seqs <= 32;
  if (small) {
    if (lane < n_seqs) q.load(p, lane, R);
    small = __all_sync(0xffffffffu, static_cast<int64_t>(p.c.heads) * q.tiles * (q.steps + kSegmentUnits) < (1 << 25));
  }
  if (small) {
    const int mine = p.c.heads * q.tiles;
    const int segments = __reduce_add_sync(0xffffffffu, mine), steps = __reduce_add_sync(0xffffffffu, mine * q.steps);
    lay(segments, steps);
    if (c0 >= total) return;
    const int size = line.size(q), units = mine * size, per = static_cast<int>(line.per);
    int x = units;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, x, o);
      if (lane >= o) x += y;
    }
    const int first = x - units, all = __shfl_sync(0xffffffffu, x, 31);
    total = all;
    if (c0 >= total) return;
    // The cuts of this warp's run, by lanes 0 and 1: in the last sequence that begins at or before them.
    const int64_t cut0 = c0 + warp * per, cut1 = cut0 + per;
    const int at0 = 31 - __clz(__ballot_sync(0xffffffffu, lane < n_seqs && first <= cut0));
    const int at1 = 31 - __clz(__ballot_sync(0xffffffffu, lane < n_seqs && first <= cut1));
    const int64_t cut = lane & 1 ? cut1 : cut0;
    const int from = __shfl_sync(0xffffffffu, first, lane & 1 ? at1 : at0), of = __shfl_sync(0xffffffffu, size, lane & 1 ? at1 : at0);
    int cut_u = all;
    if (cut < all) {
      const int off = static_cast<int>(cut) - from, in = off % of;
      cut_u = from + off - in + static_cast<int>(line.cut_at(in, of));
    }
    u = __shfl_sync(0xffffffffu, cut_u, 0);
    u1 = __shfl_sync(0xffffffffu, cut_u, 1);
    b = at0;
    seq_at = __shfl_sync(0xffffffffu, first, at0);
    q.n0 = __shfl_sync(0xffffffffu, q.n0, at0);
    q.len = __shfl_sync(0xffffffffu, q.len, at0);
    q.rows = __shfl_sync(0xffffffffu, q.rows, at0);
    q.tiles = __shfl_sync(0xffffffffu, q.tiles, at0);
    q.first = __shfl_sync(0xffffffffu, q.first, at0);
    q.steps = __shfl_sync(0xffffffffu, q.steps, at0);
    __syncthreads();         // (what thread 0 has cleared)
  } else {
    int64_t before = 0;
    // The sum of v over the threads before this one, added to `before`, which moves on by the sum over all.
    const auto sum_before = [&](int64_t v) {
      int64_t x = v;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int64_t y = __shfl_up_sync(0xffffffffu, x, o);
        if (lane >= o) x += y;
      }
      __syncthreads();
      if (lane == 31) scan[warp] = x;
      __syncthreads();
      x += before - v;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) {
        x += w < warp ? scan[w] : 0;
        before += scan[w];
      }
      return x;
    };
    Sequence s = {};
#pragma unroll 1
    for (int pass = 0; pass < 2; ++pass) {
      int64_t segments = 0, steps = 0;
#pragma unroll 1
      for (int64_t i0 = 0; i0 < n_seqs; i0 += kThreads) {
        const int64_t i = i0 + threadIdx.x;
        if (pass == 0 || n_seqs > kThreads) {
          s = Sequence{};
          if (i < n_seqs) s.load(p, i, R);
        }
        if (pass == 0) {
          segments += static_cast<int64_t>(p.c.heads) * s.tiles;
          steps += static_cast<int64_t>(p.c.heads) * s.tiles * s.steps;
          continue;
        }
        const int size = line.size(s);
        const int64_t x = sum_before(line.units(s, p.c.heads));
        first_unit[threadIdx.x] = x;
        segment_size[threadIdx.x] = size;
        __syncthreads();
        // Threads 0..kWarps look for their cut among these sequences: the last that begins at or before it.
        const int64_t cut = c0 + threadIdx.x * line.per;
        if (threadIdx.x <= kWarps && cut >= first_unit[0] && cut < before) {
          int lo = 0, hi = static_cast<int>(min(static_cast<int64_t>(kThreads), n_seqs - i0));
          while (hi - lo > 1) {
            const int mid = (lo + hi) >> 1;
            if (first_unit[mid] <= cut) lo = mid;
            else hi = mid;
          }
          const int64_t seg = first_unit[lo] + quotient(cut - first_unit[lo], segment_size[lo]) * segment_size[lo];
          cut_b[threadIdx.x] = i0 + lo;
          cut_seq[threadIdx.x] = first_unit[lo];
          cut_u[threadIdx.x] = seg + line.cut_at(cut - seg, segment_size[lo]);
        }
      }
      if (pass == 0) {
        sum_before(segments);
        segments = before;
        before = 0;
        sum_before(steps);
        steps = before;
        before = 0;
        lay(segments, steps);
        if (c0 >= total) return;
      }
    }
    total = before;
    if (c0 >= total) return;
    __syncthreads();
    if (threadIdx.x <= kWarps && c0 + threadIdx.x * line.per >= total) cut_u[threadIdx.x] = total;
    __syncthreads();
    u = cut_u[warp], b = cut_b[warp], seq_at = cut_seq[warp];
    u1 = cut_u[warp + 1];
    if (u < u1) q.load(p, b, R);
  }

  uint32_t phases = 0;       // of each stage's next copy
  int stages = S;            // that copies go to; a held piece takes the last kHeld

  while (u < u1) {
    {                        // a run may begin where a sequence ends, and goes on through others
      int64_t n = line.units(q, p.c.heads);
      while (u >= seq_at + n) {
        seq_at += n;
        q.load(p, ++b, R);
        n = line.units(q, p.c.heads);
      }
    }
    // The segment that u lies in: [at, end) of the line.
    const int size = line.size(q);
    const int seg = static_cast<int>(quotient(u - seq_at, size));
    const int64_t at = seq_at + static_cast<int64_t>(seg) * size, end = at + size;
    const int h = q.tiles == 1 ? seg : divide(seg, q.tiles), tile = seg - h * q.tiles;
    const bool begins = u == at, ends = end <= u1;
    int t0 = q.first + line.steps_before(u - at, q), t1 = q.first + line.steps_before(min(end, u1) - at, q);

    // Row r of the tile: new row i = r' / group, head r' % group, r' = tile * R + r. It sees [low, seen).
    const int rows = q.rows * p.group;
    auto row_of = [&](int r, int& i, int& hq) {
      const int rr = tile * R + r;
      i = divide(rr, p.group);
      hq = h * p.group + rr - i * p.group;
      return rr < rows;
    };
    auto seen_of = [&](int i) { return q.len - q.rows + 1 + i; };
    auto low_of = [&](int seen) { return p.a.window > 0 ? static_cast<int>(max(int64_t(0), seen - p.a.window)) : 0; };
    const int seen_least = seen_of(divide(tile * R, p.group)), seen_most = seen_of(divide(min(tile * R + R, rows) - 1, p.group));
    const int low_least = low_of(seen_least), low_most = low_of(seen_most);
    // Steps of the run that a row of this tile sees, and those of them that all of its rows see whole.
    t0 = max(t0, low_least >> 5);
    t1 = min(t1, ((seen_most - 1) >> 5) + 1);            // (a sum of 31 could pass 2^31)
    const int mine = max(0, t1 - t0);
    const int whole0 = ((low_most - 1) >> 5) + 1, wholes = max(0, (seen_least >> 5) - whole0);

    // Granules of this warp's steps: lane k % 32 has the two of step t0 + k (-1: one that no row sees, whose page may be gone, or its
    // page is out of range), and makes their copies, as one where they lie side by side.
    const int per_page = p.c.page_shift - 4;
    const int32_t* table = p.c.table + b * p.c.ldt;
    const int first_granule = low_least >> 4, last_granule = (seen_most - 1) >> 4;
    auto granule_at = [&](int g) -> int {
      const int64_t i = static_cast<int64_t>(g) >> per_page;
      const int page = g >= first_granule && g <= last_granule && i < p.c.ldt ? table[i] : -1;
      if (page < 0 || page >= p.c.n_pages) return -1;
      return static_cast<int>(((static_cast<int64_t>(page) * p.c.heads + h) << per_page) + (g & ((1 << per_page) - 1)));
    };
    int ga = -1, gb = -1;
    auto look_up = [&](int k) {          // of the steps k + lane
      ga = gb = -1;
      if (k + lane < mine) {
        const int g = 2 * (t0 + k + lane);
        ga = granule_at(g);
        gb = per_page > 0 && g < last_granule && ga >= 0 ? ga + 1 : granule_at(g + 1);
        if ((ga < 0 && g >= first_granule) || (gb < 0 && g < last_granule)) report_error(p.err, ERR_PAGE);
      }
    };
    auto issue = [&](int to) {
      uint64_t* bar = &full[warp][to];
      uint8_t* dst = ring + to * Sh::kStep;
      const uint8_t* a = p.c.data + static_cast<int64_t>(ga) * Gr::kBytes;
      if (gb == ga + 1 && ga >= 0) {
        mbar_expect_tx(bar, Sh::kStep);
        bulk_g2s(dst, a, Sh::kStep, bar);
      } else {
        mbar_expect_tx(bar, (ga >= 0 ? Gr::kBytes : 0) + (gb >= 0 ? Gr::kBytes : 0));
        if (ga >= 0) bulk_g2s(dst, a, Gr::kBytes, bar);
        if (gb >= 0) bulk_g2s(dst + Gr::kBytes, p.c.data + static_cast<int64_t>(gb) * Gr::kBytes, Gr::kBytes, bar);
      }
    };
    Raw8<T> raw[G];          // of the queries: the first rows' are on their way while the pages are looked up
    auto load_rows = [&](int nt) {
      int i, hq;
      if (row_of(8 * nt + gid, i, hq)) {
        const T* src = static_cast<const T*>(p.a.Q) + (q.n0 + i) * p.a.ldq + static_cast<int64_t>(hq) * D + 8 * tig;
#pragma unroll
        for (int g = 0; g < G; ++g) {
          if (p.vec) raw[g].template load<true>(src + 32 * g);
          else raw[g].template load<false>(src + 32 * g);
        }
      }
    };
    load_rows(0);
    if (lane < R) {
      int i, hq;
      row_of(lane, i, hq);
      range[warp][lane] = make_int2(low_of(seen_of(i)), seen_of(i));
    }
    look_up(0);
    if (lane < min(stages - 1, mine)) issue(lane);

    // Queries as operands: lane (gid, tig) has of row gid the elements 32 g + 8 tig + 0..7, times 2^a with the
    // row's largest between 2^14 and 2^15 (so that fp16 and bf16 queries are exact), the odd ones
    // also times 2^-4 for the codes that are four bits higher.
    uint32_t qb[NT][G][2][2], qs[NT][(G + 3) / 4][2];
    [[maybe_unused]] uint32_t ql[kSplitQ ? NT : 1][kSplitQ ? G : 1][2][2];
    float factor[NT][2];                                              // of the scores of columns 2 tig, 2 tig + 1
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      int i, hq;
      const bool here = row_of(8 * nt + gid, i, hq);
      if (nt > 0) load_rows(nt);
      float most = 0.f, sums[G];
#pragma unroll
      for (int g = 0; g < G; ++g)
#pragma unroll
        for (int j = 0; j < 8; ++j) most = fmaxf(most, here ? fabsf(raw[g][j]) : 0.f);
      most = fmaxf(most, __shfl_xor_sync(0xffffffffu, most, 1));
      most = fmaxf(most, __shfl_xor_sync(0xffffffffu, most, 2));
      // 2^e <= most < 2^(e + 1); rows below 2^-86 have scores of nothing, and those beyond 2^118 are NaN all over.
      const int e = max(-86, min(127, static_cast<int>(__float_as_uint(most) >> 23) - 127));
      const float up1 = pow2((14 - e) >> 1), up2 = pow2(14 - e - ((14 - e) >> 1));
#pragma unroll
      for (int g = 0; g < G; ++g) {
        float v[8];
        sums[g] = 0.f;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          v[j] = here ? raw[g][j] * up1 * up2 : 0.f;
          sums[g] += v[j];
          if (j & 1) v[j] *= 0.0625f;
        }
        sums[g] += __shfl_xor_sync(0xffffffffu, sums[g], 1);
        sums[g] += __shfl_xor_sync(0xffffffffu, sums[g], 2);
        sums[g] *= 0x1p-6f;
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          qb[nt][g][k][0] = pack_half2(v[2 * k], v[2 * k + 4]);
          qb[nt][g][k][1] = pack_half2(v[2 * k + 1], v[2 * k + 5]);
          if constexpr (kSplitQ) {
            ql[nt][g][k][0] = pack_half2(low_part(v[2 * k]), low_part(v[2 * k + 4]));
            ql[nt][g][k][1] = pack_half2(low_part(v[2 * k + 1]), low_part(v[2 * k + 5]));
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
      const float f = seen_of(i) <= 0 ? 0.f : most < 0x1p118f ? p.a.scale * 1.44269504f * pow2(10 + min(e, 117)) : NAN;
#pragma unroll
      for (int c = 0; c < 2; ++c) factor[nt][c] = __shfl_sync(0xffffffffu, f, 4 * (2 * tig + c));
    }

    float o[NT][G][2][4], om[NT][4], top[NT][2];
    int sigma = kSplit ? -24 : 0;                                     // products with s are relative to 2^sigma
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      top[nt][0] = top[nt][1] = kLow;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        // A row whose scores all lie below fp32's range has no weights, as one that sees nothing, but is not a row of zeros: with
        // this total, which no weight leaves anything of, it becomes 0 / 0. (A score is its factor times less than 2^20.)
        om[nt][j] = j >= 2 && fabsf(factor[nt][j & 1]) > 0x1p100f ? 0x1p-140f : 0.f;
#pragma unroll
        for (int g = 0; g < G; ++g) o[nt][g][0][j] = o[nt][g][1][j] = 0.f;
      }
    }

    // A step of 32 places, two granules. Rows 0..15 of the operands are a granule's places in this order, so that the value codes of
    // lanes side by side lie in different banks: row r is place r / 2 + 4 (r % 2), of the lower or upper eight.
    const int ta = (gid >> 1) + 4 * (gid & 1);
    const int k_at = ta * (D / 2) + tig * (4 * G), p_at = Gr::kCodes + ta * (4 * G);
    const int v_at = Gr::kValues + tig * (D / 2) + gid * (2 * G);
    const int m_at = Gr::kValues + Gr::kCodes + (D >= 128 ? ((lane & 8) + ((lane >> 1) & 3) + 4 * (lane & 1)) * (4 * G) : tig * (4 * G));
    const auto step = [&](auto edge_tag, const uint8_t* st, int place0, int hide) {
      const bool kEdge = edge_tag;               // some row does not see all of its places
      float s[2][NT][4];
#pragma unroll
      for (int w = 0; w < 2; ++w) {
        const uint8_t* gr = st + w * Gr::kBytes;
        uint32_t ka[G], kb[G], pa[G], pb[G];                          // pa, pb: G / 2 words of s, then G / 2 of m
        auto words = [](uint32_t (&w)[G], const uint8_t* src) {
          if constexpr (G == 2) {
            *reinterpret_cast<uint2*>(w) = *reinterpret_cast<const uint2*>(src);
          } else {
#pragma unroll
            for (int i = 0; i < G / 4; ++i) *reinterpret_cast<uint4*>(w + 4 * i) = reinterpret_cast<const uint4*>(src)[i];
          }
        };
        words(ka, gr + k_at);
        words(kb, gr + k_at + 8 * (D / 2));
        words(pa, gr + p_at);
        words(pb, gr + p_at + 8 * (4 * G));
        float sm[NT][4];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          if constexpr (G == 2) {
            mma_f16_zero(sm[nt], pa[1], pb[1], 0u, 0u, qs[nt][0][0], 0u);
          } else {
            mma_f16_zero(sm[nt], pa[G / 2], pb[G / 2], pa[G / 2 + 1], pb[G / 2 + 1], qs[nt][0][0], qs[nt][0][1]);
            if constexpr (G == 8) mma_f16(sm[nt], pa[6], pb[6], pa[7], pb[7], qs[nt][1][0], qs[nt][1][1]);
          }
#pragma unroll
          for (int j = 0; j < 4; ++j) s[w][nt][j] = sm[nt][j] * 0x1p-18f;
        }
#pragma unroll
        for (int g = 0; g < G; ++g) {
          const float2 sa2 = __half22float2(bits_half2(pa[g / 2])), sb2 = __half22float2(bits_half2(pb[g / 2]));
          const float sa = g & 1 ? sa2.y : sa2.x, sb = g & 1 ? sb2.y : sb2.x;
          const uint32_t a0 = ka[g] & M0, a1 = kb[g] & M0, a2 = ka[g] & M1, a3 = kb[g] & M1;
          const uint32_t c0 = (ka[g] >> 8) & M0, c1 = (kb[g] >> 8) & M0, c2 = (ka[g] >> 8) & M1, c3 = (kb[g] >> 8) & M1;
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) {
            float acc[4];
            mma_f16_zero(acc, a0, a1, a2, a3, qb[nt][g][0][0], qb[nt][g][0][1]);
            mma_f16(acc, c0, c1, c2, c3, qb[nt][g][1][0], qb[nt][g][1][1]);
            if constexpr (kSplitQ) {
              mma_f16(acc, a0, a1, a2, a3, ql[nt][g][0][0], ql[nt][g][0][1]);
              mma_f16(acc, c0, c1, c2, c3, ql[nt][g][1][0], ql[nt][g][1][1]);
            }
            s[w][nt][0] = fmaf(sa, acc[0], s[w][nt][0]);
            s[w][nt][1] = fmaf(sa, acc[1], s[w][nt][1]);
            s[w][nt][2] = fmaf(sb, acc[2], s[w][nt][2]);
            s[w][nt][3] = fmaf(sb, acc[3], s[w][nt][3]);
          }
        }
        // Sum s acc is of 2^(a - 24) q . (k - m), sm of 2^(a - 6) q . m.
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int j = 0; j < 4; ++j) s[w][nt][j] *= factor[nt][j & 1];
        if (kEdge) {
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int c = 0; c < 2; ++c) {
              const int2 sees = range[warp][8 * nt + 2 * tig + c];
              const int place = place0 + 16 * w + ta, hidden = hide >> w & 1;
              if (place < sees.x || place >= sees.y || hidden) s[w][nt][c] = -INFINITY;
              if (place + 8 < sees.x || place + 8 >= sees.y || hidden) s[w][nt][c + 2] = -INFINITY;
            }
        }
      }

      // The values' parameters, two places a word, in the order of the operand's rows 2 tig, 2 tig + 1: m0 (lower eight places)
      // and m1 (upper eight) as an operand whose rows g (4 + g for 128 elements) are the blocks' m + 8 s; for rows of 16 bits also va and
      // vb, their s. fp32 rows: s of two blocks a word, of places ta and ta + 8. Places that no row of the tile sees: 0.
      uint32_t m0[2], m1[2], sizes = 0;
      uint32_t s0[2], s1[2];                                          // the s in the places of the m
      uint32_t va[2][kSplit ? G / 2 : G], vb[2][kSplit ? G / 2 : G];
#pragma unroll
      for (int w = 0; w < 2; ++w) {
        const uint8_t* row = st + w * Gr::kBytes + m_at;
        const auto unseen = [&](int place) {
          return kEdge && (place0 + 16 * w + place < low_least || place0 + 16 * w + place >= seen_most || (hide >> w & 1));
        };
        uint32_t keep0 = 0xffffffffu, keep1 = 0xffffffffu;
        if (kEdge) {
          keep0 = (unseen(tig) ? 0u : 0xffffu) | (unseen(tig + 4) ? 0u : 0xffff0000u);
          keep1 = (unseen(tig + 8) ? 0u : 0xffffu) | (unseen(tig + 12) ? 0u : 0xffff0000u);
        }
        if constexpr (D >= 128) {
          load_transposed(m0[w], m1[w], row + (D == 256 ? 2 * G : 0));
          m0[w] &= keep0, m1[w] &= keep1;
          uint32_t t0 = m0[w], t1 = m1[w];                            // of 128 elements: rows 0..3 of the same matrices
          if constexpr (D == 256) {
            load_transposed(t0, t1, row);
            t0 &= keep0, t1 &= keep1;
          }
          if constexpr (!kSplit) {
            sizes |= t0 | t1;
#pragma unroll
            for (int g = 0; g < G; ++g) {
              va[w][g] = __shfl_sync(0xffffffffu, t0, 4 * g + tig);
              vb[w][g] = __shfl_sync(0xffffffffu, t1, 4 * g + tig);
            }
          }
          s0[w] = D == 256 ? t0 : __shfl_xor_sync(0xffffffffu, t0, 16);
          s1[w] = D == 256 ? t1 : __shfl_xor_sync(0xffffffffu, t1, 16);
        } else {
          const auto words = [&](int place) { return *reinterpret_cast<const uint2*>(row + place * 8); };
          const uint2 x = words(0), y = words(4), z = words(8), t = words(12);
          if constexpr (!kSplit) {
            va[w][0] = __byte_perm(x.x, y.x, 0x5410) & keep0, va[w][1] = __byte_perm(x.x, y.x, 0x7632) & keep0;
            vb[w][0] = __byte_perm(z.x, t.x, 0x5410) & keep1, vb[w][1] = __byte_perm(z.x, t.x, 0x7632) & keep1;
            sizes |= va[w][0] | va[w][1] | vb[w][0] | vb[w][1];
          }
          const uint32_t pick = gid == 0 ? 0x5410u : 0x7632u;
          m0[w] = gid < G ? __byte_perm(x.y, y.y, pick) & keep0 : 0u;
          m1[w] = gid < G ? __byte_perm(z.y, t.y, pick) & keep1 : 0u;
          s0[w] = gid < G ? __byte_perm(x.x, y.x, pick) & keep0 : 0u;
          s1[w] = gid < G ? __byte_perm(z.x, t.x, pick) & keep1 : 0u;
        }
        if (kEdge) {                                        // a NaN (m is 0 there) reaches rows by the codes' weights
          s0[w] &= __heq2_mask(bits_half2(s0[w]), bits_half2(s0[w]));
          s1[w] &= __heq2_mask(bits_half2(s1[w]), bits_half2(s1[w]));
        }
        if constexpr (kSplit) {
          const uint8_t* vp = st + w * Gr::kBytes + Gr::kValues + p_at;
#pragma unroll
          for (int i = 0; i < G / 2; ++i) {
            va[w][i] = unseen(ta) ? 0u : reinterpret_cast<const uint32_t*>(vp)[i];
            vb[w][i] = unseen(ta + 8) ? 0u : reinterpret_cast<const uint32_t*>(vp + 8 * (4 * G))[i];
          }
        }
      }
      if constexpr (!kSplit && D >= 128) sizes = gid < G ? sizes : 0;

      // Scores less their columns' offset; the maximum is moved where one passes it by kAhead, sigma where an s passes 2^sigma.
      // Rows of 16 bits have sigma 0 until an s is 2 or more (its exponent's highest bit is set). Split weights are taken times
      // 2^-sigma (exactly, in fp32) from the first.
      float x[2][NT][4];
      const auto sigma_x = [&] { return kSplit ? static_cast<float>(sigma) : 0.f; };
      const auto shift = [&] {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          const float off[2] = {top[nt][0] + (sigma_x() - kTop), top[nt][1] + (sigma_x() - kTop)};
#pragma unroll
          for (int w = 0; w < 2; ++w)
#pragma unroll
            for (int j = 0; j < 4; ++j) x[w][nt][j] = s[w][nt][j] - off[j & 1];
        }
      };
      shift();
      float ahead = x[0][0][0];
#pragma unroll
      for (int w = 0; w < 2; ++w)
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int j = 0; j < 4; ++j) ahead = fmaxf(ahead, x[w][nt][j]);
      float largest = 0.f;
      const auto find_largest = [&] {                                 // a NaN counts for nothing
        __half2 big = __habs2(bits_half2(va[0][0]));
#pragma unroll
        for (int w = 0; w < 2; ++w)
#pragma unroll
          for (int i = 0; i < (kSplit ? G / 2 : G); ++i)
            big = __hmax2(big, __hmax2(__habs2(bits_half2(va[w][i])), __habs2(bits_half2(vb[w][i]))));
        largest = fminf(fmaxf(fmaxf(__low2float(big), __high2float(big)), 0.f), 65504.f);
      };
      if constexpr (kSplit) find_largest();
      if (__any_sync(0xffffffffu, ahead > kTop + kAhead - sigma_x() ||
                                      (kSplit ? largest > pow2(sigma) : (sizes & 0x40004000u) != 0))) {
        if constexpr (!kSplit) {
          find_largest();
          if (largest < 2.f) largest = 0.f;
        }
        const uint32_t bits = __reduce_max_sync(0xffffffffu, __float_as_uint(largest));
        const int want = max(sigma, static_cast<int>((bits + 0x007fffffu) >> 23) - 127);   // the power of two not below it
        const float by = pow2(max(-126, sigma - want));
        sigma = want;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            float m = fmaxf(fmaxf(s[0][nt][c], s[0][nt][c + 2]), fmaxf(s[1][nt][c], s[1][nt][c + 2]));
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
        shift();
      }

      float os[NT][4];                                                // this step's sums of m + 8 s, and of the weights
      const float scale_m = sigma > 0 ? 0.0625f : 0.5f;
#pragma unroll
      for (int w = 0; w < 2; ++w) {
        // Weights, transposed as operands. Rows of 16 bits: the weights times 2^kTop rounded to fp16, and for each block's codes these
        // times 2^-sigma and s (at most 2^15: s is below 2 with sigma 0, else s / 2^sigma at most 1; what 2^-sigma takes from a weight
        // is below 2^(sigma - 35) of the largest, and does not show in the total). fp32 rows: products with s taken in fp32, and the
        // weights times 2^kTop, all in two halves.
        uint32_t pw[NT][2];
        [[maybe_unused]] uint32_t pl[kSplit ? NT : 1][2];
        [[maybe_unused]] __half2 ps[kSplit ? 1 : NT][2];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
          for (int j = 0; j < 4; ++j) x[w][nt][j] = exp2_fast(x[w][nt][j]);
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            if constexpr (kSplit) {
              const float up = pow2(sigma), y = x[w][nt][2 * k] * up, z = x[w][nt][2 * k + 1] * up;
              pw[nt][k] = transpose8(pack_half2(y, z));
              pl[nt][k] = transpose8(pack_half2(low_part(y), low_part(z)));
            } else {
              pw[nt][k] = transpose8(pack_half2(x[w][nt][2 * k], x[w][nt][2 * k + 1]));
              ps[nt][k] = __hmul2(bits_half2(pw[nt][k]), __float2half2_rn(pow2(-sigma)));
            }
          }
        }
        // The m + 8 s (times 1/2, or 1/16 where s may be 2 and more: in fp16's range), and a row of ones (row 8).
        [[maybe_unused]] uint32_t l0 = 0, l1 = 0;                     // what rounding them to fp16 leaves
        if constexpr (kSplit) {
          const auto both = [&](uint32_t& m, uint32_t& l, uint32_t s) {
            const float2 a = __half22float2(bits_half2(m)), b = __half22float2(bits_half2(s));
            const float u = fmaf(b.x, 8.f, a.x) * scale_m, v = fmaf(b.y, 8.f, a.y) * scale_m;
            m = pack_half2(u, v);
            l = pack_half2(low_part(u), low_part(v));
          };
          both(m0[w], l0, s0[w]);
          both(m1[w], l1, s1[w]);
        } else {
          const __half2 eight = __float2half2_rn(8.f * scale_m), by = __float2half2_rn(scale_m);
          m0[w] = half2_bits(__hfma2(bits_half2(s0[w]), eight, __hmul2(bits_half2(m0[w]), by)));
          m1[w] = half2_bits(__hfma2(bits_half2(s1[w]), eight, __hmul2(bits_half2(m1[w]), by)));
        }
        const uint32_t one = gid == 0 ? 0x3c003c00u : 0u;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          if (w == 0) mma_f16_zero(os[nt], m0[w], one, m1[w], one, pw[nt][0], pw[nt][1]);
          else mma_f16(os[nt], m0[w], one, m1[w], one, pw[nt][0], pw[nt][1]);
          if constexpr (kSplit) {
            mma_f16(os[nt], m0[w], one, m1[w], one, pl[nt][0], pl[nt][1]);
            mma_f16(os[nt], l0, 0u, l1, 0u, pw[nt][0], pw[nt][1]);
          }
          if (w == 1) {
#pragma unroll
            for (int j = 0; j < 2; ++j) {
              om[nt][j] = fmaf(os[nt][j], sigma > 0 ? 16.f : 2.f, om[nt][j]);
              om[nt][j + 2] += os[nt][j + 2];
            }
          }
        }
        // The values' codes: of places tig, tig + 4, tig + 8, tig + 12 four elements of each block (row gid of the operand
        // the first of them, row gid + 8 the second, and so on). A NaN of a place that a row does not see is left out.
        const uint8_t* vc = st + w * Gr::kBytes + v_at;
        uint32_t cw[4][G / 2];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          if constexpr (G == 2) {
            cw[k][0] = *reinterpret_cast<const uint32_t*>(vc + 4 * k * (D / 2));
          } else {
#pragma unroll
            for (int i = 0; i < G / 4; ++i)
              *reinterpret_cast<uint2*>(&cw[k][2 * i]) = reinterpret_cast<const uint2*>(vc + 4 * k * (D / 2))[i];
          }
        }
#pragma unroll
        for (int g = 0; g < G; ++g) {
          const uint32_t pick = g & 1 ? 0x7632u : 0x5410u;
          const uint32_t y = __byte_perm(cw[0][g / 2], cw[1][g / 2], pick), z = __byte_perm(cw[2][g / 2], cw[3][g / 2], pick);
          const auto even = [](uint32_t w) { return kSplit ? codes_less_8<0>(w) : w & M0; };
          const auto odd = [](uint32_t w) { return kSplit ? codes_less_8<4>(w) : w & M1; };
          const uint32_t a0 = even(y), a1 = odd(y), a2 = even(z), a3 = odd(z);
          const uint32_t c0 = even(y >> 8), c1 = odd(y >> 8), c2 = even(z >> 8), c3 = odd(z >> 8);
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) {
            if constexpr (kSplit) {
              const float2 sa2 = __half22float2(bits_half2(va[w][g / 2])), sb2 = __half22float2(bits_half2(vb[w][g / 2]));
              const float sa = g & 1 ? sa2.y : sa2.x, sb = g & 1 ? sb2.y : sb2.x;
              float t[4] = {x[w][nt][0] * sa, x[w][nt][1] * sa, x[w][nt][2] * sb, x[w][nt][3] * sb};
              if (kEdge) {
#pragma unroll
                for (int j = 0; j < 4; ++j) t[j] = x[w][nt][j] == 0.f ? 0.f : t[j];
              }
              const uint32_t b0 = transpose8(pack_half2(t[0], t[1])), b1 = transpose8(pack_half2(t[2], t[3]));
              const uint32_t d0 = transpose8(pack_half2(low_part(t[0]), low_part(t[1])));
              const uint32_t d1 = transpose8(pack_half2(low_part(t[2]), low_part(t[3])));
              float of[2][4];
#pragma unroll
              for (int k = 0; k < 2; ++k) {
                mma_f16_zero(of[k], k ? c0 : a0, k ? c1 : a1, k ? c2 : a2, k ? c3 : a3, d0, d1);
                mma_f16(of[k], k ? c0 : a0, k ? c1 : a1, k ? c2 : a2, k ? c3 : a3, b0, b1);
#pragma unroll
                for (int j = 0; j < 4; ++j) o[nt][g][k][j] += of[k][j];
              }
            } else {
              uint32_t b0 = half2_bits(__hmul2(ps[nt][0], bits_half2(va[w][g])));
              uint32_t b1 = half2_bits(__hmul2(ps[nt][1], bits_half2(vb[w][g])));
              if (kEdge) {
                b0 &= __hne2_mask(bits_half2(pw[nt][0]), __half2half2(__ushort_as_half(0)));
                b1 &= __hne2_mask(bits_half2(pw[nt][1]), __half2half2(__ushort_as_half(0)));
              }
              mma_f16(o[nt][g][0], kEven, kOdd, kEven, kOdd, b0, b1);
              mma_f16(o[nt][g][1], kEven, kOdd, kEven, kOdd, b0, b1);
              mma_f16(o[nt][g][0], a0, a1, a2, a3, b0, b1);
              mma_f16(o[nt][g][1], c0, c1, c2, c3, b0, b1);
            }
          }
        }
      }
    };

    // Bit k % 32 of a, b: the first, the second granule of step k has no page (next: of the 32 steps that copies are at).
    uint32_t hidden_a = __ballot_sync(0xffffffffu, ga < 0 && lane < mine);
    uint32_t hidden_b = __ballot_sync(0xffffffffu, gb < 0 && lane < mine), next_a = 0, next_b = 0;
    int stage = 0, to = min(stages - 1, mine) % stages, made = min(stages - 1, mine);
#pragma unroll 1
    for (int k = 0; k < mine; ++k) {
      uint64_t* bar = &full[warp][stage];
      const uint32_t phase = (phases >> stage) & 1;
      if (!mbar_try_wait(bar, phase)) mbar_wait(bar, phase, &abort, p.err);
      __syncwarp();                               // every lane is past the step before this one: its stage is free
      if ((k & 31) == 0 && k > 0) {
        hidden_a = next_a;
        hidden_b = next_b;
      }
      const int t = t0 + k, hide = (hidden_a >> (k & 31) & 1) | (hidden_b >> (k & 31) & 1) << 1;
      if (made < mine) {
        if ((made & 31) == 0) {                   // the next 32 steps' pages
          look_up(made);
          next_a = __ballot_sync(0xffffffffu, ga < 0 && made + lane < mine);
          next_b = __ballot_sync(0xffffffffu, gb < 0 && made + lane < mine);
        }
        if (lane == (made & 31)) issue(to);
        ++made;
        to = to + 1 == stages ? 0 : to + 1;
      }
      const uint8_t* st = ring + stage * Sh::kStep;
      phases ^= 1u << stage;
      stage = stage + 1 == stages ? 0 : stage + 1;
      const bool edge = static_cast<unsigned>(t - whole0) >= static_cast<unsigned>(wholes) || hide != 0;
      // One copy of the step's code, or one more for the steps that all rows see whole. With many short sequences the code that a
      // CTA runs through bounds rows of 16 bits (256 of up to 900 places: 37.5 us with one copy, 42.8 with two; 32 of up to
      // 32768: 74.2 and 73.5). Where a step has more registers at work, the branches cost more (16 of 64 fp32 elements: 60 and 51).
      if constexpr (!FINE && NT == 1) {
        step(edge, st, 32 * t, hide);
      } else {
        if (edge) step(std::true_type{}, st, 32 * t, hide);
        else step(std::false_type{}, st, 32 * t, 0);
      }
    }

    // The piece's sums as rows: where a held piece goes, or over the first stages.
    const bool first_piece = !begins, whole = begins && ends;
    float* sums = reinterpret_cast<float*>(ring + (first_piece ? (S - Sh::kHeld) * Sh::kStep : 0));
    float(&most_of)[R] = stat[warp][first_piece ? 0 : 1][0];
    float(&total_of)[R] = stat[warp][first_piece ? 0 : 1][1];
    const float up = pow2(sigma + (kSplit ? 0 : 24)), up_odd = pow2(sigma + (kSplit ? 0 : 20));
    __syncwarp();
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        const int r = 8 * nt + 2 * tig + c;
        if (gid == 0) {
          most_of[r] = top[nt][c];
          total_of[r] = om[nt][c + 2];
        }
#pragma unroll
        for (int g = 0; g < G; ++g) {
          const float m = __shfl_sync(0xffffffffu, om[nt][c], 4 * ((D == 128 ? 4 : 0) + g) + tig);
          *reinterpret_cast<float4*>(sums + r * Sh::kPitch + 32 * g + 4 * gid) =
              make_float4(fmaf(o[nt][g][0][c], up, m), fmaf(o[nt][g][0][c + 2], up_odd, m),
                          fmaf(o[nt][g][1][c], up, m), fmaf(o[nt][g][1][c + 2], up_odd, m));
        }
      }
    __syncwarp();
    if (whole) {
#pragma unroll 2
      for (int r0 = 0; r0 < R && tile * R + r0 < rows; r0 += 32 / L) {
        const int r = r0 + lane / L, l8 = lane % L;
        int i, hq;
        const bool here = row_of(r, i, hq);
        const float sum = total_of[r], inv = sum == 0.f ? 0.f : __fdiv_rn(1.0f, sum);    // a row that sees nothing
        float v[8];
#pragma unroll
        for (int j = 0; j < 2; ++j)
          *reinterpret_cast<float4*>(v + 4 * j) = *reinterpret_cast<const float4*>(sums + r * Sh::kPitch + 8 * l8 + 4 * j);
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] = sum == 0.f ? 0.f : v[j] * inv;
        store_row<T, D>(p, here, q.n0 + i, hq, l8, v);
      }
      fence_proxy_async_smem();      // the stages are written by copies again
      __syncwarp();
    } else {
      if (first_piece) stages = S - Sh::kHeld;
      if (lane == 0) {
        int parts = 0;
        if (begins) {
          // The CTA whose runs have the segment's last unit: that of the last cut within it that was not moved to its end.
          int64_t last = quotient(end - 1, line.per);
          while (line.cut_at(last * line.per - at, size) == size) --last;
          parts = static_cast<int>(quotient(last, kWarps) - blockIdx.x) + 1;
        }
        piece[warp][first_piece ? 0 : 1] = Piece{q.n0, h, tile, parts, rows, begins, ends};
        atomicOr(&there, 1u << (2 * warp + (first_piece ? 0 : 1)));
      }
    }
    u = min(end, u1);
  }
  if (abort) {               // copies that a wait gave up on land before the CTA ends
    for (int k = 0; k < S; ++k) mbar_wait_bounded(&full[warp][k], ((phases >> k) & 1) ^ 1);
  }
  __syncthreads();
  if (there == 0) return;

  // The pieces of segments that several warps had, in the order of the line; each group of lanes does it for its rows. A segment
  // that was begun and ended in this CTA is done with; what another CTA began (part 0) or ends (part 1) is left as a part.
  float* parts = p.parts + 2 * static_cast<int64_t>(blockIdx.x) * kPart<D, R>;
#pragma unroll 1
  for (int r0 = warp * (32 / L); r0 < R; r0 += kWarps * (32 / L)) {
    const int r = r0 + lane / L, l8 = lane % L;
    float v[8], most = kLow, sum = 0.f;
    bool open = false, begun = false;
    const Piece* now = nullptr;
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = 0.f;
    auto close = [&](bool ended) {
      const float inv = sum == 0.f ? 0.f : __fdiv_rn(1.0f, sum);
      if (begun && ended) {
        const int rr = now->tile * R + r, i = divide(rr, p.group), hq = now->h * p.group + rr - i * p.group;
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] = sum == 0.f ? 0.f : v[j] * inv;
        store_row<T, D>(p, rr < now->rows, now->n0 + i, hq, l8, v);
      } else {
        float* part = parts + (begun ? kPart<D, R> : 0);
#pragma unroll
        for (int j = 0; j < 2; ++j)
          *reinterpret_cast<float4*>(part + r * D + 8 * l8 + 4 * j) = *reinterpret_cast<const float4*>(v + 4 * j);
        if (l8 == 0) {
          part[R * D + r] = most;
          part[R * D + R + r] = sum;
        }
        if (begun && threadIdx.x == 0) {
          p.meta[2 * blockIdx.x] = make_int4(now->h, now->tile, now->parts, 0);
          p.meta[2 * blockIdx.x + 1] = make_int4(static_cast<int>(now->n0), now->rows, 0, 0);
        }
      }
      open = false;
    };
#pragma unroll 1
    for (uint32_t left = there; left; left &= left - 1) {
      const int w = __ffs(left) - 1;
      const Piece& pc = piece[w >> 1][w & 1];
      const float* src = reinterpret_cast<const float*>(smem + (w >> 1) * Sh::kRing + (w & 1 ? 0 : (S - Sh::kHeld) * Sh::kStep)) +
                         r * Sh::kPitch + 8 * l8;
      if (!open) {
        open = true;
        begun = pc.begins;
        now = &pc;
        most = kLow;
        sum = 0.f;
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] = 0.f;
      }
      const float m = stat[w >> 1][w & 1][0][r], more = fmaxf(most, m), f = exp2_fast(most - more), g = exp2_fast(m - more);
      sum = fmaf(sum, f, stat[w >> 1][w & 1][1][r] * g);
      most = more;
#pragma unroll
      for (int j = 0; j < 8; ++j) v[j] = fmaf(v[j], f, src[j] * g);
      if (pc.ends) close(true);
    }
    if (open) close(false);
  }
}

// The segments that several CTAs had parts of. Every CTA makes the list of the CTAs that began one, and takes rows of
// their tiles: a row by one warp where there are rows enough for all, else by up to eight that share its parts.
constexpr int kJoinWarps = 8, kJoinThreads = 32 * kJoinWarps;

template <typename T, int D, int R>
__global__ void __launch_bounds__(kJoinThreads) attn_q4_join_kernel(const Attn p, int ctas) {
  constexpr int E = D / 32;                                           // elements of a lane
  extern __shared__ int4 list[];                                      // [ctas][2]: the CTA, and what it left in meta
  __shared__ float sums[kJoinWarps][D];
  __shared__ int found[kJoinWarps];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  pdl_enter();
  int n = 0;
  for (int c0 = 0; c0 < ctas; c0 += kJoinThreads) {
    const int c = c0 + threadIdx.x;
    int4 a = make_int4(-1, 0, 0, 0), b = a;
    if (c < ctas) a = p.meta[2 * c], b = p.meta[2 * c + 1];
    const uint32_t all = __ballot_sync(0xffffffffu, a.x >= 0);
    if (c0 > 0) __syncthreads();
    if (lane == 0) found[warp] = __popc(all);
    __syncthreads();
    int at = n;
#pragma unroll
    for (int w = 0; w < kJoinWarps; ++w) {
      if (w < warp) at += found[w];
      n += found[w];
    }
    if (a.x >= 0) {
      at += __popc(all & ((1u << lane) - 1));
      a.w = c;
      list[2 * at] = a;
      list[2 * at + 1] = b;
    }
  }
  if (n == 0) return;
  __syncthreads();
  const int items = n * R;
  int W = 1;                                                          // warps of a row
  while (W < kJoinWarps && items * 2 * W <= static_cast<int>(gridDim.x) * kJoinWarps) W *= 2;
  const int each = kJoinWarps / W, group = warp / W, part0 = warp % W;
  for (int first = blockIdx.x * each; first < items; first += gridDim.x * each) {
    const int item = first + group;
    int i = 0, hq = 0, n0 = 0;
    bool here = false;
    float sum = 0.f, acc[E];
#pragma unroll
    for (int e = 0; e < E; ++e) acc[e] = 0.f;
    if (item < items) {
      const int4 a = list[2 * (item / R)], b = list[2 * (item / R) + 1];
      const int r = item % R, rr = a.y * R + r, count = a.z;
      i = divide(rr, p.group);
      hq = a.x * p.group + rr - i * p.group;
      n0 = b.x;
      here = rr < b.y;
      const float* base = p.parts + 2 * static_cast<int64_t>(a.w) * kPart<D, R>;
      auto part = [&](int k) { return base + (k == 0 ? 1 : 2 * static_cast<int64_t>(k)) * kPart<D, R>; };
      if (here) {
        // Parts k0 + lane: their maxima and totals; the sums relative to the largest so far.
        float most = kLow;
        for (int k0 = 0; k0 < count; k0 += 32) {
          const int k = k0 + lane, some = min(32, count - k0);
          float m = kLow, t = 0.f;
          if (k < count) m = part(k)[R * D + r], t = part(k)[R * D + R + r];
          float more = m;
#pragma unroll
          for (int o = 16; o > 0; o >>= 1) more = fmaxf(more, __shfl_xor_sync(0xffffffffu, more, o));
          more = fmaxf(more, most);
          const float by = exp2_fast(most - more), f = k < count ? exp2_fast(m - more) : 0.f;
          most = more;
          sum = sum * by + f * t;
#pragma unroll
          for (int e = 0; e < E; ++e) acc[e] *= by;
#pragma unroll 4
          for (int t = part0; t < some; t += W) {
            const float g = __shfl_sync(0xffffffffu, f, t);
            const float* src = part(k0 + t) + r * D + E * lane;
            float v[E];
            if constexpr (E == 2) {
              *reinterpret_cast<float2*>(v) = *reinterpret_cast<const float2*>(src);
            } else {
#pragma unroll
              for (int e = 0; e < E / 4; ++e) reinterpret_cast<float4*>(v)[e] = reinterpret_cast<const float4*>(src)[e];
            }
#pragma unroll
            for (int e = 0; e < E; ++e) acc[e] = fmaf(g, v[e], acc[e]);
          }
        }
        sum = warp_sum_f(sum);
      }
    }
#pragma unroll
    for (int e = 0; e < E; ++e) sums[warp][E * lane + e] = acc[e];
    __syncthreads();
    if (part0 == 0) {
      const float inv = sum == 0.f ? 0.f : __fdiv_rn(1.0f, sum);
      float v[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        v[j] = 0.f;
        if (lane < D / 8)
          for (int w = 0; w < W; ++w) v[j] += sums[warp + w][8 * lane + j];
        v[j] = sum == 0.f ? 0.f : v[j] * inv;
      }
      store_row<T, D>(p, here && lane < D / 8, static_cast<int64_t>(n0) + i, hq, lane, v);
    }
    __syncthreads();
  }
}

// Rows of a tile: 8, or 16 where a sequence has more than 64 (row, query head) pairs of a key head on the average. 16 unpack a
// step once for two columns of operands, but leave a warp more registers and so eight warps in place of twelve. us with 8 and 16
// rows, 8 key heads of 128: 64 sequences of up to 4096 places with 12 pairs 38.0 and 46.1, 16 of up to 8192 with 32 pairs 41.5
// and 43.8, with 64 pairs 57.3 and 57.2 (fp32 rows 83 and 100), 4 with 256 pairs 102 and 88 (fp32 160 and 151). Heads of
// 256 elements always 8: their sums are 128 registers for 16 rows.
int tile_rows(int group, int D, int64_t N, int64_t n_seqs) { return D == 256 || group * N <= 64 * n_seqs ? 8 : 16; }

template <typename T, int D, int NT, bool FINE>
cudaError_t run(const Attn& p, int num_sms, cudaStream_t s) {
  using Sh = Shape<T, D, NT, FINE>;
  static std::atomic<uint64_t> allowed{0};                            // devices on which the shared memory is set
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev >= 64 || !(allowed.load(std::memory_order_acquire) >> dev & 1)) {
    e = cudaFuncSetAttribute(attn_q4_kernel<T, D, NT, FINE>, cudaFuncAttributeMaxDynamicSharedMemorySize, Sh::kSmem);
    if (e != cudaSuccess) return e;
    if (dev < 64) allowed.fetch_or(uint64_t(1) << dev, std::memory_order_release);
  }
  const int grid = num_sms;
  e = launch_pdl(attn_q4_kernel<T, D, NT, FINE>, dim3(grid), dim3(Sh::kThreads), Sh::kSmem, s, p);
  if (e != cudaSuccess) return e;
  return launch_pdl(attn_q4_join_kernel<T, D, Sh::R>, dim3(num_sms), dim3(kJoinThreads), grid * 2 * sizeof(int4), s, p, grid);
}

template <typename T, bool FINE>
cudaError_t run(const Attn& p, int num_sms, cudaStream_t s) {
  const bool wide = tile_rows(p.group, p.c.D, p.a.N, p.c.n_seqs) == 16;
  if (p.c.D == 64) return wide ? run<T, 64, 2, FINE>(p, num_sms, s) : run<T, 64, 1, FINE>(p, num_sms, s);
  if (p.c.D == 128) return wide ? run<T, 128, 2, FINE>(p, num_sms, s) : run<T, 128, 1, FINE>(p, num_sms, s);
  return run<T, 256, 1, FINE>(p, num_sms, s);
}

template <typename T>
cudaError_t run(const Attn& p, int num_sms, cudaStream_t s) {
  return sizeof(T) == 4 || p.a.Xq ? run<T, true>(p, num_sms, s) : run<T, false>(p, num_sms, s);
}
template <>
cudaError_t run<float>(const Attn& p, int num_sms, cudaStream_t s) {
  return run<float, true>(p, num_sms, s);
}

}  // namespace

size_t attn_q4_workspace(int n_q, int n_kv, int D, int64_t N, int64_t n_seqs, int num_sms) {
  const int R = tile_rows(n_q / n_kv, D, N, n_seqs);
  const size_t ctas = static_cast<size_t>(num_sms);
  return ctas * (2 * sizeof(int4) + 2 * sizeof(float) * (static_cast<size_t>(R) * D + 2 * R));
}

cudaError_t launch_attn_q4(int dtype, const AttnArgs& a, const KvCache& c, void* ws, int* err, int num_sms, cudaStream_t s) {
  const int64_t size = dtype == KQ_F32 ? 4 : 2;
  Attn p = {a, c, nullptr, static_cast<int4*>(ws), a.n_q / c.heads,
            a.ldq * size % 16 == 0 && (!a.O || a.ldo * size % 16 == 0), err};
  p.parts = reinterpret_cast<float*>(p.meta + 2 * num_sms);
  if (dtype == KQ_F16) return run<__half>(p, num_sms, s);
  if (dtype == KQ_BF16) return run<__nv_bfloat16>(p, num_sms, s);
  return run<float>(p, num_sms, s);
}

}  // namespace kq
