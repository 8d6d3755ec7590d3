// Products of Q8_1 activations with 4-bit weights that carry group scales:
//
//   y[m] = Sum_b d_b * s(m, b) * ( Sum_k c[m][k] q[k] - z(m, b) * Sum_k q[k] )
//
// over the 32-element blocks b, c the 4-bit codes, s and z the scale and zero
// point of the block's group, d and q the block's Q8_1 scale and codes. The two
// sums over a block are exact in 32-bit integers (dp4a); the products with the
// scales and the sum over the blocks are fp32.
#include <cuda_bf16.h>

#include <algorithm>
#include <cstdlib>

#include "kq_internal.h"
#include "kq_types.cuh"

namespace kq {
namespace {

constexpr int G4_WARPS = 8;
constexpr unsigned FULL_MASK = 0xffffffffu;

template <typename S>
__device__ __forceinline__ float scale_at(const void* scales, int64_t i) {
  return to_f32(static_cast<const S*>(scales)[i]);
}

// One warp per output row and activation row; lane l takes the blocks l, l + 32, ...
template <typename S, bool MOE>
__global__ void __launch_bounds__(G4_WARPS * 32) g4_simple_kernel(G4Weights w, const int32_t* __restrict__ ids,
                                                                  int n_experts, int top_k, bool x_per_slot,
                                                                  const uint8_t* __restrict__ Xq, float* __restrict__ Y,
                                                                  int64_t M, int blocks, int64_t rows, int* err) {
  pdl_enter();
  const int lane = threadIdx.x & 31;
  const int64_t m = static_cast<int64_t>(blockIdx.x) * G4_WARPS + (threadIdx.x >> 5);
  if (m >= M) return;
  for (int64_t p = blockIdx.y; p < rows; p += gridDim.y) {
    int64_t r = m, xr = p;
    if (MOE) {
      const int e = ids[p];
      if (e < 0 || e >= n_experts) {
        if (lane == 0) {
          if (m == 0) report_error(err, ERR_EXPERT_ID);
          Y[p * M + m] = 0.f;
        }
        continue;
      }
      r = static_cast<int64_t>(e) * M + m;
      xr = x_per_slot ? p : p / top_k;
    }
    const uint4* codes = reinterpret_cast<const uint4*>(w.codes) + r * blocks;
    const uint8_t* xrow = Xq + xr * blocks * Q8_1_BYTES;
    float acc = 0.f;
    for (int b = lane; b < blocks; b += 32) {
      const uint4 c = codes[b];
      const int64_t gi = r * w.groups + (b >> w.group_shift);
      const float s = scale_at<S>(w.scales, gi);
      const int z = w.zeros ? w.zeros[gi] : 8;
      const uint32_t* xb = reinterpret_cast<const uint32_t*>(xrow + static_cast<int64_t>(b) * Q8_1_BYTES);
      const float d = __low2float(bits_half2(xb[0]));
      const uint32_t cw[4] = {c.x, c.y, c.z, c.w};
      int dot = 0, sum = 0;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const uint32_t x0 = xb[1 + 2 * i], x1 = xb[2 + 2 * i];  // elements 8i..8i+3, 8i+4..8i+7
        dot = dp4a_us(cw[i] & 0x0f0f0f0fu, static_cast<int>(__byte_perm(x0, x1, 0x6420)), dot);
        dot = dp4a_us((cw[i] >> 4) & 0x0f0f0f0fu, static_cast<int>(__byte_perm(x0, x1, 0x7531)), dot);
        sum = __dp4a(static_cast<int>(x0), 0x01010101, sum);
        sum = __dp4a(static_cast<int>(x1), 0x01010101, sum);
      }
      acc = fmaf(s * d, static_cast<float>(dot - z * sum), acc);
    }
    acc = warp_sum_f(acc);
    if (lane == 0) Y[p * M + m] = acc;
  }
}

// ---------------------------------------------------------------------------
// Several activation rows: tensor-core form
// ---------------------------------------------------------------------------
// Weights read once for up to 8 * NT activation rows, with m16n8k16 fp16 MMAs
// whose operands are small integers, so that every block's dot product is exact
// in the fp32 accumulator.
//
// Weight codes are not converted: a nibble or-ed into the mantissa of fp16 1024
// is 1024 + c (low nibbles of a 16-bit field) or 1024 + 16 c (the next ones), one
// logic operation for two codes. The even k of a block go through one MMA as
// (1024 + c) * q, the odd k through a second as (1024 + 16 c) * (q / 16), both
// exact; their sum is Sum c q + 1024 Sum_even q + 64 Sum_odd q, an integer below
// 32 * 1039 * 128 < 2^24. The excess depends on the activation row alone and is
// taken off by starting the accumulator at its negative (with 8 Sum q too where
// there are no zero points).
//
// k is permuted within a block: lane (g = lane / 4, t = lane % 4) of a warp
// takes word t (k = 8t..8t+7) of its rows' 16-byte blocks for A and the same k of
// activation row g for B.
//
// A CTA's four warps take 32 weight rows each and share the activations: the
// B fragments of a panel of K (g4_panel(NT) / NT blocks) are made once, by all warps,
// into shared memory. Over a panel each warp runs on its own: its weights and
// scales come by cp.async into a ring of its own, a few chunks (128 k) deep,
// which keeps filling while fragments are made. Where there are too few row
// tiles for the SMs, a cluster of CTAs splits K; their sums are added in rank
// order through distributed shared memory.
constexpr int G4_CHUNK = 4;        // 32-element blocks per chunk
// Chunks of weights in flight per warp: as many as leave room for four CTAs on an SM.
__host__ __device__ constexpr int g4_stages(bool FINE) { return FINE ? 3 : 4; }
constexpr int G4_ROWS = 128;       // weight rows of a CTA, 32 per warp
// Fragments (of one block and 8 activation rows) per panel.
__host__ __device__ constexpr int g4_panel(int NT) { return NT == 4 ? 32 : 16; }
constexpr int G4_SPAN = 16;        // groups whose scales are fetched together: a 32-byte sector of a row
constexpr int G4_LIST = 256;       // rows of one expert collected at a time

struct alignas(16) G4Frag {    // of one block and 8 activation rows
  uint4 b[32];     // lane (g, t) at frag_at(g, t): even k (two registers), odd k / 16 (two registers)
  float4 init[4];  // per t: start of the accumulators of rows 2t, 2t + 1, 2t, 2t + 1
  float2 d[4];     // per t: scales of rows 2t, 2t + 1
  float2 sum[4];   // per t: Sum q of rows 2t, 2t + 1 (with zero points)
};
// Written for one t and all g at a time and read for all t and two g by eight
// lanes at a time: both touch eight different 16-byte bank groups.
__device__ __forceinline__ int frag_at(int g, int t) { return t * 8 + ((g + 2 * t) & 7); }

template <bool FINE>
struct alignas(16) G4Warp {    // a warp's own
  uint8_t w[g4_stages(FINE)][32][G4_CHUNK * 16];
  uint8_t raw[2][32][G4_SPAN * 3];                 // as in memory: G4_SPAN scales, then G4_SPAN zero points
  float2 scale[FINE ? G4_CHUNK : 1][FINE ? 32 : 1];   // scale and zero point of a chunk's blocks (FINE)
};
template <int NT, bool FINE>
struct G4Smem {
  G4Warp<FINE> warp[4];
  G4Frag frag[g4_panel(NT)];
  int count, list[G4_LIST];                       // the expert's pairs
};
// cp.async and ldmatrix take 16-byte rows at 16-byte boundaries.
static_assert(sizeof(G4Warp<true>) % 16 == 0 && sizeof(G4Warp<false>) % 16 == 0 && sizeof(G4Frag) == 640 && G4_SPAN % 16 == 0);
static_assert(offsetof(G4Warp<false>, raw) % 16 == 0);

__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, uint32_t bytes) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}
__device__ __forceinline__ void cp_async4(uint32_t dst, const void* src, uint32_t bytes) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}
__device__ __forceinline__ void cp_async8(uint32_t dst, const void* src) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 8;" ::"r"(dst), "l"(src) : "memory");
}
// `bytes` (at most a multiple of 4 per row) of a row whose address and length are
// multiples of 4, in pieces as large as its alignment allows.
__device__ __forceinline__ void cp_async_row(uint32_t dst, const uint8_t* src, int bytes, int align) {
  if (align % 16 == 0) {
    for (int o = 0; o < bytes; o += 16) cp_async16(dst + o, src + o, 16);
  } else if (align % 8 == 0) {
    for (int o = 0; o < bytes; o += 8) cp_async8(dst + o, src + o);
  } else {
    for (int o = 0; o < bytes; o += 4) cp_async4(dst + o, src + o, 4);
  }
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_async_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }

__device__ __forceinline__ void ldmatrix4(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr));
}
__device__ __forceinline__ void mma16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1, float c0,
                                         float c1, float c2, float c3) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%11,%12,%13};"
      : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(c0), "f"(c1), "f"(c2), "f"(c3));
}
__device__ __forceinline__ float ld_cluster_f32(uint32_t addr) {
  float v;
  asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(addr) : "memory");
  return v;
}
// (v & mask) | 0x6400'6400 in one operation.
__device__ __forceinline__ uint32_t with_1024(uint32_t v, uint32_t mask) {
  uint32_t r;
  asm("lop3.b32 %0, %1, %2, %3, 0xea;" : "=r"(r) : "r"(v), "r"(mask), "r"(0x64006400u));
  return r;
}
constexpr uint32_t H2_M1152 = 0xe480e480u, H2_M72 = 0xd480d480u, H2_SIXTEENTH = 0x2c002c00u;   // fp16 pairs

struct G4Args {
  G4Weights w;
  const uint8_t* Xq;
  float* Y;
  const int32_t* ids;   // null: one matrix, rows 0..rows-1 of Xq
  int n_experts, top_k;
  bool x_per_slot, by_pair;
  int64_t M;
  int64_t rows;         // activation rows, or (token, slot) pairs
  int blocks;           // 32-element blocks per row
  int splits;           // CTAs of a cluster, over K
  int* err;
};

// Byte i of v as fp32, exactly: 2^23 + byte, less 2^23.
__device__ __forceinline__ float byte_f32(uint32_t v, int i) {
  return __uint_as_float(__byte_perm(v, 0x4b000000u, 0x7440 + i)) - 8388608.0f;
}

// FINE: a group is shorter than a chunk, so every block has its own scale; else
// one scale serves a chunk. ZEROS: zero points are given.
template <int NT, bool FINE, bool ZEROS>
__global__ void __launch_bounds__(128, NT == 4 ? 3 : 4) g4_mma_kernel(G4Args a) {
  extern __shared__ __align__(16) uint8_t smem_raw[];
  G4Smem<NT, FINE>& sm = *reinterpret_cast<G4Smem<NT, FINE>*>(smem_raw);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  G4Warp<FINE>& my = sm.warp[warp];
  const int g = lane >> 2, t = lane & 3;
  constexpr int TOK = NT * 8;
  constexpr int G4_STAGES = g4_stages(FINE);
  constexpr int PANEL = g4_panel(NT) / NT / G4_CHUNK;   // chunks
  static_assert(sizeof(sm.frag) >= TOK * G4_ROWS * sizeof(float));   // the sums take the fragments' place
  const int rank = a.splits > 1 ? static_cast<int>(cluster_ctarank()) : 0;
  const int64_t m0 = static_cast<int64_t>(blockIdx.x / a.splits) * G4_ROWS;
  const int rows = static_cast<int>(min(a.M - m0, static_cast<int64_t>(G4_ROWS)));   // of this tile

  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  // One matrix: its weights are on their way before the previous kernel's end.
  if (a.ids) asm volatile("griddepcontrol.wait;" ::: "memory");
  int expert = 0;
  int64_t scan = 0;     // next pair to look at
  if (a.ids) {
    if (a.by_pair) {
      // One cluster per pair; the first pair of an expert takes all of its pairs.
      expert = a.ids[blockIdx.y];
      if (expert < 0 || expert >= a.n_experts) {
        if (tid == 0 && blockIdx.x == 0) report_error(a.err, ERR_EXPERT_ID);
        if (rank == 0 && tid < rows) a.Y[blockIdx.y * a.M + m0 + tid] = 0.f;
        return;
      }
      int earlier = 0;
      for (int p = tid; p < static_cast<int>(blockIdx.y); p += 128) earlier |= a.ids[p] == expert;
      if (__syncthreads_or(earlier)) return;
      scan = blockIdx.y;
    } else {
      expert = blockIdx.y;
      // Invalid ids belong to no expert: expert 0's CTAs write their zeros.
      if (expert == 0 && rank == 0) {
        for (int64_t p = tid; p < a.rows; p += 128) {
          const int e = a.ids[p];
          if (e < 0 || e >= a.n_experts) {
            if (blockIdx.x == 0) report_error(a.err, ERR_EXPERT_ID);
            for (int m = 0; m < rows; ++m) a.Y[p * a.M + m0 + m] = 0.f;
          }
        }
      }
    }
  }
  const int64_t row0 = static_cast<int64_t>(expert) * a.M + m0;
  const int64_t row_bytes = static_cast<int64_t>(a.blocks) * 16;
  const int chunks = (a.blocks + G4_CHUNK - 1) / G4_CHUNK;
  const int c_begin = static_cast<int>(static_cast<int64_t>(chunks) * rank / a.splits);
  const int c_end = static_cast<int>(static_cast<int64_t>(chunks) * (rank + 1) / a.splits);
  const bool even = a.blocks % G4_CHUNK == 0;   // whole chunks
  const int64_t xbytes = static_cast<int64_t>(a.blocks) * Q8_1_BYTES;
  // This lane copies 16-byte piece t of its warp's rows g + 8 i, and fetches the
  // scales of its row `lane` (a row past the tile's last is that row again; its
  // sums are not written).
  const uint8_t* wsrc0[4];
#pragma unroll
  for (int i = 0; i < 4; ++i)
    wsrc0[i] = a.w.codes + (row0 + min(warp * 32 + g + 8 * i, rows - 1)) * row_bytes + t * 16 + static_cast<int64_t>(c_begin) * 64;
  const uint32_t wdst = smem_u32(&my.w[0][g][(t ^ ((g >> 1) & 3)) << 4]);
  const int64_t srow = (row0 + min(tid, rows - 1)) * a.w.groups;
  // ldmatrix: lane l gives the address of row l % 8 of matrix l / 8: rows 0-7, 8-15 of
  // the first and then of the second 16-row tile.
  uint32_t arow[G4_CHUNK];   // of each block of a chunk
#pragma unroll
  for (int b = 0; b < G4_CHUNK; ++b) arow[b] = smem_u32(&my.w[0][lane][(b ^ ((lane >> 1) & 3)) << 4]);
  const int frag = frag_at(g, t);
  auto scale_f = [&](uint16_t bits) {
    return a.w.scale_dtype == KQ_F16 ? __half2float(__ushort_as_half(bits)) : __uint_as_float(static_cast<uint32_t>(bits) << 16);
  };

  for (;;) {
    int have;
    if (a.ids) {
      // Collect this expert's pairs (in any order: each output depends on its own pair alone).
      __syncthreads();
      if (tid == 0) sm.count = 0;
      __syncthreads();
      bool more = scan < a.rows;
      while (more) {
        const int64_t p = scan + tid;
        if (p < a.rows && a.ids[p] == expert) sm.list[atomicAdd(&sm.count, 1)] = static_cast<int>(p);
        scan += 128;
        __syncthreads();
        have = *reinterpret_cast<volatile int*>(&sm.count);
        more = scan < a.rows && have + 128 <= G4_LIST;
        __syncthreads();
      }
      have = *reinterpret_cast<volatile int*>(&sm.count);
      if (a.splits > 1) {
        // The clusters' CTAs use the list of rank 0: theirs may be in another order.
        cluster_sync();
        if (rank != 0)
          for (int i = tid; i < have; i += 128) {
            int v;
            asm volatile("ld.shared::cluster.s32 %0, [%1];" : "=r"(v) : "r"(mapa_shared(&sm.list[i], 0)) : "memory");
            sm.list[i] = v;
          }
        cluster_sync();
      }
      if (have == 0) return;
    } else {
      have = static_cast<int>(min(a.rows - static_cast<int64_t>(blockIdx.y) * TOK, static_cast<int64_t>(TOK)));
    }
    for (int n0 = 0; n0 < have; n0 += TOK) {
      const int nn = min(TOK, have - n0);
      // A thread makes one (activation row, block) of a panel's fragments, or two: row
      // tid % TOK of this pass, the panel's blocks tid / TOK, ... Their nine words are
      // loaded a panel ahead.
      constexpr int MINE = g4_panel(NT) * 8 / 128;
      const int xn = tid % TOK;
      const uint32_t* xr = nullptr;
      if (xn < nn) {
        int64_t r = static_cast<int64_t>(blockIdx.y) * TOK + xn;
        if (a.ids) {
          const int p = sm.list[n0 + xn];
          r = a.x_per_slot ? p : p / a.top_k;
        }
        xr = reinterpret_cast<const uint32_t*>(a.Xq + r * xbytes);
      }
      const uint8_t* wsrc[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) wsrc[i] = wsrc0[i];
      int span_chunk = c_begin;      // the next chunk whose scales are in a new span
      // The copies of chunk c (called for c_begin, c_begin + 1, ...) into a slot.
      auto fill = [&](int c, int slot) {
        const uint32_t wd = wdst + slot * (32 * 64);
        if (even || c + 1 < chunks) {
#pragma unroll
          for (int i = 0; i < 4; ++i) cp_async16(wd + i * 512, wsrc[i], 16);
        } else {
#pragma unroll
          for (int i = 0; i < 4; ++i) {   // blocks past K: zero
            const bool in = c * G4_CHUNK + t < a.blocks;
            cp_async16(wd + i * 512, in ? wsrc[i] : a.w.codes, in ? 16 : 0);
          }
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) wsrc[i] += 64;
        // The scales of the next G4_SPAN groups with the first chunk that needs them; the
        // span before the last is out of use by then.
        if (c == span_chunk) {
          const int span = (c * G4_CHUNK >> a.w.group_shift) / G4_SPAN;
          span_chunk = static_cast<int>(min((static_cast<int64_t>(span + 1) * G4_SPAN << a.w.group_shift) / G4_CHUNK, static_cast<int64_t>(chunks)));
          const int n = static_cast<int>(min(a.w.groups - span * G4_SPAN, static_cast<int64_t>(G4_SPAN)));
          const int64_t at = srow + span * G4_SPAN;
          uint8_t* raw = my.raw[span & 1][lane];
          const uint16_t* ss = static_cast<const uint16_t*>(a.w.scales) + at;
          for (int i = n; i < G4_SPAN; ++i) {   // blocks past K get scale 0
            reinterpret_cast<uint16_t*>(raw)[i] = 0;
            raw[2 * G4_SPAN + i] = 0;
          }
          if (a.w.groups % 2 == 0) {
            cp_async_row(smem_u32(raw), reinterpret_cast<const uint8_t*>(ss), 2 * n, static_cast<int>(2 * a.w.groups & 31));
          } else {
            for (int i = 0; i < n; ++i) reinterpret_cast<uint16_t*>(raw)[i] = __ldg(ss + i);
          }
          if (ZEROS) {
            if (a.w.groups % 4 == 0) {
              cp_async_row(smem_u32(raw) + 2 * G4_SPAN, a.w.zeros + at, n, static_cast<int>(a.w.groups & 31));
            } else {
              for (int i = 0; i < n; ++i) raw[2 * G4_SPAN + i] = __ldg(a.w.zeros + at + i);
            }
          }
        }
      };
      uint32_t px[MINE][9];
      auto load = [&](int c) {
#pragma unroll
        for (int k = 0; k < MINE; ++k) {
          const int b = c * G4_CHUNK + tid / TOK + k * (128 / TOK);
#pragma unroll
          for (int j = 0; j < 9; ++j) px[k][j] = 0;
          if (xr && b < a.blocks) {
#pragma unroll
            for (int j = 0; j < 9; ++j) px[k][j] = __ldg(xr + static_cast<int64_t>(b) * 9 + j);
          }
        }
      };
      auto make = [&](int k) {
        G4Frag& f = sm.frag[(tid / TOK + k * (128 / TOK)) * NT + xn / 8];
        const int fg = xn & 7;
        int se = 0, so = 0;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const uint32_t x0 = px[k][1 + 2 * j], x1 = px[k][2 + 2 * j];
          const uint32_t ev = __byte_perm(x0, x1, 0x6240), od = __byte_perm(x0, x1, 0x7351);
          se = __dp4a(static_cast<int>(ev), 0x01010101, se);
          so = __dp4a(static_cast<int>(od), 0x01010101, so);
          const uint32_t ue = ev ^ 0x80808080u, uo = od ^ 0x80808080u;    // codes + 128
          f.b[frag_at(fg, j)] = make_uint4(
              half2_bits(__hadd2(bits_half2(__byte_perm(ue, 0x64646464u, 0x4140)), bits_half2(H2_M1152))),
              half2_bits(__hadd2(bits_half2(__byte_perm(ue, 0x64646464u, 0x4342)), bits_half2(H2_M1152))),
              half2_bits(__hfma2(bits_half2(__byte_perm(uo, 0x64646464u, 0x4140)), bits_half2(H2_SIXTEENTH), bits_half2(H2_M72))),
              half2_bits(__hfma2(bits_half2(__byte_perm(uo, 0x64646464u, 0x4342)), bits_half2(H2_SIXTEENTH), bits_half2(H2_M72))));
        }
        float* c = reinterpret_cast<float*>(&f.init[fg >> 1]) + (fg & 1);
        c[0] = c[2] = static_cast<float>(ZEROS ? -(1024 * se + 64 * so) : -(1032 * se + 72 * so));
        reinterpret_cast<float*>(&f.d[fg >> 1])[fg & 1] = __low2float(bits_half2(px[k][0]));
        if (ZEROS) reinterpret_cast<float*>(&f.sum[fg >> 1])[fg & 1] = static_cast<float>(se + so);
      };

      float acc[2][NT][4] = {};
      for (int i = 0; i < G4_STAGES - 1; ++i) {
        if (c_begin + i < c_end) fill(c_begin + i, i);
        cp_async_commit();
      }
      if (!a.ids) asm volatile("griddepcontrol.wait;" ::: "memory");
      load(c_begin);
      int slot = 0;   // of chunk c
      for (int c = c_begin, p_begin = c_begin, p_end = c_begin; c < c_end; ++c) {
        if (c == p_end) {
          p_begin = c;
          p_end = min(c + PANEL, c_end);
          __syncthreads();   // the last panel is used up
#pragma unroll
          for (int k = 0; k < MINE; ++k) make(k);
          load(p_end);
          __syncthreads();
        }
        cp_async_wait<G4_STAGES - 2>();
        __syncwarp();
        uint32_t wc[G4_CHUNK][4];
#pragma unroll
        for (int b = 0; b < G4_CHUNK; ++b) ldmatrix4(wc[b], arow[b] + slot * (32 * 64));
        if (c + G4_STAGES - 1 < c_end) fill(c + G4_STAGES - 1, slot == 0 ? G4_STAGES - 1 : slot - 1);
        cp_async_commit();
        slot = slot == G4_STAGES - 1 ? 0 : slot + 1;
        const G4Frag* pf = &sm.frag[(c - p_begin) * (G4_CHUNK * NT)];
        float2 s[4];   // scale and zero point of rows g, g + 8, g + 16, g + 24
        if (FINE) {
          // Lane: row; the four blocks' scales converted once. A chunk has four groups or two.
          const int gr = c * G4_CHUNK >> a.w.group_shift;
          const uint8_t* raw = my.raw[(gr / G4_SPAN) & 1][lane];
          const uint16_t* rs = reinterpret_cast<const uint16_t*>(raw) + gr % G4_SPAN;
          const uint8_t* rz = raw + 2 * G4_SPAN + gr % G4_SPAN;
          uint2 sb;
          uint32_t zb;
          if (a.w.group_shift == 0) {
            sb = *reinterpret_cast<const uint2*>(rs);
            zb = *reinterpret_cast<const uint32_t*>(rz);
          } else {
            const uint32_t two = *reinterpret_cast<const uint32_t*>(rs), zz = *reinterpret_cast<const uint16_t*>(rz);
            sb = make_uint2(__byte_perm(two, 0, 0x1010), __byte_perm(two, 0, 0x3232));
            zb = __byte_perm(zz, 0, 0x1100);
          }
          my.scale[0][lane] = make_float2(scale_f(sb.x & 0xffff), ZEROS ? byte_f32(zb, 0) : 0.f);
          my.scale[1][lane] = make_float2(scale_f(sb.x >> 16), ZEROS ? byte_f32(zb, 1) : 0.f);
          my.scale[2][lane] = make_float2(scale_f(sb.y & 0xffff), ZEROS ? byte_f32(zb, 2) : 0.f);
          my.scale[3][lane] = make_float2(scale_f(sb.y >> 16), ZEROS ? byte_f32(zb, 3) : 0.f);
          __syncwarp();
        } else {
          const int gr = (c * G4_CHUNK) >> a.w.group_shift;
          const uint8_t* raw = my.raw[(gr / G4_SPAN) & 1][g];
#pragma unroll
          for (int i = 0; i < 4; ++i)
            s[i] = make_float2(scale_f(reinterpret_cast<const uint16_t*>(raw + i * (8 * G4_SPAN * 3))[gr % G4_SPAN]),
                               ZEROS ? byte_f32(raw[i * (8 * G4_SPAN * 3) + 2 * G4_SPAN + gr % G4_SPAN], 0) : 0.f);
        }
        float part[2][NT][4];   // of this chunk, before the chunk's scale (not FINE)
#pragma unroll
        for (int b = 0; b < G4_CHUNK; ++b) {
          const uint32_t (&w)[4] = wc[b];
          uint32_t L[2][4], U[2][4];
#pragma unroll
          for (int m = 0; m < 2; ++m) {
            const uint32_t v0 = w[2 * m] >> 8, v1 = w[2 * m + 1] >> 8;
            L[m][0] = with_1024(w[2 * m], 0x000f000fu);
            L[m][1] = with_1024(w[2 * m + 1], 0x000f000fu);
            L[m][2] = with_1024(v0, 0x000f000fu);
            L[m][3] = with_1024(v1, 0x000f000fu);
            U[m][0] = with_1024(w[2 * m], 0x00f000f0u);
            U[m][1] = with_1024(w[2 * m + 1], 0x00f000f0u);
            U[m][2] = with_1024(v0, 0x00f000f0u);
            U[m][3] = with_1024(v1, 0x00f000f0u);
          }
          if (FINE) {
#pragma unroll
            for (int i = 0; i < 4; ++i) s[i] = my.scale[b][8 * i + g];
          }
#pragma unroll
          for (int n = 0; n < NT; ++n) {
            const G4Frag& f = pf[b * NT + n];
            const uint4 bf = f.b[frag];
            const float4 c0 = f.init[t];
            const float2 d = f.d[t];
            float2 sq = make_float2(0.f, 0.f);
            if (ZEROS) sq = f.sum[t];
#pragma unroll
            for (int m = 0; m < 2; ++m) {
              float r[4];
              mma16816(r, L[m], bf.x, bf.y, c0.x, c0.y, c0.z, c0.w);
              mma16816(r, U[m], bf.z, bf.w, r[0], r[1], r[2], r[3]);
              if (ZEROS) {
                r[0] = fmaf(-s[2 * m].y, sq.x, r[0]);
                r[1] = fmaf(-s[2 * m].y, sq.y, r[1]);
                r[2] = fmaf(-s[2 * m + 1].y, sq.x, r[2]);
                r[3] = fmaf(-s[2 * m + 1].y, sq.y, r[3]);
              }
              if (FINE) {
                acc[m][n][0] = fmaf(r[0] * d.x, s[2 * m].x, acc[m][n][0]);
                acc[m][n][1] = fmaf(r[1] * d.y, s[2 * m].x, acc[m][n][1]);
                acc[m][n][2] = fmaf(r[2] * d.x, s[2 * m + 1].x, acc[m][n][2]);
                acc[m][n][3] = fmaf(r[3] * d.y, s[2 * m + 1].x, acc[m][n][3]);
              } else {
                part[m][n][0] = b == 0 ? r[0] * d.x : fmaf(r[0], d.x, part[m][n][0]);
                part[m][n][1] = b == 0 ? r[1] * d.y : fmaf(r[1], d.y, part[m][n][1]);
                part[m][n][2] = b == 0 ? r[2] * d.x : fmaf(r[2], d.x, part[m][n][2]);
                part[m][n][3] = b == 0 ? r[3] * d.y : fmaf(r[3], d.y, part[m][n][3]);
              }
            }
          }
        }
        if (!FINE) {
#pragma unroll
          for (int m = 0; m < 2; ++m) {
            const float f0 = s[2 * m].x, f1 = s[2 * m + 1].x;
#pragma unroll
            for (int n = 0; n < NT; ++n) {
              acc[m][n][0] = fmaf(part[m][n][0], f0, acc[m][n][0]);
              acc[m][n][1] = fmaf(part[m][n][1], f0, acc[m][n][1]);
              acc[m][n][2] = fmaf(part[m][n][2], f1, acc[m][n][2]);
              acc[m][n][3] = fmaf(part[m][n][3], f1, acc[m][n][3]);
            }
          }
        }
      }
      cp_async_wait<0>();
      __syncthreads();  // the fragments make room for the sums of this CTA, [activation row][weight row]
      float* red = reinterpret_cast<float*>(sm.frag);
#pragma unroll
      for (int m = 0; m < 2; ++m)
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int k = 0; k < 4; ++k)
            red[(n * 8 + 2 * t + (k & 1)) * G4_ROWS + warp * 32 + m * 16 + g + 8 * (k >> 1)] = acc[m][n][k];
      if (a.splits > 1) cluster_sync(); else __syncthreads();
      // Each rank adds up and writes its share of the tile's rows.
      const int sh = 31 - __clz(G4_ROWS / a.splits);
      for (int i = tid; i < nn << sh; i += 128) {
        const int n = i >> sh, m = (rank << sh) + (i & ((1 << sh) - 1));
        if (m >= rows) continue;
        float v = red[n * G4_ROWS + m];
        if (a.splits > 1) {
          v = 0.f;
          for (int r = 0; r < a.splits; ++r) v += ld_cluster_f32(mapa_shared(red + n * G4_ROWS + m, r));
        }
        const int64_t out = a.ids ? sm.list[n0 + n] : static_cast<int64_t>(blockIdx.y) * TOK + n;
        a.Y[out * a.M + m0 + m] = v;
      }
      if (a.splits > 1) cluster_sync(); else __syncthreads();
    }
    if (!a.ids || scan >= a.rows) return;
  }
}

template <bool MOE>
cudaError_t launch_simple(const G4Weights& w, const int32_t* ids, int n_experts, int top_k, bool x_per_slot,
                          const uint8_t* Xq, float* Y, int64_t M, int64_t K, int64_t rows, int* err, cudaStream_t s) {
  const dim3 grid(static_cast<unsigned>((M + G4_WARPS - 1) / G4_WARPS),
                  static_cast<unsigned>(std::min<int64_t>(rows, 65535)));
  auto k = w.scale_dtype == KQ_F16 ? g4_simple_kernel<__half, MOE> : g4_simple_kernel<__nv_bfloat16, MOE>;
  return launch_pdl(k, grid, dim3(G4_WARPS * 32), 0, s, w, ids, n_experts, top_k, x_per_slot, Xq, Y, M,
                    static_cast<int>(K / 32), rows, err);
}

template <int NT, bool FINE, bool ZEROS>
cudaError_t launch_mma(const G4Args& a, unsigned grid_y, int slot, cudaStream_t s) {
  void (*k)(G4Args) = g4_mma_kernel<NT, FINE, ZEROS>;
  cudaError_t e = allow_max_smem(reinterpret_cast<const void*>(k), slot);
  if (e != cudaSuccess) return e;
  const int64_t tiles = (a.M + G4_ROWS - 1) / G4_ROWS;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(tiles * a.splits), grid_y);
  cfg.blockDim = dim3(128);
  cfg.dynamicSmemBytes = sizeof(G4Smem<NT, FINE>);
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim = {static_cast<unsigned>(a.splits), 1, 1};
  cfg.attrs = attr;
  cfg.numAttrs = a.splits > 1 ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, k, a);
}

template <int NT>
cudaError_t launch_mma_nt(const G4Args& a, unsigned grid_y, int slot, cudaStream_t s) {
  const bool zeros = a.w.zeros != nullptr;
  if (a.w.group_shift < 2)
    return zeros ? launch_mma<NT, true, true>(a, grid_y, slot, s) : launch_mma<NT, true, false>(a, grid_y, slot + 1, s);
  return zeros ? launch_mma<NT, false, true>(a, grid_y, slot + 2, s) : launch_mma<NT, false, false>(a, grid_y, slot + 3, s);
}

// NT: 8-row tiles of activations per CTA; grid_y: token tiles, pairs or experts.
cudaError_t launch_rows(G4Args a, unsigned grid_y, int64_t active_y, int NT, int num_sms, cudaStream_t s) {
  const int chunks = (a.blocks + G4_CHUNK - 1) / G4_CHUNK;
  const int64_t tiles = (a.M + G4_ROWS - 1) / G4_ROWS * active_y;
  a.splits = 1;
  while (a.splits < 8 && tiles * a.splits < 2 * num_sms && chunks >= 4 * a.splits) a.splits *= 2;
  if (const char* v = getenv("G4_SPLITS")) a.splits = atoi(v);
  if (NT == 1) return launch_mma_nt<1>(a, grid_y, kSmemG4, s);
  if (NT == 2) return launch_mma_nt<2>(a, grid_y, kSmemG4 + 4, s);
  return launch_mma_nt<4>(a, grid_y, kSmemG4 + 8, s);
}

}  // namespace

cudaError_t launch_matvec_g4(const G4Weights& w, const uint8_t* Xq, float* Y, int64_t M, int64_t K, int64_t N,
                             int num_sms, cudaStream_t s) {
  const char* tv = getenv("G4_MIN");
  if (N >= (tv ? atoi(tv) : 3)) {
    const int NT = N > 16 ? 4 : N > 8 ? 2 : 1;
    const G4Args a{w, Xq, Y, nullptr, 0, 1, false, false, M, N, static_cast<int>(K / 32), 1, nullptr};
    const int64_t tok = (N + NT * 8 - 1) / (NT * 8);
    return launch_rows(a, static_cast<unsigned>(tok), tok, NT, num_sms, s);
  }
  return launch_simple<false>(w, nullptr, 0, 1, false, Xq, Y, M, K, N, nullptr, s);
}

cudaError_t launch_moe_matvec_g4(const G4Weights& w, int n_experts, const int32_t* ids, int top_k, bool x_per_slot,
                                 const uint8_t* Xq, float* Y, int64_t M, int64_t K, int64_t T, int* err, int num_sms,
                                 cudaStream_t s) {
  const int64_t pairs = T * top_k;
  if (T > 1) {
    const bool by_pair = pairs <= n_experts;
    const G4Args a{w, Xq, Y, ids, n_experts, top_k, x_per_slot, by_pair, M, pairs, static_cast<int>(K / 32), 1, err};
    const int64_t y = by_pair ? pairs : n_experts;
    const int64_t each = pairs / n_experts;
    return launch_rows(a, static_cast<unsigned>(y), y, each > 16 ? 4 : each > 4 ? 2 : 1, num_sms, s);
  }
  return launch_simple<true>(w, ids, n_experts, top_k, x_per_slot, Xq, Y, M, K, T * top_k, err, s);
}

}  // namespace kq
