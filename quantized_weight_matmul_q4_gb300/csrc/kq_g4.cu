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
#include <atomic>

#include "kq_decode.h"
#include "kq_types.cuh"

namespace kq {
namespace {

constexpr unsigned FULL_MASK = 0xffffffffu;

struct G4Args {
  G4Weights w;
  const uint8_t* Xq;
  float* Y;
  const int32_t* ids;   // null: one matrix, rows 0..rows-1 of Xq
  int n_experts, top_k;
  bool x_per_slot;
  bool eager;           // nearly every expert has pairs: its weights are asked for before they are known
  int64_t M;
  int64_t rows;         // activation rows, or (token, slot) pairs
  int blocks;           // 32-element blocks per row
  int splits;           // CTAs of a cluster, over K
  int parts;            // clusters that share an expert's rows
  int* err;
};

__device__ __forceinline__ float scale_f32(bool fp16, uint16_t bits) {
  return fp16 ? __half2float(__ushort_as_half(bits)) : __uint_as_float(static_cast<uint32_t>(bits) << 16);
}

// ---------------------------------------------------------------------------
// One activation row: weight stream with dp4a
// ---------------------------------------------------------------------------
// The CTA unpacks the activation row once into shared memory: per 32-element block
// the even codes and the odd codes (16 bytes each, as the weights' low and high
// nibbles pair up), the scale and the sum of the codes. Then its warps stream
// weights: 2^lanes_log2 lanes share a row, each taking every 2^lanes_log2-th 16-byte
// block of it, U rows at a time, with the next four 16-byte loads of a lane in
// flight while it works on the last four. A block costs a lane some 68 instructions
// (counted on 152064 x 3584): 20 to unpack and multiply, the others read the activations from
// shared memory, convert and apply the scales, and make addresses and bounds. Unpacking costs less
// with dp4a than in the tensor-core form below, and without tiles no row is idle.
//
// Bound by HBM for large matrices (152064 x 3584: 45.5 us, 281 MB, 6.2 TB/s = 0.91 of the
// measured copy; issue slots 67 % busy) and by the launch and the first loads' latency for
// small ones (4096 x 4096: 3.3 us, launch included;
// eight experts' 1536 x 2048: 5.5 us, 2.4 TB/s).
constexpr int G4_DP_WARPS = 8;
constexpr int G4_DP_CTAS = 3;   // per SM

template <int NX, int U, bool ZEROS>
__global__ void __launch_bounds__(G4_DP_WARPS * 32, G4_DP_CTAS) g4_dp_kernel(G4Args a, int lanes_log2) {
  extern __shared__ __align__(16) uint8_t smem_raw[];
  uint4* xe = reinterpret_cast<uint4*>(smem_raw);       // [NX][blocks]
  uint4* xo = xe + NX * a.blocks;
  float2* xs = reinterpret_cast<float2*>(xo + NX * a.blocks);   // scale, sum (as an integer)
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  constexpr int JU = 4 / U;
  const int L = 1 << lanes_log2, l = lane & (L - 1), sub = lane >> lanes_log2, per = 32 >> lanes_log2;
  const bool fp16 = a.w.scale_dtype == KQ_F16;

  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  // One matrix: its first weights are on their way before the previous kernel's end.
  if (a.ids) asm volatile("griddepcontrol.wait;" ::: "memory");
  int64_t expert = 0;
  if (a.ids) {
    expert = a.ids[blockIdx.y];
    if (expert < 0 || expert >= a.n_experts) {
      if (tid == 0 && blockIdx.x == 0) report_error(a.err, ERR_EXPERT_ID);
      for (int64_t m = static_cast<int64_t>(blockIdx.x) * blockDim.x + tid; m < a.M; m += static_cast<int64_t>(gridDim.x) * blockDim.x)
        a.Y[blockIdx.y * a.M + m] = 0.f;
      return;
    }
  }
  const uint4* codes = reinterpret_cast<const uint4*>(a.w.codes) + expert * a.M * a.blocks + l;
  const uint16_t* scales = static_cast<const uint16_t*>(a.w.scales) + expert * a.M * a.w.groups;
  const uint8_t* zeros = a.w.zeros + expert * a.M * a.w.groups;
  const int64_t tiles = (a.M + per * U - 1) / (per * U);
  const int steps = (a.blocks + L * JU - 1) / (L * JU);   // of JU blocks per row
  const int64_t first = static_cast<int64_t>(blockIdx.x) * G4_DP_WARPS + warp;
  const int64_t stride = static_cast<int64_t>(gridDim.x) * G4_DP_WARPS;
  // This lane group's first row of a tile. The last tile is moved back to be whole
  // (U > 1 needs M >= per * U); a row computed twice gets the same value twice.
  auto row_of = [&](int64_t tile) {
    return min(min(tile * (per * U), max(a.M - per * U, static_cast<int64_t>(0))) + sub, a.M - 1);
  };
  const int64_t u_codes = static_cast<int64_t>(per) * a.blocks, u_scales = per * a.w.groups;

  uint4 wn[U][JU];
  uint16_t sn[U][JU];
  uint8_t zn[U][JU] = {};   // apart: nothing here waits for a load
  auto fetch = [&](int64_t row, int step) {
    const uint4* pc = codes + row * a.blocks;
    const int64_t ps = row * a.w.groups;
#pragma unroll
    for (int j = 0; j < JU; ++j) {
      const int b = (step * JU + j) * L;
      const bool in = b + l < a.blocks;
      const int64_t gr = ps + ((b + l) >> a.w.group_shift);
#pragma unroll
      for (int u = 0; u < U; ++u) {
        wn[u][j] = make_uint4(0, 0, 0, 0);
        sn[u][j] = 0;
        if (in) {
          wn[u][j] = __ldcs(pc + b + u * u_codes);
          sn[u][j] = __ldg(scales + gr + u * u_scales);
          if (ZEROS) zn[u][j] = __ldg(zeros + gr + u * u_scales);
        }
      }
    }
  };
  int64_t row = row_of(first);
  if (first < tiles) fetch(row, 0);

  if (!a.ids) asm volatile("griddepcontrol.wait;" ::: "memory");
  // A thread unpacks a block. (Ordinary loads: the previous kernel may have written it after this one
  // began, which the read-only path does not allow.)
  const int64_t xrow = a.ids ? (a.x_per_slot ? blockIdx.y : blockIdx.y / a.top_k) : 0;
  for (int i = tid; i < NX * a.blocks; i += blockDim.x) {
    const uint32_t* xb = reinterpret_cast<const uint32_t*>(a.Xq + (xrow * a.blocks + i) * Q8_1_BYTES);
    uint32_t e[4], o[4];
    int s = 0;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const uint32_t x0 = xb[1 + 2 * k], x1 = xb[2 + 2 * k];
      e[k] = __byte_perm(x0, x1, 0x6420);
      o[k] = __byte_perm(x0, x1, 0x7531);
      s = __dp4a(static_cast<int>(x0), 0x01010101, s);
      s = __dp4a(static_cast<int>(x1), 0x01010101, s);
    }
    xe[i] = make_uint4(e[0], e[1], e[2], e[3]);
    xo[i] = make_uint4(o[0], o[1], o[2], o[3]);
    xs[i] = make_float2(__low2float(bits_half2(xb[0])), __int_as_float(s));
  }
  __syncthreads();

  for (int64_t tile = first; tile < tiles; tile += stride) {
    const int64_t m = row;
    float acc[U][NX] = {};
    for (int step = 0; step < steps; ++step) {
      uint4 w[U][JU];
      uint16_t sc[U][JU];
      uint8_t zp[U][JU];
#pragma unroll
      for (int u = 0; u < U; ++u)
#pragma unroll
        for (int j = 0; j < JU; ++j) {
          w[u][j] = wn[u][j];
          sc[u][j] = sn[u][j];
          zp[u][j] = ZEROS ? zn[u][j] : 8;
        }
      if (step + 1 < steps) {
        fetch(row, step + 1);
      } else if (tile + stride < tiles) {
        row = row_of(tile + stride);
        fetch(row, 0);
      }
#pragma unroll
      for (int j = 0; j < JU; ++j) {
        // A block past the row's end: its weights and scale are zero, any x will do.
        const int b = min((step * JU + j) * L + l, a.blocks - 1);
#pragma unroll
        for (int n = 0; n < NX; ++n) {
          const uint4 e = xe[n * a.blocks + b], o = xo[n * a.blocks + b];
          const float2 ds = xs[n * a.blocks + b];
          const int sum = __float_as_int(ds.y);
#pragma unroll
          for (int u = 0; u < U; ++u) {
            const uint4 c = w[u][j];
            int dot = dp4a_us(c.x & 0x0f0f0f0fu, static_cast<int>(e.x), 0);
            int dot2 = dp4a_us((c.x >> 4) & 0x0f0f0f0fu, static_cast<int>(o.x), 0);
            dot = dp4a_us(c.y & 0x0f0f0f0fu, static_cast<int>(e.y), dot);
            dot2 = dp4a_us((c.y >> 4) & 0x0f0f0f0fu, static_cast<int>(o.y), dot2);
            dot = dp4a_us(c.z & 0x0f0f0f0fu, static_cast<int>(e.z), dot);
            dot2 = dp4a_us((c.z >> 4) & 0x0f0f0f0fu, static_cast<int>(o.z), dot2);
            dot = dp4a_us(c.w & 0x0f0f0f0fu, static_cast<int>(e.w), dot);
            dot2 = dp4a_us((c.w >> 4) & 0x0f0f0f0fu, static_cast<int>(o.w), dot2);
            const int t = dot + dot2 - static_cast<int>(zp[u][j]) * sum;
            acc[u][n] = fmaf(scale_f32(fp16, sc[u][j]) * ds.x, static_cast<float>(t), acc[u][n]);
          }
        }
      }
    }
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
      for (int n = 0; n < NX; ++n) {
        float v = acc[u][n];
        for (int o = L >> 1; o > 0; o >>= 1) v += __shfl_xor_sync(FULL_MASK, v, o);
        if (l == 0) a.Y[(static_cast<int64_t>(blockIdx.y) + n) * a.M + m + u * per] = v;
      }
  }
}

// ---------------------------------------------------------------------------
// Several activation rows: tensor-core form
// ---------------------------------------------------------------------------
// Weights read once for up to 8 * NT activation rows, with m16n8k16 fp16 MMAs
// whose operands are small integers, so that every block's dot product is exact
// in the fp32 accumulator.
//
// Weight codes become fp16 by one logic operation for two codes: a low nibble of a
// 16-bit field or-ed into the mantissa of 1024 is 1024 + c, the next nibble in that of
// 64 is 64 + c. The even k of a block go through one MMA, the odd k through a second.
// Without zero points the sum is Sum (c - 8) q + 1032 Sum_even q + 72 Sum_odd q, an
// integer below 32 * 1039 * 128 < 2^24; the excess depends on the activation row alone
// and is taken off by starting the accumulator at its negative. With zero points
// 1024 + z and 64 + z are subtracted first (packed fp16, exact), or z Sum q from the sum.
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
//
// The legacy MMA form and not tensor memory, since every block's sums are multiplied
// with two scales: here they are in registers already, from tensor memory the
// whole accumulator would be read back for every 32 k.
//
// Bound by latency, not by HBM nor by a pipe: some 270 instructions per warp and chunk (8 rows,
// groups of 128 and longer) up to 620 (16 rows, groups of 32 with zero points) at 46 to 59 % of the
// issue slots. 16 warps to an SM at most (128 registers a thread) wait on their own chains (copies,
// ldmatrix, unpacking, two MMAs, scales) and on the barriers around the making of fragments; taking one
// stage out (copies, unpacking, scales, fmas, fragments) took 2 to 12 % off an earlier state. A line
// through the times over K, launch included, begins at 4.0 us (4096 weight rows, 8 activation
// rows, K split in eight) or 5.7 (14336, 16 rows) and rises by 0.6 or 3.1 us (3.6 with
// groups of 32 and zero points) per 1024 of K; 4096 x 128, 8 rows: 2.3 us.
// 4096 x 4096, 8 rows: 6.4 us; 14336 x 4096, 16 rows, groups of 32 with zero
// points: 20.0 us (1.8 TB/s); 128 experts' 2048 x 768, 512 (token, slot) rows, the same
// groups: 40.7 us (3.0 TB/s). Copying by TMA instead of cp.async was slower (the latter
// 46 -> 49.5 us), and so was a CTA that goes on to the next tile of its expert's rows
// with its copies running ahead (43.2 us with one tile, 43.6 with two, 57.2 with four).
constexpr int G4_CHUNK = 4;        // 32-element blocks per chunk
// Chunks of weights in flight per warp: as many as leave room for four CTAs on an SM.
__host__ __device__ constexpr int g4_stages(bool FINE, bool ZEROS) { return FINE || ZEROS ? 3 : 4; }
constexpr int G4_ROWS = 128;       // weight rows of a CTA, 32 per warp
// Fragments (of one block and 8 activation rows) per panel.
__host__ __device__ constexpr int g4_panel(int NT) { return NT == 4 ? 32 : 16; }
// Groups whose scales are fetched together: a 32-byte sector of a row, or, where a row's scales or
// zero points begin between two 4-byte words, half of one (the words that hold them).
constexpr int G4_SPAN = 16;
constexpr int G4_SPAN_LOG2 = 4;
constexpr int G4_MAX_SPLITS = 16;
constexpr int G4_LIST = 192;       // rows of one expert collected at a time (at least 128)

struct alignas(16) G4Frag {    // of one block and 8 activation rows
  uint4 b[32];     // per lane: even k (two registers), odd k (two registers)
  float4 init[4];  // per t: start of the accumulators of rows 2t, 2t + 1, 2t, 2t + 1 (without zero points)
  float4 d[4];     // per t: scales of rows 2t, 2t + 1, sums of their codes
  float4 pad[1];   // 656 bytes: eight threads that write eight blocks' fragments meet different banks
};
template <bool FINE, bool ZEROS>
struct alignas(16) G4Warp {    // a warp's own
  uint8_t w[g4_stages(FINE, ZEROS)][32][G4_CHUNK * 16];
  uint8_t raw[2][32][G4_SPAN * (ZEROS ? 3 : 2)];   // as in memory: scales, from byte 2 * G4_SPAN zero points
  // Of a chunk's blocks (FINE): the scale, and -(1024 + zero point) as an fp16 pair.
  float2 scale[FINE ? G4_CHUNK : 1][FINE ? 32 : 1];
};
template <int NT, bool FINE, bool ZEROS>
struct G4Smem {
  G4Warp<FINE, ZEROS> warp[4];
  G4Frag frag[g4_panel(NT)];
  // The next panel's activations as in memory, row after row, from the 16-byte boundary that each begins behind.
  alignas(16) uint8_t x[g4_panel(NT) * 8 * Q8_1_BYTES + NT * 8 * 16];
  const uint8_t* xrow[NT * 8];                    // activation rows of this pass
  unsigned counts[4];                             // of a warp's pairs
  int list[G4_LIST];                              // the expert's pairs
};
// cp.async and ldmatrix take 16-byte rows at 16-byte boundaries.
static_assert(sizeof(G4Warp<true, true>) % 16 == 0 && sizeof(G4Warp<false, false>) % 16 == 0 && sizeof(G4Frag) == 656 && G4_SPAN % 16 == 0);

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
#pragma unroll 1
    for (int o = 0; o < bytes; o += 16) cp_async16(dst + o, src + o, 16);
  } else if (align % 8 == 0) {
#pragma unroll 1
    for (int o = 0; o < bytes; o += 8) cp_async8(dst + o, src + o);
  } else {
#pragma unroll 1
    for (int o = 0; o < bytes; o += 4) cp_async4(dst + o, src + o, 4);
  }
}
// The `bytes` from `src` on, as the WORDS aligned words that hold them (zeros past the end). The bytes
// before src in its word have to be readable; `any` is an address for copies of nothing.
template <int WORDS>
__device__ __forceinline__ void cp_async_words(uint32_t dst, const void* src, int bytes, const void* any) {
  const int off = static_cast<int>(reinterpret_cast<uintptr_t>(src) & 3);
  const uint8_t* p = static_cast<const uint8_t*>(src) - off;
#pragma unroll
  for (int w = 0; w < WORDS; ++w) {
    const int n = min(max(bytes + off - 4 * w, 0), 4);
    cp_async4(dst + 4 * w, n > 0 ? p + 4 * w : any, n);
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
// (v & mask) | magic in one operation.
template <uint32_t MASK, uint32_t MAGIC>
__device__ __forceinline__ uint32_t codes_f16(uint32_t v) {
  uint32_t r;
  asm("lop3.b32 %0, %1, %2, %3, 0xea;" : "=r"(r) : "r"(v), "r"(MASK), "r"(MAGIC));
  return r;
}
__device__ __forceinline__ uint32_t add_f16x2(uint32_t a, uint32_t b) { return half2_bits(__hadd2(bits_half2(a), bits_half2(b))); }
constexpr uint32_t H2_M1152 = 0xe480e480u, H2_960 = 0x63806380u;   // fp16 pairs

// Byte i of v.
__device__ __forceinline__ float byte_f32(uint32_t v, int i) {
  return __uint_as_float(__byte_perm(v, 0x4b000000u, 0x7440 + i)) - 8388608.f;
}
// -(1024 + byte i of v) as an fp16 pair.
__device__ __forceinline__ uint32_t zero_f16x2(uint32_t v, int i) { return __byte_perm(v, 0xe4e4e4e4u, 0x4040 + 0x0101 * i); }

// FINE: a group is shorter than a chunk, so every block has its own scale; else
// one scale serves a chunk. ZEROS: zero points are given.
template <int NT, bool FINE, bool ZEROS>
__global__ void __launch_bounds__(128, NT == 4 ? 3 : 4) g4_mma_kernel(G4Args a) {
  extern __shared__ __align__(16) uint8_t smem_raw[];
  G4Smem<NT, FINE, ZEROS>& sm = *reinterpret_cast<G4Smem<NT, FINE, ZEROS>*>(smem_raw);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  G4Warp<FINE, ZEROS>& my = sm.warp[warp];
  const int g = lane >> 2, t = lane & 3;
  constexpr int TOK = NT * 8;
  constexpr int G4_STAGES = g4_stages(FINE, ZEROS);
  constexpr int PANEL = g4_panel(NT) / NT / G4_CHUNK;   // chunks
  // Zero points times the sum of the activations' codes are taken from the blocks' sums, exactly as well, where
  // that is cheaper than subtracting them from the codes: with eight rows and a zero point to
  // a block (128 experts of 2048 x 768, 64 tokens: 39.9 us against 42.6; 16 rows, 14336 x 4096:
  // 20.4 against 19.4; groups of 128, 8 rows: 13.7 against 13.3).
  constexpr bool LATE = ZEROS && FINE && NT == 1;
  static_assert(NT == 4 || sizeof(sm) <= 228 * 1024 / 4 - 1024);   // four CTAs on an SM
  static_assert(sizeof(sm.frag) >= TOK * G4_ROWS * sizeof(float));   // the sums take the fragments' place
  const int rank = a.splits > 1 ? static_cast<int>(cluster_ctarank()) : 0;
  const int64_t m0 = static_cast<int64_t>(blockIdx.x / a.splits) * G4_ROWS;
  const int rows = static_cast<int>(min(a.M - m0, static_cast<int64_t>(G4_ROWS)));   // of this tile

  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  if (!a.eager) asm volatile("griddepcontrol.wait;" ::: "memory");
  const int part = a.ids ? static_cast<int>(blockIdx.y) % a.parts : 0;
  const int expert = a.ids ? static_cast<int>(blockIdx.y) / a.parts : 0;
  int64_t scan = 0;     // next pair to look at
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
  const uint32_t wdst = smem_u32(&my.w[0][g][(t ^ ((g >> 1) & 3)) << 4]);
  const int64_t srow = (row0 + min(tid, rows - 1)) * a.w.groups;
  // Every row's scales and zero points begin on a 4-byte word; else those of row `lane`, and those of
  // the rows g + 8 i alike, this many behind one (in the words copied).
  const bool wide = a.w.groups % 2 == 0 && (!ZEROS || a.w.groups % 4 == 0);
  const int span_log2 = wide ? G4_SPAN_LOG2 : G4_SPAN_LOG2 - 1;
  const int off = static_cast<int>(FINE ? srow : (row0 + warp * 32 + g) * a.w.groups) & 3;
  // ldmatrix: lane l gives the address of row l % 8 of matrix l / 8: rows 0-7, 8-15 of
  // the first and then of the second 16-row tile.
  uint32_t arow[G4_CHUNK];   // of each block of a chunk
#pragma unroll
  for (int b = 0; b < G4_CHUNK; ++b) arow[b] = smem_u32(&my.w[0][lane][(b ^ ((lane >> 1) & 3)) << 4]);
  auto scale_f = [&](uint16_t bits) {
    return a.w.scale_dtype == KQ_F16 ? __half2float(__ushort_as_half(bits)) : __uint_as_float(static_cast<uint32_t>(bits) << 16);
  };

  // LATE: the zero point; else -(1024 + it) as an fp16 pair.
  auto zero = [](uint32_t v, int i) {
    return LATE ? byte_f32(v, i) : ZEROS ? __uint_as_float(zero_f16x2(v, i)) : 0.f;
  };

  const uint8_t* wsrc[4];
  int span_chunk;      // the next chunk whose scales are in a new span
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
    // The scales of the next span of groups with the first chunk that needs them; the
    // span before the last is out of use by then (a span is G4_STAGES - 1 chunks at least).
    if (c == span_chunk) {
      const int span = c * G4_CHUNK >> a.w.group_shift >> span_log2;
      span_chunk = static_cast<int>(min((static_cast<int64_t>(span + 1) << span_log2 << a.w.group_shift) / G4_CHUNK, static_cast<int64_t>(chunks)));
      const int n = static_cast<int>(min(a.w.groups - (static_cast<int64_t>(span) << span_log2), static_cast<int64_t>(1) << span_log2));
      const int64_t at = srow + (static_cast<int64_t>(span) << span_log2);
      uint8_t* raw = my.raw[span & 1][lane];
      const uint16_t* ss = static_cast<const uint16_t*>(a.w.scales) + at;
      if (wide) {
#pragma unroll 1
        for (int i = n; i < G4_SPAN; ++i) {   // blocks past K get scale 0
          reinterpret_cast<uint16_t*>(raw)[i] = 0;
          if (ZEROS) raw[2 * G4_SPAN + i] = 0;
        }
        cp_async_row(smem_u32(raw), reinterpret_cast<const uint8_t*>(ss), 2 * n, static_cast<int>(2 * a.w.groups & 31));
        if (ZEROS) cp_async_row(smem_u32(raw) + 2 * G4_SPAN, a.w.zeros + at, n, static_cast<int>(a.w.groups & 31));
      } else {
        cp_async_words<G4_SPAN / 4 + 1>(smem_u32(raw), ss, 2 * n, a.w.codes);
        if (ZEROS) cp_async_words<G4_SPAN / 8 + 1>(smem_u32(raw) + 2 * G4_SPAN, a.w.zeros + at, n, a.w.codes);
      }
    }
  };
  auto begin = [&] {   // of a pass over K: the first copies
#pragma unroll
    for (int i = 0; i < 4; ++i)
      wsrc[i] = a.w.codes + (row0 + min(warp * 32 + g + 8 * i, rows - 1)) * row_bytes + t * 16 + static_cast<int64_t>(c_begin) * 64;
    span_chunk = c_begin;
#pragma unroll 1
    for (int i = 0; i < G4_STAGES - 1; ++i) {
      if (c_begin + i < c_end) fill(c_begin + i, i);
      cp_async_commit();
    }
  };
  // Weights that are surely needed, or nearly so, are on their way before the previous
  // kernel's end.
  bool begun = a.eager;
  if (a.eager) {
    begin();
    asm volatile("griddepcontrol.wait;" ::: "memory");
  }
  // Invalid ids belong to no expert: expert 0's CTAs write their zeros.
  if (a.ids && blockIdx.y == 0 && rank == 0) {
    for (int64_t p = tid; p < a.rows; p += 128) {
      const int e = a.ids[p];
      if (e < 0 || e >= a.n_experts) {
        if (blockIdx.x == 0) report_error(a.err, ERR_EXPERT_ID);
        for (int m = 0; m < rows; ++m) a.Y[p * a.M + m0 + m] = 0.f;
      }
    }
  }

  for (;;) {
    int have;
    if (a.ids) {
      // Collect this expert's pairs in their order, which all CTAs of the expert share: 512 at a time;
      // where so many are this expert's that the list would overflow, 128 at a time.
      have = 0;
      while (scan < a.rows) {
        unsigned mine[4], counts = 0;   // a byte for each 128
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const int64_t p = scan + tid + 128 * k;
          mine[k] = __ballot_sync(FULL_MASK, p < a.rows && a.ids[p] == expert);
          counts |= static_cast<unsigned>(__popc(mine[k])) << (8 * k);
        }
        __syncthreads();   // the last counts, or the last pass, are done with
        if (lane == 0) sm.counts[warp] = counts;
        __syncthreads();
        unsigned before = 0, all = 0;
#pragma unroll
        for (int w = 0; w < 4; ++w) {
          if (w < warp) before += sm.counts[w];
          all += sm.counts[w];
        }
        const int found = static_cast<int>((all & 255) + (all >> 8 & 255) + (all >> 16 & 255) + (all >> 24));
        const bool fits = have + found <= G4_LIST;
        if (!fits && have > 0) break;   // those are enough for now: these again next time
        int at = have;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          if (k > 0 && !fits) break;
          if (mine[k] >> lane & 1)
            sm.list[at + (before >> (8 * k) & 255) + __popc(mine[k] & ((1u << lane) - 1))] = static_cast<int>(scan + tid + 128 * k);
          at += static_cast<int>(all >> (8 * k) & 255);
        }
        have = at;
        scan += fits ? 512 : 128;
        if (!fits && have > 0) break;
      }
      __syncthreads();
      if (have == 0) {
        cp_async_wait<0>();
        return;
      }
    } else {
      have = static_cast<int>(min(a.rows - static_cast<int64_t>(blockIdx.y) * TOK, static_cast<int64_t>(TOK)));
    }
    for (int n0 = part * TOK; n0 < have; n0 += a.parts * TOK) {
      const int nn = min(TOK, have - n0);
      if (tid < TOK) {
        const uint8_t* p = nullptr;
        if (tid < nn) {
          int64_t r = static_cast<int64_t>(blockIdx.y) * TOK + tid;
          if (a.ids) {
            const int pair = sm.list[n0 + tid];
            r = a.x_per_slot ? pair : pair / a.top_k;
          }
          p = a.Xq + r * xbytes;
        }
        sm.xrow[tid] = p;
      }
      // The activations of the panel at chunk c, in 16-byte pieces from the boundary that the row
      // begins at or behind (`even`: at). Piece tid + 128 k is `xat` bytes behind the panel's first.
      constexpr int PIECES = PANEL * G4_CHUNK * Q8_1_BYTES / 16;   // of a row, and one more where rows begin between boundaries
      constexpr int XP = (TOK * (PIECES + 1) + 127) / 128;
      const int pieces = even ? PIECES : PIECES + 1;
      __syncthreads();   // sm.xrow
      const uint8_t* xsrc[XP];
      int xat[XP];
#pragma unroll
      for (int k = 0; k < XP; ++k) {
        const int i = tid + 128 * k, r = even ? i / PIECES : i / (PIECES + 1);
        const uint8_t* p = r < TOK ? sm.xrow[r] : nullptr;
        const int o = (i - r * pieces) * 16 - static_cast<int>(reinterpret_cast<uintptr_t>(p) & 15);
        xat[k] = p ? o : 1 << 28;
        xsrc[k] = p ? p + o + static_cast<int64_t>(c_begin) * (G4_CHUNK * Q8_1_BYTES) : a.Xq;
      }
      auto load = [&](int c) {
        const int left = static_cast<int>(min(xbytes - static_cast<int64_t>(c) * (G4_CHUNK * Q8_1_BYTES), static_cast<int64_t>(1) << 24));
#pragma unroll
        for (int k = 0; k < XP; ++k) {
          const int i = tid + 128 * k;
          if (i >= TOK * pieces) break;
          const int n = min(max(left - xat[k], 0), 16);
          cp_async16(smem_u32(sm.x) + i * 16, n > 0 ? xsrc[k] : a.Xq, n);
          xsrc[k] += PIECES * 16;
        }
      };
      // A thread makes one (activation row, block) of a panel's fragments, or two.
      constexpr int MINE = g4_panel(NT) * 8 / 128;
      int xbyte[MINE];   // its first byte in sm.x
#pragma unroll
      for (int k = 0; k < MINE; ++k) {
        const int xn = (tid + 128 * k) / (PANEL * G4_CHUNK), blk = tid % (PANEL * G4_CHUNK);
        xbyte[k] = xn * (pieces * 16) + blk * Q8_1_BYTES + static_cast<int>(reinterpret_cast<uintptr_t>(sm.xrow[xn]) & 15);
      }
      auto make = [&](int k) {
        constexpr int PB = PANEL * G4_CHUNK;   // blocks
        const int xn = (tid + 128 * k) / PB, blk = tid % PB;
        const uint32_t* px = reinterpret_cast<const uint32_t*>(sm.x + xbyte[k]);
        G4Frag& f = sm.frag[blk * NT + xn / 8];
        const int fg = xn & 7;
        int se = 0, so = 0;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const uint32_t x0 = px[1 + 2 * j], x1 = px[2 + 2 * j];
          const uint32_t ev = __byte_perm(x0, x1, 0x6240), od = __byte_perm(x0, x1, 0x7351);
          if (!ZEROS || LATE) {
            se = __dp4a(static_cast<int>(ev), 0x01010101, se);
            so = __dp4a(static_cast<int>(od), 0x01010101, so);
          }
          const uint32_t ue = ev ^ 0x80808080u, uo = od ^ 0x80808080u;    // codes + 128, then 1024 + that
          f.b[fg * 4 + j] = make_uint4(add_f16x2(__byte_perm(ue, 0x64646464u, 0x4140), H2_M1152),
                                       add_f16x2(__byte_perm(ue, 0x64646464u, 0x4342), H2_M1152),
                                       add_f16x2(__byte_perm(uo, 0x64646464u, 0x4140), H2_M1152),
                                       add_f16x2(__byte_perm(uo, 0x64646464u, 0x4342), H2_M1152));
        }
        if (!ZEROS || LATE) {
          float* c = reinterpret_cast<float*>(&f.init[fg >> 1]) + (fg & 1);
          c[0] = c[2] = static_cast<float>(LATE ? -(1024 * se + 64 * so) : -(1032 * se + 72 * so));
        }
        float* fd = reinterpret_cast<float*>(&f.d[fg >> 1]) + (fg & 1);
        fd[0] = __low2float(bits_half2(px[0]));
        if (LATE) fd[2] = static_cast<float>(se + so);
      };

      float acc[2][NT][4] = {};
      if (!begun) begin();
      begun = false;
      load(c_begin);
      cp_async_commit();
      int slot = 0;   // of chunk c
      for (int c = c_begin, p_begin = c_begin, p_end = c_begin; c < c_end; ++c) {
        if (c == p_end) {
          p_begin = c;
          p_end = min(c + PANEL, c_end);
          // The panel's activations: their copies were followed by those of the chunks of
          // the panel before but one.
          if (c == c_begin) cp_async_wait<0>(); else cp_async_wait<PANEL - 1>();
          __syncthreads();   // everyone's; the last panel is used up
#pragma unroll
          for (int k = 0; k < MINE; ++k) make(k);
          __syncthreads();
          if (p_end < c_end) load(p_end);   // with this chunk's group
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
        float s[4];       // scales of rows g, g + 8, g + 16, g + 24
        uint32_t z[4];    // their -(1024 + zero point), fp16 pairs
        if (FINE) {
          // Lane: row; the four blocks' scales converted once. A chunk has four groups or two.
          const int gr = c * G4_CHUNK >> a.w.group_shift;
          const uint8_t* raw = my.raw[(gr >> span_log2) & 1][lane];
          const int at = gr & ((1 << span_log2) - 1);
          const uint16_t* rs = reinterpret_cast<const uint16_t*>(raw) + at;
          const uint8_t* rz = raw + 2 * G4_SPAN + at;
          uint2 sb;
          uint32_t zb;
          if (!wide) {
            rs += off & 1;
            rz += off;
            const int b1 = 1 >> a.w.group_shift, b2 = 2 >> a.w.group_shift, b3 = 3 >> a.w.group_shift;
            sb = make_uint2(rs[0] | static_cast<uint32_t>(rs[b1]) << 16, rs[b2] | static_cast<uint32_t>(rs[b3]) << 16);
            zb = ZEROS ? rz[0] | rz[b1] << 8 | rz[b2] << 16 | static_cast<uint32_t>(rz[b3]) << 24 : 0;
          } else if (a.w.group_shift == 0) {
            sb = *reinterpret_cast<const uint2*>(rs);
            zb = ZEROS ? *reinterpret_cast<const uint32_t*>(rz) : 0;
          } else {
            const uint32_t two = *reinterpret_cast<const uint32_t*>(rs), zz = ZEROS ? *reinterpret_cast<const uint16_t*>(rz) : 0;
            sb = make_uint2(__byte_perm(two, 0, 0x1010), __byte_perm(two, 0, 0x3232));
            zb = __byte_perm(zz, 0, 0x1100);
          }
          my.scale[0][lane] = make_float2(scale_f(sb.x & 0xffff), zero(zb, 0));
          my.scale[1][lane] = make_float2(scale_f(sb.x >> 16), zero(zb, 1));
          my.scale[2][lane] = make_float2(scale_f(sb.y & 0xffff), zero(zb, 2));
          my.scale[3][lane] = make_float2(scale_f(sb.y >> 16), zero(zb, 3));
          __syncwarp();
        } else {
          const int gr = (c * G4_CHUNK) >> a.w.group_shift;
          const int at = gr & ((1 << span_log2) - 1);
          const uint8_t* raw = my.raw[(gr >> span_log2) & 1][g] + 2 * at + (wide ? 0 : 2 * (off & 1));
          const int to_zero = 2 * G4_SPAN - at + (wide ? 0 : off - 2 * (off & 1));
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const uint8_t* r = raw + i * (8 * sizeof(my.raw[0][0]));
            s[i] = scale_f(*reinterpret_cast<const uint16_t*>(r));
            if (ZEROS) z[i] = __float_as_uint(zero(r[to_zero], 0));
          }
        }
        float part[2][NT][4];   // of this chunk, before the chunk's scale (not FINE)
#pragma unroll
        for (int b = 0; b < G4_CHUNK; ++b) {
          const uint32_t (&w)[4] = wc[b];
          if (FINE) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const float2 v = my.scale[b][8 * i + g];
              s[i] = v.x;
              z[i] = __float_as_uint(v.y);
            }
          }
          uint32_t L[2][4], U[2][4];
#pragma unroll
          for (int m = 0; m < 2; ++m)
#pragma unroll
            for (int h = 0; h < 2; ++h) {   // rows g and g + 8 of the 16
              const uint32_t v = w[2 * m + h], v8 = v >> 8;
              L[m][h] = codes_f16<0x000f000fu, 0x64006400u>(v);
              L[m][h + 2] = codes_f16<0x000f000fu, 0x64006400u>(v8);
              U[m][h] = codes_f16<0x00f000f0u, 0x54005400u>(v);
              U[m][h + 2] = codes_f16<0x00f000f0u, 0x54005400u>(v8);
              if (ZEROS && !LATE) {
                const uint32_t zl = z[2 * m + h], zu = add_f16x2(zl, H2_960);
                L[m][h] = add_f16x2(L[m][h], zl);
                L[m][h + 2] = add_f16x2(L[m][h + 2], zl);
                U[m][h] = add_f16x2(U[m][h], zu);
                U[m][h + 2] = add_f16x2(U[m][h + 2], zu);
              }
            }
#pragma unroll
          for (int n = 0; n < NT; ++n) {
            const G4Frag& f = pf[b * NT + n];
            const uint4 bf = f.b[lane];
            float4 c0 = make_float4(0.f, 0.f, 0.f, 0.f);
            if (!ZEROS || LATE) c0 = f.init[t];
            const float4 d = f.d[t];
#pragma unroll
            for (int m = 0; m < 2; ++m) {
              float r[4];
              mma16816(r, L[m], bf.x, bf.y, c0.x, c0.y, c0.z, c0.w);
              mma16816(r, U[m], bf.z, bf.w, r[0], r[1], r[2], r[3]);
#pragma unroll
              for (int k = 0; k < 4; ++k) {
                if (LATE) r[k] = fmaf(-__uint_as_float(z[2 * m + (k >> 1)]), k & 1 ? d.w : d.z, r[k]);
                const float v = r[k] * (k & 1 ? d.y : d.x);
                if (FINE) acc[m][n][k] = fmaf(v, s[2 * m + (k >> 1)], acc[m][n][k]);
                else part[m][n][k] = b == 0 ? v : fmaf(r[k], k & 1 ? d.y : d.x, part[m][n][k]);
              }
            }
          }
        }
        if (!FINE) {
#pragma unroll
          for (int m = 0; m < 2; ++m) {
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
              for (int k = 0; k < 4; ++k) acc[m][n][k] = fmaf(part[m][n][k], s[2 * m + (k >> 1)], acc[m][n][k]);
          }
        }
      }
      if (a.splits == 1) {
        // A warp's store writes whole sectors: eight weight rows (g) of four activation rows.
        const int64_t m = m0 + warp * 32 + g;
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            const int col = n * 8 + 2 * t + k;
            if (col >= nn) continue;
            float* y = a.Y + (a.ids ? sm.list[n0 + col] : static_cast<int64_t>(blockIdx.y) * TOK + col) * a.M + m;
#pragma unroll
            for (int i = 0; i < 4; ++i)
              if (m + 8 * i < a.M) y[8 * i] = acc[i >> 1][n][2 * (i & 1) + k];
          }
        if (n0 + a.parts * TOK < have) __syncthreads();   // before the next rows' fragments
        continue;
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
      cluster_sync();
      // Each rank adds up and writes its share of the tile's rows.
      const int sh = 31 - __clz(G4_ROWS / a.splits);
      for (int i = tid; i < nn << sh; i += 128) {
        const int n = i >> sh, m = (rank << sh) + (i & ((1 << sh) - 1));
        if (m >= rows) continue;
        float v = 0.f;
#pragma unroll 1
        for (int r0 = 0; r0 < a.splits; r0 += 8) {
          float part[8];   // all on their way before the first is added
#pragma unroll
          for (int r = 0; r < 8; ++r)
            part[r] = r0 + r < a.splits ? ld_cluster_f32(mapa_shared(red + n * G4_ROWS + m, r0 + r)) : 0.f;
#pragma unroll
          for (int r = 0; r < 8; ++r) v += part[r];
        }
        const int64_t out = a.ids ? sm.list[n0 + n] : static_cast<int64_t>(blockIdx.y) * TOK + n;
        a.Y[out * a.M + m0 + m] = v;
      }
      cluster_sync();   // the others have read this CTA's sums
    }
    if (!a.ids || scan >= a.rows) {
      cp_async_wait<0>();   // of a part without rows
      return;
    }
  }
}

// Raises a kernel's dynamic shared-memory limit to the maximum and lets it have clusters of sixteen,
// once per device: later calls only read a flag. 24 slots: 12 of the tensor-core form, 12 of the
// weight stream.
constexpr int G4_SLOTS = 24, G4_DEVICES = 64;
std::atomic<uint8_t> g_ready[G4_SLOTS][G4_DEVICES];
cudaError_t prepare(const void* kernel, int slot) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (slot < 0 || slot >= G4_SLOTS || dev < 0 || dev >= G4_DEVICES) return cudaErrorInvalidValue;
  if (g_ready[slot][dev].load(std::memory_order_acquire)) return cudaSuccess;
  e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, 227 * 1024);
  if (e == cudaSuccess && slot < 12) e = cudaFuncSetAttribute(kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
  if (e == cudaSuccess) g_ready[slot][dev].store(1, std::memory_order_release);
  return e;
}

constexpr size_t G4_DP_SMEM = 72 * 1024;   // the activation row that g4_dp_kernel may hold (three CTAs per SM)
size_t g4_dp_smem(int64_t NX, int64_t blocks) { return static_cast<size_t>(NX * blocks) * 40; }

template <int NX, int U>
cudaError_t launch_dp(const G4Args& a, unsigned grid_x, unsigned grid_y, int lanes_log2, int slot, cudaStream_t s) {
  auto k = a.w.zeros ? g4_dp_kernel<NX, U, true> : g4_dp_kernel<NX, U, false>;
  const size_t smem = g4_dp_smem(NX, a.blocks);
  if (smem > 48 * 1024) {
    const cudaError_t e = prepare(reinterpret_cast<const void*>(k), slot + (a.w.zeros ? 1 : 0));
    if (e != cudaSuccess) return e;
  }
  return launch_pdl(k, dim3(grid_x, grid_y), dim3(G4_DP_WARPS * 32), smem, s, a, lanes_log2);
}

// NX activation rows of one matrix (pairs == 0), or `pairs` (token, slot) pairs on their own.
template <int NX>
cudaError_t launch_stream(const G4Args& a, int64_t pairs, int num_sms, cudaStream_t s) {
  // Lanes per row: the most that leave at most an eighth of a row's lanes idle at its
  // end (else the fewest idle).
  int lanes_log2 = 5;
  int64_t best = INT64_MAX;
  for (int k = 5; k >= 3; --k) {
    const int64_t padded = (a.blocks + (1 << k) - 1) >> k << k;
    if (padded < best) {
      best = padded;
      lanes_log2 = k;
    }
    if (8 * best <= 9 * static_cast<int64_t>(a.blocks)) break;
  }
  const int per = 32 >> lanes_log2;
  const int64_t y = pairs ? pairs : 1;
  const int64_t row_warps = (a.M + per - 1) / per * y;   // warps at one row per lane group
  const int64_t slots = static_cast<int64_t>(num_sms) * G4_DP_CTAS * G4_DP_WARPS;
  const int64_t q = best >> lanes_log2;                  // blocks of a lane per row
  // Rows per lane: as many as fill its four loads, and four where the rows are many (of 4096
  // codes, one activation row: 4096 rows 3.3 us by one and 5.9 by four, 11008 5.8 and 6.3,
  // 14336 7.1 and 6.7, 28672 12.9 and 11.7, 152064 59 and 51).
  int U = q >= 4 ? 1 : q >= 2 ? 2 : 4;
  if (NX == 1 && 2 * row_warps >= 7 * slots) U = 4;
  if (a.M < per * U) U = 1;
  const int64_t tiles = (a.M + per * U - 1) / (per * U);
  const int64_t ctas = (tiles + G4_DP_WARPS - 1) / G4_DP_WARPS;
  // CTAs per pair: as many as run at once, or, where the pairs do not divide those well, as run in
  // two to four rounds: the first number of rounds that fills nine tenths of its places (384
  // experts of 2048 x 768, 240 pairs: 70.5 us in one round, 47.9 in two, 44.8 in four; 128
  // experts of 1536 x 2048, 128 pairs: 47.7 in one, 42.3 in two; 64 pairs, which fit: 22.6
  // and 25.0).
  int64_t most = 1;
  for (int64_t rounds = 1, best_used = 0; rounds <= 4; ++rounds) {
    const int64_t places = static_cast<int64_t>(num_sms) * G4_DP_CTAS * rounds, each = places / y;
    const int64_t used = 1000 * each * y / places;
    if (used <= best_used) continue;
    best_used = used;
    most = each;
    if (used >= 900) break;
  }
  const unsigned gx = static_cast<unsigned>(std::min(ctas, most)), gy = static_cast<unsigned>(y);
  const int slot = 12 + 6 * (NX - 1);
  if (U == 1) return launch_dp<NX, 1>(a, gx, gy, lanes_log2, slot, s);
  if (U == 2) return launch_dp<NX, 2>(a, gx, gy, lanes_log2, slot + 2, s);
  return launch_dp<NX, 4>(a, gx, gy, lanes_log2, slot + 4, s);
}

template <int NT, bool FINE, bool ZEROS>
cudaError_t launch_mma(const G4Args& a, unsigned grid_y, int num_sms, int slot, cudaStream_t s) {
  void (*k)(G4Args) = g4_mma_kernel<NT, FINE, ZEROS>;
  const cudaError_t e = prepare(reinterpret_cast<const void*>(k), slot);
  if (e != cudaSuccess) return e;
  const int64_t tiles = (a.M + G4_ROWS - 1) / G4_ROWS;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(tiles * a.splits), grid_y);
  cfg.blockDim = dim3(128);
  size_t smem = sizeof(G4Smem<NT, FINE, ZEROS>);
  if (a.splits > 1) {
    // Clusters are packed onto as few SMs as hold them (4096 x 4096, 8 rows, 256 CTAs: 7.5 us
    // against 6.6 spread). So ask for the shared memory that leaves an SM its even share
    // of the CTAs only, if that leaves a tenth of the places free: clusters need places
    // near one another. With one place to an SM, clusters of eight need more free (2048 x 4096,
    // 128 CTAs on 152 SMs: 9.5 us, as they do not all run at once; 5.6 with two places). (An SM has
    // 228 KB, each CTA's reservation 1 KB.)
    const int64_t ctas = tiles * a.splits * grid_y;
    int64_t share = (ctas * 10 + 9 * num_sms - 1) / (9 * num_sms);
    if (share == 1 && (a.splits == 16 || (a.splits == 8 && 4 * ctas > 3 * num_sms))) share = 2;
    if (share <= 4) smem = std::max<size_t>(smem, std::min<size_t>(227 * 1024, 228 * 1024 / share - 1024) / 16 * 16);
  }
  cfg.dynamicSmemBytes = smem;
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
cudaError_t launch_mma_nt(const G4Args& a, unsigned grid_y, int num_sms, int slot, cudaStream_t s) {
  const bool zeros = a.w.zeros != nullptr;
  if (a.w.group_shift < 2)
    return zeros ? launch_mma<NT, true, true>(a, grid_y, num_sms, slot, s) : launch_mma<NT, true, false>(a, grid_y, num_sms, slot + 1, s);
  return zeros ? launch_mma<NT, false, true>(a, grid_y, num_sms, slot + 2, s) : launch_mma<NT, false, false>(a, grid_y, num_sms, slot + 3, s);
}

// CTAs that run at once (by shared memory and registers).
int64_t g4_places(int NT, int num_sms) { return static_cast<int64_t>(num_sms) * (NT == 4 ? 3 : 4); }

// K is split while all clusters still run at once, a tenth of the places left free for
// clusters of four and eight, which need places near one another. (Of 4096 codes a row,
// without zero points. Eight rows: 4096 x 4096 17.2 us in one part, 10.6 in two, 7.1 in four, 6.4
// in eight; 9600 x 4096 12.2 in two, 10.2 in four, 13.1 in the eight that no longer run at
// once; 28672 x 4096 33.6 in one, 21.1 in two, 22.9 in four.) Sixteen parts where those CTAs are no
// more than the SMs (four rows: 512 x 7168 5.8 in eight, 4.7 in sixteen; 1024 x 4096 4.7 and 4.5;
// 2048 x 4096, 256 CTAs, 5.3 and 8.8). A part keeps two chunks at least.
int g4_splits(int64_t tiles, int64_t blocks, int NT, int num_sms) {
  const int64_t chunks = (blocks + G4_CHUNK - 1) / G4_CHUNK, places = g4_places(NT, num_sms);
  int splits = 1;
  while (splits < G4_MAX_SPLITS && chunks >= 4 * splits &&
         (splits == 1   ? tiles * 2 <= places
          : splits == 8 ? tiles * 16 <= num_sms
                        : 20 * tiles * splits <= 9 * places))
    splits *= 2;
  return splits;
}

// rows: activation rows of a product (an expert's, on average); products: how many (experts).
cudaError_t launch_rows(G4Args a, int64_t rows, int64_t products, int num_sms, cudaStream_t s) {
  // Rows per CTA: 8, 16 or 32 (14336 x 4096: 16 rows 17.9 us by 16 and 21.8 by 8; 32 rows 31.1
  // by 16 and 33.8 by 32; 64 rows 51.8 by 16 and 44.6 by 32; 256 rows 152 by 16 and 142
  // by 32). The 32 cost where they leave places empty (8192 x 4096, 128 rows: 52.0 by 16, 71.7
  // by 32 on 256 of 456 places; 14336 x 4096, 96 rows, 336 of 456: 72 by either).
  // Experts' CTAs take twice the average at once, so that few experts need a second pass over their
  // weights (128 experts of 2048 x 768, pairs per expert: 4 39.8 us by 8 and 51.1 by 16; 8 62.7 by
  // 8 and 55.9 by 16; 32 127 by 16 and 133 by 32; 64 229 by 16 and 225 by 32).
  const int64_t m_tiles = (a.M + G4_ROWS - 1) / G4_ROWS;
  int NT = rows > (a.ids ? 4 : 8) ? 2 : 1;
  if (rows > 32) {
    const int64_t tiles = m_tiles * ((rows + 31) / 32) * products, places = g4_places(4, num_sms);
    const int64_t ctas = tiles * g4_splits(tiles, a.blocks, 4, num_sms);
    if (4 * ctas >= 3 * ((ctas + places - 1) / places * places)) NT = 4;
  }
  int64_t y = a.ids ? products : (rows + NT * 8 - 1) / (NT * 8);
  a.splits = g4_splits(m_tiles * y, a.blocks, NT, num_sms);
  if (a.ids) {
    // An expert's passes side by side where there are places (11 experts of 218 x 800, 41 rows
    // each: 9.4 us against 23.2).
    const int64_t passes = (2 * rows + NT * 8 - 1) / (NT * 8);
    a.parts = static_cast<int>(std::max<int64_t>(1, std::min(passes, g4_places(NT, num_sms) * 9 / 10 / (m_tiles * y * a.splits))));
    y *= a.parts;
  }
  const unsigned grid_y = static_cast<unsigned>(y);
  if (NT == 1) return launch_mma_nt<1>(a, grid_y, num_sms, 0, s);
  if (NT == 2) return launch_mma_nt<2>(a, grid_y, num_sms, 4, s);
  return launch_mma_nt<4>(a, grid_y, num_sms, 8, s);
}

}  // namespace

cudaError_t launch_matvec_g4(const G4Weights& w, const uint8_t* Xq, float* Y, int64_t M, int64_t K, int64_t N,
                             int num_sms, cudaStream_t s) {
  G4Args a{w, Xq, Y, nullptr, 0, 1, false, true, M, N, static_cast<int>(K / 32), 1, 1, nullptr};
  // One or two rows: the weight stream, where a row's copy leaves three CTAs on an SM (4096 x 4096,
  // two rows: 4.7 us against 6.0 of the tensor-core form; three rows as a stream took 6.6); two
  // rows of a matrix that keeps every SM busy go to the tensor cores (28672 x 4096:
  // 17.4 against 20.3, 57344 x 4096: 32.6 against 35.8, 65536 x 4096: 36.7 against 35.3, 152064 x
  // 3584: 68.2 against 61.5).
  if ((N == 1 || (N == 2 && M <= 400 * static_cast<int64_t>(num_sms))) && g4_dp_smem(N, a.blocks) <= G4_DP_SMEM)
    return N == 1 ? launch_stream<1>(a, 0, num_sms, s) : launch_stream<2>(a, 0, num_sms, s);
  constexpr int64_t MOST = 65535 * 8;   // grid.y
  for (int64_t n0 = 0; n0 < N; n0 += MOST) {
    a.rows = std::min(N - n0, MOST);
    a.Xq = Xq + n0 * a.blocks * Q8_1_BYTES;
    a.Y = Y + n0 * M;
    const cudaError_t e = launch_rows(a, a.rows, 1, num_sms, s);
    if (e != cudaSuccess) return e;
  }
  return cudaSuccess;
}

cudaError_t launch_moe_matvec_g4(const G4Weights& w, int n_experts, const int32_t* ids, int top_k, bool x_per_slot,
                                 const uint8_t* Xq, float* Y, int64_t M, int64_t K, int64_t T, int* err, int num_sms,
                                 cudaStream_t s) {
  const int64_t pairs = T * top_k;
  G4Args a{w, Xq, Y, ids, n_experts, top_k, x_per_slot, pairs >= n_experts, M, pairs, static_cast<int>(K / 32), 1, 1, err};
  // About one pair to an expert: each is a weight stream of its own, although an expert's weights are then read
  // once per pair (128 experts of 2048 x 768: 64 pairs 15.3 us against 22.1 of the
  // tensor-core form, 112 pairs 20.8 and 27.4, 128 pairs 26.6 and 28.7; of 1536 x 2048: 64 pairs
  // 22.5 and 30.6, 96 pairs 34.7 and 35.9, 128 pairs 42.3 and 37.9). The tensor-core form leaves places
  // empty where the experts are few (4096 x 4096: 8 experts, 8 pairs 16.6 and 21.6, 12 pairs
  // 21.4 and 21.7, 16 pairs 26.7 and 21.6; 16 experts, 16 pairs 26.9 and 35.6, 24 pairs 36.8 and 35.8).
  const bool few = pairs <= std::max<int64_t>(7 * n_experts / 8, std::min<int64_t>(24, 3 * n_experts / 2));
  if ((T == 1 || few) && pairs <= 65535 && g4_dp_smem(1, a.blocks) <= G4_DP_SMEM)
    return launch_stream<1>(a, pairs, num_sms, s);
  return launch_rows(a, pairs / n_experts, n_experts, num_sms, s);
}

}  // namespace kq
