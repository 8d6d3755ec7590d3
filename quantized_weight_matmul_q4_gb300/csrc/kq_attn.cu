// Attention over the 4-bit paged cache, for the new tokens of a decode step.
//
//   o = Sum_t softmax_t(scale q . k_t) v_t   over the places t that a row sees
//
// Row i of a sequence's n new rows sees the places below kv_len - n + 1 + i and, with a window, the
// last `window` of those; a row that sees none gives zeros.
#include <cuda_bf16.h>

#include <algorithm>

#include "kq_kv4.cuh"
#include "kq_types.cuh"

namespace kq {
namespace {

struct Attn {
  AttnArgs a;
  KvCache c;
  float* ws;
  int* err;
};

// A warp per row and query head, a token at a time, D / 32 elements a lane (one of each block).
template <typename T, int D>
__global__ void __launch_bounds__(128) attn_q4_rows_kernel(const Attn p) {
  pdl_enter();
  using Gr = Granule<D>;
  constexpr int G = D / 32;
  const int lane = threadIdx.x & 31;
  const int64_t item = (static_cast<int64_t>(blockIdx.x) * 128 + threadIdx.x) >> 5;
  if (item >= p.a.N * p.a.n_q) return;
  const int64_t n = item / p.a.n_q;
  const int hq = static_cast<int>(item - n * p.a.n_q), h = hq / (p.a.n_q / p.c.heads);
  int64_t b = n, len = 0, i = 0, rows = 1;
  if (p.a.q_start) {
    b = -1;
    for (int64_t k = 0; k < p.c.n_seqs; ++k)
      if (n >= p.a.q_start[k] && n < p.a.q_start[k + 1]) b = k;
    if (b < 0) return;
    i = n - p.a.q_start[b];
    rows = p.a.q_start[b + 1] - p.a.q_start[b];
  }
  len = p.a.kv_len[b];
  const int64_t end = len - rows + 1 + i, begin = p.a.window > 0 ? max(int64_t(0), end - p.a.window) : 0;
  const T* q = static_cast<const T*>(p.a.Q) + n * p.a.ldq + static_cast<int64_t>(hq) * D;
  float qv[G], o[G], m = -INFINITY, l = 0.f;
#pragma unroll
  for (int g = 0; g < G; ++g) qv[g] = to_f32(q[32 * g + lane]) * p.a.scale, o[g] = 0.f;
  for (int64_t t = begin; t < end; ++t) {
    const int64_t at = granule_of(p.c, b, t);
    if (at < 0) {
      if (lane == 0) report_error(p.err, ERR_PAGE);
      continue;
    }
    const uint8_t* gr = p.c.data + (at + (static_cast<int64_t>(h) << (p.c.page_shift - 4))) * Gr::kBytes;
    const int r = static_cast<int>(t & 15);
    const __half* kp = reinterpret_cast<const __half*>(gr + Gr::kCodes + r * 4 * G);
    const __half* vp = reinterpret_cast<const __half*>(gr + Gr::kValues + Gr::kCodes + r * 4 * G);
    float s = 0.f, v[G];
#pragma unroll
    for (int g = 0; g < G; ++g) {
      const uint8_t kc = gr[r * (D / 2) + 4 * G * (lane >> 3) + 4 * g + ((lane & 7) >> 1)];
      const uint8_t vc = gr[Gr::kValues + r * (D / 2) + 2 * G * (lane >> 2) + 2 * g + ((lane & 3) >> 1)];
      const int sh = 4 * (lane & 1);
      s = fmaf(qv[g], fmaf(static_cast<float>((kc >> sh) & 15), __half2float(kp[g]), __half2float(kp[G + g])), s);
      v[g] = fmaf(static_cast<float>((vc >> sh) & 15), __half2float(vp[g]), __half2float(vp[G + g]));
    }
    s = warp_sum_f(s);
    const float mn = fmaxf(m, s), f = expf(m - mn), e = expf(s - mn);
    l = fmaf(l, f, e);
#pragma unroll
    for (int g = 0; g < G; ++g) o[g] = fmaf(o[g], f, e * v[g]);
    m = mn;
  }
  const float inv = end > begin ? 1.f / l : 0.f;
#pragma unroll
  for (int g = 0; g < G; ++g) o[g] = end > begin ? o[g] * inv : 0.f;
  if (p.a.O) {
    T* out = static_cast<T*>(p.a.O) + n * p.a.ldo + static_cast<int64_t>(hq) * D;
#pragma unroll
    for (int g = 0; g < G; ++g) out[32 * g + lane] = from_f32<T>(o[g]);
  }
  if (p.a.Xq) {
#pragma unroll
    for (int g = 0; g < G; ++g) {
      float x = fabsf(o[g]);
      for (int k = 16; k > 0; k >>= 1) {
        const float y = __shfl_xor_sync(0xffffffffu, x, k);
        x = (x > y || x != x) ? x : y;
      }
      const float d = __fdiv_rn(x, 127.f), di = d > 1e-38f ? __fdiv_rn(1.f, d) : 0.f;
      const int c = __float2int_rn(__fmul_rn(o[g], di));
      const int sum = warp_sum_i(c);
      uint8_t* blk = p.a.Xq + ((n * p.a.n_q + hq) * G + g) * Q8_1_BYTES;
      blk[4 + lane] = static_cast<uint8_t>(c);
      if (lane == 0) {
        const __half dh = __float2half_rn(d);
        reinterpret_cast<__half*>(blk)[0] = dh;
        reinterpret_cast<__half*>(blk)[1] = __float2half_rn(__half2float(dh) * static_cast<float>(sum));
      }
    }
  }
}

template <typename T>
cudaError_t rows(const Attn& p, cudaStream_t s) {
  const dim3 grid(static_cast<unsigned>((p.a.N * p.a.n_q + 3) / 4));
  if (p.c.D == 64) return launch_pdl(attn_q4_rows_kernel<T, 64>, grid, dim3(128), 0, s, p);
  if (p.c.D == 128) return launch_pdl(attn_q4_rows_kernel<T, 128>, grid, dim3(128), 0, s, p);
  return launch_pdl(attn_q4_rows_kernel<T, 256>, grid, dim3(128), 0, s, p);
}

}  // namespace

size_t attn_q4_workspace(int, int, int, int64_t, int64_t, int) { return 16; }

cudaError_t launch_attn_q4(int dtype, const AttnArgs& a, const KvCache& c, void* ws, int* err, int, cudaStream_t s) {
  const Attn p = {a, c, static_cast<float*>(ws), err};
  if (dtype == KQ_F16) return rows<__half>(p, s);
  if (dtype == KQ_BF16) return rows<__nv_bfloat16>(p, s);
  return rows<float>(p, s);
}

}  // namespace kq
