// C ABI of the attention-side operators of a decode step and of sampling: argument checks and
// dispatch to the kernels. Declarations and contracts: include/kq.h.
#include "kq_attn.h"

namespace kq {
namespace {

inline bool aligned(const void* p, unsigned to) { return (reinterpret_cast<uintptr_t>(p) & (to - 1)) == 0; }
inline bool aligned16(const void* p) { return aligned(p, 16); }
constexpr int64_t kMaxDim = (int64_t(1) << 31) - 1;
constexpr int64_t kMaxValues = int64_t(1) << 38;
constexpr int64_t kMaxHeads = int64_t(1) << 30;

kq_status finish(cudaError_t e) { return e == cudaSuccess ? KQ_OK : KQ_ERR_CUDA; }

bool valid_dtype(int t) { return t == KQ_F32 || t == KQ_F16 || t == KQ_BF16; }
// Row strides in elements: an output's rows do not overlap; an input's may be one row (0).
bool valid_ld_out(int64_t ld, int64_t K) { return ld >= K && ld <= kMaxDim; }
bool valid_ld_in(int64_t ld, int64_t K) { return ld == 0 || valid_ld_out(ld, K); }
bool valid_size(int64_t n) { return n > 0 && n <= kMaxDim; }

// The checks of a table of cosines and sines for heads of D elements; fills *r.
kq_status rope_of(const float* cos_sin, int32_t rot, int64_t n_positions, int pairing, int D, Rope* r) {
  *r = Rope{cos_sin, 0, 0, false};
  if (!cos_sin) return KQ_OK;
  if (pairing != KQ_ROPE_HALF && pairing != KQ_ROPE_PAIRS) return KQ_ERR_TYPE;
  if (rot < 16 || rot > D || rot % 16 != 0 || !valid_size(n_positions)) return KQ_ERR_SHAPE;
  r->rot = rot;
  r->n_positions = n_positions;
  r->pairs = pairing == KQ_ROPE_PAIRS;
  return KQ_OK;
}

// The checks of a 4-bit cache and its table; fills *c.
kq_status cache_of(const void* cache, int64_t n_pages, int32_t page_size, int32_t heads, int32_t D, const int32_t* table,
                   int64_t ldt, int64_t n_seqs, KvCache* c) {
  if (!cache || !table) return KQ_ERR_NULL;
  if ((D != 64 && D != 128 && D != 256) || heads <= 0 || heads > 4096 || page_size < 16 || page_size > 65536 ||
      (page_size & (page_size - 1)) != 0 || !valid_size(n_pages) || !valid_size(ldt) || !valid_size(n_seqs))
    return KQ_ERR_SHAPE;
  int shift = 4;
  while ((1 << shift) < page_size) ++shift;
  *c = KvCache{static_cast<uint8_t*>(const_cast<void*>(cache)), table, ldt, n_seqs, n_pages, shift, heads, D};
  return KQ_OK;
}
bool cache_aligned(const KvCache& c) { return aligned16(c.data) && aligned(c.table, 4); }

}  // namespace
}  // namespace kq

using namespace kq;

extern "C" {

kq_status kq_qk_norm_rope(int dtype, const void* Q, int64_t ldq, int32_t n_q_heads, const void* K, int64_t ldk,
                          int32_t n_k_heads, int32_t head_dim, const float* q_gamma, const float* k_gamma, float eps,
                          const float* cos_sin, int32_t rot_dim, int64_t n_positions, int pairing, const int32_t* positions,
                          int out_dtype, void* Qo, int64_t ldqo, void* Ko, int64_t ldko, int64_t N, kq_stream_t stream) {
  if (!valid_dtype(dtype) || !valid_dtype(out_dtype) || (dtype != KQ_F32 && out_dtype != dtype)) return KQ_ERR_TYPE;
  if (!Q || !Qo || (n_k_heads > 0 && (!K || !Ko))) return KQ_ERR_NULL;
  if (n_q_heads <= 0 || n_q_heads > 65536 || n_k_heads < 0 || n_k_heads > 65536 || head_dim < 16 || head_dim > 256 ||
      head_dim % 16 != 0 || !valid_size(N) || N * (n_q_heads + n_k_heads) > kMaxHeads ||
      !(eps >= 0.f && eps < 1e30f))  // also rejects NaN
    return KQ_ERR_SHAPE;
  const int64_t q = static_cast<int64_t>(n_q_heads) * head_dim, k = static_cast<int64_t>(n_k_heads) * head_dim;
  if (!valid_ld_in(ldq, q) || !valid_ld_out(ldqo, q) || (k && (!valid_ld_in(ldk, k) || !valid_ld_out(ldko, k))))
    return KQ_ERR_SHAPE;
  Rope rope;
  const kq_status st = rope_of(cos_sin, rot_dim, n_positions, pairing, head_dim, &rope);
  if (st != KQ_OK) return st;
  if (!aligned16(Q) || !aligned16(Qo) || !aligned16(q_gamma) || !aligned16(cos_sin) || !aligned(positions, 4) ||
      (k && (!aligned16(K) || !aligned16(Ko) || !aligned16(k_gamma))))
    return KQ_ERR_ALIGN;
  int dev, sms;
  int* err;
  if (device_context(&dev, &sms, &err) != cudaSuccess) return KQ_ERR_CUDA;
  return finish(launch_qk_norm_rope(dtype, Q, ldq, n_q_heads, K, ldk, n_k_heads, head_dim, q_gamma, k_gamma, eps, rope,
                                    positions, out_dtype, Qo, ldqo, Ko, ldko, N, err, sms,
                                    reinterpret_cast<cudaStream_t>(stream)));
}

kq_status kq_kv_append_q4(int dtype, const void* K, int64_t ldk, const void* V, int64_t ldv, int32_t n_heads,
                          int32_t head_dim, const float* cos_sin, int32_t rot_dim, int64_t n_positions, int pairing,
                          const int32_t* positions, const int32_t* seq_ids, const int32_t* block_table, int64_t ldt,
                          int64_t n_seqs, void* cache, int64_t n_pages, int32_t page_size, int64_t N, kq_stream_t stream) {
  if (!valid_dtype(dtype)) return KQ_ERR_TYPE;
  if (!K || !V || !positions) return KQ_ERR_NULL;
  KvCache c;
  kq_status st = cache_of(cache, n_pages, page_size, n_heads, head_dim, block_table, ldt, n_seqs, &c);
  if (st != KQ_OK) return st;
  const int64_t row = static_cast<int64_t>(n_heads) * head_dim;
  if (!valid_size(N) || 2 * N * n_heads > kMaxHeads || !valid_ld_in(ldk, row) || !valid_ld_in(ldv, row) ||
      (!seq_ids && N > n_seqs))
    return KQ_ERR_SHAPE;
  Rope rope;
  st = rope_of(cos_sin, rot_dim, n_positions, pairing, head_dim, &rope);
  if (st != KQ_OK) return st;
  if (!aligned16(K) || !aligned16(V) || !aligned16(cos_sin) || !aligned(positions, 4) || !aligned(seq_ids, 4) ||
      !cache_aligned(c))
    return KQ_ERR_ALIGN;
  int dev, sms;
  int* err;
  if (device_context(&dev, &sms, &err) != cudaSuccess) return KQ_ERR_CUDA;
  return finish(launch_kv_append_q4(dtype, K, ldk, V, ldv, rope, positions, seq_ids, c, N, err, sms,
                                    reinterpret_cast<cudaStream_t>(stream)));
}

kq_status kq_kv_gather_q4(const void* cache, int64_t n_pages, int32_t page_size, int32_t n_heads, int32_t head_dim,
                          const int32_t* block_table, int64_t ldt, int64_t n_seqs, const int32_t* positions,
                          const int32_t* seq_ids, int dtype, void* K, int64_t ldk, void* V, int64_t ldv, int64_t N,
                          kq_stream_t stream) {
  if (!valid_dtype(dtype)) return KQ_ERR_TYPE;
  if (!K || !V || !positions) return KQ_ERR_NULL;
  KvCache c;
  const kq_status st = cache_of(cache, n_pages, page_size, n_heads, head_dim, block_table, ldt, n_seqs, &c);
  if (st != KQ_OK) return st;
  const int64_t row = static_cast<int64_t>(n_heads) * head_dim;
  if (!valid_size(N) || 2 * N * n_heads > kMaxHeads || !valid_ld_out(ldk, row) || !valid_ld_out(ldv, row) ||
      (!seq_ids && N > n_seqs))
    return KQ_ERR_SHAPE;
  if (!aligned16(K) || !aligned16(V) || !aligned(positions, 4) || !aligned(seq_ids, 4) || !cache_aligned(c))
    return KQ_ERR_ALIGN;
  int dev, sms;
  int* err;
  if (device_context(&dev, &sms, &err) != cudaSuccess) return KQ_ERR_CUDA;
  return finish(launch_kv_gather_q4(c, positions, seq_ids, dtype, K, ldk, V, ldv, N, err, sms,
                                    reinterpret_cast<cudaStream_t>(stream)));
}

size_t kq_attn_q4_workspace_bytes(int32_t n_q_heads, int32_t n_kv_heads, int32_t head_dim, int64_t N, int64_t n_seqs) {
  if (n_kv_heads <= 0 || n_kv_heads > 4096 || n_q_heads <= 0 || n_q_heads % n_kv_heads != 0 || n_q_heads > 65536 ||
      (head_dim != 64 && head_dim != 128 && head_dim != 256) || !valid_size(N) || !valid_size(n_seqs))
    return 0;
  int dev, sms;
  int* err;
  if (device_context(&dev, &sms, &err) != cudaSuccess) sms = 152;
  return attn_q4_workspace(n_q_heads, n_kv_heads, head_dim, N, n_seqs, sms);
}

kq_status kq_attn_q4(int dtype, const void* Q, int64_t ldq, int32_t n_q_heads, const void* cache, int64_t n_pages,
                     int32_t page_size, int32_t n_kv_heads, int32_t head_dim, const int32_t* block_table, int64_t ldt,
                     int64_t n_seqs, const int32_t* kv_len, const int32_t* q_start, float scale, int64_t window, void* O,
                     int64_t ldo, void* Xq, int64_t N, void* ws, size_t ws_bytes, kq_stream_t stream) {
  if (!valid_dtype(dtype)) return KQ_ERR_TYPE;
  if (!Q || !kv_len || (!O && !Xq) || !ws) return KQ_ERR_NULL;
  KvCache c;
  const kq_status st = cache_of(cache, n_pages, page_size, n_kv_heads, head_dim, block_table, ldt, n_seqs, &c);
  if (st != KQ_OK) return st;
  const int64_t row = static_cast<int64_t>(n_q_heads) * head_dim;
  if (n_q_heads <= 0 || n_q_heads > 65536 || n_q_heads % n_kv_heads != 0 || !valid_size(N) || N * row > kMaxValues ||
      N * n_q_heads > (int64_t(1) << 30) ||
      (!q_start && N != n_seqs) || !valid_ld_in(ldq, row) || (O && !valid_ld_out(ldo, row)) ||
      !(scale > -1e30f && scale < 1e30f) || window < 0)
    return KQ_ERR_SHAPE;
  if (!aligned16(Q) || !aligned16(O) || !aligned16(Xq) || !aligned16(ws) || !aligned(kv_len, 4) || !aligned(q_start, 4) ||
      !cache_aligned(c))
    return KQ_ERR_ALIGN;
  int dev, sms;
  int* err;
  if (device_context(&dev, &sms, &err) != cudaSuccess) return KQ_ERR_CUDA;
  if (ws_bytes < attn_q4_workspace(n_q_heads, n_kv_heads, head_dim, N, n_seqs, sms)) return KQ_ERR_WORKSPACE;
  const AttnArgs a = {Q, ldq, n_q_heads, scale, window, q_start, kv_len, O, ldo, static_cast<uint8_t*>(Xq), N};
  return finish(launch_attn_q4(dtype, a, c, ws, err, sms, reinterpret_cast<cudaStream_t>(stream)));
}

kq_status kq_sample(int dtype, const void* logits, int64_t ld, const float* temperature, const int32_t* top_k,
                    const float* top_p, const float* min_p, const float* u, int32_t* ids, float* probs, int64_t V, int64_t N,
                    kq_stream_t stream) {
  if (!valid_dtype(dtype)) return KQ_ERR_TYPE;
  if (!logits || !u || !ids) return KQ_ERR_NULL;
  if (V <= 0 || V > SAMPLE_MAX_V || !valid_size(N) || N * V > (int64_t(1) << 40) || !valid_ld_in(ld, V)) return KQ_ERR_SHAPE;
  if (!aligned16(logits) || !aligned(temperature, 4) || !aligned(top_k, 4) || !aligned(top_p, 4) || !aligned(min_p, 4) ||
      !aligned(u, 4) || !aligned(ids, 4) || !aligned(probs, 4))
    return KQ_ERR_ALIGN;
  int dev, sms;
  int* err;
  if (device_context(&dev, &sms, &err) != cudaSuccess) return KQ_ERR_CUDA;
  const SampleArgs a = {logits, ld, temperature, top_k, top_p, min_p, u, ids, probs, V, N};
  return finish(launch_sample(dtype, a, sms, reinterpret_cast<cudaStream_t>(stream)));
}

}  // extern "C"
