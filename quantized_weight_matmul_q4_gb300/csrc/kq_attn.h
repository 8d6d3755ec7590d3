// Internal interface of the attention-side operators of a decode step (head norms and rotation, the
// 4-bit paged cache and its attention, sampling): their checks and entry points are in
// kq_attn_api.cu, their kernels in kq_heads.cu, kq_attn.cu and kq_sample.cu.
#pragma once

#include "kq_internal.h"

namespace kq {

constexpr int ERR_POSITION = KQ_DEVERR_POSITION;
constexpr int ERR_PAGE = KQ_DEVERR_PAGE;

// Rotation by a table of cosines and sines; cos_sin null: none.
struct Rope {
  const float* cos_sin;      // [n_positions][rot]
  int rot;                   // elements turned, a multiple of 16
  int64_t n_positions;
  bool pairs;                // elements 2i and 2i + 1, not i and i + rot / 2
};

// The 4-bit cache: bytes [n_pages][heads][page / 16][20 * D].
struct KvCache {
  uint8_t* data;
  const int32_t* table;      // [n_seqs][ldt]: page of places [i * page, (i + 1) * page) of a sequence
  int64_t ldt;               // pages a row of the table has
  int64_t n_seqs;
  int64_t n_pages;
  int page_shift;            // log2 of the places of a page
  int heads;
  int D;
};

cudaError_t launch_qk_norm_rope(int dtype, const void* Q, int64_t ldq, int n_q, const void* K, int64_t ldk, int n_k, int D,
                                const float* q_gamma, const float* k_gamma, float eps, const Rope& rope,
                                const int32_t* positions, int out_dtype, void* Qo, int64_t ldqo, void* Ko, int64_t ldko,
                                int64_t N, int* err, int num_sms, cudaStream_t s);

cudaError_t launch_kv_append_q4(int dtype, const void* K, int64_t ldk, const void* V, int64_t ldv, const Rope& rope,
                                const int32_t* positions, const int32_t* seq_ids, const KvCache& c, int64_t N, int* err,
                                int num_sms, cudaStream_t s);
cudaError_t launch_kv_gather_q4(const KvCache& c, const int32_t* positions, const int32_t* seq_ids, int dtype, void* K,
                                int64_t ldk, void* V, int64_t ldv, int64_t N, int* err, int num_sms, cudaStream_t s);

struct AttnArgs {
  const void* Q;
  int64_t ldq;
  int n_q;                   // query heads, a multiple of the cache's
  float scale;
  int64_t window;            // 0: none
  const int32_t* q_start;    // [n_seqs + 1] or null (row n belongs to sequence n)
  const int32_t* kv_len;     // [n_seqs]
  void* O;                   // dtype of Q, or null
  int64_t ldo;
  uint8_t* Xq;               // Q8_1 rows of n_q * D, or null
  int64_t N;
};
size_t attn_q4_workspace(int n_q, int n_kv, int D, int64_t N, int64_t n_seqs, int num_sms);
cudaError_t launch_attn_q4(int dtype, const AttnArgs& a, const KvCache& c, void* ws, int* err, int num_sms, cudaStream_t s);

// Row parameters may be null: temperature 1, no limit.
struct SampleArgs {
  const void* logits;
  int64_t ld;
  const float* temperature;
  const int32_t* top_k;
  const float* top_p;
  const float* min_p;
  const float* u;
  int32_t* ids;
  float* probs;              // or null
  int64_t V, N;
};
constexpr int64_t SAMPLE_MAX_V = 1 << 19;
cudaError_t launch_sample(int dtype, const SampleArgs& a, int num_sms, cudaStream_t s);

}  // namespace kq
