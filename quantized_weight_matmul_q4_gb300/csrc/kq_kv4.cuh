// Where a token's codes and parameters are in the 4-bit cache.
#pragma once

#include "kq_attn.h"
#include "kq_common.cuh"

namespace kq {

// The granule of 16 places of one head: key codes [16][D / 2], key parameters [16][D / 32 s, D / 32 m],
// value codes, value parameters.
template <int D>
struct Granule {
  static constexpr int G = D / 32;          // blocks of a head
  static constexpr int kCodes = 8 * D;      // bytes of 16 tokens' codes
  static constexpr int kParams = 2 * D;     // and of their parameters
  static constexpr int kValues = kCodes + kParams;
  static constexpr int kBytes = 2 * kValues;
};

// The granule that holds place `pos` of sequence `seq` for head 0, or -1 where the table or the
// cache has no such place. Heads are (page / 16) granules apart.
__device__ __forceinline__ int64_t granule_of(const KvCache& c, int64_t seq, int64_t pos) {
  const int64_t i = pos >> c.page_shift;
  if (seq < 0 || seq >= c.n_seqs || pos < 0 || i >= c.ldt) return -1;
  const int64_t page = c.table[seq * c.ldt + i];
  if (page < 0 || page >= c.n_pages) return -1;
  const int per = c.page_shift - 4;
  return ((page * c.heads) << per) + ((pos & ((int64_t(1) << c.page_shift) - 1)) >> 4);
}

}  // namespace kq
