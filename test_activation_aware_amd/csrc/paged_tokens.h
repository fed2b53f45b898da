// Where a token of a ragged batch stands, for the kernels that take the
// batch's rows one by one.
#pragma once

#include "ttq_internal.h"

namespace ttq {

// The sequence of token `tok`, -1 when it is none's.  By a whole wave with one
// token: 64 starts a step, by ballot.
__device__ __forceinline__ int sequence_of(const Places& p, int tok) {
  const int lane = threadIdx.x & 63;
  int n = 0;
  for (int c = 0; c < p.n_seqs; c += 64) {
    const int i = c + lane;
    const unsigned long long b = __ballot(i < p.n_seqs && p.q_start[min(i, p.n_seqs - 1)] <= tok);
    n += __popcll(b);
    if (b != ~0ull) break;
  }
  const int s = __builtin_amdgcn_readfirstlane(n - 1);
  return s < 0 || tok >= p.q_start[s + 1] ? -1 : s;
}

// The position of token `tok` of sequence s; may be negative.
__device__ __forceinline__ int64_t position_of(const Places& p, int s, int tok) {
  return (int64_t)p.kv_len[s] - ((int64_t)p.q_start[s + 1] - tok);
}

// The page of position pos of sequence s; false when it has none.
__device__ __forceinline__ bool page_of(const Places& p, int s, int64_t pos, uint32_t& page) {
  if (pos < 0 || (pos >> p.page_shift) >= p.n_blocks) return false;
  page = (uint32_t)p.table[s * p.table_stride + (pos >> p.page_shift)];
  return page < p.n_pages;
}

}  // namespace ttq
