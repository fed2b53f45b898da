// Paged attention: the number of splits along the keys, and the dispatch on
// type and head size (one translation unit for each).
#include "paged_attention.h"

#include <algorithm>

#include "ttq_internal.h"

namespace ttq {

// Few tiles leave most of the 256 CUs idle: the keys of each are then split
// until there are two workgroups for each CU, each split with at least two
// tiles of 64 keys of the longest sequence.
int attn_splits(int64_t total_q, int n_seqs, int n_kv, int group, int64_t max_kv_len) {
  const int64_t tiles = (total_q * group / kAttnRows + n_seqs) * n_kv;
  const int64_t want = 512 / std::max<int64_t>(tiles, 1), most = max_kv_len / 128;
  return (int)std::max<int64_t>(1, std::min<int64_t>({want, most, 64}));
}

hipError_t launch_paged_attention(const AttnArgs& a, bool bf16, int head_dim, hipStream_t s) {
  switch (head_dim) {
    case 64: return bf16 ? launch_attn<__bf16, 64>(a, s) : launch_attn<_Float16, 64>(a, s);
    case 128: return bf16 ? launch_attn<__bf16, 128>(a, s) : launch_attn<_Float16, 128>(a, s);
    default: return bf16 ? launch_attn<__bf16, 256>(a, s) : launch_attn<_Float16, 256>(a, s);
  }
}

}  // namespace ttq
