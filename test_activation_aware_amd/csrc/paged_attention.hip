// Paged attention: the number of splits along the keys, and the dispatch on
// type and head size (one translation unit for each).
#include "paged_attention.h"

#include <algorithm>
#include <cstdlib>

#include "ttq_internal.h"

namespace ttq {

namespace {

int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

}  // namespace

int attn_plan(AttnArgs& a, int head_dim, int64_t max_q_len, int64_t max_kv_len) {
  const int64_t max_rows = max_q_len * a.group;
  const bool rows = max_rows > kAttnKeyRows, keys = !rows || a.n_seqs > 1;
  a.skip_rows = rows && keys ? kAttnKeyRows : 0;
  // keys that one row can see; a prefix's length is not known here
  const int64_t span = std::max<int64_t>(1, a.window > 0 && a.prefix == nullptr ? std::min<int64_t>(max_kv_len, a.window) : max_kv_len);
  a.key_splits = a.row_splits = 0;
  a.key_per = a.row_per = 1;
  a.key_waves = 1;
  if (keys) {
    const int64_t tiles = ceil_div(span + kAttnKeyRows, 32), items = (int64_t)a.n_seqs * a.n_kv;
    a.key_waves = items >= 512 && tiles < 16 ? 1 : 4;
    int64_t want = std::min((head_dim == 64 ? 512 : 256) / items, tiles / 6);
    const char* e1 = getenv("KW"); const char* e2 = getenv("KS");
    if (e1) a.key_waves = atoi(e1);
    if (e2) want = std::min<int64_t>(atoi(e2), tiles);
    want = std::max<int64_t>(want, 1);
    a.key_per = (int)ceil_div(tiles, want);
    a.key_splits = (int)ceil_div(tiles, a.key_per);
  }
  if (rows) {
    const int64_t tiles = ceil_div(span + std::min<int64_t>(max_rows, kAttnRows) / a.group, 64);
    const int64_t items = (a.total_q * (int64_t)a.group / kAttnRows + 1) * a.n_kv;
    const char* e2 = getenv("RS");
    int64_t want = e2 ? atoi(e2) : std::max<int64_t>(1, 512 / items);
    want = std::min(want, std::max<int64_t>(1, tiles / 2));
    a.row_per = (int)ceil_div(tiles, want);
    a.row_splits = (int)ceil_div(tiles, a.row_per);
  }
  return std::max(a.key_splits, a.row_splits);
}

hipError_t launch_paged_attention(const AttnArgs& a, bool bf16, int head_dim, hipStream_t s) {
  switch (head_dim) {
    case 64: return bf16 ? launch_attn<__bf16, 64>(a, s) : launch_attn<_Float16, 64>(a, s);
    case 128: return bf16 ? launch_attn<__bf16, 128>(a, s) : launch_attn<_Float16, 128>(a, s);
    default: return bf16 ? launch_attn<__bf16, 256>(a, s) : launch_attn<_Float16, 256>(a, s);
  }
}

}  // namespace ttq
