// Paged attention: the number of splits along the keys, and the dispatch on
// type and head size (one translation unit for each).
#include "paged_attention.h"

#include <algorithm>

#include "ttq_internal.h"

namespace ttq {

namespace {

int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

}  // namespace

// Sequences of at most 32 rows (decode tokens: heads of a group times tokens)
// take the key form, all others the row form; a batch takes the form of its
// longest sequence, since two launches one after the other cost more than
// short sequences lose in the row form (24 sequences, chunks of up to 512
// among decode tokens, 16/8 heads of 256, capped, window 1024: 82 us in the
// row form alone, 157 us with both).
//
// Key form.  A workgroup's four waves (two for heads of 256) share one item (a
// sequence and a key head): one workgroup fills a CU's LDS, so up to 256 are
// wanted (twice as many for heads of 64), in one round: 3 sequences of up to
// 131072 keys with 8 key heads take 177 us in 8 splits, 192 workgroups, and
// 237 us in 12.  A split keeps two tiles a wave (1 sequence of 4000 keys, 8
// key heads: 14.1 us in 8 or 16 splits, 17.6 in 32), and more than 16 splits
// are worth their join only when each is long.  Many short items need no
// sharing: a wave each (128 sequences of 500 keys: 42.6 us against 47.5).
//
// Row form.  Two workgroups fit a CU; where there are fewer, the keys are
// split, six tiles of 64 or more a split (512 tokens over 2000, 12 heads of
// 64: 31.8 us in one, 24.9 in 4, 28.3 in 8; 64 tokens over 16000, 32/8 heads
// of 128: 292 us in one, 41 in 21).
int attn_plan(AttnArgs& a, int head_dim, int64_t max_q_len, int64_t max_kv_len) {
  const int64_t max_rows = max_q_len * a.group;
  // keys that one query can see; a prefix's length is not known here
  const int64_t span = std::max<int64_t>(
      1, a.window > 0 && a.prefix == nullptr ? std::min<int64_t>(max_kv_len, a.window) : max_kv_len);
  a.key_splits = a.row_splits = 0;
  a.key_per = a.row_per = 1;
  a.key_waves = 1;
  if (max_rows <= kAttnKeyRows) {
    const int64_t tiles = ceil_div(span + max_q_len, 32), items = (int64_t)a.n_seqs * a.n_kv;
    a.key_waves = items >= 512 && tiles < 32 ? 1 : head_dim == 256 ? 2 : 4;
    int64_t want = std::min((head_dim == 64 ? 512 : 256) / items, std::max<int64_t>(16, tiles / 64));
    want = std::min(want, tiles / (2 * a.key_waves));
    if (want < 3) want = 1;  // a join costs more than half of so little work
    a.key_per = (int)ceil_div(tiles, want);
    a.key_splits = (int)ceil_div(tiles, a.key_per);
  } else {
    const int keys = head_dim == 256 ? 32 : 64;
    const int64_t tiles = ceil_div(span + std::min<int64_t>(max_rows, kAttnRows) / a.group, keys);
    const int64_t items = (a.total_q * (int64_t)a.group / kAttnRows + 1) * a.n_kv;
    const int64_t want = std::max<int64_t>(1, std::min(512 / items, tiles * keys / 384));
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
