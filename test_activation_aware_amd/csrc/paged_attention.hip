// Paged attention: the number of splits along the keys, and the dispatch on
// type and head size (one translation unit for each).
#include "paged_attention.h"

#include <algorithm>

#include "ttq_internal.h"

namespace ttq {

namespace {

int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

}  // namespace

// Two forms.  In the row form 128 rows (heads of a group times tokens) share
// every key tile that they load; in the key form 32 rows are worked on by
// several waves, each with keys of its own.  A wave needs about 1 us for a key
// tile, 32 keys or 64, if it has the SIMD to itself, so that a long chain of
// tiles costs more than loading keys again: with decode tokens (at most 32 rows
// a sequence) and with few rows otherwise (up to 128 workgroups of the row
// form) the key form wins (4 x 64 tokens over 1000, 32/8 heads of 128: 15.7 us
// against 29.8; 1000 tokens, 12 heads of 64: 11.1 against 22.5; but 5 x 800
// tokens, 16 heads of 64, 512 workgroups: 31.0 against 22.2, and 64 tokens over
// 16000, 32/8 heads of 128: 51.8 against 44.2).  One launch has one form: a batch of chunks and decode tokens takes the row form for both (24
// sequences, chunks of up to 512, 16/8 heads of 256, capped, window 1024: 82
// us, 157 in two launches).
//
// Key form.  A workgroup's four waves (two for heads of 256) share one item (a
// tile of rows and a key head): one workgroup fills a CU's LDS, so up to 256
// are wanted (twice as many for heads of 64), in one round: 3 sequences of up
// to 131072 keys with 8 key heads take 177 us in 8 splits, 192 workgroups, and
// 237 us in 12.  A split keeps two tiles a wave (1 sequence of 4000 keys, 8 key
// heads: 14.1 us in 8 or 16 splits, 17.6 in 32), and more than 16 splits are
// worth their join only when each is long.  Many short items need no sharing: a
// wave each (128 sequences of 500 keys: 42.6 us against 47.5).
//
// Row form.  Two workgroups fit a CU; where there are fewer, the keys are
// split, 384 keys or more a split (512 tokens over 2000, 12 heads of 64: 31.8
// us in one, 24.9 in 4, 28.3 in 8).  A few rounds of long chains end sooner
// when a CU's waves share one workgroup, in two halves (4096 tokens, 16/8 heads
// of 256: 163 us against 203; 2 x 1024 tokens over 6000, 32/8 heads of 128: 190
// against 247; 4000 tokens, 16 heads of 64: 53 against 60); short chains and
// many rounds do not (8 x 512 tokens, 32/8 heads of 128: 49 against 39; 16384
// tokens, 64/8: 4282 against 3986).
int attn_plan(AttnArgs& a, int head_dim, int64_t max_q_len, int64_t max_kv_len) {
  const int64_t max_rows = max_q_len * a.group, all_rows = a.total_q * (int64_t)a.group;
  // keys that one query can see (a prefix's length is not known here)
  const int64_t span = std::max<int64_t>(
      1, a.window > 0 && a.prefix == nullptr ? std::min<int64_t>(max_kv_len, a.window) : max_kv_len);
  const int64_t row_items = (all_rows / kAttnRows + 1) * a.n_kv;
  a.key_splits = a.row_splits = 0;
  if (max_rows <= kAttnKeyRows || (row_items <= 128 && span <= 8192)) {
    const int64_t tiles = ceil_div(span + std::min<int64_t>(max_q_len, kAttnKeyRows), 32);
    a.key_tiles = (int)(all_rows / kAttnKeyRows) + a.n_seqs;  // enough wherever the sequences begin
    const int64_t items = (max_rows <= kAttnKeyRows ? a.n_seqs : all_rows / kAttnKeyRows + 1) * a.n_kv;
    a.key_waves = items >= 512 && tiles < 32 ? 1 : head_dim == 256 ? 2 : 4;
    int64_t want = std::min((head_dim == 64 ? 512 : 256) / items, std::max<int64_t>(16, tiles / 64));
    want = std::min(want, tiles / (2 * a.key_waves));
    if (want < 3) want = 1;  // a join costs more than half of so little work
    a.key_per = (int)ceil_div(tiles, want);
    a.key_splits = (int)ceil_div(tiles, a.key_per);
  } else {
    const int keys = head_dim == 256 ? 32 : 64;
    const int64_t tiles = ceil_div(span + kAttnRows / a.group, keys);
    const int64_t want = std::max<int64_t>(1, std::min(512 / row_items, tiles * keys / 384));
    a.row_tiles = (int)(all_rows / kAttnRows) + a.n_seqs;
    a.row_per = (int)ceil_div(tiles, want);
    a.row_splits = (int)ceil_div(tiles, a.row_per);
    a.row_halves = span >= 2048 && row_items >= 512 && row_items < 1280 ? 2 : 1;
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
