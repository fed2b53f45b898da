// Paged attention: the number of splits along the keys, and the dispatch on
// type and head size (one translation unit for each).
#include "paged_attention.h"

#include <algorithm>

#include "ttq_internal.h"

namespace ttq {

namespace {

int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

// tiles that `rows` rows of n sequences have at most, however they are divided
int most_tiles(int64_t rows, int n, int bm) { return (int)((rows + (int64_t)n * (bm - 1)) / bm); }

// keys that one query can see (a prefix's length is not known here)
int64_t keys_seen(const AttnArgs& a, int64_t max_kv_len) {
  return std::max<int64_t>(1, a.window > 0 && a.prefix == nullptr ? std::min<int64_t>(max_kv_len, a.window) : max_kv_len);
}

}  // namespace

// Two forms.  In the row form 128 rows (heads of a group times tokens) share
// every key tile that they load; in the key form 32 rows are worked on by
// several waves, each with keys of its own.  A wave needs about 1 us for a key
// tile, 32 keys or 64, if it has the SIMD to itself, so that a long chain of
// tiles costs more than loading keys again: the key form takes decode tokens
// (at most 32 rows a sequence) and otherwise few rows over few keys, where the
// row form would not fill half the CUs (4 x 64 tokens over 1000, 32/8 heads of
// 128: 15.7 us against 29.8; 512 tokens over 2512, 16 heads of 64: 21.8 against
// 28.8).  Loading the keys for every 32 rows ends that at work (rows times
// keys) which is less the wider the heads, two waves being all that fit a CU
// at 256: 250 tokens over 20000, 16 heads of 64: 56 us against 47; 64 over
// 16000, 32/8 heads of 128: 56 against 42; 256 over 2256, 16/8 heads of 256: 65
// against 49.  One launch has one form: a batch of chunks and decode tokens
// takes the row form for both (24 sequences, chunks of up to 512, 16/8 heads of
// 256, capped, window 1024: 84 us, 157 in two launches).  That holds for contexts
// of like length; one far beyond the others' is a chain that the batch's one
// split count leaves whole (32/8 heads of 128: 512 tokens beside a decode token
// over 131072 1900 us, 16 and 107 in two calls; 64 decode tokens over 1000 of
// which one has 131072 1180 us, 44 without).
//
// Key form.  A workgroup's four waves (two for heads of 256) share one item (a
// tile of rows and a key head): one workgroup fills a CU's LDS, so up to 256
// are wanted (twice as many for heads of 64), in one round: 3 sequences of up
// to 131072 keys with 8 key heads take 177 us in 8 splits, 192 workgroups, and
// 237 us in 12.  A split keeps two tiles a wave (1 sequence of 4000 keys, 8 key
// heads: 14.1 us in 8 or 16 splits, 17.6 in 32), and more than 16 splits are
// worth their join only when each is long.  Two are not taken, whatever the
// length: the rule comes from short contexts, where a join costs more than half
// of the work, and long ones lose by it (over 100000 keys 10 sequences in three
// splits read 6.1 TB/s, 11 in one 4.5, 16 in one 5.8).  Many short items need no
// sharing: a wave each (128 sequences of 500 keys: 42.6 us against 47.5).
//
// Row form.  A CU holds eight waves of it (sixteen for heads of 64): two
// workgroups, or one whose halves take every other tile, which is a shorter
// chain.  Up to one workgroup a CU the halves always win (1000 tokens over
// 3000, 32/8 heads of 128: 57 us against 68; 2000 tokens, 16/8 heads of 256: 72
// against 100), and with fewer workgroups the keys are split as well, 384 or
// more a split, until each CU has one (64 tokens over 16000, 32/8 heads of 128:
// 41.7 us in 10 splits, 50.2 in 21).  Beyond that, long chains gain at about
// two rounds of the CUs (2 x 1024 tokens over 6000, 32/8 heads of 128, 520
// workgroups: 190 us against 247; 4000 tokens over 6000, 16/8 heads of 256, 504:
// 288 against 328; the rule takes 480 to 799 for that, and nothing between 520
// and 799 was measured) and lose where one more round begins or chains are short
// (3 x 800 tokens over 3000, 16/8 heads of 256, 308 workgroups: 174 against 152;
// 5 x 800 tokens: 67 against 53; 10000 tokens: 880 against 848).  With heads of
// 64 two such workgroups fit a CU and the limits are wider (4000 tokens, 16
// heads: 54 against 63; 12 x 500 tokens over 2500: 82 against 97, over 500: 25.4
// against 22.8; 20 x 800 tokens: 66 against 60).
int attn_plan(AttnArgs& a, int head_dim, int64_t max_q_len, int64_t max_kv_len) {
  const int64_t max_rows = max_q_len * a.group, all_rows = a.total_q * (int64_t)a.group;
  const int64_t span = keys_seen(a, max_kv_len);
  const int64_t row_items = (all_rows / kAttnRows + 1) * a.n_kv;
  a.key_splits = a.row_splits = 0;
  a.rows_from = 0;
  a.rows_to = 0x7FFFFFFF;
  const int64_t few = head_dim == 64 ? 1 << 19 : head_dim == 128 ? 1 << 18 : 1 << 16;
  if (max_rows <= kAttnKeyRows || (row_items <= 128 && row_items * span <= few)) {
    const int64_t tiles = ceil_div(span + std::min<int64_t>(max_q_len, kAttnKeyRows), 32);
    a.key_tiles = most_tiles(all_rows, a.n_seqs, kAttnKeyRows);
    const int64_t items = (max_rows <= kAttnKeyRows ? a.n_seqs : all_rows / kAttnKeyRows + 1) * a.n_kv;
    a.key_waves = items >= 512 && tiles < 32 ? 1 : head_dim == 256 ? 2 : 4;
    int64_t want = std::min((head_dim == 64 ? 512 : 256) / items, std::max<int64_t>(16, tiles / 64));
    want = std::min({want, tiles / (2 * a.key_waves), 0x7FFFFFFF / ((int64_t)a.key_tiles * a.n_kv)});
    if (want < 3) want = 1;
    a.key_per = (int)ceil_div(tiles, want);
    a.key_splits = (int)ceil_div(tiles, a.key_per);
  } else {
    attn_plan_rows(a, head_dim, max_kv_len);
  }
  return std::max(a.key_splits, a.row_splits);
}

void attn_plan_rows(AttnArgs& a, int head_dim, int64_t max_kv_len) {
  const int64_t all_rows = a.total_q * (int64_t)a.group, span = keys_seen(a, max_kv_len);
  const int keys = head_dim == 256 ? 32 : 64;
  const int64_t tiles = ceil_div(span + kAttnRows / a.group, keys);
  a.row_tiles = most_tiles(all_rows, a.n_seqs, kAttnRows);
  // about as many workgroups have rows: half a tile is lost on a sequence of
  // many rows, and one of few has a tile
  const int64_t groups = std::max<int64_t>(1, (2 * all_rows / kAttnRows + a.n_seqs) * a.n_kv / 2);
  const int64_t want = std::max<int64_t>(1, std::min(256 / groups, tiles * keys / 384));
  a.row_per = (int)ceil_div(tiles, want);
  a.row_splits = (int)ceil_div(tiles, a.row_per);
  const bool even = span >= 2048 && (head_dim == 64 ? groups < 1280 : groups >= 480 && groups < 800);
  a.row_halves = groups <= (head_dim == 64 ? 640 : 288) || even ? 2 : 1;
}

int64_t attn_threads(const AttnArgs& a) {
  const int64_t work = a.key_splits > 0 ? (int64_t)a.key_tiles * a.key_splits * a.n_kv * a.key_waves * 64
                                        : (int64_t)a.row_tiles * a.row_splits * a.n_kv * a.row_halves * 256;
  return std::max(work, std::max(a.key_splits, a.row_splits) > 1 ? (int64_t)a.total_q * a.n_heads * 256 : 0);
}

hipError_t launch_paged_attention(const AttnArgs& a, bool bf16, int head_dim, hipStream_t s) {
  switch (head_dim) {
    case 64: return bf16 ? launch_attn<__bf16, 64>(a, s) : launch_attn<_Float16, 64>(a, s);
    case 128: return bf16 ? launch_attn<__bf16, 128>(a, s) : launch_attn<_Float16, 128>(a, s);
    default: return bf16 ? launch_attn<__bf16, 256>(a, s) : launch_attn<_Float16, 256>(a, s);
  }
}

}  // namespace ttq
