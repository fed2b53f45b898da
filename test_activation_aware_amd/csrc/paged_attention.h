// Arguments and launch forms of the paged attention, shared by its
// translation units.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace ttq {

// Rows of a workgroup of the row form and of the key form.
constexpr int kAttnRows = 128;
constexpr int kAttnKeyRows = 32;

// One call, as the kernels take it.  Row r of sequence s stands for new token
// r / group and query head kvh * group + r % group: the heads that share a
// key head lie side by side, so that a tile of rows reads each key once.
struct AttnArgs {
  const void* q;
  int64_t ldq;
  void* o;
  int64_t ldo;
  float* lse;  // may be NULL
  const char* k;
  const char* v;
  int64_t page_bytes;
  uint32_t n_pages;
  const int32_t* table;
  int64_t table_stride;
  int n_blocks;
  const int32_t* q_start;
  const int32_t* kv_len;
  const int32_t* prefix;  // may be NULL
  const float* slopes;    // may be NULL
  int n_seqs;
  int total_q;
  int n_heads, n_kv, group;
  int page_shift;
  float scale_log2;  // scale * log2(e): scores are kept in units of log 2
  float cap_in;      // 2 scale log2(e) / cap, or 0 without a cap
  float cap_out;     // cap * log2(e)
  bool cap_wide;     // a cap beyond 64: the form that keeps small scores
  int window;        // 0: none
  // How the work is cut (attn_plan); the form with no splits is not used.
  int key_tiles, key_splits, key_per, key_waves;  // key form: tiles of 32 rows; key tiles of 32 in a split
  int row_tiles, row_splits, row_per, row_halves;  // row form: tiles of 128 rows; key tiles in a split
  int rows_from, rows_to;  // sequences of rows_from <= rows < rows_to are this launch's
  float* part_o;    // [splits][total_q * n_heads][D]
  float2* part_ml;  // [splits][total_q * n_heads] running maximum (log 2 units), sum
  int* part_n;      // [total_q * n_heads] splits of the row; NULL without splits
};

// The attention of one head size and type, the join of the splits included.
template <typename T, int D>
hipError_t launch_attn(const AttnArgs& a, hipStream_t s);

// The row form with keys and values in fp16, queries and outputs in bf16.
template <int D>
hipError_t launch_prompts(const AttnArgs& a, hipStream_t s);

// The row form's cut alone: a.row_tiles, row_splits, row_per, row_halves.
void attn_plan_rows(AttnArgs& a, int head_dim, int64_t max_kv_len);

// The same over a cache held in 4 bits (packed_cache.h) by kernels of its own, for
// the sequences of few rows that `a` names.  Either a.key_splits > 0 shares of the
// work of each key head, joined by a second launch (part_o [n_kv][shares][2]
// [rows_of_tile][D], part_ml alike), or a.key_tiles workgroups a key head with a
// tile of rows each.
constexpr int kPackedShare = 12;  // places of a share, at least
struct PackedArgs {
  AttnArgs a;
  bool bf16;         // queries and outputs
  bool once;         // a sequence has one tile of rows: 16, and its keys are read once
  int rows_of_tile;  // 16, or where not once 32 for heads of 64 and 128
};
template <int D>
hipError_t launch_packed(const PackedArgs& p, hipStream_t s);

// Pages of a 4-bit cache, as far as the sequences of a.rows_from rows or more
// read them, in fp16: k, v [pages][kv heads][page size][head dim].
struct ExpandArgs {
  AttnArgs a;  // of the 4-bit cache
  char* k;
  char* v;
  int64_t page_bytes;  // of the 16-bit pages
  int32_t* table;      // [n_seqs][n_blocks], written: block b of sequence s is page s * n_blocks + b; NULL: pages keep their numbers
  int per_seq;         // workgroups of a sequence
  int* part_n;         // of the launch over the 16-bit pages, set to 0 for the other sequences; NULL: it has no splits
};

// One call over a 4-bit cache: sequences of few rows by the kernels for them,
// those of many over 16-bit pages by the row form of the 16-bit attention.
struct PackedCall {
  PackedArgs few;
  bool has_few, has_many;  // either may be left out
  ExpandArgs expand;
  AttnArgs rows;
};
// Fills in how the work is cut, from few.a as made for the 4-bit cache.  `rows` and
// `expand` lack their 16-bit pages.
void packed_plan(PackedCall& c, int head_dim, int64_t max_q_len, int64_t max_kv_len);
int64_t packed_threads(const PackedCall& c);
hipError_t launch_packed_attention(const PackedCall& c, int head_dim, hipStream_t s);

}  // namespace ttq
