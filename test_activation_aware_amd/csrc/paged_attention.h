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
  float* part_o;    // [splits][total_q * n_heads][D]
  float2* part_ml;  // [splits][total_q * n_heads] running maximum (log 2 units), sum
  int* part_n;      // [total_q * n_heads] splits of the row; NULL without splits
};

// The attention of one head size and type, the join of the splits included.
template <typename T, int D>
hipError_t launch_attn(const AttnArgs& a, hipStream_t s);

}  // namespace ttq
