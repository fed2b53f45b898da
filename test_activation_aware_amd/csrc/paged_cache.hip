// Moves of the paged key-value cache: new rows into their pages, and copies
// of whole pages with the rewrite of a block table.  Both only move bytes.
#include "paged_tokens.h"

namespace ttq {

namespace {

// One wave per new token: finds its sequence (64 starts a step, by ballot),
// its page and place, and copies its key and value rows, 16 bytes a lane.  No
// token waits for another.  Bound by memory for prompts (9588 tokens, 8 heads
// of 128: 78.5 MB moved in 15.4 us, 5.1 TB/s), by the chain of four dependent
// loads for a decode step (64 tokens: 3.1 us).
__global__ __launch_bounds__(256) void cache_write_kernel(const char* __restrict__ k, int64_t ldk,
                                                          const char* __restrict__ v, int64_t ldv, char* kc, char* vc,
                                                          int64_t page_bytes, int n_kv, int row_bytes, Places at) {
  const int lane = threadIdx.x & 63;
  const int tok = __builtin_amdgcn_readfirstlane((int)(blockIdx.x * 4 + (threadIdx.x >> 6)));
  if (tok >= at.total_q) return;
  const int s = sequence_of(at, tok);
  if (s < 0) return;  // a token of no sequence
  const int64_t pos = position_of(at, s, tok);
  uint32_t page;
  if (!page_of(at, s, pos, page)) return;  // no place for it
  const int slot = (int)(pos & ((1 << at.page_shift) - 1));
  const int per_head = row_bytes / 16, chunks = n_kv * per_head;
  for (int c = lane; c < chunks; c += 64) {
    const int h = c / per_head, in = c - h * per_head;
    const int64_t to = page * page_bytes + (((int64_t)h << at.page_shift) + slot) * row_bytes + in * 16;
    const uint4 a = *reinterpret_cast<const uint4*>(k + tok * ldk + (int64_t)c * 16);
    const uint4 b = *reinterpret_cast<const uint4*>(v + tok * ldv + (int64_t)c * 16);
    *reinterpret_cast<uint4*>(kc + to) = a;
    *reinterpret_cast<uint4*>(vc + to) = b;
  }
}

constexpr int kPiece = 8192;         // bytes that a workgroup copies
constexpr int kRemapEntries = 4096;  // table entries of a workgroup
constexpr int kRemapPairs = 2048;    // pairs in LDS at a time
constexpr int kSlots = 4096;         // of the hash table of their sources

// Blocks below copy_blocks: one piece of one page of one layer, keys or
// values, bound by memory.  Small pieces in many workgroups keep most loads
// in flight (700 pages of 128 KiB in 4 layers, keys and values, 1.47 GB moved:
// 290 us with 8 KiB a workgroup, 421 with 4, 318 with 16, 408 with 32), and
// stores past the caches leave these to the reads (285 us, 5.15 TB/s; 16 pages
// of 32 KiB in 16 layers 5.1 us against 5.8).
//
// The rest rewrite the block table: each holds 4096 entries in registers and
// looks them up in a hash of the pairs' sources (open addressing in LDS, 2048
// pairs at a time; of equal sources the lowest pair counts, whatever the order
// of the atomics).
typedef uint32_t u4 __attribute__((ext_vector_type(4)));
__global__ __launch_bounds__(256) void copy_pages_kernel(char* k, char* v, int64_t layer_bytes, int64_t page_bytes,
                                                         uint32_t n_pages, int64_t bytes, const int32_t* src,
                                                         const int32_t* dst, int n_pairs, int pieces, int layers,
                                                         unsigned copy_blocks, int32_t* table, int rows, int cols,
                                                         int64_t table_stride) {
  const int tid = threadIdx.x;
  if (blockIdx.x < copy_blocks) {
    unsigned b = blockIdx.x;
    const int piece = b % pieces;
    b /= pieces;
    char* const m = (b & 1) ? v : k;
    b /= 2;
    const int layer = b % layers, pair = b / layers;
    const uint32_t from = (uint32_t)src[pair], to = (uint32_t)dst[pair];
    if (from >= n_pages || to >= n_pages || from == to) return;
    char* const at = m + layer * layer_bytes + (int64_t)piece * kPiece + tid * 16;
    const int n = (int)min<int64_t>(kPiece, bytes - (int64_t)piece * kPiece) - tid * 16;
    const char* s = at + from * page_bytes;
    char* d = at + to * page_bytes;
    constexpr int U = kPiece / 4096;
    u4 x[U];
#pragma unroll
    for (int u = 0; u < U; ++u)
      if (u * 4096 < n) x[u] = *reinterpret_cast<const u4*>(s + u * 4096);
#pragma unroll
    for (int u = 0; u < U; ++u)
      if (u * 4096 < n) __builtin_nontemporal_store(x[u], reinterpret_cast<u4*>(d + u * 4096));
    return;
  }
  __shared__ int key[kSlots], val[kSlots];
  const int64_t total = (int64_t)rows * cols, e0 = (int64_t)(blockIdx.x - copy_blocks) * kRemapEntries;
  constexpr int E = kRemapEntries / 256;
  int32_t entry[E];
  bool found[E];
#pragma unroll
  for (int i = 0; i < E; ++i) {
    const int64_t e = e0 + i * 256 + tid;
    entry[i] = e < total ? table[e / cols * table_stride + e % cols] : -1;
    found[i] = entry[i] < 0;
  }
  for (int p0 = 0; p0 < n_pairs; p0 += kRemapPairs) {
    const int np = min(kRemapPairs, n_pairs - p0);
    for (int i = tid; i < kSlots; i += 256) {
      key[i] = -1;
      val[i] = 0x7FFFFFFF;
    }
    __syncthreads();
    for (int i = tid; i < np; i += 256) {
      const int from = src[p0 + i];
      if ((uint32_t)from >= n_pages || (uint32_t)dst[p0 + i] >= n_pages) continue;
      unsigned h = ((unsigned)from * 2654435761u) >> 20;
      for (;;) {  // at most half of the slots are taken
        const int was = atomicCAS(&key[h], -1, from);
        if (was == -1 || was == from) break;
        h = (h + 1) & (kSlots - 1);
      }
      atomicMin(&val[h], p0 + i);
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < E; ++i) {
      if (found[i]) continue;
      unsigned h = ((unsigned)entry[i] * 2654435761u) >> 20;
      while (key[h] != -1 && key[h] != entry[i]) h = (h + 1) & (kSlots - 1);
      if (key[h] == entry[i]) {
        const int64_t e = e0 + i * 256 + tid;
        table[e / cols * table_stride + e % cols] = dst[val[h]];
        found[i] = true;
      }
    }
    __syncthreads();
  }
}

}  // namespace

int64_t cache_write_threads(int64_t total_q) { return (total_q + 3) / 4 * 256; }

hipError_t launch_cache_write(const void* k, int64_t ldk, const void* v, int64_t ldv, void* kc, void* vc,
                              int64_t page_bytes, int n_kv, int row_bytes, const Places& at, hipStream_t s) {
  cache_write_kernel<<<(unsigned)((at.total_q + 3) / 4), 256, 0, s>>>(
      static_cast<const char*>(k), ldk * 2, static_cast<const char*>(v), ldv * 2, static_cast<char*>(kc),
      static_cast<char*>(vc), page_bytes, n_kv, row_bytes, at);
  return hipGetLastError();
}

int64_t copy_pages_blocks(int64_t bytes, int layers, int n_pairs, int64_t table_entries) {
  return (bytes + kPiece - 1) / kPiece * 2 * layers * n_pairs + (table_entries + kRemapEntries - 1) / kRemapEntries;
}

hipError_t launch_copy_pages(void* k, void* v, int64_t layer_bytes, int layers, int64_t page_bytes, int64_t n_pages,
                             int64_t bytes, const int32_t* src, const int32_t* dst, int n_pairs, int32_t* table,
                             int rows, int cols, int64_t table_stride, hipStream_t s) {
  const int pieces = (int)((bytes + kPiece - 1) / kPiece);
  const int64_t copies = copy_pages_blocks(bytes, layers, n_pairs, 0);
  const int64_t all = copy_pages_blocks(bytes, layers, n_pairs, table != nullptr ? (int64_t)rows * cols : 0);
  copy_pages_kernel<<<(unsigned)all, 256, 0, s>>>(static_cast<char*>(k), static_cast<char*>(v), layer_bytes,
                                                  page_bytes, (uint32_t)n_pages, bytes, src, dst, n_pairs, pieces,
                                                  layers, (unsigned)copies, table, rows, cols, table_stride);
  return hipGetLastError();
}

}  // namespace ttq
