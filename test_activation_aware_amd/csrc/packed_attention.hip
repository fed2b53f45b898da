// Attention over a cache held in 4 bits: how a call is cut, and the pages in 16
// bits that its prompts read.
#include <algorithm>

#include "packed_cache.h"
#include "paged_attention_tiles.h"
#include "ttq_internal.h"

namespace ttq {

namespace {

typedef uint32_t u4 __attribute__((ext_vector_type(4)));

int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

// eight codes of one word as 16-bit values: scale * code + lo in 32 bits
template <typename T>
__device__ __forceinline__ u4 values_of(uint32_t w, float scale, float lo) {
  u4 x;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float a = __builtin_fmaf(scale, (float)(w >> (4 * i) & 15u), lo);
    const float b = __builtin_fmaf(scale, (float)(w >> (4 * i + 16) & 15u), lo);
    x[i] = pack2<T>(a, b);
  }
  return x;
}

__device__ __forceinline__ float half_of(uint32_t x, int i) {
  return (float)__builtin_bit_cast(_Float16, (uint16_t)(x >> (16 * i)));
}

// The keys and values of one page and key head a step; a thread reads 16 bytes of
// codes and as much of scales and los, and writes 64 bytes: of K four pieces of a
// token's row, of V the same channels of four tokens.  Bound by the writes.
template <typename T, int D>
__global__ __launch_bounds__(256) void packed_expand_kernel(ExpandArgs e) {
  const AttnArgs& a = e.a;
  constexpr int C = D < 128 ? D : 128, B = D / C, W = C / 32;
  const int s = blockIdx.x / e.per_seq, size = 1 << a.page_shift;
  const int q0 = clampi(a.q_start[s], 0, a.total_q), q1 = clampi(a.q_start[s + 1], 0, a.total_q);
  const int q_len = max(q1 - q0, 0);
  if (q_len * a.group < a.rows_from) return;
  const int kv_len = (int)min<int64_t>(max(a.kv_len[s], 0), min<int64_t>((int64_t)a.n_blocks << a.page_shift, 0x7FFF0000));
  const int prefix = a.prefix != nullptr ? clampi(a.prefix[s], 0, kv_len) : 0;
  // the blocks that some query sees, and the rest of their tiles of 64 keys: the
  // prefix's, then from the first window on
  const int first = (window_begin(kv_len - q_len, a.window) & ~63) >> a.page_shift, end = (kv_len + size - 1) >> a.page_shift;
  const int pre = min((min((prefix + 63) & ~63, kv_len) + size - 1) >> a.page_shift, first);
  const int64_t n = (int64_t)(pre + end - first) * a.n_kv;
  for (int64_t i = blockIdx.x - (int64_t)s * e.per_seq; i < n; i += e.per_seq) {
    const int kvh = (int)(i % a.n_kv), at = (int)(i / a.n_kv), block = at < pre ? at : first + (at - pre);
    const uint32_t from = (uint32_t)a.table[s * a.table_stride + block];
    int64_t to = from;
    if (e.table != nullptr) {
      to = (int64_t)s * a.n_blocks + block;
      if (kvh == 0 && threadIdx.x == 0) e.table[to] = from < a.n_pages ? (int32_t)to : -1;
    }
    if (from >= a.n_pages) continue;
    const int64_t in = from * a.page_bytes + ((int64_t)kvh << a.page_shift) * (D * 5 / 8);
    const int64_t out = to * e.page_bytes + ((int64_t)kvh << a.page_shift) * (D * 2);
    // a unit of 16 tokens holds 16 * B * 4 such pieces of K and as many of V / 16 B
    for (int x = threadIdx.x; x < size * B * 4; x += 256) {
      const int h = x & 3, b = (x >> 2) % B, tok = (x >> 2) / B, t = tok & 15;
      const char* p = a.k + in + (tok & ~15) * (D * 5 / 8) + b * 10 * C;
      char* o = e.k + out + (int64_t)tok * (D * 2) + (b * C + h * 8) * 2;
      uint32_t w[W], q[W];
      if constexpr (W == 4) {
        const u4 y = *reinterpret_cast<const u4*>(p + t * 64 + h * 16), z = *reinterpret_cast<const u4*>(p + 8 * C + t * 16);
#pragma unroll
        for (int k = 0; k < W; ++k) w[k] = y[k], q[k] = z[k];
      } else {
        const uint2 y = *reinterpret_cast<const uint2*>(p + t * 32 + h * 8), z = *reinterpret_cast<const uint2*>(p + 8 * C + t * 8);
        w[0] = y.x, w[1] = y.y, q[0] = z.x, q[1] = z.y;
      }
#pragma unroll
      for (int k = 0; k < W; ++k)
        *reinterpret_cast<u4*>(o + k * 64) = values_of<T>(w[k], half_of(q[k], 0), half_of(q[k], 1));
    }
    for (int x = threadIdx.x; x < size / 4 * (D / 8); x += 256) {
      const int v = x % (D / 8), quad = x / (D / 8), b = v / (C / 8), col = v % (C / 8);
      const char* p = a.v + in + quad / 4 * 16 * (D * 5 / 8) + b * 10 * C;
      char* o = e.v + out + (int64_t)quad * 4 * (D * 2) + v * 16;
      const u4 w = *reinterpret_cast<const u4*>(p + (quad % 4 * (C / 8) + col) * 16);
      const u4 q = *reinterpret_cast<const u4*>(p + 8 * C + (quad % 4 * W + col / 4) * 16);
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const uint32_t word = w[k], sc = q[k / 2], lo = q[2 + k / 2];
        *reinterpret_cast<u4*>(o + k * (D * 2)) = values_of<T>(word, half_of(sc, k & 1), half_of(lo, k & 1));
      }
    }
  }
}

template <typename T>
hipError_t expand(const ExpandArgs& e, int head_dim, hipStream_t s) {
  const unsigned grid = (unsigned)e.a.n_seqs * e.per_seq;
  if (head_dim == 64) packed_expand_kernel<T, 64><<<grid, 256, 0, s>>>(e);
  else if (head_dim == 128) packed_expand_kernel<T, 128><<<grid, 256, 0, s>>>(e);
  else packed_expand_kernel<T, 256><<<grid, 256, 0, s>>>(e);
  return hipGetLastError();
}

}  // namespace

int packed_plan(PackedCall& c, int head_dim, int64_t max_q_len, int64_t max_kv_len) {
  AttnArgs& a = c.few.a;
  const int64_t max_rows = max_q_len * a.group, all_rows = a.total_q * (int64_t)a.group;
  int64_t few = 128;  // rows of a sequence from which its pages are brought to 16 bits
  c.many = max_rows > few;
  c.rows = c.expand.a = a;
  a.rows_from = 0;
  a.rows_to = c.many ? (int)few + 1 : 0x7FFFFFFF;
  a.row_splits = a.other_splits = 0;
  const int64_t rows = std::min(max_rows, few);
  c.few.rows_of_tile = rows <= 16 ? 16 : head_dim == 256 || rows <= 32 ? 32 : 64;
  const int bm = c.few.rows_of_tile;
  const int64_t most = ceil_div(all_rows + (int64_t)a.n_seqs * (bm - 1), bm);
  a.key_tiles = (int)(c.many ? std::min(most, a.n_seqs * ceil_div(few, bm)) : most);
  const int64_t span = std::max<int64_t>(
      1, a.window > 0 && a.prefix == nullptr ? std::min<int64_t>(max_kv_len, a.window) : max_kv_len);
  const int64_t tiles = ceil_div(span + std::min<int64_t>(max_q_len, bm), 32);
  const int64_t items = std::max<int64_t>(1, std::min<int64_t>(all_rows / bm + a.n_seqs, a.n_seqs * ceil_div(rows, bm))) * a.n_kv;
  a.key_waves = items >= 2048 && tiles < 32 ? 1 : 4;
  int64_t groups = 256 * (head_dim == 256 ? (bm == 16 ? 2 : 1) : bm == 16 ? 4 : bm == 32 ? (head_dim == 64 ? 4 : 2) : head_dim == 64 ? 2 : 1);
  int64_t want = std::min({groups / items, tiles / (2 * a.key_waves), 0x7FFFFFFF / ((int64_t)a.key_tiles * a.n_kv)});
  if (want < 2) want = 1;
  a.key_per = (int)ceil_div(tiles, want);
  a.key_splits = (int)ceil_div(tiles, a.key_per);
  c.few.join = !c.many;
  if (!c.many) return a.key_splits;

  c.rows.key_splits = c.rows.key_tiles = 0;
  attn_plan_rows(c.rows, head_dim, max_kv_len);
  c.rows.rows_from = (int)few + 1;
  c.rows.rows_to = 0x7FFFFFFF;
  c.rows.other_splits = a.key_splits;
  c.expand.a.rows_from = (int)few + 1;
  // about 16 workgroups a CU if every sequence has all its blocks
  const int64_t steps = ceil_div(span + max_q_len, int64_t(1) << a.page_shift) * a.n_kv;
  c.expand.per_seq = (int)std::max<int64_t>(1, std::min<int64_t>(steps, 4096 / a.n_seqs));
  return std::max(a.key_splits, c.rows.row_splits);
}

int64_t packed_threads(const PackedCall& c) {
  const AttnArgs& a = c.few.a;
  int64_t n = (int64_t)a.key_tiles * a.key_splits * a.n_kv * a.key_waves * 64;
  if (c.many) n = std::max({n, attn_threads(c.rows), (int64_t)a.n_seqs * c.expand.per_seq * 256});
  else if (a.key_splits > 1) n = std::max(n, (int64_t)a.total_q * a.n_heads * 256);
  return n;
}

hipError_t launch_packed_attention(const PackedCall& c, int head_dim, hipStream_t s) {
  hipError_t e;
  switch (head_dim) {
    case 64: e = launch_packed<64>(c.few, s); break;
    case 128: e = launch_packed<128>(c.few, s); break;
    default: e = launch_packed<256>(c.few, s);
  }
  if (e != hipSuccess || !c.many) return e;
  e = c.few.bf16 ? expand<__bf16>(c.expand, head_dim, s) : expand<_Float16>(c.expand, head_dim, s);
  if (e != hipSuccess) return e;
  return launch_paged_attention(c.rows, c.few.bf16, head_dim, s);
}

}  // namespace ttq
