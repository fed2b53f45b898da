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

// eight codes of one word as fp16 values: scale * code + lo in 32 bits
__device__ __forceinline__ u4 values_of(uint32_t w, float scale, float lo) {
  u4 x;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float a = __builtin_fmaf(scale, (float)(w >> (4 * i) & 15u), lo);
    const float b = __builtin_fmaf(scale, (float)(w >> (4 * i + 16) & 15u), lo);
    x[i] = pack2<_Float16>(a, b);
  }
  return x;
}

__device__ __forceinline__ float half_of(uint32_t x, int i) {
  return (float)__builtin_bit_cast(_Float16, (uint16_t)(x >> (16 * i)));
}

// A wave takes one page of one key head at a time; a lane reads 16 bytes of codes
// and as much of scales and los, and writes 64 bytes: of K four pieces of a
// token's row, of V the same channels of four tokens.  Bound by the writes: 10000
// tokens of 8 heads of 128, 41 MB written, in 11 to 14 us, the launch among it.  The
// pages are fp16 whatever the type of the queries is: bf16 would cost the values
// three of its bits (outputs 3.9e-3 from 64 bits instead of 1.7e-3).
template <int D>
__global__ __launch_bounds__(256) void packed_expand_kernel(ExpandArgs e) {
  const AttnArgs& a = e.a;
  constexpr int C = D < 128 ? D : 128, B = D / C, W = C / 32;
  const int s = blockIdx.x / e.per_seq, size = 1 << a.page_shift;
  const int q0 = clampi(a.q_start[s], 0, a.total_q), q1 = clampi(a.q_start[s + 1], 0, a.total_q);
  const int q_len = max(q1 - q0, 0);
  if (q_len * a.group < a.rows_from) {
    // the other launches' rows: the join of the prompts' splits has nothing to do with them
    if (e.part_n != nullptr)
      for (int i = (blockIdx.x - s * e.per_seq) * 256 + threadIdx.x; i < q_len * a.n_heads; i += e.per_seq * 256)
        e.part_n[(int64_t)q0 * a.n_heads + i] = 0;
    return;
  }
  const int kv_len = (int)min<int64_t>(max(a.kv_len[s], 0), min<int64_t>((int64_t)a.n_blocks << a.page_shift, 0x7FFF0000));
  const int prefix = a.prefix != nullptr ? clampi(a.prefix[s], 0, kv_len) : 0;
  // the blocks that some query sees, and the rest of their tiles of 64 keys: the
  // prefix's, then from the first window on
  const int first = (window_begin(kv_len - q_len, a.window) & ~63) >> a.page_shift, end = (kv_len + size - 1) >> a.page_shift;
  const int pre = min((min((prefix + 63) & ~63, kv_len) + size - 1) >> a.page_shift, first);
  const int64_t n = (int64_t)(pre + end - first) * a.n_kv;
  const int lane = threadIdx.x & 63, wave = uniform((int)threadIdx.x >> 6);
  for (int64_t i = ((int64_t)blockIdx.x - (int64_t)s * e.per_seq) * 4 + wave; i < n; i += (int64_t)e.per_seq * 4) {
    const int kvh = (int)(i % a.n_kv), at = (int)(i / a.n_kv), block = at < pre ? at : first + (at - pre);
    const uint32_t from = (uint32_t)a.table[s * a.table_stride + block];
    int64_t to = from;
    if (e.table != nullptr) {
      to = (int64_t)s * a.n_blocks + block;
      if (kvh == 0 && lane == 0) e.table[to] = from < a.n_pages ? (int32_t)to : -1;
    }
    if (from >= a.n_pages) continue;
    const int64_t in = from * a.page_bytes + ((int64_t)kvh << a.page_shift) * (D * 5 / 8);
    const int64_t out = to * e.page_bytes + ((int64_t)kvh << a.page_shift) * (D * 2);
    // a unit of 16 tokens holds 16 * B * 4 such pieces of K and as many of V / 16 B
    for (int x = lane; x < size * B * 4; x += 64) {
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
        *reinterpret_cast<u4*>(o + k * 64) = values_of(w[k], half_of(q[k], 0), half_of(q[k], 1));
    }
    for (int x = lane; x < size / 4 * (D / 8); x += 64) {
      const int v = x % (D / 8), quad = x / (D / 8), b = v / (C / 8), col = v % (C / 8);
      const char* p = a.v + in + quad / 4 * 16 * (D * 5 / 8) + b * 10 * C;
      char* o = e.v + out + (int64_t)quad * 4 * (D * 2) + v * 16;
      const u4 w = *reinterpret_cast<const u4*>(p + (quad % 4 * (C / 8) + col) * 16);
      const u4 q = *reinterpret_cast<const u4*>(p + 8 * C + (quad % 4 * W + col / 4) * 16);
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const uint32_t word = w[k], sc = q[k / 2], lo = q[2 + k / 2];
        *reinterpret_cast<u4*>(o + k * (D * 2)) = values_of(word, half_of(sc, k & 1), half_of(lo, k & 1));
      }
    }
  }
}

hipError_t expand(const ExpandArgs& e, int head_dim, hipStream_t s) {
  const unsigned grid = (unsigned)e.a.n_seqs * e.per_seq;
  if (head_dim == 64) packed_expand_kernel<64><<<grid, 256, 0, s>>>(e);
  else if (head_dim == 128) packed_expand_kernel<128><<<grid, 256, 0, s>>>(e);
  else packed_expand_kernel<256><<<grid, 256, 0, s>>>(e);
  return hipGetLastError();
}

}  // namespace

// Two ways.  The kernels for few rows turn the codes into numbers for every 16 or
// 32 rows again; they reach about a third of the matrix cores' rate, and need no
// pages in 16 bits.  The row form of the 16-bit attention has twice that rate when
// there is much to do, behind a pass that writes the pages (3.2 times the bytes of
// the 4-bit ones).  So a call with little work altogether, rows times keys times
// key heads, takes the first way whatever its rows are (16 heads of 64: 1000
// tokens over 3000, twice, 50 us against 53; 4 times 91 against 78.  32/8 heads of
// 128: 1500 tokens 45 against 48; 4 x 1000 94 against 78.  16/8 heads of 256:
// 2000 tokens 81 against 82, 2 x 1000 53 against 56, 8 x 600 95 against 72), twice
// as much where the batch is not of prompts alone: the second way then has three
// launches, none of which fills the GPU.  Of 58 batches of 4 to 32 sequences over up
// to 1500, 3000 or 6000 keys, a quarter to three quarters of them chunks, with 1.1
// to 1.9 times that work, the first way took 0.84 of the second's time with heads of
// 64 (14 batches, 0.64 to 1.16), 0.87 with 128 (21, 0.71 to 1.18) and 0.73 with 256
// (23, 0.53 to 1.05); it was the slower one where one or two long chunks were nearly
// all of the work (32/8 heads of 64, 1363 tokens beside three decode tokens over
// 3000: 44 us against 38; 8 chunks of up to 141 beside 8 over 6000: 97 against 125).
// Beyond that sequences of more rows than `few` go the second way (64/8 heads of
// 128: 16 x 64 tokens over 4000, 512 rows each, 222 us against 229; 4 x 128 tokens,
// 1024 rows, 116 against 96; 16/8 heads of 256: 8 x 128 tokens over 2000, 256 rows,
// 76 against 108; 8 x 200 120 against 109).
//
// Few rows: 16 a tile when every sequence has one such tile, which then reads its
// keys past the caches (64 decode tokens over up to 8192, 64/8 heads of 128: 83 us
// against 125; 16 x 4 tokens over 4000, 32/8 heads: 30 against 35), and otherwise 32
// (16 for heads of 256, whose sums fill the registers; 16 x 4 tokens over 4000, 64/8
// heads: 41 us against 43; 16 x 16 tokens: 63 against 109).  A workgroup takes one tile and all its keys where that is a short
// chain or where there are many such tiles (q tokens over k keys, n sequences, heads;
// first all keys, then shares: 1 x 1000, n = 8, 32/8 of 128: 11.3 and 11.6 us; 64 x
// 1000, n = 4: 15 and 31; 128 x 2000, n = 4, 16 of 64: 19 and 31; 1 x up to 2000, n =
// 128, 32/8 of 128: 42 and 52; 1 x up to 4096, n = 256: 130 and 143).  Otherwise the
// work of each key head is cut into equal shares across the sequences, and a second
// launch joins what ends inside a tile (shares, then all keys: n = 1, 4000 keys: 12
// and 32; 64 x up to 8192, 64/8 of 128: 82 and 100; 8 x up to 8192, n = 16: 56 and
// 78), as many as two or three workgroups a CU have (64 x up to 8192: 512 shares 83
// us, 768 84, 1024 87; 3 x up to 131072: 74, 77 and 82), four with heads of 64, whose
// tiles are half the bytes (4 x 100000: 1024 shares 106 us, 768 110, 512 131).  One
// wave a workgroup where a sequence has two tiles of keys at most and there are many
// (300 x 60, 32/8 heads of 128: 12 us against 18 with four; 128 x 100, four tiles: 9.6
// against 8.5).
void packed_plan(PackedCall& c, int head_dim, int64_t max_q_len, int64_t max_kv_len) {
  AttnArgs& a = c.few.a;
  const int64_t max_rows = max_q_len * a.group, all_rows = a.total_q * (int64_t)a.group;
  const int64_t span = std::max<int64_t>(
      1, a.window > 0 && a.prefix == nullptr ? std::min<int64_t>(max_kv_len, a.window) : max_kv_len);
  const int64_t few = head_dim == 256 ? 256 : 512;
  const int64_t little = (head_dim == 64 ? 100000000 : head_dim == 128 ? 60000000 : 36000000) *
                         (2 * (int64_t)a.total_q <= a.n_seqs * max_q_len ? 2 : 1);
  c.has_many = max_rows > few && all_rows * a.n_kv > little / span;
  // one sequence is of either kind, whatever the bounds say: it takes one of the two
  c.has_few = !c.has_many || a.n_seqs > 1;
  c.rows = c.expand.a = a;
  a.rows_from = 0;
  a.rows_to = c.has_many ? (int)few + 1 : 0x7FFFFFFF;
  a.row_splits = a.key_splits = 0;
  if (c.has_few) {
    const int64_t rows = c.has_many ? std::min(max_rows, few) : max_rows;
    c.few.once = rows <= 16;
    c.few.rows_of_tile = head_dim == 256 || c.few.once ? 16 : 32;
    const int bm = c.few.rows_of_tile;
    const int64_t most = ceil_div(all_rows + (int64_t)a.n_seqs * (bm - 1), bm);
    a.key_tiles = (int)(c.has_many ? std::min(most, a.n_seqs * ceil_div(few, bm)) : most);
    const int64_t tiles = ceil_div(span + std::min<int64_t>(max_q_len, bm), 32);
    // tiles with rows, about: how many sequences of few rows there are beside prompts is not known
    const int64_t items = a.n_kv * (c.has_many ? a.n_seqs : std::min(all_rows / bm + a.n_seqs, a.n_seqs * ceil_div(rows, bm)));
    const int64_t whole = items >= (c.few.once ? 2048 : 512) ? INT64_MAX : items >= (c.few.once ? 512 : 256) ? 80 : 32;
    if (tiles <= whole) {
      a.key_waves = tiles <= 2 && items >= 1024 ? 1 : 4;
    } else {
      a.key_waves = 4;
      const int groups = head_dim != 64 ? 512 : c.few.once ? 1024 : 768;
      a.key_splits = std::max(1, groups / a.n_kv);
    }
  }
  if (!c.has_many) return;

  c.rows.key_splits = c.rows.key_tiles = 0;
  attn_plan_rows(c.rows, head_dim, max_kv_len);
  c.rows.rows_from = c.expand.a.rows_from = c.has_few ? (int)few + 1 : 0;
  c.rows.rows_to = 0x7FFFFFFF;
  // about 16 workgroups a CU if every sequence has all its blocks
  const int64_t steps = ceil_div(ceil_div(span + max_q_len, int64_t(1) << a.page_shift) * a.n_kv, 4);
  c.expand.per_seq = (int)std::max<int64_t>(1, std::min<int64_t>(steps, 4096 / a.n_seqs));
}

int64_t packed_threads(const PackedCall& c) {
  const AttnArgs& a = c.few.a;
  int64_t n = 0;
  if (c.has_few) {
    n = (int64_t)(a.key_splits > 0 ? a.key_splits : a.key_tiles) * a.n_kv * a.key_waves * 64;
  }
  if (c.has_many) n = std::max({n, attn_threads(c.rows), (int64_t)a.n_seqs * c.expand.per_seq * 256});
  return n;
}

hipError_t launch_packed_attention(const PackedCall& c, int head_dim, hipStream_t s) {
  hipError_t e = hipSuccess;
  if (c.has_few) e = head_dim == 64 ? launch_packed<64>(c.few, s) : head_dim == 128 ? launch_packed<128>(c.few, s) : launch_packed<256>(c.few, s);
  if (e != hipSuccess || !c.has_many) return e;
  e = expand(c.expand, head_dim, s);
  if (e != hipSuccess) return e;
  if (!c.few.bf16) return launch_paged_attention(c.rows, false, head_dim, s);
  return head_dim == 64 ? launch_prompts<64>(c.rows, s) : head_dim == 128 ? launch_prompts<128>(c.rows, s) : launch_prompts<256>(c.rows, s);
}

}  // namespace ttq
