// What the kernels of attention over the paged cache have in common, whatever
// the cache holds: how a batch is cut into tiles of rows, tiles of keys and
// splits, what becomes of a score, and where the sums of a row go.
#pragma once

#include "paged_attention.h"

namespace ttq {

namespace {

typedef _Float16 h8 __attribute__((ext_vector_type(8)));
typedef __bf16 b8 __attribute__((ext_vector_type(8)));
typedef float f2v __attribute__((ext_vector_type(2)));
typedef float f16x __attribute__((ext_vector_type(16)));
typedef short s4v __attribute__((ext_vector_type(4)));
typedef short s8v __attribute__((ext_vector_type(8)));
typedef uint32_t u4v __attribute__((ext_vector_type(4)));

template <typename T>
struct Vec;
template <>
struct Vec<_Float16> {
  typedef _Float16 v2 __attribute__((ext_vector_type(2)));
  typedef h8 v8;
  static constexpr uint32_t INF = 0x7C00;
  static __device__ __forceinline__ float dot_zero(uint32_t x, float c) {
    return __builtin_amdgcn_fdot2(__builtin_bit_cast(v2, x), v2{0, 0}, c, false);
  }
};
template <>
struct Vec<__bf16> {
  typedef __bf16 v2 __attribute__((ext_vector_type(2)));
  typedef b8 v8;
  static constexpr uint32_t INF = 0x7F80;
  static __device__ __forceinline__ float dot_zero(uint32_t x, float c) {
    return __builtin_amdgcn_fdot2_f32_bf16(__builtin_bit_cast(v2, x), v2{(__bf16)0.f, (__bf16)0.f}, c, false);
  }
};

__device__ __forceinline__ f16x mfma(h8 a, h8 b, f16x c) {
  return __builtin_amdgcn_mfma_f32_32x32x16_f16(a, b, c, 0, 0, 0);
}
__device__ __forceinline__ f16x mfma(b8 a, b8 b, f16x c) {
  return __builtin_amdgcn_mfma_f32_32x32x16_bf16(a, b, c, 0, 0, 0);
}

// two floats rounded to nearest even, as one register
template <typename T>
__device__ __forceinline__ uint32_t pack2(float a, float b) {
  const f2v v = {a, b};
  return __builtin_bit_cast(uint32_t, __builtin_convertvector(v, typename Vec<T>::v2));
}

// Infinities and NaN in a pair of 16-bit values: the top bit of each that is one.
template <typename T>
__device__ __forceinline__ uint32_t not_finite(uint32_t x) {
  return ((x & 0x7FFF7FFFu) + (0x8000u - Vec<T>::INF) * 0x10001u) & 0x80008000u;
}

// the other half of the wave's value of the same lane column, joined
__device__ __forceinline__ float half_max(float x) {
  const uint32_t u = __builtin_bit_cast(uint32_t, x);
  const auto r = __builtin_amdgcn_permlane32_swap(u, u, false, false);
  return fmaxf(__builtin_bit_cast(float, (uint32_t)r[0]), __builtin_bit_cast(float, (uint32_t)r[1]));
}
__device__ __forceinline__ float half_sum(float x) {
  const uint32_t u = __builtin_bit_cast(uint32_t, x);
  const auto r = __builtin_amdgcn_permlane32_swap(u, u, false, false);
  return __builtin_bit_cast(float, (uint32_t)r[0]) + __builtin_bit_cast(float, (uint32_t)r[1]);
}

constexpr float kLog2e = 1.44269504088896341f, kLn2 = 0.693147180559945309f;

__device__ __forceinline__ float exp2_fast(float x) { return __builtin_amdgcn_exp2f(x); }

// The power of two that a row of bf16 queries is divided by to meet keys in fp16;
// most: the row's largest magnitude, as its bits.  It comes to 2^15 .. 65280, so
// that values down to 2^-29 of it keep their 8 bits.  Rows whose largest is an
// infinity are divided by the most; the least, 2^-64, keeps biases finite, and the
// queries that lose bits by it have scores too small to matter.
__device__ __forceinline__ int shift_of(uint32_t most) {
  return (int)min(max(most >> 7, 78u), 254u) - 142;
}

__device__ __forceinline__ int clampi(int x, int lo, int hi) { return min(max(x, lo), hi); }

// a value of an index array at a place that is the same for the whole wave:
// a scalar load, which does not wait for the vector loads in flight
__device__ __forceinline__ int uniform_load(const int32_t* p, int64_t i) {
  typedef const __attribute__((address_space(4))) int32_t* constant_ptr;
  return ((constant_ptr)(uintptr_t)p)[i];
}
__device__ __forceinline__ int uniform(int x) { return __builtin_amdgcn_readfirstlane(x); }
__device__ __forceinline__ void* uniform_ptr(const char* p) {
  const uint64_t u = (uint64_t)(uintptr_t)p;
  return (void*)(uintptr_t)(((uint64_t)(uint32_t)uniform((int)(u >> 32)) << 32) | (uint32_t)uniform((int)(uint32_t)u));
}

// A tile of BM rows of one sequence.
struct SeqTile {
  int s;        // sequence, -1: none
  int row0;     // first row of the tile in its sequence
  int n_rows;   // rows of the sequence
  int q0;       // first new token of the sequence in Q
  int q_len, kv_len, prefix;
};
// sum over the lanes up to this one
__device__ __forceinline__ int wave_scan(int x) {
  x += __builtin_amdgcn_update_dpp(0, x, 0x111, 0xF, 0xF, false);  // within rows of 16 lanes: from 1, 2, 4, 8 before
  x += __builtin_amdgcn_update_dpp(0, x, 0x112, 0xF, 0xF, false);
  x += __builtin_amdgcn_update_dpp(0, x, 0x114, 0xF, 0xF, false);
  x += __builtin_amdgcn_update_dpp(0, x, 0x118, 0xF, 0xF, false);
  x += __builtin_amdgcn_update_dpp(0, x, 0x142, 0xA, 0xF, false);  // the last lane of row 0 to row 1, of 2 to 3
  x += __builtin_amdgcn_update_dpp(0, x, 0x143, 0xC, 0xF, false);  // lane 31 to rows 2 and 3
  return x;
}
// The tile at `order`, counted from the last one of the last sequence.  The
// tiles are counted, 64 sequences a step, so that those of a grid that has
// none, an upper bound's rest, come last and together: strewn among the others
// they leave the CUs unevenly filled (32 x 128 tokens over 1300, 16/8 heads of
// 256, window 1024, 512 workgroups where two fit a CU: 97 us against 142).
template <int BM>
__device__ __forceinline__ SeqTile find_tile(const AttnArgs& a, int order, int lane) {
  SeqTile t;
  t.s = -1;
  int back = 0;  // tiles of the sequences before these, counted from the end
  for (int base = 0; base < a.n_seqs; base += 64) {
    // all of a sequence's numbers in one round of loads
    const int i = a.n_seqs - 1 - (base + lane), ic = max(i, 0);
    const int q0 = clampi(a.q_start[ic], 0, a.total_q), q1 = clampi(a.q_start[ic + 1], 0, a.total_q);
    const int kv = a.kv_len[ic], pre = a.prefix != nullptr ? a.prefix[ic] : 0;
    const int q_len = max(q1 - q0, 0);
    const int rows = q_len * a.group;
    const bool mine = i >= 0 && rows >= a.rows_from && rows < a.rows_to;
    const int upto = back + wave_scan(mine ? (rows + BM - 1) / BM : 0);
    const unsigned long long hit = __ballot(upto > order);
    if (hit != 0) {
      const int at = uniform(__builtin_ctzll(hit));
      auto of = [&](int x) { return __builtin_amdgcn_readlane(x, at); };
      t.s = a.n_seqs - 1 - (base + at);
      t.q0 = of(q0);
      t.q_len = of(q_len);
      t.n_rows = t.q_len * a.group;
      t.row0 = (of(upto) - 1 - order) * BM;
      const int64_t room = (int64_t)a.n_blocks << a.page_shift;
      t.kv_len = (int)min<int64_t>(max(of(kv), 0), min<int64_t>(room, 0x7FFF0000));
      t.prefix = clampi(of(pre), 0, t.kv_len);
      return t;
    }
    back = __builtin_amdgcn_readlane(upto, 63);
  }
  return t;
}
// The tile of this workgroup.  The last tiles of a sequence see most keys and
// go first.  Where two workgroups fit a CU (PAIRED), every other round of the
// 256 CUs goes the other way, so that a CU has a long and a short one (5
// prompts, 3316 tokens, 16 heads of 64: 27.3 us against 30.7; 24 chunks and
// decode tokens over up to 4096: 57.1 against 65.2).
template <int BM, bool PAIRED>
__device__ __forceinline__ SeqTile tile_of_block(const AttnArgs& a, int order, int tiles, int lane) {
  if constexpr (PAIRED) {
    const int round = max(1, 256 / a.n_kv), begin = order / round * round;
    if ((order / round) & 1) order = min(begin + round, tiles) - 1 - (order - begin);
  }
  return find_tile<BM>(a, order, lane);
}

// The key tiles (KT keys each) that some row of a tile sees: na tiles from 0
// (the prefix), then tiles first, first + 1, ...; n in all.
struct KeyTiles {
  int na, first, n;
  int all_lo, all_hi;  // keys all_lo .. all_hi - 1 are seen by all rows, besides the prefix
  __device__ __forceinline__ int at(int j) const { return j < na ? j : first + (j - na); }
  // some row does not see some key of the n at k0
  __device__ __forceinline__ bool mixed(const SeqTile& t, int k0, int n) const {
    const int end = min(k0 + n, t.kv_len);
    return !(end <= all_hi && k0 >= all_lo) && end > t.prefix;
  }
};
// The first key that a query at pos sees through the window.  Queries before
// position 0 see none through it; their positions stay out of the difference,
// which would pass 32 bits with a window of nearly 2^31.
__device__ __forceinline__ int window_begin(int pos, int window) {
  return window > 0 ? max(0, max(pos, 0) - window + 1) : 0;
}
template <int KT>
__device__ __forceinline__ KeyTiles key_tiles(const AttnArgs& a, const SeqTile& t, int bm) {
  const int p0 = t.kv_len - t.q_len + t.row0 / a.group;  // first and last query position
  const int p1 = t.kv_len - t.q_len + (min(t.row0 + bm, t.n_rows) - 1) / a.group;
  const int hi = max(p1 + 1, 0), lo = window_begin(p0, a.window);
  KeyTiles k;
  k.na = (t.prefix + KT - 1) / KT;
  k.first = max(k.na, lo / KT);
  k.n = k.na + max(0, (hi + KT - 1) / KT - k.first);
  k.all_lo = window_begin(p1, a.window);
  k.all_hi = p0 + 1;
  return k;
}

// One split's share of a tile's n key tiles: at least one split is active.
struct Share {
  int j0, j1;
  int active;  // splits that have keys (1 also when there are none)
};
__device__ __forceinline__ Share share_of(int n, int per, int splits, int split) {
  Share s;
  s.active = max(1, min((n + per - 1) / per, splits));
  s.j0 = min(split * per, n);
  s.j1 = split == splits - 1 ? n : min(s.j0 + per, n);  // the last one takes what a too small bound left over
  return s;
}

// What a score becomes besides scaled: bits of the kernels' MODS.
constexpr int kCap = 1, kBias = 2, kWideCap = 4;  // one of the caps at most

// Where the sums of one row go: the output itself when its keys were not
// split, the workspace otherwise.
template <typename T, int D>
struct Sink {
  const AttnArgs& a;
  int64_t index;  // of the row: token * n_heads + head
  float m, l, inv;
  bool last;  // no other split
  T* out;
  float* part;
  __device__ __forceinline__ Sink(const AttnArgs& args, int tok, int head, int split, int active, float max, float sum)
      : a(args), index((int64_t)tok * args.n_heads + head), m(max), l(sum), last(active == 1) {
    inv = l > 0.f ? 1.f / l : l != l ? l : 0.f;
    out = static_cast<T*>(a.o) + (int64_t)tok * a.ldo + (int64_t)head * D;
    part = a.part_o + ((int64_t)split * a.total_q * a.n_heads + index) * D;
  }
  __device__ __forceinline__ void four(int d, float x, float y, float z, float w) const {
    if (last) *reinterpret_cast<uint2*>(out + d) = make_uint2(pack2<T>(x * inv, y * inv), pack2<T>(z * inv, w * inv));
    else *reinterpret_cast<float4*>(part + d) = make_float4(x, y, z, w);
  }
  // by one lane of the row
  __device__ __forceinline__ void sums(int split, int active) const {
    if (last) {
      if (a.lse != nullptr) a.lse[index] = (m + __builtin_log2f(l)) * kLn2;
    } else {
      a.part_ml[(int64_t)split * a.total_q * a.n_heads + index] = make_float2(m, l);
    }
    if (a.part_n != nullptr && split == 0) a.part_n[index] = active;
  }
};

// The score q k, capped: cap tanh(x) = cap - 2 cap / (exp(2 x) + 1), in units
// of log 2.  Its error is about 3e-7 cap whatever the score.
__device__ __forceinline__ float capped(const AttnArgs& a, float s) {
  return __builtin_fmaf(-2.f * a.cap_out, __builtin_amdgcn_rcpf(exp2_fast(s * a.cap_in) + 1.f), a.cap_out);
}
// The same for caps beyond 64, where that error would pass 2e-5.  Below half of
// the cap z tanh(x) / x by tanh's series in x^2, whose next term is 9e-8 at 1/4;
// beyond it 1 - 2 / (exp(2 x) + 1) is 0.46 or more.  A kernel of its own: the
// series costs registers (24 chunks and decode tokens over up to 4096, 16/8
// heads of 256, window 1024: 80 us with the form above, 117 with this one, 136
// and 155 with a branch between them in one kernel).
__device__ __forceinline__ float wide_capped(const AttnArgs& a, float s) {
  const float y = s * a.cap_in, x = y * (0.5f * kLn2), w = x * x;
  float p = __builtin_fmaf(w, 21844.f / 6081075.f, -1382.f / 155925.f);
  p = __builtin_fmaf(w, p, 62.f / 2835.f);
  p = __builtin_fmaf(w, p, -17.f / 315.f);
  p = __builtin_fmaf(w, p, 2.f / 15.f);
  p = __builtin_fmaf(w, p, -1.f / 3.f);
  p = __builtin_fmaf(w, p, 1.f);
  const float far = a.cap_out * __builtin_fmaf(-2.f, __builtin_amdgcn_rcpf(exp2_fast(y) + 1.f), 1.f);
  return w < 0.25f ? s * a.scale_log2 * p : far;
}

// Joins the splits of a row: a workgroup per row, its 1024 / D groups of D / 4
// lanes take every group-th split, so that a row of many splits is read with
// as many loads in flight.
template <typename T, int D>
__global__ __launch_bounds__(256) void attn_join_kernel(AttnArgs a) {
  constexpr int G = 1024 / D, L = D / 4;
  __shared__ float4 sums[G][L];
  __shared__ float weight[G];
  const int64_t rows = (int64_t)a.total_q * a.n_heads, at = blockIdx.x;
  const int n = min(uniform_load(a.part_n, at), max(a.key_splits, a.row_splits));
  const int tok = (int)(at / a.n_heads);
  // rows of no sequence have no splits, whatever the workspace holds there
  if (tok < uniform_load(a.q_start, 0) || tok >= uniform_load(a.q_start, a.n_seqs)) return;
  if (n <= 1) return;  // written where it belongs already
  const int g = threadIdx.x / L, lane = threadIdx.x % L;
  float m = -INFINITY;
  for (int s = 0; s < n; ++s) m = fmaxf(m, a.part_ml[s * rows + at].x);
  const float mu = m == -INFINITY ? 0.f : m;
  float l = 0.f;
  float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
  for (int s = g; s < n; s += G) {
    const float2 ml = a.part_ml[s * rows + at];
    const float4 p = *reinterpret_cast<const float4*>(a.part_o + (s * rows + at) * D + lane * 4);
    const float w = exp2_fast(ml.x - mu);
    l += w * ml.y;
    // an infinity of a split whose weight is 0 stays one, as within a split
    auto of = [&](float v) { return w == 0.f && v * 0.f != 0.f ? v : w * v; };
    x.x += of(p.x);
    x.y += of(p.y);
    x.z += of(p.z);
    x.w += of(p.w);
  }
  sums[g][lane] = x;
  if (lane == 0) weight[g] = l;
  __syncthreads();
  if (g != 0) return;
  for (int i = 1; i < G; ++i) {
    const float4 y = sums[i][lane];
    x.x += y.x;
    x.y += y.y;
    x.z += y.z;
    x.w += y.w;
    l += weight[i];
  }
  const float inv = l > 0.f ? 1.f / l : l != l ? l : 0.f;
  T* out = static_cast<T*>(a.o) + tok * a.ldo + (at - (int64_t)tok * a.n_heads) * D + lane * 4;
  *reinterpret_cast<uint2*>(out) = make_uint2(pack2<T>(x.x * inv, x.y * inv), pack2<T>(x.z * inv, x.w * inv));
  if (a.lse != nullptr && lane == 0) a.lse[at] = (m + __builtin_log2f(l)) * kLn2;
}

}  // namespace

}  // namespace ttq
