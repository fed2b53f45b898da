// Attention of a ragged batch of new tokens over a paged cache:
//   z_ij = scale q_i . k_j, capped: cap tanh(z / cap), biased: z - slope |i - j|
//   o_i = sum_j softmax_j(z_ij) v_j   over the keys j that query i sees
// in one pass over the keys with a running maximum and sum (32 bits).
//
// The scores are formed transposed, S^T = K Q^T (MFMA 32x32x16: keys are the
// rows, queries the columns), so that a lane holds 16 scores of one query per
// 32 keys: maximum and sum are in-lane but for one exchange between the wave's
// halves, the rescale factor of a query is a register of its own lane, and the
// probabilities, rounded to the operand type, are the B operand of
// O^T += V^T P^T without leaving their lane: the MFMA sums over 16 keys in any
// order, so half h takes the keys {4h..4h+3, 8+4h..8+4h+3} that it holds, and
// V is read in the same order by the transposing LDS read.
//
// Keys and values come through LDS by direct-to-LDS loads, the next stage in
// flight while one is worked on.  A load instruction moves 1 KB: whole rows of
// one page (pages hold 16 tokens or more).  Its buffer resource ends at the
// sequence's last key, so that what a page holds beyond it reaches LDS as zeros
// (never NaN), and a page number outside the cache reads nothing.  Infinities
// and NaN among the values of a tile that only some of the rows see are taken
// out in LDS, since 0 x inf would bring them to the other rows; after the last
// tile the rows that see them get them (settle_not_finite).  16-byte chunks are permuted within a row through the source
// addresses: K by the row's low bits (the A operand reads one chunk of 32
// rows), V in groups of 64 bytes (the transposing read takes 64 bytes of 4
// rows), both free of bank conflicts in the 64-bank LDS.
#pragma once

#include <type_traits>
#include <utility>

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

template <int N>
__device__ __forceinline__ void wait_loads() {  // at most N vector loads still in flight
  static_assert(N >= 0 && N < 64, "vmcnt field");
  __builtin_amdgcn_s_waitcnt((N & 15) | ((N >> 4) << 14) | 0x0F70);
}

__device__ __forceinline__ void wait_lds() {  // this wave's LDS operations are done
  asm volatile("" ::: "memory");
  __builtin_amdgcn_s_waitcnt(0xC07F);
}

__device__ __forceinline__ void barrier_only() {
  asm volatile("" ::: "memory");
  __builtin_amdgcn_s_barrier();
  asm volatile("" ::: "memory");
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
    const int upto = back + wave_scan(i >= 0 ? (q_len * a.group + BM - 1) / BM : 0);
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

// KT keys of one key head: K and V into LDS, a wave's share of the loads.
//
// The loads are inline asm: they write no register, and the compiler, which
// cannot tell the stages apart, would otherwise wait for the stage in flight
// before every LDS read.  wait_loads() is the wait for them.
template <int D, int KT, int NW>
struct Loader {
  static constexpr int ROWB = 2 * D, CPR = D / 8, RPL = 1024 / ROWB;
  static constexpr int ROWS = KT / NW;        // rows of a wave
  static constexpr int GR = ROWS < 16 ? ROWS : 16;  // 16 rows lie in one page
  static constexpr int GROUPS = ROWS / GR;
  static constexpr int LPG = GR / RPL;        // loads of a group, K or V
  static constexpr int LOADS = GROUPS * LPG;  // loads of a wave per matrix
  static constexpr int MAT = KT * ROWB;       // bytes of a stage of K or of V
  static_assert(LPG % 2 == 0 && ROWS % GR == 0 && KT % NW == 0 && GR % 4 == 0, "load split");
  const char *k, *v;  // of the key head
  const int32_t* table;
  int kv_len, row0, kvoff[LPG], vvoff;

  static __device__ __forceinline__ int swz_k(int row) { return D == 64 ? (row >> 1) & 7 : row & 15; }
  static __device__ __forceinline__ int swz_v(int row) { return D == 64 ? ((row >> 1) & 1) << 2 : (row & 3) << 2; }

  __device__ __forceinline__ void setup(const AttnArgs& a, const SeqTile& t, int kvh, int share, int lane) {
    const int64_t off = ((int64_t)kvh << a.page_shift) * ROWB;
    k = a.k + off;
    v = a.v + off;
    table = a.table + (int64_t)t.s * a.table_stride;
    kv_len = t.kv_len;
    row0 = share * ROWS;
    const int lrow = lane / CPR, pc = lane % CPR;
#pragma unroll
    for (int i = 0; i < LPG; ++i) kvoff[i] = (i * RPL + lrow) * ROWB + ((pc ^ swz_k(row0 + i * RPL + lrow)) << 4);
    vvoff = lrow * ROWB + ((pc ^ swz_v(lrow)) << 4);
    static_assert(RPL % 4 == 0 || D == 256, "the V permutation repeats every load");
  }
  // the pages of a tile's rows, fetched ahead of issue()
  __device__ __forceinline__ void pages(const AttnArgs& a, int tile, int (&id)[GROUPS]) const {
#pragma unroll
    for (int g = 0; g < GROUPS; ++g)
      id[g] = uniform_load(table, min((tile * KT + row0 + g * GR) >> a.page_shift, a.n_blocks - 1));
  }
  // Two loads.  m0: the LDS address; nothing else in these kernels uses it.
  // s_nop 4: the compiler may have written a register of the resource on the
  // vector unit just before, and a vector memory instruction reads such a
  // register right only five wait states later; nothing but this block sees to
  // that.  A second load from the same resource has them behind it.
  static __device__ __forceinline__ void dma2(__attribute__((ext_vector_type(4))) int rsrc, int voff0, int voff1,
                                              uint32_t lds0, uint32_t lds1) {
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 4\n\tbuffer_load_dwordx4 %2, %4, 0 offen lds\n\t"
                 "s_mov_b32 m0, %1\n\ts_nop 0\n\tbuffer_load_dwordx4 %3, %4, 0 offen lds"
                 :
                 : "s"(lds0), "s"(lds1), "v"(voff0), "v"(voff1), "s"(rsrc)
                 : "memory");
  }
  // K (or V) rows of a tile into the stage
  template <bool IS_V>
  __device__ __forceinline__ void issue(const AttnArgs& a, int tile, const int (&ids)[GROUPS], const char* stage) const {
    typedef int i4 __attribute__((ext_vector_type(4)));
    const uint32_t lds = (uint32_t)(uintptr_t)(__attribute__((address_space(3))) const char*)stage;
#pragma unroll
    for (int g = 0; g < GROUPS; ++g) {
      const int pos = tile * KT + row0 + g * GR;
      const uint32_t id = (uint32_t)ids[g];
      const bool bad = id >= a.n_pages;
      const int rec = uniform(bad ? 0 : clampi(kv_len - pos, 0, GR) * ROWB);
      const uint64_t at = (uint64_t)(uintptr_t)(IS_V ? v : k) + (uint64_t)(bad ? 0 : id) * (uint64_t)a.page_bytes +
                          (uint32_t)((pos & ((1 << a.page_shift) - 1)) * ROWB);
      const i4 r = {uniform((int)(uint32_t)at), uniform((int)((at >> 32) & 0xFFFF)), rec, 0x00020000};
      const uint32_t to = (uint32_t)uniform((int)(lds + (row0 + g * GR) * ROWB));
      auto off = [&](int i) {
        if constexpr (IS_V) return D == 256 && (i & 1) ? (vvoff ^ (8 << 4)) + i * 1024 : vvoff + i * 1024;
        else return kvoff[i];
      };
#pragma unroll
      for (int i = 0; i < LPG; i += 2) dma2(r, off(i), off(i + 1), to + i * 1024, to + (i + 1) * 1024);
    }
  }
};

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

// Infinities and NaN in a pair of 16-bit values: the top bit of each that is one.
template <typename T>
__device__ __forceinline__ uint32_t not_finite(uint32_t x) {
  return ((x & 0x7FFF7FFFu) + (0x8000u - Vec<T>::INF) * 0x10001u) & 0x80008000u;
}
// Zeros in their place in N bytes of LDS, by the wave that loaded them.
// Returns whether there were any: 0 x is NaN for them alone, and a dot product
// with zeros looks at two values in one operation.
template <typename T, int N>
__device__ __forceinline__ bool take_out_not_finite(char* lv, int lane) {
  float c = 0.f;
#pragma unroll
  for (int i = 0; i < N / 1024; ++i) {
    const u4v x = *reinterpret_cast<const u4v*>(lv + i * 1024 + lane * 16);
#pragma unroll
    for (int e = 0; e < 4; ++e) c = Vec<T>::dot_zero(x[e], c);
  }
  if (!__any(c != c)) return false;
#pragma unroll 1
  for (int i = lane * 16; i < N; i += 1024) {
    u4v x = *reinterpret_cast<const u4v*>(lv + i);
#pragma unroll
    for (int e = 0; e < 4; ++e) x[e] &= ~((not_finite<T>(x[e]) >> 15) * 0xFFFFu);
    *reinterpret_cast<u4v*>(lv + i) = x;
  }
  return true;
}
// The lowest n bits of 32, n of any size.
__device__ __forceinline__ uint32_t low_bits(int n) { return n <= 0 ? 0u : n >= 32 ? ~0u : (1u << n) - 1u; }
// The infinities and NaN among V[.][d .. d + 3] of the keys of a share's tiles
// (of the mixed ones alone, or of all) that a query at qpos sees: three bits an
// element, +inf, -inf, NaN.  By a whole wave, each half with a d of its own: a
// lane reads one key of 32, and every row picks those that it sees out of the
// ballots.
template <typename T, int D, int KT>
__device__ __forceinline__ int not_finite_seen(const AttnArgs& a, const SeqTile& t, const KeyTiles& kt, const Share& sh,
                                               int kvh, int qpos, int d, bool mixed_only) {
  constexpr int PER = KT / 32, U = 4;  // steps of a tile; steps whose loads are in flight together
  const int lane = threadIdx.x & 63, lo = window_begin(qpos, a.window);
  const int32_t* table = a.table + (int64_t)t.s * a.table_stride;
  const char* v = a.v + ((int64_t)kvh << a.page_shift) * (2 * D) + d * 2;
  const int steps = (sh.j1 - sh.j0) * PER;
  int kinds = 0;
#pragma unroll 1
  for (int s = 0; s < steps; s += U) {
    uint2 x[U];
    int p0[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int tile = kt.at(sh.j0 + (s + u) / PER) * KT;
      x[u] = make_uint2(0, 0);
      p0[u] = tile + (s + u) % PER * 32;
      const int pos = p0[u] + (lane & 31);
      if (s + u >= steps || pos >= t.kv_len || (mixed_only && !kt.mixed(t, tile, KT))) continue;
      const uint32_t id = (uint32_t)table[pos >> a.page_shift];
      if (id < a.n_pages)
        x[u] = *reinterpret_cast<const uint2*>(v + (int64_t)id * a.page_bytes +
                                               (int64_t)(pos & ((1 << a.page_shift) - 1)) * (2 * D));
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (!__any((not_finite<T>(x[u].x) | not_finite<T>(x[u].y)) != 0)) continue;
      const uint32_t seen = ((low_bits(qpos + 1 - p0[u]) & ~low_bits(lo - p0[u])) | low_bits(t.prefix - p0[u])) &
                            low_bits(t.kv_len - p0[u]);
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const uint32_t bits = (e < 2 ? x[u].x : x[u].y) >> (16 * (e & 1)) & 0xFFFFu;
        auto of_half = [&](bool is) { return ((uint32_t)(__ballot(is) >> (lane & 32)) & seen) != 0; };
        kinds |= (int)of_half(bits == Vec<T>::INF) << 3 * e;
        kinds |= (int)of_half(bits == (Vec<T>::INF | 0x8000u)) << (3 * e + 1);
        kinds |= (int)of_half((bits & 0x7FFFu) > Vec<T>::INF) << (3 * e + 2);
      }
    }
  }
  return kinds;
}
// What one lane has stored of one row (4 elements at d, d + step, ...), set right
// for infinities and NaN among the values that the row sees: those taken out of
// mixed tiles are added, and an element that is not finite gets the sum of them
// all, since in a tile that every row sees 0 x inf, of a probability that has
// become 0, is NaN.  So neither depends on where tiles, halves and shares end.
// A row whose sum is no number (NaN scores) stays as it is.  By whole waves;
// `row`: the lane has one.  Rare, and slow: a second pass over V for each eight
// elements of a wave that are not finite (4096 tokens over 10000, 64/8 heads of
// 128: 1350 us when every head has an infinity at an early key, 1150 without, 6900
// when 128 elements of one have; a scan by each row for itself took 7800 and
// 90000).
template <typename T, int D, int KT>
__device__ __forceinline__ void settle_not_finite(const AttnArgs& a, const SeqTile& t, const KeyTiles& kt, const Share& sh,
                                                  int kvh, int split, int tok, int head, int qpos, int d, int step,
                                                  bool row, bool taken_out, bool number) {
  const int64_t index = (int64_t)(t.q0 + tok) * a.n_heads + head;
  T* out = static_cast<T*>(a.o) + (int64_t)(t.q0 + tok) * a.ldo + (int64_t)head * D;
  float* part = a.part_o + ((int64_t)split * a.total_q * a.n_heads + index) * D;
  auto value = [](int kind) {
    return kind == 0 ? 0.f : kind == 1 ? INFINITY : kind == 2 ? -INFINITY : __builtin_nanf("");
  };
#pragma unroll 1
  for (int i = 0; i < D; i += step, d += step) {
    float x[4] = {0.f, 0.f, 0.f, 0.f};
    if (row && sh.active == 1) {
      const uint2 w = *reinterpret_cast<const uint2*>(out + d);
#pragma unroll
      for (int e = 0; e < 4; ++e)
        x[e] = (float)__builtin_bit_cast(T, (uint16_t)((e < 2 ? w.x : w.y) >> (16 * (e & 1))));
    } else if (row) {
      const float4 w = *reinterpret_cast<const float4*>(part + d);
      x[0] = w.x, x[1] = w.y, x[2] = w.z, x[3] = w.w;
    }
    int set = 0;
    if (taken_out) {
      set = not_finite_seen<T, D, KT>(a, t, kt, sh, kvh, qpos, d, true);
#pragma unroll
      for (int e = 0; e < 4; ++e) x[e] += value(set >> 3 * e & 7);
    }
    if (__any(row && number && (x[0] + x[1] + x[2] + x[3]) * 0.f != 0.f)) {
      int all = not_finite_seen<T, D, KT>(a, t, kt, sh, kvh, qpos, d, false);
      if (!number) all = 0;
#pragma unroll
      for (int e = 0; e < 4; ++e) x[e] = (all >> 3 * e & 7) != 0 ? value(all >> 3 * e & 7) : x[e];
      set |= all;
    }
    if (set == 0 || !row) continue;
    if (sh.active == 1) *reinterpret_cast<uint2*>(out + d) = make_uint2(pack2<T>(x[0], x[1]), pack2<T>(x[2], x[3]));
    else *reinterpret_cast<float4*>(part + d) = make_float4(x[0], x[1], x[2], x[3]);
  }
}

// A wave's 32 query rows: their queries, running maximum and sum, and output
// sums (one row per lane column, its halves in two lanes), and the work on one
// key tile.
template <typename T, int D, int KT, int MODS>
struct Core {
  typedef typename Vec<T>::v8 v8;
  static constexpr int KF = KT / 32, DS = D / 16, DF = D / 32, ROWB = 2 * D;
  static constexpr bool CAP = (MODS & (kCap | kWideCap)) != 0;
  typedef Loader<D, KT, 1> L;
  typedef f16x Scores[KF];
  typedef uint32_t Probs[KF][8];
  v8 q[DS];
  f16x o[DF];
  float m, l, slope;
  int row, qpos, head, tok;
  int hh, first_pos, last_pos, first_lo, full_lo, ksw, kaddr, vaddr, vsw, vchunk;

  __device__ __forceinline__ void setup(const AttnArgs& a, const SeqTile& t, int kvh, int row0, int lane) {
    const int l32 = lane & 31;
    hh = lane >> 5;
    row = row0 + l32;
    const int rc = min(row, t.n_rows - 1);
    tok = rc / a.group;
    head = kvh * a.group + (rc - tok * a.group);
    qpos = t.kv_len - t.q_len + tok;
    const T* p = static_cast<const T*>(a.q) + (int64_t)(t.q0 + tok) * a.ldq + (int64_t)head * D + hh * 8;
#pragma unroll
    for (int s = 0; s < DS; ++s) q[s] = *reinterpret_cast<const v8*>(p + s * 16);
    slope = 0.f;
    if constexpr ((MODS & kBias) != 0) slope = a.slopes[head] * (CAP ? kLog2e : kLog2e / a.scale_log2);
    m = -INFINITY;
    l = 0.f;
#pragma unroll
    for (int d = 0; d < DF; ++d)
#pragma unroll
      for (int e = 0; e < 16; ++e) o[d][e] = 0.f;
    // the wave's first and last query positions, and the first keys that these
    // two see through the window: full_lo .. first_pos are seen by all its rows
    first_pos = uniform(t.kv_len - t.q_len + min(row0, t.n_rows - 1) / a.group);
    last_pos = uniform(t.kv_len - t.q_len + (min(row0 + 32, t.n_rows) - 1) / a.group);
    first_lo = window_begin(first_pos, a.window);
    full_lo = window_begin(last_pos, a.window);
    ksw = L::swz_k(l32);
    kaddr = l32 * ROWB;
    const int kk = (lane & 15) >> 2, c = lane & 3;
    vaddr = (4 * hh + kk) * ROWB + (c & 1) * 8;
    vsw = L::swz_v(kk);
    vchunk = ((lane >> 4) & 1) * 2 + (c >> 1);
  }

  // the key of a lane's score e of fragment f, past 4 * hh
  static __device__ __forceinline__ constexpr int key(int f, int e) { return f * 32 + 8 * (e / 4) + (e & 3); }

  // S^T = K Q^T of the key tile at lk.  A bias without a cap is what the sums
  // start from: z = scale (q k + b), so b = -slope |i - j| / scale.
  __device__ __forceinline__ void scores(const char* lk, int k0, Scores& s) const {
#pragma unroll
    for (int f = 0; f < KF; ++f)
#pragma unroll
      for (int e = 0; e < 16; ++e) s[f][e] = 0.f;
    if constexpr (MODS == kBias) add_bias(k0, s);
#pragma unroll
    for (int st = 0; st < DS; ++st)
#pragma unroll
      for (int f = 0; f < KF; ++f)
        // the permutation is of 16 chunks: the second half of a row of 256 is at a fixed offset
        s[f] = mfma(*reinterpret_cast<const v8*>(lk + f * 32 * ROWB + st / 8 * 256 + kaddr + ((((2 * st) % 16 + hh) ^ ksw) << 4)),
                    q[st], s[f]);
  }
  __device__ __forceinline__ void add_bias(int k0, Scores& s) const {
    if (k0 + KT <= first_pos + 1) {  // no key after any of the queries: linear in the key
      const float b = slope * (float)(k0 + 4 * hh - qpos);
#pragma unroll
      for (int f = 0; f < KF; ++f)
#pragma unroll
        for (int e = 0; e < 16; ++e) s[f][e] += __builtin_fmaf(slope, (float)key(f, e), b);
    } else {
      const float i = (float)(qpos - k0 - 4 * hh);
#pragma unroll
      for (int f = 0; f < KF; ++f)
#pragma unroll
        for (int e = 0; e < 16; ++e) s[f][e] -= slope * fabsf(i - (float)key(f, e));
    }
  }

  // The score q k, capped: cap tanh(x) = cap - 2 cap / (exp(2 x) + 1), in units
  // of log 2.  Its error is about 3e-7 cap whatever the score.
  static __device__ __forceinline__ float cap(const AttnArgs& a, float s) {
    return __builtin_fmaf(-2.f * a.cap_out, __builtin_amdgcn_rcpf(exp2_fast(s * a.cap_in) + 1.f), a.cap_out);
  }
  // The same for caps beyond 64, where that error would pass 2e-5.  Below half of
  // the cap z tanh(x) / x by tanh's series in x^2, whose next term is 9e-8 at 1/4;
  // beyond it 1 - 2 / (exp(2 x) + 1) is 0.46 or more.  A kernel of its own: the
  // series costs registers (24 chunks and decode tokens over up to 4096, 16/8
  // heads of 256, window 1024: 80 us with the form above, 117 with this one, 136
  // and 155 with a branch between them in one kernel).
  static __device__ __forceinline__ float wide_cap(const AttnArgs& a, float s) {
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

  // Cap, bias and mask of the scores; then the running maximum, and with it
  // the sums so far.  Returns the maximum to subtract.
  __device__ __forceinline__ float limit(const AttnArgs& a, const SeqTile& t, int k0, Scores& s) {
    if constexpr (CAP) {
#pragma unroll
      for (int f = 0; f < KF; ++f)
#pragma unroll
        for (int e = 0; e < 16; ++e) s[f][e] = (MODS & kWideCap) != 0 ? wide_cap(a, s[f][e]) : cap(a, s[f][e]);
      if constexpr ((MODS & kBias) != 0) add_bias(k0, s);
    }
    if (!((k0 + KT <= first_pos + 1 && k0 >= full_lo) || k0 + KT <= t.prefix)) {  // not seen by all rows
      const int base = k0 + 4 * hh, hi = qpos - base, lo = window_begin(qpos, a.window) - base, pre = t.prefix - base;
#pragma unroll
      for (int f = 0; f < KF; ++f)
#pragma unroll
        for (int e = 0; e < 16; ++e) {
          const int j = key(f, e);
          const bool seen = (j <= hi && j >= lo) || j < pre;
          s[f][e] = seen ? s[f][e] : -INFINITY;
        }
    }
    float mx = s[0][0];
#pragma unroll
    for (int f = 0; f < KF; ++f)
#pragma unroll
      for (int e = 0; e < 16; ++e) mx = fmaxf(mx, s[f][e]);
    mx = half_max(mx);
    if constexpr (!CAP) mx *= a.scale_log2;
    // The sums are rescaled only when a maximum has grown by more than 8: the
    // probabilities then stay below 2^8, which both operand types hold as well.
    // Each row goes by its own maximum (the others' factor is 1), so that no bit
    // of its output depends on what else its wave works on.
    if (__any(mx > m + 8.f)) {
      const float mn = mx > m + 8.f ? mx : m;
      const float al = mn == -INFINITY ? 1.f : exp2_fast(m - mn);
      l *= al;
#pragma unroll
      for (int d = 0; d < DF; ++d)
#pragma unroll
        for (int e = 0; e < 16; ++e) o[d][e] *= al;
      m = mn;
    }
    return m == -INFINITY ? 0.f : m;
  }

  // The probabilities, summed in 32 bits and rounded to the operand type, two
  // keys to a register.
  __device__ __forceinline__ void probs(const AttnArgs& a, const Scores& s, float mu, Probs& p) {
    const float c = CAP ? 1.f : a.scale_log2;
#pragma unroll
    for (int f = 0; f < KF; ++f)
#pragma unroll
      for (int e = 0; e < 16; e += 2) {
        const float x = exp2_fast(__builtin_fmaf(s[f][e], c, -mu));
        const float y = exp2_fast(__builtin_fmaf(s[f][e + 1], c, -mu));
        l += x + y;
        p[f][e / 2] = pack2<T>(x, y);
      }
  }

  // O^T += V^T P^T
  __device__ __forceinline__ void outputs(const char* lv, const Probs& p) {
#pragma unroll
    for (int f = 0; f < KF; ++f)
#pragma unroll
      for (int st = 0; st < 2; ++st) {
        const uint4 pu = make_uint4(p[f][st * 4], p[f][st * 4 + 1], p[f][st * 4 + 2], p[f][st * 4 + 3]);
#pragma unroll
        for (int d = 0; d < DF; ++d) {
          const char* at = lv + (f * 32 + st * 16) * ROWB + d / 4 * 256 + vaddr + (((d % 4 * 4 + vchunk) ^ vsw) << 4);
          const s4v x = __builtin_amdgcn_ds_read_tr16_b64_v4i16(
              (__attribute__((address_space(3))) s4v*)const_cast<char*>(at));
          const s4v y = __builtin_amdgcn_ds_read_tr16_b64_v4i16(
              (__attribute__((address_space(3))) s4v*)const_cast<char*>(at + 8 * ROWB));
          const v8 vf = __builtin_bit_cast(v8, __builtin_shufflevector(x, y, 0, 1, 2, 3, 4, 5, 6, 7));
          o[d] = mfma(vf, __builtin_bit_cast(v8, pu), o[d]);
        }
      }
  }

  // Key tile `tile`, its K at lk and its V at lv.
  __device__ __forceinline__ void work(const AttnArgs& a, const SeqTile& t, const char* lk, const char* lv, int tile) {
    const int k0 = tile * KT;
    if (k0 >= t.prefix && (k0 > last_pos || k0 + KT <= first_lo)) return;  // seen by other waves' rows only
    Scores s;
    Probs p;
    scores(lk, k0, s);
    const float mu = limit(a, t, k0, s);
    probs(a, s, mu, p);
    outputs(lv, p);
  }

  // What a wave that has all of its rows' keys (of a split) leaves.  Returns
  // whether some of the lane's sums are not finite, and whether the row's sum is
  // a number.
  struct Left {
    bool bad, number;
  };
  __device__ __forceinline__ Left store(const AttnArgs& a, const SeqTile& t, int split, int active) const {
    const float sum = half_sum(l);
    if (row >= t.n_rows) return {false, false};
    const Sink<T, D> to(a, t.q0 + tok, head, split, active, m, sum);
#pragma unroll
    for (int d = 0; d < DF; ++d)
#pragma unroll
      for (int g = 0; g < 4; ++g)
        to.four(d * 32 + g * 8 + hh * 4, o[d][4 * g], o[d][4 * g + 1], o[d][4 * g + 2], o[d][4 * g + 3]);
    if (hh == 0) to.sums(split, active);
    float zero = 0.f;
#pragma unroll
    for (int d = 0; d < DF; ++d)
#pragma unroll
      for (int e = 0; e < 16; ++e) zero = __builtin_fmaf(o[d][e], 0.f, zero);
    return {zero != 0.f, sum == sum};
  }
};

// Row form: four waves of 32 rows share a key tile of KT keys in two stages.
// With HALVES = 2 another four, the second wave of each SIMD, take the same
// rows through every other tile: half the chain of tiles of two workgroups that
// each go through all of them, with as many waves.  The halves are joined in
// LDS.
//
// Bound by the matrix cores, the exponentials and the chip's power together:
// 4096 tokens over 10000, 64/8 heads of 128 in fp16 take 1040 to 1100 us from
// card to card, 0.97 to 1.03 PFLOP/s where a large library product reaches 1.33;
// the matrix cores are busy in 52 % of the cycles, and the same cycles with zeros
// for inputs take 762 us, at a higher clock.  64 rows a wave (a key read feeds two products, one wave a
// SIMD) took 1400 us and more, eight waves on one tile 1015 to 1061 but a
// quarter more on small grids, groups of waves that alternate products and
// exponentials 1204, three or four stages no less than two.  64 keys a tile (32
// for heads of 256) leave two workgroups a CU their two stages each.
template <typename T, int D, int KT, int HALVES, int MODS>
__global__ __launch_bounds__(256 * HALVES, 2) void attn_rows_kernel(AttnArgs a) {
  typedef Loader<D, KT, 4> L;
  constexpr int STAGE = 2 * L::MAT;  // K, then V
  __shared__ __attribute__((aligned(16))) char lds[HALVES * 2 * STAGE];
  __shared__ int left_out[HALVES * 4];
  const int lane = threadIdx.x & 63, wave = uniform((int)threadIdx.x >> 6), half = wave >> 2;
  const int kvh = blockIdx.x % a.n_kv, item = blockIdx.x / a.n_kv, split = item % a.row_splits;
  const SeqTile t = tile_of_block<kAttnRows, HALVES == 1 || D == 64>(a, item / a.row_splits, a.row_tiles, lane);
  if (t.s < 0) return;
  const KeyTiles kt = key_tiles<KT>(a, t, kAttnRows);
  const Share sh = share_of(kt.n, a.row_per, a.row_splits, split);
  if (split >= sh.active) return;

  L ld;
  ld.setup(a, t, kvh, wave & 3, lane);
  Core<T, D, KT, MODS> c;
  c.setup(a, t, kvh, t.row0 + (wave & 3) * 32, lane);
  char* mine = lds + half * 2 * STAGE;
  const int j0 = sh.j0 + half;
  int id[L::GROUPS];
  ld.pages(a, kt.at(j0), id);
  wait_loads<0>();  // the queries, once: their first use is inside the loop
  auto load = [&](int j, const char* stage) {
    ld.template issue<false>(a, kt.at(j), id, stage);
    ld.template issue<true>(a, kt.at(j), id, stage + L::MAT);
    ld.pages(a, kt.at(j + HALVES), id);
  };
  if (j0 < sh.j1) load(j0, mine);
  // a wave past the sequence's rows only loads: its SIMD is the others'
  const bool any_rows = t.row0 + (wave & 3) * 32 < t.n_rows;
  bool left = false;  // some of the loaded values were not finite
  // The barrier says that a tile has landed and that nobody reads the other
  // stage any more: the loads of the next tile go there.
  auto step = [&](int j, char* stage, char* other) {
    wait_loads<0>();
    asm volatile("" ::: "memory");
    if (j < sh.j1 && kt.mixed(t, kt.at(j) * KT, KT) &&
        take_out_not_finite<T, L::ROWS * L::ROWB>(stage + L::MAT + ld.row0 * L::ROWB, lane))
      left = true;
    // what was taken out is out, and the reads of the other stage have returned
    // (their products may still wait: s_barrier itself waits for no LDS read)
    wait_lds();
    barrier_only();
    if (j + HALVES < sh.j1) load(j + HALVES, other);
    if (any_rows && j < sh.j1) c.work(a, t, stage, stage + L::MAT, kt.at(j));
  };
  // both halves take as many steps: the second one's last may be of no tile
  for (int j = j0; j - half < sh.j1; j += 2 * HALVES) {
    step(j, mine, mine + STAGE);
    if (j - half + HALVES < sh.j1) step(j + HALVES, mine + STAGE, mine);
  }
  if (lane == 0) left_out[wave] = left;
  if constexpr (HALVES == 2) {
    static_assert(4 * 32 * D * 4 <= 4 * STAGE, "the sums fit the stages");
    __shared__ float2 ml[4][64];
    float4* sums = reinterpret_cast<float4*>(lds) + (wave & 3) * 32 * D / 4;  // [d / 4][row][4]
    __syncthreads();
    if (half == 1) {
#pragma unroll
      for (int d = 0; d < D / 32; ++d)
#pragma unroll
        for (int g = 0; g < 4; ++g)
          sums[(d * 8 + g * 2 + c.hh) * 32 + (lane & 31)] =
              make_float4(c.o[d][4 * g], c.o[d][4 * g + 1], c.o[d][4 * g + 2], c.o[d][4 * g + 3]);
      ml[wave & 3][lane] = make_float2(c.m, c.l);
    }
    __syncthreads();
    if (half == 1) return;
    const float2 other = ml[wave][lane];
    const float m = fmaxf(c.m, other.x), mu = m == -INFINITY ? 0.f : m;
    const float w0 = exp2_fast(c.m - mu), w1 = exp2_fast(other.x - mu);
    c.m = m;
    c.l = c.l * w0 + other.y * w1;
#pragma unroll
    for (int d = 0; d < D / 32; ++d)
#pragma unroll
      for (int g = 0; g < 4; ++g) {
        const float4 x = sums[(d * 8 + g * 2 + c.hh) * 32 + (lane & 31)];
        c.o[d][4 * g] = c.o[d][4 * g] * w0 + x.x * w1;
        c.o[d][4 * g + 1] = c.o[d][4 * g + 1] * w0 + x.y * w1;
        c.o[d][4 * g + 2] = c.o[d][4 * g + 2] * w0 + x.z * w1;
        c.o[d][4 * g + 3] = c.o[d][4 * g + 3] * w0 + x.w * w1;
      }
  }
  const auto stored = c.store(a, t, split, sh.active);
  if constexpr (HALVES == 1) {
    wait_lds();
    __syncthreads();
  }
  int any = 0;
#pragma unroll
  for (int i = 0; i < HALVES * 4; ++i) any |= left_out[i];
  if (any != 0 || __any(stored.bad))
    settle_not_finite<T, D, KT>(a, t, kt, sh, kvh, split, c.tok, c.head, c.qpos, c.hh * 4, 8, c.row < t.n_rows, any != 0,
                                stored.number);
}

// Key form, for decode tokens and other small batches: NW waves share 32 rows
// and split the keys, 32 a tile, each with stages of its own and no barrier
// until their sums are joined at the end.
//
// Bound by memory: 64 decode tokens, contexts of up to 8192, 64/8 heads of 128
// read 1.03 GB in 194 us, 5.3 TB/s; 3 of up to 131072 with 32/8 heads 1.05 GB
// in 179, 5.9 TB/s, the join of 5.6 us in it (a copy moves 4.9).
template <typename T, int D, int NW, int MODS>
__global__ __launch_bounds__(NW * 64, 1) void attn_keys_kernel(AttnArgs a) {
  constexpr int KT = 32;
  typedef Loader<D, KT, 1> L;
  constexpr int STAGE = 2 * L::MAT;  // K, then V
  __shared__ __attribute__((aligned(16))) char lds[NW * 2 * STAGE];
  __shared__ float2 ml[NW][32];
  __shared__ int left_out[NW];
  const int lane = threadIdx.x & 63, wave = uniform((int)threadIdx.x >> 6);
  const int kvh = blockIdx.x % a.n_kv, item = blockIdx.x / a.n_kv, split = item % a.key_splits;
  const SeqTile t = tile_of_block<kAttnKeyRows, false>(a, item / a.key_splits, a.key_tiles, lane);
  if (t.s < 0) return;
  const KeyTiles kt = key_tiles<KT>(a, t, kAttnKeyRows);
  const Share sh = share_of(kt.n, a.key_per, a.key_splits, split);
  if (split >= sh.active) return;

  L ld;
  ld.setup(a, t, kvh, 0, lane);
  char* mine = lds + wave * 2 * STAGE;
  Core<T, D, KT, MODS> c;
  c.setup(a, t, kvh, t.row0, lane);
  int id[L::GROUPS];
  const int j0 = sh.j0 + wave;
  ld.pages(a, kt.at(j0), id);
  wait_loads<0>();  // the queries, once: their first use is inside the loop
  auto load = [&](int j, const char* stage) {
    ld.template issue<false>(a, kt.at(j), id, stage);
    ld.template issue<true>(a, kt.at(j), id, stage + L::MAT);
    ld.pages(a, kt.at(j + NW), id);
  };
  if (j0 < sh.j1) load(j0, mine);
  bool left = false;  // some of the loaded values were not finite
  auto step = [&](int j, char* stage, char* other) {
    if (j + NW < sh.j1) {
      wait_lds();  // this wave's reads of the other stage have returned
      load(j + NW, other);
      wait_loads<2 * L::LOADS>();
    } else {
      wait_loads<0>();
    }
    asm volatile("" ::: "memory");
    if (kt.mixed(t, kt.at(j) * KT, KT) && take_out_not_finite<T, L::MAT>(stage + L::MAT, lane)) left = true;
    c.work(a, t, stage, stage + L::MAT, kt.at(j));
    asm volatile("" ::: "memory");
  };
  for (int j = j0; j < sh.j1; j += 2 * NW) {
    step(j, mine, mine + STAGE);
    if (j + NW < sh.j1) step(j + NW, mine + STAGE, mine);
  }

  if constexpr (NW == 1) {
    const auto stored = c.store(a, t, split, sh.active);
    if (left || __any(stored.bad))
      settle_not_finite<T, D, KT>(a, t, kt, sh, kvh, split, c.tok, c.head, c.qpos, c.hh * 4, 8, c.row < t.n_rows, left,
                                  stored.number);
  } else {
    const float sum = half_sum(c.l);
    // the waves' sums through their own stages, [d / 4][row][4]
    float4* mo = reinterpret_cast<float4*>(mine);
#pragma unroll
    for (int d = 0; d < D / 32; ++d)
#pragma unroll
      for (int g = 0; g < 4; ++g)
        mo[(d * 8 + g * 2 + c.hh) * 32 + (lane & 31)] =
            make_float4(c.o[d][4 * g], c.o[d][4 * g + 1], c.o[d][4 * g + 2], c.o[d][4 * g + 3]);
    if (c.hh == 0) ml[wave][lane] = make_float2(c.m, sum);
    if (lane == 0) left_out[wave] = left;
    __syncthreads();
    const int row = threadIdx.x & 31;
    const bool is_row = t.row0 + row < t.n_rows;
    float m = -INFINITY, l = 0.f, w[NW];
#pragma unroll
    for (int i = 0; i < NW; ++i) m = fmaxf(m, ml[i][row].x);
    const float mu = m == -INFINITY ? 0.f : m;
#pragma unroll
    for (int i = 0; i < NW; ++i) {
      w[i] = exp2_fast(ml[i][row].x - mu);
      l += w[i] * ml[i][row].y;
    }
    const Sink<T, D> to(a, t.q0 + c.tok, c.head, split, sh.active, m, l);
    float zero = 0.f;
    for (int d4 = is_row ? threadIdx.x >> 5 : D; d4 < D / 4; d4 += NW * 2) {
      float x = 0.f, y = 0.f, z = 0.f, u = 0.f;
#pragma unroll
      for (int i = 0; i < NW; ++i) {
        const float4 v = reinterpret_cast<const float4*>(lds + i * 2 * STAGE)[d4 * 32 + row];
        x += w[i] * v.x;
        y += w[i] * v.y;
        z += w[i] * v.z;
        u += w[i] * v.w;
      }
      to.four(d4 * 4, x, y, z, u);
      zero = __builtin_fmaf(x, 0.f, __builtin_fmaf(y, 0.f, __builtin_fmaf(z, 0.f, __builtin_fmaf(u, 0.f, zero))));
    }
    if (threadIdx.x < 32 && is_row) to.sums(split, sh.active);
    int any = 0;
#pragma unroll
    for (int i = 0; i < NW; ++i) any |= left_out[i];
    if (any != 0 || __any(zero != 0.f))
      settle_not_finite<T, D, KT>(a, t, kt, sh, kvh, split, c.tok, c.head, c.qpos, (threadIdx.x >> 5) * 4, NW * 8, is_row,
                                  any != 0, l == l);
  }
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

template <typename T, int D, int MODS>
hipError_t launch_mods(const AttnArgs& a, hipStream_t s) {
  if (a.key_splits > 0) {
    const unsigned grid = (unsigned)a.key_tiles * a.key_splits * a.n_kv;
    constexpr int NW = D == 256 ? 2 : 4;  // 128 KiB of stages, 64 for heads of 64
    if (a.key_waves > 1) attn_keys_kernel<T, D, NW, MODS><<<grid, NW * 64, 0, s>>>(a);
    else attn_keys_kernel<T, D, 1, MODS><<<grid, 64, 0, s>>>(a);
  } else {
    const unsigned grid = (unsigned)a.row_tiles * a.row_splits * a.n_kv;
    constexpr int KT = D == 256 ? 32 : 64;
    if (a.row_halves == 2) attn_rows_kernel<T, D, KT, 2, MODS><<<grid, 512, 0, s>>>(a);
    else attn_rows_kernel<T, D, KT, 1, MODS><<<grid, 256, 0, s>>>(a);
  }
  hipError_t e = hipGetLastError();
  if (e != hipSuccess || (a.key_splits <= 1 && a.row_splits <= 1)) return e;
  attn_join_kernel<T, D><<<(unsigned)(a.total_q * a.n_heads), 256, 0, s>>>(a);
  return hipGetLastError();
}

}  // namespace

template <typename T, int D>
hipError_t launch_attn(const AttnArgs& a, hipStream_t s) {
  if (a.cap_in == 0.f) return a.slopes != nullptr ? launch_mods<T, D, kBias>(a, s) : launch_mods<T, D, 0>(a, s);
  if (a.cap_wide)
    return a.slopes != nullptr ? launch_mods<T, D, kWideCap | kBias>(a, s) : launch_mods<T, D, kWideCap>(a, s);
  return a.slopes != nullptr ? launch_mods<T, D, kCap | kBias>(a, s) : launch_mods<T, D, kCap>(a, s);
}

}  // namespace ttq
