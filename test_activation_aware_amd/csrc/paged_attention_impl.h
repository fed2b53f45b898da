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

#include "paged_attention_tiles.h"

namespace ttq {

namespace {

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
template <typename T, int D, int KT, typename IO>
__device__ __forceinline__ void settle_not_finite(const AttnArgs& a, const SeqTile& t, const KeyTiles& kt, const Share& sh,
                                                  int kvh, int split, int tok, int head, int qpos, int d, int step,
                                                  bool row, bool taken_out, bool number) {
  const int64_t index = (int64_t)(t.q0 + tok) * a.n_heads + head;
  IO* out = static_cast<IO*>(a.o) + (int64_t)(t.q0 + tok) * a.ldo + (int64_t)head * D;
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
        x[e] = (float)__builtin_bit_cast(IO, (uint16_t)((e < 2 ? w.x : w.y) >> (16 * (e & 1))));
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
    if (sh.active == 1) *reinterpret_cast<uint2*>(out + d) = make_uint2(pack2<IO>(x[0], x[1]), pack2<IO>(x[2], x[3]));
    else *reinterpret_cast<float4*>(part + d) = make_float4(x[0], x[1], x[2], x[3]);
  }
}

// A wave's 32 query rows: their queries, running maximum and sum, and output
// sums (one row per lane column, its halves in two lanes), and the work on one
// key tile.  Queries and outputs are of type IO: bf16 queries that meet keys in
// fp16 are brought into its range by a power of two of their row's largest value,
// which the scores get back.
template <typename T, int D, int KT, int MODS, typename IO = T>
struct Core {
  typedef typename Vec<T>::v8 v8;
  static constexpr bool SCALED = !std::is_same<T, IO>::value;
  static constexpr int KF = KT / 32, DS = D / 16, DF = D / 32, ROWB = 2 * D;
  static constexpr bool CAP = (MODS & (kCap | kWideCap)) != 0;
  typedef Loader<D, KT, 1> L;
  typedef f16x Scores[KF];
  typedef uint32_t Probs[KF][8];
  v8 q[DS];
  f16x o[DF];
  float m, l, slope, up;  // up: SCALED, what a row's queries were divided by
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
    const IO* p = static_cast<const IO*>(a.q) + (int64_t)(t.q0 + tok) * a.ldq + (int64_t)head * D + hh * 8;
    if constexpr (SCALED) load_scaled(p);
    else
#pragma unroll
      for (int s = 0; s < DS; ++s) q[s] = *reinterpret_cast<const v8*>(p + s * 16);
    slope = 0.f;
    if constexpr ((MODS & kBias) != 0) slope = a.slopes[head] * (CAP ? kLog2e : kLog2e / scale(a));
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

  // bf16 queries at p, in fp16
  __device__ __forceinline__ void load_scaled(const IO* p) {
    u4v x[DS];
    uint32_t most = 0;
#pragma unroll
    for (int s = 0; s < DS; ++s) {
      x[s] = *reinterpret_cast<const u4v*>(p + s * 16);
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const uint32_t w = x[s][e];
        most = max(most, max(w & 0x7FFFu, w >> 16 & 0x7FFFu));
      }
    }
    most = max(most, (uint32_t)__shfl_xor((int)most, 32));
    const int shift = shift_of(most);
    up = __builtin_ldexpf(1.f, shift);
#pragma unroll
    for (int s = 0; s < DS; ++s) {
      v8 f;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const uint32_t w = x[s][e];
        f[2 * e] = (T)__builtin_ldexpf(__builtin_bit_cast(float, w << 16), -shift);
        f[2 * e + 1] = (T)__builtin_ldexpf(__builtin_bit_cast(float, w & 0xFFFF0000u), -shift);
      }
      q[s] = f;
    }
  }
  // what a score has to be multiplied by, in units of log 2
  __device__ __forceinline__ float scale(const AttnArgs& a) const {
    if constexpr (SCALED) return a.scale_log2 * up;
    else return a.scale_log2;
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

  // Cap, bias and mask of the scores; then the running maximum, and with it
  // the sums so far.  Returns the maximum to subtract.
  __device__ __forceinline__ float limit(const AttnArgs& a, const SeqTile& t, int k0, Scores& s) {
    if constexpr (CAP) {
#pragma unroll
      for (int f = 0; f < KF; ++f)
#pragma unroll
        for (int e = 0; e < 16; ++e) {
          const float z = SCALED ? s[f][e] * up : s[f][e];
          s[f][e] = (MODS & kWideCap) != 0 ? wide_capped(a, z) : capped(a, z);
        }
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
    if constexpr (!CAP) mx *= scale(a);
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
    const float c = CAP ? 1.f : scale(a);
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
    const Sink<IO, D> to(a, t.q0 + tok, head, split, active, m, sum);
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
template <typename T, int D, int KT, int HALVES, int MODS, typename IO = T>
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
  Core<T, D, KT, MODS, IO> c;
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
    settle_not_finite<T, D, KT, IO>(a, t, kt, sh, kvh, split, c.tok, c.head, c.qpos, c.hh * 4, 8, c.row < t.n_rows, any != 0,
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
      settle_not_finite<T, D, KT, T>(a, t, kt, sh, kvh, split, c.tok, c.head, c.qpos, c.hh * 4, 8, c.row < t.n_rows, left,
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
      settle_not_finite<T, D, KT, T>(a, t, kt, sh, kvh, split, c.tok, c.head, c.qpos, (threadIdx.x >> 5) * 4, NW * 8, is_row,
                                  any != 0, l == l);
  }
}

template <typename T, int D, int MODS, typename IO>
hipError_t launch_rows(const AttnArgs& a, hipStream_t s) {
  const unsigned grid = (unsigned)a.row_tiles * a.row_splits * a.n_kv;
  constexpr int KT = D == 256 ? 32 : 64;
  if (a.row_halves == 2) attn_rows_kernel<T, D, KT, 2, MODS, IO><<<grid, 512, 0, s>>>(a);
  else attn_rows_kernel<T, D, KT, 1, MODS, IO><<<grid, 256, 0, s>>>(a);
  return hipGetLastError();
}
template <typename T, int D>
hipError_t launch_join(const AttnArgs& a, hipStream_t s) {
  attn_join_kernel<T, D><<<(unsigned)(a.total_q * a.n_heads), 256, 0, s>>>(a);
  return hipGetLastError();
}

template <typename T, int D, int MODS>
hipError_t launch_mods(const AttnArgs& a, hipStream_t s) {
  hipError_t e;
  if (a.key_splits > 0) {
    const unsigned grid = (unsigned)a.key_tiles * a.key_splits * a.n_kv;
    constexpr int NW = D == 256 ? 2 : 4;  // 128 KiB of stages, 64 for heads of 64
    if (a.key_waves > 1) attn_keys_kernel<T, D, NW, MODS><<<grid, NW * 64, 0, s>>>(a);
    else attn_keys_kernel<T, D, 1, MODS><<<grid, 64, 0, s>>>(a);
    e = hipGetLastError();
  } else {
    e = launch_rows<T, D, MODS, T>(a, s);
  }
  if (e != hipSuccess || (a.key_splits <= 1 && a.row_splits <= 1)) return e;
  return launch_join<T, D>(a, s);
}

}  // namespace

template <typename T, int D>
hipError_t launch_attn(const AttnArgs& a, hipStream_t s) {
  if (a.cap_in == 0.f) return a.slopes != nullptr ? launch_mods<T, D, kBias>(a, s) : launch_mods<T, D, 0>(a, s);
  if (a.cap_wide)
    return a.slopes != nullptr ? launch_mods<T, D, kWideCap | kBias>(a, s) : launch_mods<T, D, kWideCap>(a, s);
  return a.slopes != nullptr ? launch_mods<T, D, kCap | kBias>(a, s) : launch_mods<T, D, kCap>(a, s);
}

// The row form with fp16 keys and values and bf16 queries and outputs.
template <int D>
hipError_t launch_prompts(const AttnArgs& a, hipStream_t s) {
  hipError_t e;
  const bool bias = a.slopes != nullptr;
  if (a.cap_in == 0.f) e = bias ? launch_rows<_Float16, D, kBias, __bf16>(a, s) : launch_rows<_Float16, D, 0, __bf16>(a, s);
  else if (a.cap_wide)
    e = bias ? launch_rows<_Float16, D, kWideCap | kBias, __bf16>(a, s) : launch_rows<_Float16, D, kWideCap, __bf16>(a, s);
  else e = bias ? launch_rows<_Float16, D, kCap | kBias, __bf16>(a, s) : launch_rows<_Float16, D, kCap, __bf16>(a, s);
  if (e != hipSuccess || a.row_splits <= 1) return e;
  return launch_join<__bf16, D>(a, s);
}

}  // namespace ttq
