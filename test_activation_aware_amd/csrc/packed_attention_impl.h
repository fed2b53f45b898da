// Attention over a paged cache held in 4 bits, for decode tokens and other few
// rows: the keys and values are turned into 16 bits in registers, where the
// matrix instructions want them, and never pass through LDS.
//
// As in 16 bits (paged_attention_impl.h) the scores are formed transposed, here
// with MFMA 16x16x32: S^T = K Q^T for 16 keys and 16 rows (heads of a group times
// tokens), then O^T += V^T P^T over 32 keys.  Lane (n, h) of the wave, n = lane %
// 16, h = lane / 16, has
//   of K   key n of 16, channels 32 t + 8 h .. + 7 for t = 0, 1, ..: a word for
//          each of the instructions over t, 16 bytes in one load;
//   of S   keys 4 h .. 4 h + 3 and row n: maxima, exponentials and sums are the
//          lane's own, and two such tiles of 16 keys, rounded to 16 bits, are the
//          B operand of the second product as they are;
//   of V   the four keys of each of the two tiles, 4 h .. 4 h + 3, and the 8
//          channels of column n, 16 bytes in one load: byte permutations gather a
//          byte of the four keys, so that the eight instructions over the channels
//          of a column take their A operand from one key order;
//   of O   row n and channels 8 (4 h + i) .. + 7, i = 0 .. 3: 32 in a row.
// (packed_cache.h lays the pages out for this.)  A code becomes a number by the
// conversion of fp8, exactly, then one fused multiply-add with scale and lo,
// rounded to 16 bits once: 11 instructions for 8 values of K, 13 of V.  That is
// fp16 whatever the type of the queries; bf16 queries are brought into its range
// by a power of two of their row's largest value, which the scores get back.
//
// No waves share anything until they join their sums in LDS at the end: each has
// key tiles of its own.
// The maximum is followed when one of a row's four lanes has seen it grow by more
// than 8 (in log 2), so that a key tile needs no exchange between lanes at all.
#pragma once

#include "packed_cache.h"
#include "paged_attention_tiles.h"

namespace ttq {

namespace {

typedef _Float16 h2v __attribute__((ext_vector_type(2)));
typedef float f4v __attribute__((ext_vector_type(4)));
typedef uint32_t u2v __attribute__((ext_vector_type(2)));

__device__ __forceinline__ f4v mfma16(h8 a, h8 b, f4v c) { return __builtin_amdgcn_mfma_f32_16x16x32_f16(a, b, c, 0, 0, 0); }

__device__ __forceinline__ h2v pair(uint32_t x) { return __builtin_bit_cast(h2v, x); }
__device__ __forceinline__ h2v twice(_Float16 x) { return h2v{x, x}; }

// Two neighbouring codes of four that a word holds in a byte each, as numbers: a
// byte of 0 to 15 is an fp8 (e4m3) number of 2^-9 times that, and the conversion
// multiplies by a power of two.  Exact, and one instruction for two, where or-ing
// the codes into a mantissa and subtracting that takes three.
template <bool UPPER>
__device__ __forceinline__ h2v numbers(uint32_t bytes) {
  return __builtin_amdgcn_cvt_scalef32_pk_f16_fp8((int)bytes, 512.f, UPPER);
}
__device__ __forceinline__ h8 join4(h2v a, h2v b, h2v c, h2v d) { return h8{a[0], a[1], b[0], b[1], c[0], c[1], d[0], d[1]}; }
constexpr uint32_t kNibbles = 0x0F0F0F0Fu;

// Channels 0 to 7 in the order that PackedTile::keys leaves them in.
__device__ __forceinline__ h8 in_order(h8 x) { return __builtin_shufflevector(x, x, 0, 4, 1, 5, 2, 6, 3, 7); }
// Slot of a word that holds channel c of its eight.
__device__ __forceinline__ constexpr int slot_of(int c) { return (c & 1) * 4 + c / 2; }

// One tile of 32 keys, as loaded: two halves of 16 tokens.  ONCE: nobody else reads
// them, and the caches are left to others.
template <int D, bool ONCE>
struct PackedTile {
  static constexpr int C = D < 128 ? D : 128, B = D / C;  // channels of a block, blocks of a row
  static constexpr int T = C / 32;                        // instructions over a block's channels
  static constexpr int AUX = ONCE ? 2 : 0;                // nt
  u4v kc[2][B], kp[2][B];  // words of K over t; scale, lo pairs over t
  u4v vc[2][B], vp[2][B];  // words of four keys; scales of four keys, los of four keys

  // Pages of the two halves.
  static __device__ __forceinline__ void pages(const AttnArgs& a, const int32_t* table, int tile, int (&id)[2]) {
#pragma unroll
    for (int u = 0; u < 2; ++u)
      id[u] = uniform_load(table, min((tile * 32 + u * 16) >> a.page_shift, a.n_blocks - 1));
  }
  // Where the two halves lie, from the key head's first byte.  Page numbers outside
  // the cache and halves past the last key read as zeros.
  struct Place {
    int64_t at[2];
    int size[2];
  };
  static __device__ __forceinline__ Place place(const AttnArgs& a, const SeqTile& t, int tile, const int (&ids)[2]) {
    Place p;
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      const int pos = tile * 32 + u * 16;
      const uint32_t id = (uint32_t)ids[u];
      const bool bad = id >= a.n_pages || pos >= t.kv_len;
      p.at[u] = (int64_t)(bad ? 0 : id) * a.page_bytes + (pos & ((1 << a.page_shift) - 1)) * (D * 5 / 8);
      p.size[u] = uniform(bad ? 0 : 10 * D);
    }
    return p;
  }
  static __device__ __forceinline__ __amdgpu_buffer_rsrc_t half_of(const char* head, const Place& p, int u) {
    return __builtin_amdgcn_make_buffer_rsrc(uniform_ptr(head + p.at[u]), 0, p.size[u], 0x00020000);
  }
  __device__ __forceinline__ void load_keys(const char* head, const Place& p, int n, int h) {
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      const auto r = half_of(head, p, u);
#pragma unroll
      for (int b = 0; b < B; ++b) {
        if constexpr (C == 128) {
          kc[u][b] = __builtin_amdgcn_raw_buffer_load_b128(r, n * 64 + h * 16 + b * 10 * C, 0, AUX);
          kp[u][b] = __builtin_amdgcn_raw_buffer_load_b128(r, n * 16 + 8 * C + b * 10 * C, 0, AUX);
        } else {
          const u2v x = __builtin_amdgcn_raw_buffer_load_b64(r, n * 32 + h * 8, 0, AUX);
          const u2v y = __builtin_amdgcn_raw_buffer_load_b64(r, n * 8 + 8 * C, 0, AUX);
          kc[u][b] = u4v{x[0], x[1], 0, 0};
          kp[u][b] = u4v{y[0], y[1], 0, 0};
        }
      }
    }
  }
  __device__ __forceinline__ void load_values(const char* head, const Place& p, int n, int h) {
    const int col = n % (C / 8);
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      const auto r = half_of(head, p, u);
#pragma unroll
      for (int b = 0; b < B; ++b) {
        vc[u][b] = __builtin_amdgcn_raw_buffer_load_b128(r, (h * (C / 8) + col) * 16 + b * 10 * C, 0, AUX);
        vp[u][b] = __builtin_amdgcn_raw_buffer_load_b128(r, (h * T + col / 4) * 16 + 8 * C + b * 10 * C, 0, AUX);
      }
    }
  }
  // The A operand of instruction t over block b's channels: 16 keys, the eight
  // channels of a word in the order of in_order().
  __device__ __forceinline__ h8 keys(int u, int b, int t) const {
    const uint32_t w = kc[u][b][t], p = kp[u][b][t], even = w & kNibbles, odd = w >> 4 & kNibbles;
    const h2v q = pair(p), s = twice(q[0]), lo = twice(q[1]);
    // even bytes hold slots 0 2 4 6, channels 0 4 1 5; odd ones 1 3 5 7, channels 2 6 3 7
    return join4(__builtin_elementwise_fma(numbers<false>(even), s, lo), __builtin_elementwise_fma(numbers<true>(even), s, lo),
                 __builtin_elementwise_fma(numbers<false>(odd), s, lo), __builtin_elementwise_fma(numbers<true>(odd), s, lo));
  }
  // Byte y of the four keys' words, for all four.
  __device__ __forceinline__ void columns(int u, int b, uint32_t (&out)[4]) const {
    const uint32_t w0 = vc[u][b][0], w1 = vc[u][b][1], w2 = vc[u][b][2], w3 = vc[u][b][3];
    const uint32_t a0 = __builtin_amdgcn_perm(w1, w0, 0x05010400u), a1 = __builtin_amdgcn_perm(w1, w0, 0x07030602u);
    const uint32_t b0 = __builtin_amdgcn_perm(w3, w2, 0x05010400u), b1 = __builtin_amdgcn_perm(w3, w2, 0x07030602u);
    out[0] = __builtin_amdgcn_perm(b0, a0, 0x05040100u);
    out[1] = __builtin_amdgcn_perm(b0, a0, 0x07060302u);
    out[2] = __builtin_amdgcn_perm(b1, a1, 0x05040100u);
    out[3] = __builtin_amdgcn_perm(b1, a1, 0x07060302u);
  }
  // The A operand of a channel of each column: the codes of its eight keys, four of each half.
  __device__ __forceinline__ h8 values(int b, uint32_t bytes0, uint32_t bytes1) const {
    const uint32_t s0 = vp[0][b][0], s1 = vp[0][b][1], l0 = vp[0][b][2], l1 = vp[0][b][3];
    const uint32_t s2 = vp[1][b][0], s3 = vp[1][b][1], l2 = vp[1][b][2], l3 = vp[1][b][3];
    return join4(__builtin_elementwise_fma(numbers<false>(bytes0), pair(s0), pair(l0)),
                 __builtin_elementwise_fma(numbers<true>(bytes0), pair(s1), pair(l1)),
                 __builtin_elementwise_fma(numbers<false>(bytes1), pair(s2), pair(l2)),
                 __builtin_elementwise_fma(numbers<true>(bytes1), pair(s3), pair(l3)));
  }
  // Scales and los of the keys past the last one, whatever is there, as zeros.
  __device__ __forceinline__ void end_at(int left, int h) {  // keys of the tile that there are
#pragma unroll
    for (int u = 0; u < 2; ++u)
#pragma unroll
      for (int b = 0; b < B; ++b)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int key = u * 16 + 4 * h + (i & 1) * 2;
          const uint32_t x = vp[u][b][i], keep = (key < left ? 0xFFFFu : 0u) | (key + 1 < left ? 0xFFFF0000u : 0u);
          vp[u][b][i] = x & keep;
        }
  }
  // The values of four keys of code 15; of code 0 they are lo, and the others lie between.
  __device__ __forceinline__ uint32_t most(int u, int b, int i) const {
    const uint32_t s = vp[u][b][i], lo = vp[u][b][i + 2];
    return __builtin_bit_cast(uint32_t, __builtin_elementwise_fma(twice((_Float16)15.f), pair(s), pair(lo)));
  }
  // Scales and los of keys whose values are not all fp16 numbers, as zeros: a key that a row does not see has a
  // probability of 0 there, and 0 x inf would be NaN.  A dot product with zeros looks for them, two an operation (24
  // chunks and decode tokens, heads of 256, window 1024: 129.9 us with it, 128.9 without).
  __device__ __forceinline__ void numbers_only() {
    float c = 0.f;
#pragma unroll
    for (int u = 0; u < 2; ++u)
#pragma unroll
      for (int b = 0; b < B; ++b)
#pragma unroll
        for (int i = 0; i < 2; ++i) c = Vec<_Float16>::dot_zero(most(u, b, i), c);
    if (!__any(c != c)) return;
#pragma unroll
    for (int u = 0; u < 2; ++u)
#pragma unroll
      for (int b = 0; b < B; ++b)
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const uint32_t bad = not_finite<_Float16>(most(u, b, i)), keep = ~((bad - (bad >> 15)) | bad);
          const uint32_t s = vp[u][b][i], lo = vp[u][b][i + 2];
          vp[u][b][i] = s & keep;
          vp[u][b][i + 2] = lo & keep;
        }
  }
};

// 16 R rows of a tile in one wave: queries, running maxima and sums, output sums.
template <int D, int R, int MODS, bool ONCE>
struct PackedCore {
  typedef PackedTile<D, ONCE> Tile;
  static constexpr int B = Tile::B, T = Tile::T;
  static constexpr int O = D / 16;  // instructions over the channels of V: 8 a block, 4 for heads of 64
  static constexpr bool CAP = (MODS & (kCap | kWideCap)) != 0;
  h8 q[R][B][T];
  f4v o[R][O];
  float m[R], l[R], up[R], slope[R];  // m: in the scores' own units, so that a score less the maximum is exact
  int qpos[R];
  int first_pos, full_lo;

  // Row r * 16 + n of the tile: its token and head.
  static __device__ __forceinline__ void row_of(const AttnArgs& a, const SeqTile& t, int kvh, int row, int& tok, int& head) {
    const int rc = min(row, t.n_rows - 1);
    tok = rc / a.group;
    head = kvh * a.group + (rc - tok * a.group);
  }
  __device__ __forceinline__ void setup(const AttnArgs& a, bool bf16, const SeqTile& t, int kvh, int n, int h) {
#pragma unroll
    for (int r = 0; r < R; ++r) {
      int tok, head;
      row_of(a, t, kvh, t.row0 + r * 16 + n, tok, head);
      qpos[r] = t.kv_len - t.q_len + tok;
      const char* p = static_cast<const char*>(a.q) + ((int64_t)(t.q0 + tok) * a.ldq + (int64_t)head * D + h * 8) * 2;
      up[r] = 1.f;
      u4v x[B][T];
#pragma unroll
      for (int b = 0; b < B; ++b)
#pragma unroll
        for (int s = 0; s < T; ++s) x[b][s] = *reinterpret_cast<const u4v*>(p + (b * 128 + s * 32) * 2);
      if (bf16) {
        // the largest magnitude's power of two, over the row's four lanes
        uint32_t most = 0;
#pragma unroll
        for (int b = 0; b < B; ++b)
#pragma unroll
          for (int s = 0; s < T; ++s)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const uint32_t w = x[b][s][e];
              most = max(most, max(w & 0x7FFFu, w >> 16 & 0x7FFFu));
            }
        most = max(most, (uint32_t)__shfl_xor((int)most, 16));
        most = max(most, (uint32_t)__shfl_xor((int)most, 32));
        const int shift = shift_of(most);
        up[r] = __builtin_ldexpf(1.f, shift);
#pragma unroll
        for (int b = 0; b < B; ++b)
#pragma unroll
          for (int s = 0; s < T; ++s) {
            h8 f;
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const uint32_t w = x[b][s][e];
              f[2 * e] = (_Float16)__builtin_ldexpf(__builtin_bit_cast(float, w << 16), -shift);
              f[2 * e + 1] = (_Float16)__builtin_ldexpf(__builtin_bit_cast(float, w & 0xFFFF0000u), -shift);
            }
            q[r][b][s] = in_order(f);
          }
      } else {
#pragma unroll
        for (int b = 0; b < B; ++b)
#pragma unroll
          for (int s = 0; s < T; ++s) {
            const u4v w = x[b][s];
            q[r][b][s] = in_order(__builtin_bit_cast(h8, w));
          }
      }
      slope[r] = (MODS & kBias) != 0 ? a.slopes[head] * kLog2e : 0.f;
      m[r] = -INFINITY;
      l[r] = 0.f;
#pragma unroll
      for (int i = 0; i < O; ++i) o[r][i] = f4v{0.f, 0.f, 0.f, 0.f};
    }
    first_pos = uniform(t.kv_len - t.q_len + min(t.row0, t.n_rows - 1) / a.group);
    const int last_pos = uniform(t.kv_len - t.q_len + (min(t.row0 + 16 * R, t.n_rows) - 1) / a.group);
    full_lo = window_begin(last_pos, a.window);
  }

  // The lane's scores of row r in log 2 units times 1 / unit(): capped, biased, masked.
  __device__ __forceinline__ void limit(const AttnArgs& a, const SeqTile& t, int r, int k0, bool mixed, int h, f4v (&s)[2]) const {
    if constexpr (CAP) {
#pragma unroll
      for (int u = 0; u < 2; ++u)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float z = s[u][i] * up[r];
          s[u][i] = (MODS & kWideCap) != 0 ? wide_capped(a, z) : capped(a, z);
        }
    } else if constexpr ((MODS & kBias) != 0) {
      const float c = a.scale_log2 * up[r];
#pragma unroll
      for (int u = 0; u < 2; ++u)
#pragma unroll
        for (int i = 0; i < 4; ++i) s[u][i] *= c;
    }
    if constexpr ((MODS & kBias) != 0) {
      const float at = (float)(qpos[r] - k0 - 4 * h);
#pragma unroll
      for (int u = 0; u < 2; ++u)
#pragma unroll
        for (int i = 0; i < 4; ++i) s[u][i] -= slope[r] * fabsf(at - (float)(u * 16 + i));
    }
    if (mixed) {
      const int base = k0 + 4 * h, hi = qpos[r] - base, lo = window_begin(qpos[r], a.window) - base, pre = t.prefix - base;
#pragma unroll
      for (int u = 0; u < 2; ++u)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int j = u * 16 + i;
          const bool seen = (j <= hi && j >= lo) || j < pre;
          s[u][i] = seen ? s[u][i] : -INFINITY;
        }
    }
  }
  // What scores that are neither capped nor biased still have to be multiplied by.
  __device__ __forceinline__ float unit(const AttnArgs& a, int r) const { return MODS != 0 ? 1.f : a.scale_log2 * up[r]; }

  typedef f4v Scores[R][2];
  // S^T = K Q^T
  __device__ __forceinline__ void scores(const Tile& x, Scores& s) const {
#pragma unroll
    for (int r = 0; r < R; ++r)
#pragma unroll
      for (int u = 0; u < 2; ++u) s[r][u] = f4v{0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int u = 0; u < 2; ++u)
#pragma unroll
      for (int b = 0; b < B; ++b)
#pragma unroll
        for (int i = 0; i < T; ++i) {
          const h8 k = x.keys(u, b, i);
#pragma unroll
          for (int r = 0; r < R; ++r) s[r][u] = mfma16(k, q[r][b][i], s[r][u]);
        }
  }
  // What the scores of key tile `tile` add to the sums.
  __device__ __forceinline__ void sum_up(const AttnArgs& a, const SeqTile& t, Tile& x, Scores& s, int tile, int n, int h) {
    const int k0 = tile * 32;
    const bool mixed = !((k0 + 32 <= first_pos + 1 && k0 >= full_lo) || k0 + 32 <= t.prefix);  // not seen by all rows
    if (k0 + 32 > t.kv_len) x.end_at(t.kv_len - k0, h);
    if (mixed) x.numbers_only();
    float mx[R];
    bool grown = false;
#pragma unroll
    for (int r = 0; r < R; ++r) {
      limit(a, t, r, k0, mixed, h, s[r]);
      float y = s[r][0][0];
#pragma unroll
      for (int i = 1; i < 8; ++i) y = __builtin_elementwise_maximum(y, s[r][i / 4][i % 4]);  // NaN stays
      mx[r] = y;
      grown = grown || (y > m[r] && !((y - m[r]) * unit(a, r) <= 8.f));
    }
    // The sums are rescaled only when a maximum has grown by more than 8: the
    // probabilities then stay below 2^8.  Each row goes by its own maximum, so
    // that no bit of its output depends on what else its wave works on.
    if (__any(grown)) {
#pragma unroll
      for (int r = 0; r < R; ++r) {
        float y = mx[r];
        y = fmaxf(y, __shfl_xor(y, 16));
        y = fmaxf(y, __shfl_xor(y, 32));
        const float c = unit(a, r), mn = y > m[r] && !((y - m[r]) * c <= 8.f) ? y : m[r];
        const float al = mn == -INFINITY ? 1.f : exp2_fast((m[r] - mn) * c);
        l[r] *= al;
#pragma unroll
        for (int i = 0; i < O; ++i)
#pragma unroll
          for (int e = 0; e < 4; ++e) o[r][i][e] *= al;
        m[r] = mn;
      }
    }
    h8 p[R];
#pragma unroll
    for (int r = 0; r < R; ++r) {
      const float mu = m[r] == -INFINITY ? 0.f : m[r], c = unit(a, r);
      u4v w;
#pragma unroll
      for (int u = 0; u < 2; ++u)
#pragma unroll
        for (int i = 0; i < 4; i += 2) {
          const float y = exp2_fast((s[r][u][i] - mu) * c), z = exp2_fast((s[r][u][i + 1] - mu) * c);
          l[r] += y + z;
          w[u * 2 + i / 2] = pack2<_Float16>(y, z);
        }
      p[r] = __builtin_bit_cast(h8, w);
    }
    // O^T += V^T P^T, byte by byte of the words
    const uint32_t upper = n >= 8 ? 4 : 0;
#pragma unroll
    for (int b = 0; b < B; ++b) {
      uint32_t w0[4], w1[4];
      x.columns(0, b, w0);
      x.columns(1, b, w1);
#pragma unroll
      for (int y = 0; y < 4; ++y) {
        if constexpr (D == 64) {
          // columns 0 to 7 twice: lanes n >= 8 have the upper code of each byte
          const h8 v = x.values(b, w0[y] >> upper & kNibbles, w1[y] >> upper & kNibbles);
#pragma unroll
          for (int r = 0; r < R; ++r) o[r][y] = mfma16(v, p[r], o[r][y]);
        } else {
          const h8 v = x.values(b, w0[y] & kNibbles, w1[y] & kNibbles);
#pragma unroll
          for (int r = 0; r < R; ++r) o[r][b * 8 + 2 * y] = mfma16(v, p[r], o[r][b * 8 + 2 * y]);
          const h8 z = x.values(b, w0[y] >> 4 & kNibbles, w1[y] >> 4 & kNibbles);
#pragma unroll
          for (int r = 0; r < R; ++r) o[r][b * 8 + 2 * y + 1] = mfma16(z, p[r], o[r][b * 8 + 2 * y + 1]);
        }
      }
    }
  }

  // The sums of row r into LDS [channel / 8][row][8], rows STRIDE floats apart
  // in 8, and back out in the order of the channels.
  template <int STRIDE>
  __device__ __forceinline__ void leave(int r, float* to, int n, int h) const {
    if constexpr (D == 64) {
      // instruction y, sum i: column (4 h + i) % 8, slot 2 y or, from h = 2 on, 2 y + 1
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        float* at = to + ((4 * h + i) % 8) * STRIDE + n * 8;
#pragma unroll
        for (int y = 0; y < 4; ++y) {
          const float v = o[r][y][i];
          // slots 2 y and 2 y + 1 hold channels 0 2 | 4 6 | 1 3 | 5 7
          at[(y & 1) * 4 + y / 2 + (h >= 2 ? 2 : 0)] = v;
        }
      }
    } else {
#pragma unroll
      for (int b = 0; b < B; ++b)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          float* at = to + (b * 16 + 4 * h + i) * STRIDE + n * 8;
          float v[8];
#pragma unroll
          for (int c = 0; c < 8; ++c) v[c] = o[r][b * 8 + slot_of(c)][i];
          *reinterpret_cast<float4*>(at) = make_float4(v[0], v[1], v[2], v[3]);
          *reinterpret_cast<float4*>(at + 4) = make_float4(v[4], v[5], v[6], v[7]);
        }
    }
  }
};

// The work of a key head as one list: the batch's sequences, the tiles of 16 R
// rows of each, and for every tile the places of its key tiles.  All tiles of a
// sequence have as many places as its queries together see key tiles, and four
// more, empty, that stand for the time that beginning and ending a tile takes, in
// whole rounds of four waves.  Sequences that are not this launch's have none.
// The numbers of 64 sequences are a lane's each.
template <int BM>
struct WorkList {
  int base;             // the first of the 64
  int64_t before, end;  // places of the sequences before them, and up to their end
  int64_t incl;         // lane: places up to the end of its sequence
  int q0, q_len, kv_len, prefix, places;

  template <int CTRL, int ROWS>
  static __device__ __forceinline__ void add_from(int64_t& x) {
    const uint32_t lo = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)(uint32_t)x, CTRL, ROWS, 0xF, false);
    const uint32_t hi = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)(uint32_t)((uint64_t)x >> 32), CTRL, ROWS, 0xF, false);
    x += (int64_t)(((uint64_t)hi << 32) | lo);
  }
  static __device__ __forceinline__ int64_t of_lane(int64_t x, int lane) {
    const uint32_t lo = (uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)x, lane);
    const uint32_t hi = (uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)((uint64_t)x >> 32), lane);
    return (int64_t)(((uint64_t)hi << 32) | lo);
  }
  // The 64 sequences from base on.
  __device__ __forceinline__ void load(const AttnArgs& a, int lane) {
    const int s = min(base + lane, a.n_seqs - 1);
    q0 = clampi(a.q_start[s], 0, a.total_q);
    q_len = max(clampi(a.q_start[s + 1], 0, a.total_q) - q0, 0);
    const int kv = a.kv_len[s], pre = a.prefix != nullptr ? a.prefix[s] : 0;
    kv_len = (int)min<int64_t>(max(kv, 0), min<int64_t>((int64_t)a.n_blocks << a.page_shift, 0x7FFF0000));
    prefix = clampi(pre, 0, kv_len);
    const int na = (prefix + 31) / 32, first = max(na, window_begin(kv_len - q_len, a.window) / 32);
    places = (na + max(0, (kv_len + 31) / 32 - first) + 7) / 4 * 4;
    const int rows = q_len * a.group;
    const bool mine = base + lane < a.n_seqs && rows >= a.rows_from && rows < a.rows_to;
    incl = mine ? (int64_t)((rows + BM - 1) / BM) * places : 0;
    add_from<0x111, 0xF>(incl);  // as in wave_scan
    add_from<0x112, 0xF>(incl);
    add_from<0x114, 0xF>(incl);
    add_from<0x118, 0xF>(incl);
    add_from<0x142, 0xA>(incl);
    add_from<0x143, 0xC>(incl);
    incl += before;
    end = of_lane(incl, 63);
  }
  // All of it; leaves the last sequences in place.
  __device__ __forceinline__ int64_t total(const AttnArgs& a, int lane) {
    base = 0;
    before = 0;
    load(a, lane);
    while (base + 64 < a.n_seqs) {
      base += 64;
      before = end;
      load(a, lane);
    }
    return end;
  }
  // The tile of place `at`, which is in the list; `begin` its first place, `n` how many it has.
  __device__ __forceinline__ SeqTile find(const AttnArgs& a, int64_t at, int lane, int64_t& begin, int& n) {
    if (at < before) {
      base = 0;
      before = 0;
      load(a, lane);
    }
    while (at >= end) {
      base += 64;
      before = end;
      load(a, lane);
    }
    const int i = uniform(__builtin_ctzll(__ballot(incl > at)));
    const int64_t start = i > 0 ? of_lane(incl, i - 1) : before;
    n = __builtin_amdgcn_readlane(places, i);
    const int64_t tile = (int64_t)((uint64_t)(at - start) / (uint32_t)n);
    begin = start + tile * n;
    SeqTile t;
    t.s = base + i;
    t.q0 = __builtin_amdgcn_readlane(q0, i);
    t.q_len = __builtin_amdgcn_readlane(q_len, i);
    t.n_rows = t.q_len * a.group;
    t.kv_len = __builtin_amdgcn_readlane(kv_len, i);
    t.prefix = __builtin_amdgcn_readlane(prefix, i);
    t.row0 = (int)tile * BM;
    return t;
  }
};

// The places of a workgroup: equal shares of the list, of some rounds or more.
__device__ __forceinline__ int64_t share_size(int64_t total, int shares) {
  return max((int64_t)(((uint64_t)total + shares * 4 - 1) / (uint32_t)(shares * 4)) * 4, (int64_t)kPackedShare);
}

// Where a workgroup's sums of a part of a tile's keys go: it has two such parts
// at most, the end of one tile and the beginning of another.
__device__ __forceinline__ int64_t part_of(const AttnArgs& a, int kvh, int64_t share, int second) {
  return ((int64_t)kvh * a.key_splits + share) * 2 + second;
}

// 8 channels of a row's output, and its sum.
template <int D>
__device__ __forceinline__ void put8(const PackedArgs& p, int tok, int head, int d, const float* x, float inv) {
  char* o = static_cast<char*>(p.a.o) + ((int64_t)tok * p.a.ldo + (int64_t)head * D + d) * 2;
  u4v w;
#pragma unroll
  for (int i = 0; i < 4; ++i)
    w[i] = p.bf16 ? pack2<__bf16>(x[2 * i] * inv, x[2 * i + 1] * inv) : pack2<_Float16>(x[2 * i] * inv, x[2 * i + 1] * inv);
  *reinterpret_cast<u4v*>(o) = w;
}
__device__ __forceinline__ float inverse(float l) { return l > 0.f ? 1.f / l : l != l ? l : 0.f; }
__device__ __forceinline__ void put_sum(const AttnArgs& a, int tok, int head, float m, float l) {
  if (a.lse != nullptr) a.lse[(int64_t)tok * a.n_heads + head] = (m + __builtin_log2f(l)) * kLn2;
}

// A workgroup of NW waves has a tile of rows and a part of its keys at a time.
// SHARES: it goes through its share of the key head's list, which may begin and end
// inside a tile's keys; otherwise it has one tile and all of its keys.
//
// Bound by memory for decode tokens, with waits for loads between: 64 over up to 8192
// (276462 keys, 64/8 heads of 128) in 75 us, 4.7 TB/s of the bytes held, 3 over up to
// 131072 (233476) in 60 us, 5.0 TB/s; the loads alone take 73 us of the first, the arithmetic
// alone 56, and vector instructions keep the SIMDs busy for 40 % of the time.  One
// stage of registers a wave, keys of the next tile asked for as soon as the scores
// have taken this one's, values after the sums: four waves a SIMD hide the rest,
// while two stages leave two waves a SIMD and spill.  For more rows it is bound by
// the codes' conversion (130 us for 24 chunks and decode tokens, 16/8 heads of 256,
// capped: vector instructions for 66 % of the time).
//
// What is rounded to 16 bits: K, V and the probabilities, the operands of the matrix
// instructions, whose next wider type runs at a sixteenth of the rate.  An
// output in fp16 is 3.5e-4 to 5e-4 from 64 bits where rounding the output alone is
// 2.1e-4; in bf16 it is 1.7e-3, the output's own rounding.  Codes that are exact in
// the first product (scale and lo applied to its sums) would give 2.8e-4, at 120
// registers spilled, or with the scale in two parts a third more conversions and the
// queries' sums in a range of their own.
template <int D, int R, int NW, int MODS, bool SHARES, bool ONCE>
__global__ __launch_bounds__(NW * 64, D == 256 ? 2 : R == 1 ? 4 : D == 64 ? 3 : 2)
void packed_keys_kernel(PackedArgs p) {
  const AttnArgs& a = p.a;
  constexpr int STRIDE = 16 * 8 + 4;  // floats of 8 channels of 16 rows
  __shared__ __attribute__((aligned(16))) float sums[NW * D / 8 * STRIDE];
  __shared__ float2 ml[NW][16];
  typedef PackedCore<D, R, MODS, ONCE> Core;
  const int lane = threadIdx.x & 63, wave = uniform((int)threadIdx.x >> 6), n = lane & 15, h = lane >> 4;
  const int kvh = blockIdx.x % a.n_kv, share = blockIdx.x / a.n_kv;
  const int64_t head = ((int64_t)kvh << a.page_shift) * (D * 5 / 8);
  const char *kh = a.k + head, *vh = a.v + head;

  // keys [j0, j1) of the key tiles of tile t; second: where its sums go if that is not all
  auto work = [&](const SeqTile& t, const KeyTiles& kt, int j0, int j1, int second) {
    const int32_t* table = a.table + (int64_t)t.s * a.table_stride;
    typename Core::Tile x;
    Core c;
    int id[2];
    int j = j0 + wave;
    Core::Tile::pages(a, table, kt.at(j), id);
    auto at = Core::Tile::place(a, t, kt.at(j), id);
    Core::Tile::pages(a, table, kt.at(j + NW), id);
    if (j < j1) {
      x.load_keys(kh, at, n, h);
      x.load_values(vh, at, n, h);
    }
    c.setup(a, p.bf16, t, kvh, n, h);
    // The registers of the keys are loaded again as soon as the scores are there,
    // those of the values after the products, so that a tile is always in flight.
    for (; j < j1; j += NW) {
      const bool more = j + NW < j1;
      typename Core::Scores s;
      c.scores(x, s);
      if (more) {
        at = Core::Tile::place(a, t, kt.at(j + NW), id);
        Core::Tile::pages(a, table, kt.at(j + 2 * NW), id);
        x.load_keys(kh, at, n, h);
      }
      c.sum_up(a, t, x, s, kt.at(j), n, h);
      if (more) x.load_values(vh, at, n, h);
    }

    // 16 rows at a time: the waves' sums through LDS, joined in order.
    const bool all = j0 == 0 && j1 == kt.n;
#pragma unroll
    for (int r = 0; r < R; ++r) {
      float l = c.l[r];
      l += __shfl_xor(l, 16);
      l += __shfl_xor(l, 32);
      if (SHARES || r > 0) __syncthreads();
      c.template leave<STRIDE>(r, sums + wave * (D / 8 * STRIDE), n, h);
      if (h == 0) ml[wave][n] = make_float2(c.m[r] * c.unit(a, r), l);
      __syncthreads();
      const int row = threadIdx.x & 15, of = t.row0 + r * 16 + row;
      if (of >= t.n_rows) continue;
      int tok, hd;
      Core::row_of(a, t, kvh, of, tok, hd);
      tok += t.q0;
      float m = -INFINITY, total = 0.f, w[NW];
#pragma unroll
      for (int i = 0; i < NW; ++i) m = fmaxf(m, ml[i][row].x);
      const float mu = m == -INFINITY ? 0.f : m;
#pragma unroll
      for (int i = 0; i < NW; ++i) {
        w[i] = exp2_fast(ml[i][row].x - mu);
        total += w[i] * ml[i][row].y;
      }
      const int64_t part = part_of(a, kvh, share, second) * (16 * R) + r * 16 + row;
      for (int d8 = threadIdx.x >> 4; d8 < D / 8; d8 += NW * 4) {
        float f[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) f[e] = 0.f;
#pragma unroll
        for (int i = 0; i < NW; ++i) {
          const float4* v = reinterpret_cast<const float4*>(sums + (i * (D / 8) + d8) * STRIDE + row * 8);
          const float4 v0 = v[0], v1 = v[1];
          f[0] += w[i] * v0.x, f[1] += w[i] * v0.y, f[2] += w[i] * v0.z, f[3] += w[i] * v0.w;
          f[4] += w[i] * v1.x, f[5] += w[i] * v1.y, f[6] += w[i] * v1.z, f[7] += w[i] * v1.w;
        }
        if (!SHARES || all) {
          put8<D>(p, tok, hd, d8 * 8, f, inverse(total));
          if (d8 == 0) put_sum(a, tok, hd, m, total);
        } else {
          float4* o = reinterpret_cast<float4*>(a.part_o + part * D + d8 * 8);
          o[0] = make_float4(f[0], f[1], f[2], f[3]);
          o[1] = make_float4(f[4], f[5], f[6], f[7]);
          if (d8 == 0) a.part_ml[part] = make_float2(m, total);
        }
      }
    }
  };

  if constexpr (SHARES) {
    WorkList<16 * R> list;
    const int64_t total = list.total(a, lane), per = share_size(total, a.key_splits);
    const int64_t begin = share * per, end = min(begin + per, total);
    for (int64_t at = begin; at < end;) {
      int64_t first;
      int places;
      const SeqTile t = list.find(a, at, lane, first, places);
      const KeyTiles kt = key_tiles<32>(a, t, 16 * R);
      const int64_t last = min(first + places, end);
      const int j0 = min((int)(at - first), kt.n), j1 = min((int)(last - first), kt.n);
      if (j0 < j1 || at == first) work(t, kt, j0, j1, at > begin ? 1 : 0);
      at = last;
      if (at < end) list.load(a, lane);  // again, rather than held in registers meanwhile
    }
  } else {
    const SeqTile t = find_tile<16 * R>(a, share, lane);
    if (t.s < 0) return;
    const KeyTiles kt = key_tiles<32>(a, t, 16 * R);
    work(t, kt, 0, kt.n, 0);
  }
}

// Joins the parts of the tiles that shares end in.  The workgroup of a share has
// the tile that goes on behind its end, unless that began in an earlier one; a wave
// has every fourth row, its 256 / D groups of lanes every so many parts.  Bound by a
// launch and a chain of loads: 5 us.
template <int D, int R>
__global__ __launch_bounds__(256) void packed_join_kernel(PackedArgs p) {
  const AttnArgs& a = p.a;
  constexpr int L = D / 4, G = 64 / L;
  const int lane = threadIdx.x & 63, wave = uniform((int)threadIdx.x >> 6);
  const int kvh = blockIdx.x % a.n_kv, share = blockIdx.x / a.n_kv;
  WorkList<16 * R> list;
  const int64_t total = list.total(a, lane), per = share_size(total, a.key_splits), end = (share + 1) * per;
  if (end >= total) return;
  int64_t first;
  int places;
  const SeqTile t = list.find(a, end, lane, first, places);
  const KeyTiles kt = key_tiles<32>(a, t, 16 * R);
  if (first >= end || first < end - per || first + kt.n <= end) return;
  const int n = (int)((first + kt.n - 1) / per - share) + 1;  // shares with keys of the tile
  auto part = [&](int i, int row) {
    return part_of(a, kvh, share + i, i == 0 && first > end - per ? 1 : 0) * (16 * R) + row;
  };
  for (int row = wave; row < 16 * R && t.row0 + row < t.n_rows; row += 4) {
    // a running maximum, so that a part's maximum and its sums are one round of loads
    float m = -INFINITY, l = 0.f;
    float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
    auto add = [&](float om, float ol, float4 v) {
      const float mn = fmaxf(m, om), mu = mn == -INFINITY ? 0.f : mn;
      const float w0 = exp2_fast(m - mu), w1 = exp2_fast(om - mu);
      m = mn;
      l = l * w0 + ol * w1;
      x.x = x.x * w0 + v.x * w1;
      x.y = x.y * w0 + v.y * w1;
      x.z = x.z * w0 + v.z * w1;
      x.w = x.w * w0 + v.w * w1;
    };
    for (int i = lane / L; i < n; i += 4 * G) {
      float2 ml[4];
      float4 v[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const int64_t at = part(min(i + k * G, n - 1), row);
        ml[k] = a.part_ml[at];
        v[k] = *reinterpret_cast<const float4*>(a.part_o + at * D + lane % L * 4);
      }
#pragma unroll
      for (int k = 0; k < 4; ++k)
        if (i + k * G < n) add(ml[k].x, ml[k].y, v[k]);
    }
#pragma unroll
    for (int o = L; o < 64; o *= 2)
      add(__shfl_xor(m, o), __shfl_xor(l, o),
          make_float4(__shfl_xor(x.x, o), __shfl_xor(x.y, o), __shfl_xor(x.z, o), __shfl_xor(x.w, o)));
    if (lane >= L) continue;
    int tok, hd;
    PackedCore<D, R, 0, false>::row_of(a, t, kvh, t.row0 + row, tok, hd);
    tok += t.q0;
    const float inv = inverse(l);
    char* out = static_cast<char*>(a.o) + ((int64_t)tok * a.ldo + (int64_t)hd * D + lane * 4) * 2;
    *reinterpret_cast<uint2*>(out) =
        p.bf16 ? make_uint2(pack2<__bf16>(x.x * inv, x.y * inv), pack2<__bf16>(x.z * inv, x.w * inv))
               : make_uint2(pack2<_Float16>(x.x * inv, x.y * inv), pack2<_Float16>(x.z * inv, x.w * inv));
    if (lane == 0) put_sum(a, tok, hd, m, l);
  }
}

template <int D, int R, int MODS, bool ONCE>
hipError_t launch_packed_rows(const PackedArgs& p, hipStream_t s) {
  const AttnArgs& a = p.a;
  if (a.key_splits == 0) {
    const unsigned grid = (unsigned)a.key_tiles * a.n_kv;
    if (a.key_waves > 1) packed_keys_kernel<D, R, 4, MODS, false, ONCE><<<grid, 256, 0, s>>>(p);
    else packed_keys_kernel<D, R, 1, MODS, false, ONCE><<<grid, 64, 0, s>>>(p);
    return hipGetLastError();
  }
  const unsigned grid = (unsigned)a.key_splits * a.n_kv;
  packed_keys_kernel<D, R, 4, MODS, true, ONCE><<<grid, 256, 0, s>>>(p);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  packed_join_kernel<D, R><<<grid, 256, 0, s>>>(p);
  return hipGetLastError();
}
template <int D, int MODS>
hipError_t launch_packed_mods(const PackedArgs& p, hipStream_t s) {
  if (p.once) return launch_packed_rows<D, 1, MODS, true>(p, s);
  return launch_packed_rows<D, D == 256 ? 1 : 2, MODS, false>(p, s);
}

}  // namespace

template <int D>
hipError_t launch_packed(const PackedArgs& p, hipStream_t s) {
  const AttnArgs& a = p.a;
  const bool bias = a.slopes != nullptr;
  if (a.cap_in == 0.f) return bias ? launch_packed_mods<D, kBias>(p, s) : launch_packed_mods<D, 0>(p, s);
  if (a.cap_wide) return bias ? launch_packed_mods<D, kWideCap | kBias>(p, s) : launch_packed_mods<D, kWideCap>(p, s);
  return bias ? launch_packed_mods<D, kCap | kBias>(p, s) : launch_packed_mods<D, kCap>(p, s);
}

}  // namespace ttq
