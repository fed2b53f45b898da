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
//          channels of column n, 16 bytes in one load: a byte permutation pairs
//          two keys' codes, so that the eight instructions over the channels of a
//          column take their A operand from one key order without a transposition;
//   of O   row n and channels 8 (4 h + i) .. + 7, i = 0 .. 3: 32 in a row.
// (packed_cache.h lays the pages out for this.)  A code becomes a number by or-ing
// it into the mantissa of 1024 (or 64, four bits up), which is subtracted again:
// exact; then one fused multiply-add with scale and lo, rounded to 16 bits once.
// That is fp16 whatever the type of the queries; bf16 queries are brought into its
// range by a power of two of their row's largest value, which the scores get back.
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

// The codes at bits 0 and 16 of x, or at bits 4 and 20, as values.
__device__ __forceinline__ h2v value_low(uint32_t x, h2v scale, h2v lo) {
  const h2v c = pair((x & 0x000F000Fu) | 0x64006400u) - twice((_Float16)1024.f);
  return __builtin_elementwise_fma(c, scale, lo);
}
__device__ __forceinline__ h2v value_high(uint32_t x, h2v scale, h2v lo) {
  const h2v c = pair((x & 0x00F000F0u) | 0x54005400u) - twice((_Float16)64.f);
  return __builtin_elementwise_fma(c, scale, lo);
}
__device__ __forceinline__ h8 join4(h2v a, h2v b, h2v c, h2v d) { return h8{a[0], a[1], b[0], b[1], c[0], c[1], d[0], d[1]}; }

// Slot of a word that holds channel c of its eight.
__device__ __forceinline__ constexpr int slot_of(int c) { return (c & 1) * 4 + c / 2; }

// One tile of 32 keys, as loaded: two halves of 16 tokens.
template <int D>
struct PackedTile {
  static constexpr int C = D < 128 ? D : 128, B = D / C;  // channels of a block, blocks of a row
  static constexpr int T = C / 32;                        // instructions over a block's channels
  u4v kc[2][B], kp[2][B];  // words of K over t; scale, lo pairs over t
  u4v vc[2][B], vp[2][B];  // words of four keys; scales of four keys, los of four keys

  // Pages of the two halves.
  static __device__ __forceinline__ void pages(const AttnArgs& a, const int32_t* table, int tile, int (&id)[2]) {
#pragma unroll
    for (int u = 0; u < 2; ++u)
      id[u] = uniform_load(table, min((tile * 32 + u * 16) >> a.page_shift, a.n_blocks - 1));
  }
  // Where half u lies.  Page numbers outside the cache and halves past the last
  // key read as zeros.
  static __device__ __forceinline__ __amdgpu_buffer_rsrc_t half_at(const AttnArgs& a, const SeqTile& t, int kvh, int tile,
                                                                   int u, uint32_t id, const char* of) {
    const int pos = tile * 32 + u * 16;
    const bool bad = id >= a.n_pages || pos >= t.kv_len;
    const int64_t at = (int64_t)(bad ? 0 : id) * a.page_bytes +
                       (((int64_t)kvh << a.page_shift) + (pos & ((1 << a.page_shift) - 1))) * (D * 5 / 8);
    return __builtin_amdgcn_make_buffer_rsrc(uniform_ptr(of + at), 0, uniform(bad ? 0 : 10 * D), 0x00020000);
  }
  __device__ __forceinline__ void load_keys(const AttnArgs& a, const SeqTile& t, int kvh, int tile, const int (&ids)[2], int n,
                                            int h) {
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      const auto r = half_at(a, t, kvh, tile, u, (uint32_t)ids[u], a.k);
#pragma unroll
      for (int b = 0; b < B; ++b) {
        if constexpr (C == 128) {
          kc[u][b] = __builtin_amdgcn_raw_buffer_load_b128(r, n * 64 + h * 16 + b * 10 * C, 0, 0);
          kp[u][b] = __builtin_amdgcn_raw_buffer_load_b128(r, n * 16 + 8 * C + b * 10 * C, 0, 0);
        } else {
          const u2v x = __builtin_amdgcn_raw_buffer_load_b64(r, n * 32 + h * 8, 0, 0);
          const u2v y = __builtin_amdgcn_raw_buffer_load_b64(r, n * 8 + 8 * C, 0, 0);
          kc[u][b] = u4v{x[0], x[1], 0, 0};
          kp[u][b] = u4v{y[0], y[1], 0, 0};
        }
      }
    }
  }
  __device__ __forceinline__ void load_values(const AttnArgs& a, const SeqTile& t, int kvh, int tile, const int (&ids)[2], int n,
                                              int h) {
    const int col = n % (C / 8);
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      const auto r = half_at(a, t, kvh, tile, u, (uint32_t)ids[u], a.v);
#pragma unroll
      for (int b = 0; b < B; ++b) {
        vc[u][b] = __builtin_amdgcn_raw_buffer_load_b128(r, (h * (C / 8) + col) * 16 + b * 10 * C, 0, 0);
        vp[u][b] = __builtin_amdgcn_raw_buffer_load_b128(r, (h * T + col / 4) * 16 + 8 * C + b * 10 * C, 0, 0);
      }
    }
  }
  // The A operand of instruction t over block b's channels: 16 keys.
  __device__ __forceinline__ h8 keys(int u, int b, int t) const {
    const uint32_t w = kc[u][b][t], p = kp[u][b][t], w8 = w >> 8;
    const h2v q = pair(p), s = twice(q[0]), lo = twice(q[1]);
    return join4(value_low(w, s, lo), value_high(w, s, lo), value_low(w8, s, lo), value_high(w8, s, lo));
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
};

// 16 R rows of a tile in one wave: queries, running maxima and sums, output sums.
template <int D, int R, int MODS>
struct PackedCore {
  typedef PackedTile<D> Tile;
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
        const int exponent = (int)(most >> 7);  // infinities and NaN come through as they are
        const int shift = exponent == 0 || exponent == 255 ? 0 : exponent - 127;
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
            q[r][b][s] = f;
          }
      } else {
#pragma unroll
        for (int b = 0; b < B; ++b)
#pragma unroll
          for (int s = 0; s < T; ++s) {
            const u4v w = x[b][s];
            q[r][b][s] = __builtin_bit_cast(h8, w);
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
    float mx[R];
    bool grown = false;
#pragma unroll
    for (int r = 0; r < R; ++r) {
      limit(a, t, r, k0, mixed, h, s[r]);
      float y = fmaxf(fmaxf(s[r][0][0], s[r][0][1]), fmaxf(s[r][0][2], s[r][0][3]));
      y = fmaxf(y, fmaxf(fmaxf(s[r][1][0], s[r][1][1]), fmaxf(s[r][1][2], s[r][1][3])));
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
    // O^T += V^T P^T: byte by byte of the words, two keys paired by a permutation
    const uint32_t odd = n >= 8 ? 4 : 0;
#pragma unroll
    for (int b = 0; b < B; ++b)
#pragma unroll
      for (int y = 0; y < 4; ++y) {
        uint32_t w[4];
        h2v s4[4], l4[4];
#pragma unroll
        for (int u = 0; u < 2; ++u)
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const uint32_t w0 = x.vc[u][b][2 * i], w1 = x.vc[u][b][2 * i + 1], sc = x.vp[u][b][i], lo = x.vp[u][b][2 + i];
            w[u * 2 + i] = __builtin_amdgcn_perm(w1, w0, 0x0C040C00u + (uint32_t)y * 0x00010001u);
            s4[u * 2 + i] = pair(sc);
            l4[u * 2 + i] = pair(lo);
          }
        if constexpr (D == 64) {
          // columns 0 to 7 twice: lanes n >= 8 have the upper code of each byte
          h2v z[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) z[i] = value_low(w[i] >> odd, s4[i], l4[i]);
          const h8 v = join4(z[0], z[1], z[2], z[3]);
#pragma unroll
          for (int r = 0; r < R; ++r) o[r][y] = mfma16(v, p[r], o[r][y]);
        } else {
          h2v z[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) z[i] = value_low(w[i], s4[i], l4[i]);
          h8 v = join4(z[0], z[1], z[2], z[3]);
#pragma unroll
          for (int r = 0; r < R; ++r) o[r][b * 8 + 2 * y] = mfma16(v, p[r], o[r][b * 8 + 2 * y]);
#pragma unroll
          for (int i = 0; i < 4; ++i) z[i] = value_high(w[i], s4[i], l4[i]);
          v = join4(z[0], z[1], z[2], z[3]);
#pragma unroll
          for (int r = 0; r < R; ++r) o[r][b * 8 + 2 * y + 1] = mfma16(v, p[r], o[r][b * 8 + 2 * y + 1]);
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

template <typename T, int D>
__device__ __forceinline__ void sink8(const AttnArgs& a, int tok, int head, int split, int active, float m, float l, int d,
                                      const float* x, bool sums) {
  const Sink<T, D> to(a, tok, head, split, active, m, l);
  to.four(d, x[0], x[1], x[2], x[3]);
  to.four(d + 4, x[4], x[5], x[6], x[7]);
  if (sums) to.sums(split, active);
}

template <int D, int R, int NW, int MODS>
__global__ __launch_bounds__(NW * 64, D == 64 ? (R == 4 ? 2 : 4) : D == 128 ? (R == 4 ? 1 : R == 2 ? 2 : 4) : R == 2 ? 1 : 2)
void packed_keys_kernel(PackedArgs p) {
  const AttnArgs& a = p.a;
  constexpr int STRIDE = 16 * 8 + 4;  // floats of 8 channels of 16 rows
  __shared__ __attribute__((aligned(16))) float sums[NW * D / 8 * STRIDE];
  __shared__ float2 ml[NW][16];
  const int lane = threadIdx.x & 63, wave = uniform((int)threadIdx.x >> 6), n = lane & 15, h = lane >> 4;
  const int kvh = blockIdx.x % a.n_kv, item = blockIdx.x / a.n_kv, split = item % a.key_splits;
  const SeqTile t = find_tile<16 * R>(a, item / a.key_splits, lane);
  if (t.s < 0) return;
  const KeyTiles kt = key_tiles<32>(a, t, 16 * R);
  const Share sh = share_of(kt.n, a.key_per, a.key_splits, split);
  if (split >= sh.active) return;

  const int32_t* table = a.table + (int64_t)t.s * a.table_stride;
  typedef PackedCore<D, R, MODS> Core;
  typename Core::Tile x;
  Core c;
  int id[2], next[2];
  int j = sh.j0 + wave;
  Core::Tile::pages(a, table, kt.at(j), id);
  Core::Tile::pages(a, table, kt.at(j + NW), next);
  if (j < sh.j1) {
    x.load_keys(a, t, kvh, kt.at(j), id, n, h);
    x.load_values(a, t, kvh, kt.at(j), id, n, h);
  }
  c.setup(a, p.bf16, t, kvh, n, h);
  // The registers of the keys are loaded again as soon as the scores are there,
  // those of the values after the products, so that a tile is always in flight.
  for (; j < sh.j1; j += NW) {
    const bool more = j + NW < sh.j1;
    typename Core::Scores s;
    c.scores(x, s);
    if (more) x.load_keys(a, t, kvh, kt.at(j + NW), next, n, h);
    c.sum_up(a, t, x, s, kt.at(j), n, h);
    if (more) x.load_values(a, t, kvh, kt.at(j + NW), next, n, h);
    Core::Tile::pages(a, table, kt.at(j + 2 * NW), next);
  }

  // 16 rows at a time: the waves' sums through LDS, joined in order.
#pragma unroll
  for (int r = 0; r < R; ++r) {
    float l = c.l[r];
    l += __shfl_xor(l, 16);
    l += __shfl_xor(l, 32);
    if (r > 0) __syncthreads();
    c.template leave<STRIDE>(r, sums + wave * (D / 8 * STRIDE), n, h);
    if (h == 0) ml[wave][n] = make_float2(c.m[r] * c.unit(a, r), l);
    __syncthreads();
    const int row = threadIdx.x & 15, at = t.row0 + r * 16 + row;
    if (at >= t.n_rows) continue;
    int tok, head;
    Core::row_of(a, t, kvh, at, tok, head);
    float m = -INFINITY, total = 0.f, w[NW];
#pragma unroll
    for (int i = 0; i < NW; ++i) m = fmaxf(m, ml[i][row].x);
    const float mu = m == -INFINITY ? 0.f : m;
#pragma unroll
    for (int i = 0; i < NW; ++i) {
      w[i] = exp2_fast(ml[i][row].x - mu);
      total += w[i] * ml[i][row].y;
    }
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
      const bool first = d8 == 0;
      if (p.bf16) sink8<__bf16, D>(a, t.q0 + tok, head, split, sh.active, m, total, d8 * 8, f, first);
      else sink8<_Float16, D>(a, t.q0 + tok, head, split, sh.active, m, total, d8 * 8, f, first);
    }
  }
}

template <int D, int R, int MODS>
hipError_t launch_packed_rows(const PackedArgs& p, hipStream_t s) {
  const unsigned grid = (unsigned)p.a.key_tiles * p.a.key_splits * p.a.n_kv;
  if (p.a.key_waves > 1) packed_keys_kernel<D, R, 4, MODS><<<grid, 256, 0, s>>>(p);
  else packed_keys_kernel<D, R, 1, MODS><<<grid, 64, 0, s>>>(p);
  return hipGetLastError();
}
template <int D, int MODS>
hipError_t launch_packed_mods(const PackedArgs& p, hipStream_t s) {
  hipError_t e;
  if (p.rows_of_tile == 16) e = launch_packed_rows<D, 1, MODS>(p, s);
  else if (D == 256 || p.rows_of_tile == 32) e = launch_packed_rows<D, 2, MODS>(p, s);
  else e = launch_packed_rows<D, D == 256 ? 2 : 4, MODS>(p, s);
  if (e != hipSuccess || !p.join || splits_of(p.a) <= 1) return e;
  const unsigned rows = (unsigned)(p.a.total_q * p.a.n_heads);
  if (p.bf16) attn_join_kernel<__bf16, D><<<rows, 256, 0, s>>>(p.a);
  else attn_join_kernel<_Float16, D><<<rows, 256, 0, s>>>(p.a);
  return hipGetLastError();
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
