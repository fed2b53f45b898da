// New queries, keys and values on their way from the projection: queries and
// keys are rotated by their positions, keys and values go to their pages, in 16
// bits or in 4, and values in 4 bits come back as rows.
//
// Rotation, for channel pairs (a, b) and the table's row of the position:
//   a' = a cos - b sin,  b' = b cos + a sin
// in 32 bits, each product and sum rounded by itself (no fused multiply-add), so
// that the 4-bit codes do not depend on how a compiler contracts it.
//
// 4 bits, for the 32 channels x of a group: lo = fp16(min x), scale =
// fp16((max x - min x) / 15), code = rint((x - lo) / scale) in 0 .. 15, all in 32
// bits with IEEE division: bf16 and fp16 values lie on coarse grids, where a
// quotient by a rounded reciprocal would often miss a tie.
#include "packed_cache.h"
#include "paged_tokens.h"

namespace ttq {

namespace {

typedef uint32_t u4 __attribute__((ext_vector_type(4)));

constexpr int kThreads = 256;

template <typename T>
__device__ __forceinline__ void widen(u4 x, float* f) {
  typedef T v2 __attribute__((ext_vector_type(2)));
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t w = x[i];
    const v2 p = __builtin_bit_cast(v2, w);
    f[2 * i] = (float)p[0];
    f[2 * i + 1] = (float)p[1];
  }
}
template <typename T>
__device__ __forceinline__ u4 narrow(const float* f) {
  typedef T v2 __attribute__((ext_vector_type(2)));
  u4 x;
#pragma unroll
  for (int i = 0; i < 4; ++i) x[i] = __builtin_bit_cast(uint32_t, v2{(T)f[2 * i], (T)f[2 * i + 1]});
  return x;
}

// a' = a c - b s, b' = b c + a s
__device__ __forceinline__ void turn(float& a, float& b, float c, float s) {
#pragma clang fp contract(off)
  const float x = a * c - b * s, y = b * c + a * s;
  a = x;
  b = y;
}

// NaN to 0, infinities and what is beyond to the ends of the range
__device__ __forceinline__ float saturated(float x) { return x != x ? 0.f : fminf(fmaxf(x, -kPackMost), kPackMost); }

// the least or largest of four neighbouring lanes
template <int CTRL>
__device__ __forceinline__ float of_lane(float x) {
  return __builtin_bit_cast(
      float, __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, x), CTRL, 0xF, 0xF, true));
}
__device__ __forceinline__ float min4(float x) {
  x = fminf(x, of_lane<0xB1>(x));   // lane ^ 1
  return fminf(x, of_lane<0x4E>(x));  // lane ^ 2
}
__device__ __forceinline__ float max4(float x) {
  x = fmaxf(x, of_lane<0xB1>(x));
  return fmaxf(x, of_lane<0x4E>(x));
}

// One lane's 8 channels of a group that four neighbouring lanes hold.
__device__ __forceinline__ uint32_t pack8(float* f, _Float16& scale, _Float16& lo) {
#pragma clang fp contract(off)
  float least = f[0] = saturated(f[0]), most = least;
#pragma unroll
  for (int i = 1; i < 8; ++i) {
    f[i] = saturated(f[i]);
    least = fminf(least, f[i]);
    most = fmaxf(most, f[i]);
  }
  least = min4(least);
  most = max4(most);
  lo = (_Float16)least;
  scale = (_Float16)((most - least) / 15.f);
  // channels that are alike, or nearly: all codes are 0
  const float step = (float)scale > 0.f ? (float)scale : INFINITY, from = (float)lo;
  uint32_t w = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float c = fminf(fmaxf(rintf((f[i] - from) / step), 0.f), 15.f);
    w |= (uint32_t)c << (4 * (i / 2 + 4 * (i & 1)));
  }
  return w;
}

// A workgroup has one token and kThreads units of it at a time.  A unit is 16
// channels of one head, two vectors of 16 bytes: the two parts of eight rotated
// pairs, or neighbours.  The heads are the queries', the keys' and the values',
// in this order; the sines and cosines of a thread are the same for all its
// heads.  Reads and writes of the rows are whole and in order, and none waits for
// the lookups of sequence, position and page but the stores.
//
// Bound by memory where there is much: 19679 tokens of 32/8 heads of 128 in bf16 into
// 16 bits 91 us, 5.4 TB/s; 15853 tokens of 64/8 heads of 128 in fp16 into 4 bits 120
// us, 5.0 TB/s, with vector instructions on the SIMDs for 70 % of it (the format
// wants the codes' divisions rounded right).  A decode step is a launch and four dependent loads: 3.5 us into 16
// bits, 5.2 into 4.
template <typename T, bool PACKED>
__global__ __launch_bounds__(kThreads) void append_kernel(AppendArgs a) {
  __shared__ __attribute__((aligned(16))) float row[PACKED ? kThreads * 16 : 4];
  const int tid = threadIdx.x, dim = 1 << a.dim_shift;
  const int tok = (int)(blockIdx.x / a.slices), slice = (int)(blockIdx.x % a.slices);
  const int units = dim / 16, u = tid & (units - 1), heads = a.n_heads + 2 * a.n_kv;
  const int per = kThreads / units;  // heads of a round
  // the unit's two vectors within a head
  const bool rotated = 16 * u < a.rot_dim, apart = rotated && !a.interleaved;
  const int c0 = apart ? 8 * u : 16 * u, c1 = apart ? 8 * u + a.rot_dim / 2 : 16 * u + 8;

  const int s = sequence_of(a.at, tok);
  if (s < 0) return;
  const int64_t place = position_of(a.at, s, tok);
  float cs[8], sn[8];
  if (a.rot_dim > 0) {
    const int64_t pos = a.positions != nullptr ? a.positions[tok] : place;
    if (pos < 0 || pos >= a.n_positions) return;  // the table has no row for it
    if (rotated) {
      const float4* t = reinterpret_cast<const float4*>(a.rotation + pos * a.rot_dim + 8 * u);
      const float4* v = reinterpret_cast<const float4*>(a.rotation + pos * a.rot_dim + a.rot_dim / 2 + 8 * u);
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const float4 x = t[i], y = v[i];
        cs[4 * i] = x.x, cs[4 * i + 1] = x.y, cs[4 * i + 2] = x.z, cs[4 * i + 3] = x.w;
        sn[4 * i] = y.x, sn[4 * i + 1] = y.y, sn[4 * i + 2] = y.z, sn[4 * i + 3] = y.w;
      }
    }
  }
  uint32_t page = 0;
  const bool has_page = page_of(a.at, s, place, page);
  const int slot = (int)(place & ((1 << a.at.page_shift) - 1));

  const int rounds = (heads + per - 1) / per;
  for (int r = slice; r < rounds; r += a.slices) {
    const int h = r * per + tid / units;
    const bool is_q = h < a.n_heads, is_k = !is_q && h < a.n_heads + a.n_kv;
    const int kvh = is_q ? 0 : h - a.n_heads - (is_k ? 0 : a.n_kv);
    const bool any = h < heads && (is_q || has_page);
    float x[8], y[8];
    if (any) {
      const char* p = is_q ? a.q + tok * a.ldq : is_k ? a.k + tok * a.ldk : a.v + tok * a.ldv;
      p += ((int64_t)(is_q ? h : kvh) << a.dim_shift) * 2;
      const u4 p0 = *reinterpret_cast<const u4*>(p + c0 * 2), p1 = *reinterpret_cast<const u4*>(p + c1 * 2);
      u4 o0 = p0, o1 = p1;
      const bool turns = rotated && (is_q || is_k);
      if (turns || PACKED) {
        widen<T>(p0, x);
        widen<T>(p1, y);
        if (turns) {
          if (a.interleaved) {
#pragma unroll
            for (int i = 0; i < 4; ++i) turn(x[2 * i], x[2 * i + 1], cs[i], sn[i]);
#pragma unroll
            for (int i = 0; i < 4; ++i) turn(y[2 * i], y[2 * i + 1], cs[4 + i], sn[4 + i]);
          } else {
#pragma unroll
            for (int i = 0; i < 8; ++i) turn(x[i], y[i], cs[i], sn[i]);
          }
          o0 = narrow<T>(x);
          o1 = narrow<T>(y);
        }
      }
      if (is_q) {
        char* o = a.qr + tok * a.ldqr + ((int64_t)h << a.dim_shift) * 2;
        *reinterpret_cast<u4*>(o + c0 * 2) = o0;
        *reinterpret_cast<u4*>(o + c1 * 2) = o1;
      } else if constexpr (!PACKED) {
        char* o = (is_k ? a.kc : a.vc) + page * a.page_bytes +
                  (((((int64_t)kvh << a.at.page_shift) + slot) << a.dim_shift) * 2);
        *reinterpret_cast<u4*>(o + c0 * 2) = o0;
        *reinterpret_cast<u4*>(o + c1 * 2) = o1;
      }
    }
    if constexpr (PACKED) {
      if ((r + 1) * per <= a.n_heads) continue;  // queries alone, in all threads
      // the channels in their order: four neighbouring lanes then hold a group
      if (any && !is_q) {
        float* to = row + (tid / units << a.dim_shift);
#pragma unroll
        for (int i = 0; i < 8; i += 4) {
          *reinterpret_cast<float4*>(to + c0 + i) = make_float4(x[i], x[i + 1], x[i + 2], x[i + 3]);
          *reinterpret_cast<float4*>(to + c1 + i) = make_float4(y[i], y[i + 1], y[i + 2], y[i + 3]);
        }
      }
      __syncthreads();
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const int vec = j * kThreads + tid, vecs = dim / 8, vh = r * per + vec / vecs, v = vec & (vecs - 1);
        if (vh < a.n_heads || vh >= heads || !has_page) continue;
        float f[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) f[i] = row[vec * 8 + i];
        _Float16 scale, lo;
        const uint32_t w = pack8(f, scale, lo);
        const bool key = vh < a.n_heads + a.n_kv;
        const int kv = vh - a.n_heads - (key ? 0 : a.n_kv);
        char* o = (key ? a.kc : a.vc) + page * a.page_bytes +
                  ((((int64_t)kv << a.at.page_shift) + (slot & ~15)) << a.dim_shift) * 5 / 8;
        const int t = slot & 15;
        *reinterpret_cast<uint32_t*>(o + (key ? packed_word<true>(dim, t, v) : packed_word<false>(dim, t, v))) = w;
        if ((v & 3) != 0) continue;
        o += key ? packed_scale<true>(dim, t, v) : packed_scale<false>(dim, t, v);
        if (key) {
          typedef _Float16 h2 __attribute__((ext_vector_type(2)));
          *reinterpret_cast<uint32_t*>(o) = __builtin_bit_cast(uint32_t, h2{scale, lo});
        } else {
          *reinterpret_cast<_Float16*>(o) = scale;
          *reinterpret_cast<_Float16*>(o + kPackLo<false>) = lo;
        }
      }
      __syncthreads();
    }
  }
}

// What the 4-bit cache holds for the batch's rows, 16 bits: a workgroup has a
// token, a thread 8 channels at a time.  scale * code + lo in 32 bits, rounded
// once.  A workgroup costs 0.7 ns whatever it moves, for its lookups one after the
// other (32768 tokens of one head of 256, 44 MB: 27 us), and more heads add their
// bytes at 4.2 TB/s: 15853 tokens of 8 heads of 128, 85 MB, take 25 us, 3.4 TB/s,
// 32768 take 47 us, 3.8 TB/s.
template <typename T>
__global__ __launch_bounds__(kThreads) void packed_read_kernel(AppendArgs a) {
  const int tok = (int)blockIdx.x, dim = 1 << a.dim_shift, vecs = dim / 8;
  const int s = sequence_of(a.at, tok);
  if (s < 0) return;
  const int64_t place = position_of(a.at, s, tok);
  uint32_t page;
  if (!page_of(a.at, s, place, page)) return;
  const int slot = (int)(place & ((1 << a.at.page_shift) - 1)), t = slot & 15;
  for (int i = threadIdx.x; i < 2 * a.n_kv * vecs; i += kThreads) {
    const int h = i / vecs, v = i & (vecs - 1);
    const bool key = h < a.n_kv;
    const int kv = key ? h : h - a.n_kv;
    const char* p = (key ? a.kc : a.vc) + page * a.page_bytes +
                    ((((int64_t)kv << a.at.page_shift) + (slot & ~15)) << a.dim_shift) * 5 / 8;
    const uint32_t w = *reinterpret_cast<const uint32_t*>(p + (key ? packed_word<true>(dim, t, v) : packed_word<false>(dim, t, v)));
    p += key ? packed_scale<true>(dim, t, v) : packed_scale<false>(dim, t, v);
    const float scale = (float)*reinterpret_cast<const _Float16*>(p);
    const float lo = (float)*reinterpret_cast<const _Float16*>(p + (key ? kPackLo<true> : kPackLo<false>));
    float f[8];
#pragma unroll
    for (int c = 0; c < 8; ++c) f[c] = __builtin_fmaf(scale, (float)(w >> (4 * (c / 2 + 4 * (c & 1))) & 15u), lo);
    char* o = key ? a.kr + tok * a.ldk : a.vr + tok * a.ldv;
    *reinterpret_cast<u4*>(o + (((int64_t)kv << a.dim_shift) + v * 8) * 2) = narrow<T>(f);
  }
}

}  // namespace

// Workgroups of a token.  One while there are many: the lookups and the table's
// row once a token.  With few tokens, up to one workgroup a CU, each round of heads
// has its own (32/8 heads of 128, two rounds, us in a graph, rounds apart and in one:
// 64 tokens 3.0 and 3.3, into 4 bits 3.9 and 4.4; 170 tokens 3.4 and 3.5, 4.7 and
// 4.5; 512 tokens 4.8 and 4.3, 6.7 and 5.9).
static int slices_of(const AppendArgs& a) {
  const int per = kThreads / ((1 << a.dim_shift) / 16), rounds = (a.n_heads + 2 * a.n_kv + per - 1) / per;
  return (int64_t)a.at.total_q * rounds <= 256 ? rounds : 1;
}

int64_t append_threads(const AppendArgs& a) { return (int64_t)a.at.total_q * slices_of(a) * kThreads; }

hipError_t launch_append(AppendArgs a, bool bf16, bool packed, hipStream_t s) {
  a.slices = slices_of(a);
  const unsigned grid = (unsigned)a.at.total_q * a.slices;
  if (packed) {
    if (bf16) append_kernel<__bf16, true><<<grid, kThreads, 0, s>>>(a);
    else append_kernel<_Float16, true><<<grid, kThreads, 0, s>>>(a);
  } else {
    if (bf16) append_kernel<__bf16, false><<<grid, kThreads, 0, s>>>(a);
    else append_kernel<_Float16, false><<<grid, kThreads, 0, s>>>(a);
  }
  return hipGetLastError();
}

hipError_t launch_packed_read(const AppendArgs& a, bool bf16, hipStream_t s) {
  if (bf16) packed_read_kernel<__bf16><<<(unsigned)a.at.total_q, kThreads, 0, s>>>(a);
  else packed_read_kernel<_Float16><<<(unsigned)a.at.total_q, kThreads, 0, s>>>(a);
  return hipGetLastError();
}

}  // namespace ttq
