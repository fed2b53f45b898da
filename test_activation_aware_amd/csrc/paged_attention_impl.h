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
// Keys and values come through LDS by direct-to-LDS loads, 64 keys a stage,
// the next stage in flight while one is worked on.  A load instruction moves
// 1 KB: whole rows of one page (pages hold 16 tokens or more).  Its buffer
// resource ends at the sequence's last key, so that what a page holds beyond
// it reaches LDS as zeros (never NaN), and a page number outside the cache
// reads nothing.  16-byte chunks are permuted within a row through the source
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

template <typename T>
struct Vec;
template <>
struct Vec<_Float16> {
  typedef _Float16 v2 __attribute__((ext_vector_type(2)));
  typedef h8 v8;
};
template <>
struct Vec<__bf16> {
  typedef __bf16 v2 __attribute__((ext_vector_type(2)));
  typedef b8 v8;
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

__device__ __forceinline__ float exp2_fast(float x) { return __builtin_amdgcn_exp2f(x); }

template <int N>
__device__ __forceinline__ void wait_loads() {  // at most N vector loads still in flight
  static_assert(N >= 0 && N < 64, "vmcnt field");
  __builtin_amdgcn_s_waitcnt((N & 15) | ((N >> 4) << 14) | 0x0F70);
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

// The sequence of a tile of BM rows.  Sequence s owns the tiles from
// q_start[s] * group / BM + s on: enough for its rows wherever they begin, and
// known without a sum over the sequences before it.
struct SeqTile {
  int s;        // sequence, -1: none
  int row0;     // first row of the tile in its sequence
  int n_rows;   // rows of the sequence
  int q0;       // first new token of the sequence in Q
  int q_len, kv_len, prefix;
};
template <int BM>
__device__ __forceinline__ SeqTile find_tile(const AttnArgs& a, int tile, int lane) {
  SeqTile t;
  int n = 0;
  for (int c = 0; c < a.n_seqs; c += 64) {
    const int i = c + lane;
    bool le = false;
    if (i < a.n_seqs) le = clampi(a.q_start[i], 0, a.total_q) * a.group / BM + i <= tile;
    const unsigned long long b = __ballot(le);
    n += __popcll(b);
    if (b != ~0ull) break;
  }
  t.s = uniform(n - 1);
  if (t.s < 0) return t;
  t.q0 = clampi(uniform_load(a.q_start, t.s), 0, a.total_q);
  t.q_len = max(clampi(uniform_load(a.q_start, t.s + 1), 0, a.total_q) - t.q0, 0);
  t.n_rows = t.q_len * a.group;
  t.row0 = (tile - (t.q0 * a.group / BM + t.s)) * BM;
  if (t.row0 < 0 || t.row0 >= t.n_rows) t.s = -1;
  const int64_t room = (int64_t)a.n_blocks << a.page_shift;
  t.kv_len = (int)min<int64_t>(max(uniform_load(a.kv_len, max(t.s, 0)), 0), min<int64_t>(room, 0x7FFFFF00));
  t.prefix = a.prefix != nullptr ? clampi(uniform_load(a.prefix, max(t.s, 0)), 0, t.kv_len) : 0;
  return t;
}

// The key tiles (KT keys each) that some row of a tile sees: na tiles from 0
// (the prefix), then tiles first, first + 1, ...; n in all.
struct KeyTiles {
  int na, first, n;
  __device__ __forceinline__ int at(int j) const { return j < na ? j : first + (j - na); }
};
template <int KT>
__device__ __forceinline__ KeyTiles key_tiles(const AttnArgs& a, const SeqTile& t, int bm) {
  const int p0 = t.kv_len - t.q_len + t.row0 / a.group;  // first and last query position
  const int p1 = t.kv_len - t.q_len + (min(t.row0 + bm, t.n_rows) - 1) / a.group;
  const int hi = max(p1 + 1, 0), lo = a.window > 0 ? max(0, p0 - a.window + 1) : 0;
  KeyTiles k;
  k.na = (t.prefix + KT - 1) / KT;
  k.first = max(k.na, lo / KT);
  k.n = k.na + max(0, (hi + KT - 1) / KT - k.first);
  return k;
}

// 64 keys of one key head: K and V into LDS, this wave's share of the loads.
template <int D, int KT, int NW>
struct Loader {
  static constexpr int ROWB = 2 * D, CPR = D / 8, RPL = 1024 / ROWB;
  static constexpr int LOADS = KT / RPL / NW;  // loads of a wave per matrix
  static_assert(LOADS >= 1 && KT % (RPL * NW) == 0, "load split");
  const char *k, *v;  // of the key head
  const int32_t* table;
  int kv_len, wave, kvoff, vvoff, vxor;

  static __device__ __forceinline__ int swz_k(int row) { return D == 64 ? (row >> 1) & 7 : row & 15; }
  static __device__ __forceinline__ int swz_v(int row) { return D == 64 ? ((row >> 1) & 1) << 2 : (row & 3) << 2; }

  // the pages of a tile's loads, fetched ahead of issue()
  __device__ __forceinline__ void pages(const AttnArgs& a, int tile, int (&id)[LOADS]) const {
#pragma unroll
    for (int i = 0; i < LOADS; ++i)
      id[i] = uniform_load(table, min((tile * KT + (wave * LOADS + i) * RPL) >> a.page_shift, a.n_blocks - 1));
  }
  __device__ __forceinline__ void issue(const AttnArgs& a, int tile, const int (&ids)[LOADS], char* lk, char* lv,
                                        int lane) const {
    const int lrow = lane / CPR, pc = lane % CPR;
#pragma unroll
    for (int i = 0; i < LOADS; ++i) {
      const int r0 = (wave * LOADS + i) * RPL;
      const int pos = tile * KT + r0;
      const uint32_t id = (uint32_t)ids[i];
      const bool bad = id >= a.n_pages;
      const int rec = uniform(bad ? 0 : clampi(kv_len - pos, 0, RPL) * ROWB);
      const uint64_t off = (uint64_t)(bad ? 0 : id) * (uint64_t)a.page_bytes + (uint32_t)((pos & ((1 << a.page_shift) - 1)) * ROWB);
      const int kof = lrow * ROWB + ((pc ^ swz_k(r0 + lrow)) << 4);
      const int vof = lrow * ROWB + ((pc ^ swz_v(r0 + lrow)) << 4);
      auto rk = __builtin_amdgcn_make_buffer_rsrc(uniform_ptr(k + off), (short)0, rec, 0x00020000);
      auto rv = __builtin_amdgcn_make_buffer_rsrc(uniform_ptr(v + off), (short)0, rec, 0x00020000);
      __builtin_amdgcn_raw_ptr_buffer_load_lds(rk, (__attribute__((address_space(3))) void*)(lk + r0 * ROWB), 16, kof, 0, 0, 0);
      __builtin_amdgcn_raw_ptr_buffer_load_lds(rv, (__attribute__((address_space(3))) void*)(lv + r0 * ROWB), 16, vof, 0, 0, 0);
    }
  }
};

// Row form: NW waves of 32 RN rows each, all on the same key tiles.
template <typename T, int D, int NW, int RN, bool MODS>
__global__ __launch_bounds__(NW * 64, D == 256 ? 1 : 2) void attn_rows_kernel(AttnArgs a) {
  typedef typename Vec<T>::v8 v8;
  constexpr int KT = 64, KF = KT / 32, DS = D / 16, DF = D / 32, BM = NW * RN * 32;
  typedef Loader<D, KT, NW> L;
  constexpr int ROWB = L::ROWB, STAGE = KT * ROWB;
  __shared__ __attribute__((aligned(16))) char lk0[STAGE], lv0[STAGE], lk1[STAGE], lv1[STAGE];

  const int lane = threadIdx.x & 63, l32 = lane & 31, hh = lane >> 5;
  const int wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
  const int kvh = blockIdx.x % a.n_kv;
  const int tiles = gridDim.x / a.n_kv;
  const int split = blockIdx.y;
  const SeqTile t = find_tile<BM>(a, tiles - 1 - blockIdx.x / a.n_kv, lane);
  if (t.s < 0) return;
  const KeyTiles kt = key_tiles<KT>(a, t, BM);
  const int per = (kt.n + a.n_splits - 1) / a.n_splits;
  const int j0 = min(split * per, kt.n), j1 = min(j0 + per, kt.n);

  // this lane's queries
  int row[RN], qpos[RN], head[RN];
  v8 qf[DS][RN];
#pragma unroll
  for (int r = 0; r < RN; ++r) {
    row[r] = t.row0 + (wave * RN + r) * 32 + l32;
    const int rc = min(row[r], t.n_rows - 1);
    const int tok = rc / a.group;
    head[r] = kvh * a.group + (rc - tok * a.group);
    qpos[r] = t.kv_len - t.q_len + tok;
    const T* q = static_cast<const T*>(a.q) + (int64_t)(t.q0 + tok) * a.ldq + (int64_t)head[r] * D + hh * 8;
#pragma unroll
    for (int s = 0; s < DS; ++s) qf[s][r] = *reinterpret_cast<const v8*>(q + s * 16);
  }
  float slope[RN];
#pragma unroll
  for (int r = 0; r < RN; ++r) slope[r] = MODS && a.slopes != nullptr ? a.slopes[head[r]] * 1.44269504088896341f : 0.f;

  f16x o[DF][RN];
  float m[RN], l[RN];
#pragma unroll
  for (int r = 0; r < RN; ++r) {
    m[r] = -INFINITY;
    l[r] = 0.f;
#pragma unroll
    for (int d = 0; d < DF; ++d)
#pragma unroll
      for (int e = 0; e < 16; ++e) o[d][r][e] = 0.f;
  }

  L ld;
  {
    const int64_t hoff = ((int64_t)kvh << a.page_shift) * ROWB;
    ld.k = a.k + hoff;
    ld.v = a.v + hoff;
    ld.table = a.table + (int64_t)t.s * a.table_stride;
    ld.kv_len = t.kv_len;
    ld.wave = wave;
  }
  // tiles between these need no mask: every row of this wave sees all of them
  const int wrow0 = t.row0 + wave * RN * 32;
  const int wp0 = t.kv_len - t.q_len + min(wrow0, t.n_rows - 1) / a.group;
  const int wp1 = t.kv_len - t.q_len + (min(wrow0 + RN * 32, t.n_rows) - 1) / a.group;
  const int full_lo = a.window > 0 ? max(0, wp1 - a.window + 1) : 0;

  const int ksw = L::swz_k(l32);
  const int kaddr = l32 * ROWB;
  const int kk = (lane & 15) >> 2, vc = lane & 3, vg = (lane >> 4) & 1;
  const int vrow = (4 * hh + kk) * ROWB, vsw = L::swz_v(kk);

  auto work = [&](const char* lk, const char* lv, int tile) {
    const int k0 = tile * KT;
    f16x s[KF][RN];
#pragma unroll
    for (int f = 0; f < KF; ++f) {
#pragma unroll
      for (int r = 0; r < RN; ++r)
#pragma unroll
        for (int e = 0; e < 16; ++e) s[f][r][e] = 0.f;
#pragma unroll
      for (int st = 0; st < DS; ++st) {
        const v8 kf = *reinterpret_cast<const v8*>(lk + f * 32 * ROWB + kaddr + (((2 * st + hh) ^ ksw) << 4));
#pragma unroll
        for (int r = 0; r < RN; ++r) s[f][r] = mfma(kf, qf[st][r], s[f][r]);
      }
    }
    const bool full = (k0 + KT <= wp0 + 1 && k0 >= full_lo) || k0 + KT <= t.prefix;
    uint32_t p[KF][RN][8];
#pragma unroll
    for (int r = 0; r < RN; ++r) {
#pragma unroll
      for (int f = 0; f < KF; ++f)
#pragma unroll
        for (int e = 0; e < 16; ++e) {
          float z = s[f][r][e];
          if constexpr (MODS) {
            if (a.cap_in != 0.f)
              z = a.cap_out - 2.f * a.cap_out * __builtin_amdgcn_rcpf(exp2_fast(z * a.cap_in) + 1.f);
            else
              z *= a.scale_log2;
            const int j = k0 + f * 32 + 8 * (e / 4) + 4 * hh + (e & 3);
            z -= slope[r] * fabsf((float)(qpos[r] - j));
          }
          s[f][r][e] = z;
        }
      if (!full) {
        const int lo = a.window > 0 ? qpos[r] - a.window + 1 : 0;
#pragma unroll
        for (int f = 0; f < KF; ++f)
#pragma unroll
          for (int e = 0; e < 16; ++e) {
            const int j = k0 + f * 32 + 8 * (e / 4) + 4 * hh + (e & 3);
            const bool seen = (j <= qpos[r] && j >= lo) || j < t.prefix;
            s[f][r][e] = seen ? s[f][r][e] : -INFINITY;
          }
      }
      float mx = s[0][r][0];
#pragma unroll
      for (int f = 0; f < KF; ++f)
#pragma unroll
        for (int e = 0; e < 16; ++e) mx = fmaxf(mx, s[f][r][e]);
      mx = half_max(mx);
      if constexpr (!MODS) mx *= a.scale_log2;
      const float mn = fmaxf(m[r], mx);
      const float mu = mn == -INFINITY ? 0.f : mn;
      if (__any(mn != m[r])) {
        const float al = exp2_fast(m[r] - mu);
        l[r] *= al;
#pragma unroll
        for (int d = 0; d < DF; ++d)
#pragma unroll
          for (int e = 0; e < 16; ++e) o[d][r][e] *= al;
        m[r] = mn;
      }
      const float c = MODS ? 1.f : a.scale_log2;
      float sum = 0.f;
#pragma unroll
      for (int f = 0; f < KF; ++f)
#pragma unroll
        for (int e = 0; e < 16; e += 2) {
          const float x = exp2_fast(__builtin_fmaf(s[f][r][e], c, -mu));
          const float y = exp2_fast(__builtin_fmaf(s[f][r][e + 1], c, -mu));
          sum += x + y;
          p[f][r][e / 2] = pack2<T>(x, y);
        }
      l[r] += sum;
    }
#pragma unroll
    for (int f = 0; f < KF; ++f)
#pragma unroll
      for (int st = 0; st < 2; ++st)
#pragma unroll
        for (int d = 0; d < DF; ++d) {
          const char* at = lv + (f * 32 + st * 16) * ROWB + vrow + (((d * 4 + vg * 2 + (vc >> 1)) ^ vsw) << 4) + (vc & 1) * 8;
          const s4v x = __builtin_amdgcn_ds_read_tr16_b64_v4i16(
              (__attribute__((address_space(3))) s4v*)const_cast<char*>(at));
          const s4v y = __builtin_amdgcn_ds_read_tr16_b64_v4i16(
              (__attribute__((address_space(3))) s4v*)const_cast<char*>(at + 8 * ROWB));
          const v8 vf = __builtin_bit_cast(v8, __builtin_shufflevector(x, y, 0, 1, 2, 3, 4, 5, 6, 7));
#pragma unroll
          for (int r = 0; r < RN; ++r) {
            const uint4 pu = make_uint4(p[f][r][st * 4], p[f][r][st * 4 + 1], p[f][r][st * 4 + 2], p[f][r][st * 4 + 3]);
            o[d][r] = mfma(vf, __builtin_bit_cast(v8, pu), o[d][r]);
          }
        }
  };

  int id[L::LOADS];
  if (j0 < j1) {
    ld.pages(a, kt.at(j0), id);
    ld.issue(a, kt.at(j0), id, lk0, lv0, lane);
    ld.pages(a, kt.at(j0 + 1), id);
  }
  for (int j = j0; j < j1; j += 2) {
    if (j + 1 < j1) {
      ld.issue(a, kt.at(j + 1), id, lk1, lv1, lane);
      ld.pages(a, kt.at(j + 2), id);
      wait_loads<2 * L::LOADS>();
    } else {
      wait_loads<0>();
    }
    barrier_only();
    work(lk0, lv0, kt.at(j));
    barrier_only();
    if (j + 1 >= j1) break;
    if (j + 2 < j1) {
      ld.issue(a, kt.at(j + 2), id, lk0, lv0, lane);
      ld.pages(a, kt.at(j + 3), id);
      wait_loads<2 * L::LOADS>();
    } else {
      wait_loads<0>();
    }
    barrier_only();
    work(lk1, lv1, kt.at(j + 1));
    barrier_only();
  }

#pragma unroll
  for (int r = 0; r < RN; ++r) {
    const float sum = half_sum(l[r]);
    if (row[r] >= t.n_rows) continue;
    const int tok = row[r] / a.group;
    if (a.n_splits == 1) {
      const float inv = sum > 0.f ? 1.f / sum : sum != sum ? sum : 0.f;
      T* out = static_cast<T*>(a.o) + (int64_t)(t.q0 + tok) * a.ldo + (int64_t)head[r] * D;
#pragma unroll
      for (int d = 0; d < DF; ++d)
#pragma unroll
        for (int g = 0; g < 4; ++g) {
          const uint2 u = make_uint2(pack2<T>(o[d][r][4 * g] * inv, o[d][r][4 * g + 1] * inv),
                                     pack2<T>(o[d][r][4 * g + 2] * inv, o[d][r][4 * g + 3] * inv));
          *reinterpret_cast<uint2*>(out + d * 32 + g * 8 + hh * 4) = u;
        }
      if (a.lse != nullptr && hh == 0)
        a.lse[(int64_t)(t.q0 + tok) * a.n_heads + head[r]] = (m[r] + __builtin_log2f(sum)) * 0.693147180559945309f;
    } else {
      const int64_t at = (int64_t)split * a.total_q * a.n_heads + (int64_t)(t.q0 + tok) * a.n_heads + head[r];
      if (hh == 0) a.part_ml[at] = make_float2(m[r], sum);
      if (j0 < j1) {
        float* out = a.part_o + at * D;
#pragma unroll
        for (int d = 0; d < DF; ++d)
#pragma unroll
          for (int g = 0; g < 4; ++g)
            *reinterpret_cast<float4*>(out + d * 32 + g * 8 + hh * 4) =
                make_float4(o[d][r][4 * g], o[d][r][4 * g + 1], o[d][r][4 * g + 2], o[d][r][4 * g + 3]);
      }
    }
  }
}

// Joins the splits of a row: one wave per row, lane by lane of D.
template <typename T, int D>
__global__ __launch_bounds__(256) void attn_join_kernel(AttnArgs a) {
  const int64_t rows = (int64_t)a.total_q * a.n_heads;
  const int64_t at = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6);
  const int lane = threadIdx.x & 63;
  if (at >= rows) return;
  constexpr int E = D / 64;
  float m = -INFINITY;
  for (int s = 0; s < a.n_splits; ++s) {
    const float2 ml = a.part_ml[s * rows + at];
    m = fmaxf(m, ml.x);
  }
  const float mu = m == -INFINITY ? 0.f : m;
  float l = 0.f, acc[E];
#pragma unroll
  for (int e = 0; e < E; ++e) acc[e] = 0.f;
  for (int s = 0; s < a.n_splits; ++s) {
    const float2 ml = a.part_ml[s * rows + at];
    if (ml.y == 0.f) continue;  // an empty split has written no sums
    const float w = exp2_fast(ml.x - mu);
    l += w * ml.y;
    const float* p = a.part_o + (s * rows + at) * D + lane * E;
#pragma unroll
    for (int e = 0; e < E; ++e) acc[e] += w * p[e];
  }
  const float inv = l > 0.f ? 1.f / l : l != l ? l : 0.f;
  const int64_t tok = at / a.n_heads;
  T* out = static_cast<T*>(a.o) + tok * a.ldo + (at - tok * a.n_heads) * D + lane * E;
#pragma unroll
  for (int e = 0; e < E; ++e) out[e] = (T)(acc[e] * inv);
  if (a.lse != nullptr && lane == 0) a.lse[at] = (m + __builtin_log2f(l)) * 0.693147180559945309f;
}

}  // namespace

template <typename T, int D>
hipError_t launch_attn(const AttnArgs& a, hipStream_t s) {
  const int tiles = a.total_q * a.group / kAttnRows + a.n_seqs;
  const dim3 grid((unsigned)tiles * a.n_kv, a.n_splits);
  if (a.slopes != nullptr || a.cap_in != 0.f)
    attn_rows_kernel<T, D, 4, 1, true><<<grid, 256, 0, s>>>(a);
  else
    attn_rows_kernel<T, D, 4, 1, false><<<grid, 256, 0, s>>>(a);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess || a.n_splits == 1) return e;
  const int64_t rows = (int64_t)a.total_q * a.n_heads;
  attn_join_kernel<T, D><<<(unsigned)((rows + 3) / 4), 256, 0, s>>>(a);
  return hipGetLastError();
}

}  // namespace ttq
