// Log probabilities of given tokens, the entropy of each row and its most
// likely alternatives, from logits x [T][V] in one read of them:
//   lse = log sum_v e^(x_v),  logprob = x_token - lse,
//   H = -sum_v p_v log p_v = log(sum e^(x - m)) - sum (x - m) e^(x - m) / sum e^(x - m)
// with a running maximum m; all sums in 32 bits, relative to the maximum, so
// that a large common offset of the logits costs nothing.  The difference x - m
// is taken before its scaling to units of log 2: it is exact where it counts,
// and a scaled logit would overflow from 2.4e38 on, or differ from the scaled
// maximum by the rounding of that, which is large beside 1 from 1e8 on.  (2048 x
// 151936 in bf16 take 123.4 us with either; 7 x 50257 in fp32 10.7 us, 10.3 with
// one fma a logit.)
//
// The alternatives need no sorting of the row.  While the row streams by, the
// maximum of each group of 32 consecutive logits goes to LDS (the vector's
// own maximum, which the softmax needs anyway, and two or three steps across
// neighbouring lanes).  In the order by (value, lowest index) the `top` best
// logits lie in the `top` best groups, since every better group holds a better
// logit.  A lower bound for the groups is the top-th best of 64 buckets' best
// groups (every 64th group is a bucket's); about top groups reach it, at most
// top times a bucket's.  Ranks are counted, group against group, then logit
// against logit in the `top` groups, read again from the cache: every
// comparison is between distinct keys, so the result does not depend on any
// order of execution.  NaN ranks below everything.
//
// A row is one workgroup's; where there are few rows it is split into chunks,
// and a second kernel joins the chunks' sums and sorted lists.
//
// The continuations of beams begin with the same pass over the rows: a beam's
// best candidates are among its `keep` best logits, and another second kernel
// joins the rows of a request (beam_join_kernel).
#include "ttq_internal.h"

#include <algorithm>

namespace ttq {

namespace {

constexpr int kBuckets = 64;
constexpr int kGroup = 32;          // logits whose maximum is kept
constexpr int kMaxChunk = 262144;   // logits of a workgroup: 32 KiB of group maxima
constexpr float kLog2e = 1.44269504088896341f, kLn2 = 0.693147180559945309f;

typedef unsigned long long u64;

// a whole number that grows with x; NaN below -inf, -0 equal to 0
__device__ __forceinline__ uint32_t order_of(float x) {
  const uint32_t u = __builtin_bit_cast(uint32_t, x + 0.0f);
  if (x != x) return 0u;
  return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}
__device__ __forceinline__ float value_of(uint32_t o) {
  if (o == 0u) return __builtin_nanf("");
  return __builtin_bit_cast(float, (o & 0x80000000u) ? (o & 0x7FFFFFFFu) : ~o);
}
// larger is better: the value, then the lower index
__device__ __forceinline__ u64 key_of(uint32_t order, uint32_t index) {
  return ((u64)order << 32) | (uint32_t)~index;
}

template <typename T>
struct VecOf {  // 16 bytes of logits at any element's address
  static constexpr int N = 16 / (int)sizeof(T);
  typedef T type __attribute__((ext_vector_type(N), aligned(sizeof(T))));
};

template <int CTRL>
__device__ __forceinline__ float dpp_max(float x) {
  const int y = __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, x), CTRL, 0xF, 0xF, true);
  return fmaxf(x, __builtin_bit_cast(float, y));
}

struct Sum {
  float m, s, t;  // maximum, sum e, sum e d with d = (x - m) log2(e)
};
// How far a maximum lies below a later one mu, in units of log 2.  Cut off where
// the factor 2^d has long been 0: the sums of d take d times a count, which
// would overflow for logits masked by a large finite value, and 0 x inf is NaN.
__device__ __forceinline__ float shift_of(float m, float mu) {
  return m == -INFINITY ? 0.f : fmaxf((m - mu) * kLog2e, -1e4f);
}
__device__ __forceinline__ Sum join(Sum a, Sum b) {
  Sum r;
  r.m = fmaxf(a.m, b.m);
  const float mu = r.m == -INFINITY ? 0.f : r.m;
  const float da = shift_of(a.m, mu), db = shift_of(b.m, mu);
  const float ea = __builtin_amdgcn_exp2f(da), eb = __builtin_amdgcn_exp2f(db);
  r.s = a.s * ea + b.s * eb;
  r.t = ea * (a.t + da * a.s) + eb * (b.t + db * b.s);
  return r;
}

// log p of a logit x of the row
__device__ __forceinline__ float logprob_of(const Sum& r, float x) {
  if (r.m == -INFINITY) return r.s != r.s ? r.s : -INFINITY;
  return (x - r.m) - __builtin_log2f(r.s) * kLn2;
}

// the row's logprob and entropy from its joined sums
__device__ __forceinline__ void finish(const Sum& r, float x_tok, bool has_tok, float* logprob, float* entropy) {
  const float l2 = __builtin_log2f(r.s);
  // a row of -inf alone: no distribution; its log probabilities are -inf, its entropy 0
  const bool none = r.m == -INFINITY;
  *logprob = has_tok ? logprob_of(r, x_tok) : 0.f;
  *entropy = none ? (r.s != r.s ? r.s : 0.f) : (l2 - r.t / r.s) * kLn2;
}

// One chunk of one row.  LDS: group maxima, then the list of candidate keys.
// part: NULL where the row is whole and its results go out at once.  scores: of
// beams, or NULL; a row whose score is not finite has none, and is not read.
template <typename T, int NT>
__global__ __launch_bounds__(NT) void logprobs_kernel(const T* __restrict__ logits, int64_t ldl, int V, int chunk,
                                                      const int64_t* __restrict__ tokens, float* __restrict__ logprob,
                                                      float* __restrict__ entropy, int top,
                                                      int64_t* __restrict__ top_ids, float* __restrict__ top_lp,
                                                      Sum* __restrict__ part, u64* __restrict__ part_keys,
                                                      int groups_max, const float* __restrict__ scores) {
  extern __shared__ __attribute__((aligned(16))) char smem[];
  float* gmax = reinterpret_cast<float*>(smem);
  u64* list = reinterpret_cast<u64*>(smem + (size_t)groups_max * 4);
  __shared__ Sum wsum[NT / 64];
  __shared__ u64 best[NT];
  __shared__ u64 bound;
  __shared__ int count[2];
  __shared__ int sel[kMaxTop];

  typedef typename VecOf<T>::type vec;
  constexpr int N = VecOf<T>::N, U = 4, STEP = NT * N;
  const int tid = threadIdx.x;
  const int64_t row = blockIdx.x;
  const int c0 = blockIdx.y * chunk, len = min(chunk, V - c0);
  const T* x = logits + row * ldl + c0;
  if (scores != nullptr && !(fabsf(scores[row]) < INFINITY)) return;

  Sum r = {-INFINITY, 0.f, 0.f};
  // W vectors of each thread, the first at logit b + tid * N.  Places past the
  // row are -inf for the sums; for their group's maximum they are NaN, which
  // every logit is at least as good as (with -inf there, a last group of NaN
  // would pass for one with a number in it).
  auto take = [&](auto& f, int b) {
    constexpr int W = sizeof(f) / sizeof(f[0]);
    float bm = -INFINITY;
#pragma unroll
    for (int u = 0; u < W; ++u) {
      auto at = [&](int e) { return W > 1 || b + tid * N + e < len ? f[u][e] : __builtin_nanf(""); };
      float vm = at(0);
#pragma unroll
      for (int e = 1; e < N; ++e) vm = fmaxf(vm, at(e));
      bm = fmaxf(bm, vm);
      if (top > 0) {
        vm = dpp_max<0xB1>(vm);                         // lane ^ 1
        vm = dpp_max<0x4E>(vm);                         // lane ^ 2
        if constexpr (N == 4) vm = dpp_max<0x141>(vm);  // the other four of eight lanes
        gmax[(b + u * STEP + tid * N) / kGroup] = vm;   // the same from each lane of a group
      }
    }
    const float mn = fmaxf(r.m, bm);
    const float mu = mn == -INFINITY ? 0.f : mn;
    const float dm = shift_of(r.m, mu);
    const float al = __builtin_amdgcn_exp2f(dm);
    r.t = al * (r.t + dm * r.s);
    r.s *= al;
    r.m = mn;
    float t = r.t;
#pragma unroll
    for (int u = 0; u < W; ++u)
#pragma unroll
      for (int e = 0; e < N; ++e) {
        const float d = (f[u][e] - mu) * kLog2e;
        const float p = __builtin_amdgcn_exp2f(d);
        r.s += p;
        t = __builtin_fmaf(p, d, t);
      }
    if (t != t) {  // -inf among them: p is 0, and its term too
      t = r.t;
#pragma unroll
      for (int u = 0; u < W; ++u)
#pragma unroll
        for (int e = 0; e < N; ++e) {
          const float d = (f[u][e] - mu) * kLog2e;
          t = __builtin_fmaf(__builtin_amdgcn_exp2f(d), fmaxf(d, -1e4f), t);
        }
    }
    r.t = t;
  };
  int b = 0;
  if (len >= U * STEP) {  // whole batches, the next one requested before this one is worked on
    vec v[U];
#pragma unroll
    for (int u = 0; u < U; ++u) v[u] = *reinterpret_cast<const vec*>(x + u * STEP + tid * N);
    for (; b + U * STEP <= len; b += U * STEP) {
      float f[U][N];
#pragma unroll
      for (int u = 0; u < U; ++u)
#pragma unroll
        for (int e = 0; e < N; ++e) f[u][e] = (float)v[u][e];
      if (b + 2 * U * STEP <= len)
#pragma unroll
        for (int u = 0; u < U; ++u) v[u] = *reinterpret_cast<const vec*>(x + b + (U + u) * STEP + tid * N);
      take(f, b);
    }
  }
  for (; b < len; b += STEP) {  // what is left, a vector at a time
    float f[1][N];
    const int i = b + tid * N;
    if (i + N <= len) {
      const vec v = *reinterpret_cast<const vec*>(x + i);
#pragma unroll
      for (int e = 0; e < N; ++e) f[0][e] = (float)v[e];
    } else {
#pragma unroll
      for (int e = 0; e < N; ++e) f[0][e] = i + e < len ? (float)x[i + e] : -INFINITY;
    }
    take(f, b);
  }

  // the workgroup's sums, in a fixed order
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) {
    const Sum q = {__shfl_xor(r.m, o), __shfl_xor(r.s, o), __shfl_xor(r.t, o)};
    r = join(r, q);
  }
  if ((tid & 63) == 0) wsum[tid >> 6] = r;
  if (tid < 2) count[tid] = 0;
  __syncthreads();
  r = wsum[0];
#pragma unroll
  for (int w = 1; w < NT / 64; ++w) r = join(r, wsum[w]);
  const bool whole = part == nullptr;
  if (tid == 0) {
    if (whole) {
      const int64_t tok = tokens[row];
      const bool has = tok >= 0 && tok < V;
      finish(r, has ? (float)x[tok] : 0.f, has, logprob + row, entropy + row);
    } else {
      part[row * gridDim.y + blockIdx.y] = r;
    }
  }
  if (top <= 0) return;

  // the bound: the top-th best of the buckets' best groups (NT is a multiple
  // of 64, so a lane's groups are one bucket's)
  const int groups = (len + kGroup - 1) / kGroup;
  u64 mine = 0;
  for (int g = tid; g < groups; g += NT) {
    const u64 k = key_of(order_of(gmax[g]), (uint32_t)g);
    mine = k > mine ? k : mine;
  }
  best[tid] = mine;
  __syncthreads();
  if (tid < kBuckets) {
#pragma unroll
    for (int w = 1; w < NT / 64; ++w) {
      const u64 k = best[w * 64 + tid];
      mine = k > mine ? k : mine;
    }
    int rank = 0;
#pragma unroll
    for (int i = 0; i < kBuckets; ++i) {
      const u64 k = ((u64)(uint32_t)__builtin_amdgcn_readlane((int)(mine >> 32), i) << 32) |
                    (uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)mine, i);
      rank += k > mine;
    }
    // fewer buckets than `top` with a group: every group is a candidate
    const unsigned long long is = __ballot(mine != 0 && rank == top - 1);
    if (is == 0 ? tid == 0 : (is >> tid) & 1) bound = is == 0 ? 0 : mine;
  }
  __syncthreads();
  for (int g = tid; g < groups; g += NT) {
    const u64 k = key_of(order_of(gmax[g]), (uint32_t)g);
    if (k >= bound) list[atomicAdd(&count[0], 1)] = k;
  }
  __syncthreads();
  const int n1 = count[0];
  const int sure = min(top, n1);
  for (int i = tid; i < n1; i += NT) {
    const u64 k = list[i];
    int rank = 0;
    for (int j = 0; j < n1; ++j) rank += list[j] > k;
    if (rank < sure) sel[rank] = (int)~(uint32_t)k;
    if (rank == sure - 1) bound = k;  // nothing below this group's maximum is among the best
  }
  __syncthreads();
  const uint32_t floor_order = n1 >= top ? (uint32_t)(bound >> 32) : 0u;
  for (int i = tid; i < sure * kGroup; i += NT) {
    const int e = sel[i / kGroup] * kGroup + i % kGroup;
    if (e < len) {
      const uint32_t o = order_of((float)x[e]);
      if (o >= floor_order) list[atomicAdd(&count[1], 1)] = key_of(o, (uint32_t)(c0 + e));
    }
  }
  __syncthreads();
  const int n2 = count[1];
  for (int i = tid; i < n2; i += NT) {
    const u64 k = list[i];
    int rank = 0;
    for (int j = 0; j < n2; ++j) rank += list[j] > k;
    if (rank < top) {
      if (whole) {
        top_ids[row * top + rank] = (int64_t)(uint32_t)~(uint32_t)k;
        top_lp[row * top + rank] = logprob_of(r, value_of((uint32_t)(k >> 32)));
      } else {
        part_keys[(row * gridDim.y + blockIdx.y) * top + rank] = k;
      }
    }
  }
  // a chunk shorter than `top` logits leaves places: keys of nothing
  if (!whole)
    for (int i = n2 + tid; i < top; i += NT) part_keys[(row * gridDim.y + blockIdx.y) * top + i] = 0;
}

// Joins the chunks of a row: the sums in order, and the sorted lists, where a
// key's rank is the number of better keys in each list, found by bisection.
template <typename T>
__global__ __launch_bounds__(256) void logprobs_join_kernel(const T* __restrict__ logits, int64_t ldl, int V,
                                                            int chunks, const int64_t* __restrict__ tokens,
                                                            float* __restrict__ logprob, float* __restrict__ entropy,
                                                            int top, int64_t* __restrict__ top_ids,
                                                            float* __restrict__ top_lp, const Sum* __restrict__ part,
                                                            const u64* __restrict__ part_keys) {
  extern __shared__ __attribute__((aligned(16))) char smem[];
  u64* keys = reinterpret_cast<u64*>(smem);
  const int tid = threadIdx.x;
  const int64_t row = blockIdx.x;
  const int n = chunks * top;
  const int64_t tok = tokens[row];
  const bool has = tok >= 0 && tok < V;
  const float x = has ? (float)logits[row * ldl + tok] : 0.f;
  Sum r = {-INFINITY, 0.f, 0.f};
  if ((tid & 63) < chunks) r = part[row * chunks + (tid & 63)];  // at most 64 chunks
  for (int i = tid; i < n; i += 256) keys[i] = part_keys[row * n + i];
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) {
    const Sum q = {__shfl_xor(r.m, o), __shfl_xor(r.s, o), __shfl_xor(r.t, o)};
    r = join(r, q);
  }
  if (tid == 0) finish(r, x, has, logprob + row, entropy + row);
  __syncthreads();
  for (int i = tid; i < n; i += 256) {
    const u64 k = keys[i];
    if (k == 0) continue;
    int rank = 0;
    for (int c = 0; c < chunks; ++c) {
      int lo = 0, hi = top;  // better keys in this list
      while (lo < hi) {
        const int mid = (lo + hi) / 2;
        if (keys[c * top + mid] > k) lo = mid + 1; else hi = mid;
      }
      rank += lo;
    }
    if (rank < top) {
      top_ids[row * top + rank] = (int64_t)(uint32_t)~(uint32_t)k;
      top_lp[row * top + rank] = logprob_of(r, value_of((uint32_t)(k >> 32)));
    }
  }
}

// The candidates of a request in LDS, and their order: by total, of equal ones the
// earlier beam, then the larger logit, then the lower token.
struct Candidates {
  double* total;
  u64* key;
  int* beam;
  __device__ __forceinline__ Candidates(char* at, int n)
      : total(reinterpret_cast<double*>(at)), key(reinterpret_cast<u64*>(at + (size_t)n * 8)),
        beam(reinterpret_cast<int*>(at + (size_t)n * 16)) {}
  static constexpr int kBytes = 20;
  // How many of n are better than one of them.  The totals alone first, without a
  // branch, so that the reads of several are in flight together (with one in the
  // loop each of them took 170 ns).
  __device__ __forceinline__ int rank(int n, double t, u64 k, int w) const {
    int r = 0, same = 0;
#pragma unroll 8
    for (int b = 0; b < n; ++b) {
      const double u = total[b];
      r += u > t;
      same += u == t;
    }
    if (same > 1) {
#pragma unroll 8
      for (int b = 0; b < n; ++b) {
        const double u = total[b];
        const u64 l = key[b];
        const int v = beam[b];
        r += (u == t) & ((v < w) | ((v == w) & (l > k)));
      }
    }
    return r;
  }
};

// Places of each list that the bound is found from: four times as many as are
// kept, in all, or one each.
__host__ __device__ inline int beam_depth(int lists, int top, int keep) {
  const int deep = (4 * keep + lists - 1) / lists;
  return deep < top ? deep : top;
}
// Candidates in LDS at most: these, then those that the bound lets through, keep
// and the rest of the lists whose places are all among the best.
inline int beam_room(int lists, int top, int keep) {
  const int deep = beam_depth(lists, top, keep);
  return std::max(lists * deep, std::min(lists * top, keep + keep / deep * (top - deep)));
}

// A request's `keep` best continuations out of its beams' sorted lists, one a
// chunk of a row, and the histories that they continue.  Totals are in 64 bits:
// score + (x - lse), so that the order of two beams' candidates does not hang on
// the rounding of a sum of some tens; the rows' sums are good to a few 2^-24 of
// themselves.  Ranks are counted, one against another: first among some of each
// list, whose keep-th best is a bound, then among what reaches that.
//
// Several workgroups of a request find the same and copy a part of the histories
// each.  Bound by a launch and the chain of loads, barriers and comparisons: 13 us for
// 48 requests of 8 beams, 16 kept, histories of 500 (the pass over their 151936 logits
// in bf16: 33 us, 3.5 TB/s); 6 us for one of 4 beams.
__global__ __launch_bounds__(256) void beam_join_kernel(const float* __restrict__ scores, int beams, int chunks, int top, int keep,
                                                        int room, const Sum* __restrict__ part, const u64* __restrict__ part_keys,
                                                        float* __restrict__ out_scores, int64_t* __restrict__ parents,
                                                        int64_t* __restrict__ tokens, const int64_t* __restrict__ history,
                                                        int64_t ldh, int64_t length, int64_t* __restrict__ out_history,
                                                        int64_t ldo) {
  extern __shared__ __attribute__((aligned(16))) char smem[];
  const Candidates some(smem, room);
  __shared__ double score[kMaxBeams], lse[kMaxBeams], best_total[kMaxTop], bound_total;
  __shared__ u64 bound_key;
  __shared__ int best_beam[kMaxTop], best_token[kMaxTop], bound_beam, count;
  const int tid = threadIdx.x, lane = tid & 63;
  const int64_t request = blockIdx.x, row0 = request * beams;
  const int lists = beams * chunks, n = lists * top;
  const u64* keys = part_keys + row0 * chunks * top;

  for (int w = tid >> 6; w < beams; w += 4) {  // the row's sum, a chunk a lane: at most 64
    const float s = scores[row0 + w];
    const bool has = fabsf(s) < INFINITY && lane < chunks;
    Sum r = {-INFINITY, 0.f, 0.f};
    if (has) r = part[(row0 + w) * chunks + lane];
    float m = r.m;
#pragma unroll
    for (int o = 32; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor(m, o));
    // a factor of 2^-1e4 is 0 here too
    double sum = r.m == -INFINITY ? (double)r.s : (double)r.s * exp2((double)shift_of(r.m, m));
#pragma unroll
    for (int o = 32; o > 0; o >>= 1) sum += __shfl_xor(sum, o);
    if (lane == 0) {
      // an empty beam has left nothing: no number, whatever lies in its lists
      score[w] = fabsf(s) < INFINITY ? (double)s : __builtin_nan("");
      lse[w] = m == -INFINITY ? __builtin_nan("") : (double)m + log(sum);
    }
  }
  if (tid < keep) best_beam[tid] = -1;
  if (tid == 0) {
    bound_total = -INFINITY;
    bound_key = 0;
    bound_beam = kMaxBeams;
    count = 0;
  }
  __syncthreads();

  // -inf for keys of nothing, of NaN and of -inf, and for totals that are no number
  auto total_of = [&](u64 k, int w) {
    const double t = score[w] + ((double)value_of((uint32_t)(k >> 32)) - lse[w]);
    return k != 0 && t > -(double)INFINITY ? t : -(double)INFINITY;
  };
  const int deep = beam_depth(lists, top, keep), first = lists * deep;
  if (first >= keep) {
    for (int a = tid; a < first; a += 256) {
      const int list = a / deep, w = list / chunks;
      const u64 k = keys[list * top + a % deep];
      some.total[a] = total_of(k, w);
      some.key[a] = k;
      some.beam[a] = w;
    }
    __syncthreads();
    for (int a = tid; a < first; a += 256) {
      const double t = some.total[a];
      if (t == -(double)INFINITY || some.rank(first, t, some.key[a], some.beam[a]) != keep - 1) continue;
      bound_total = t;
      bound_key = some.key[a];
      bound_beam = some.beam[a];
    }
    __syncthreads();
  }
  const double least = bound_total;
  const u64 least_key = bound_key;
  const int least_beam = bound_beam;
  for (int i = tid; i < n; i += 256) {
    const u64 k = keys[i];
    const int w = i / top / chunks;
    const double t = total_of(k, w);
    if (t == -(double)INFINITY || t < least) continue;
    if (t == least && (w != least_beam ? w > least_beam : k < least_key)) continue;
    const int at = atomicAdd(&count, 1);
    some.total[at] = t;
    some.key[at] = k;
    some.beam[at] = w;
  }
  __syncthreads();
  const int may = count;
  for (int i = tid; i < may; i += 256) {
    const int rank = some.rank(may, some.total[i], some.key[i], some.beam[i]);
    if (rank >= keep) continue;
    best_total[rank] = some.total[i];
    best_beam[rank] = some.beam[i];
    best_token[rank] = (int)~(uint32_t)some.key[i];
  }
  __syncthreads();
  if (blockIdx.y == 0 && tid < keep) {
    const bool none = best_beam[tid] < 0;
    out_scores[request * keep + tid] = none ? -INFINITY : (float)best_total[tid];
    parents[request * keep + tid] = none ? -1 : best_beam[tid];
    tokens[request * keep + tid] = none ? -1 : best_token[tid];
  }
  if (out_history == nullptr) return;
  // rows of length + 1, the parent's and then the token; some loads of a thread in
  // flight together
  const int64_t cells = (length + 1) * keep, step = (int64_t)gridDim.y * 256;
  for (int64_t i0 = (int64_t)blockIdx.y * 256 + tid; i0 < cells; i0 += 4 * step) {
    int64_t x[4], at[4];
    int k[4];
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const int64_t i = min(i0 + u * step, cells - 1);
      k[u] = cells <= 0x7FFFFFFF ? (int)((uint32_t)i / (uint32_t)(length + 1)) : (int)(i / (length + 1));
      at[u] = i - k[u] * (length + 1);
      const int w = best_beam[k[u]];
      x[u] = w < 0 ? -1 : best_token[k[u]];
      if (w >= 0 && at[u] < length) x[u] = history[(row0 + w) * ldh + at[u]];
    }
#pragma unroll
    for (int u = 0; u < 4; ++u)
      if (i0 + u * step < cells) out_history[(request * keep + k[u]) * ldo + at[u]] = x[u];
  }
}

// Logits of a workgroup.  A row is cut only where the rows leave CUs idle and
// are long enough to pay for the join, into chunks of 24576 or more, as many as
// fill the 256 CUs once (bf16 logits of 1 x 151936: 12.5 us in 6 chunks, 16.9
// in one; 32 rows in fp32: 14.5 and 21.3; 7 x 50257 in fp32: 10.5 in one, 11.7
// in 3).
int chunk_of(int64_t T, int64_t V) {
  int64_t want = 1;
  if (V >= 4 * 24576 && T > 0) want = std::max<int64_t>(1, std::min<int64_t>({256 / T, V / 24576, 64}));
  const int64_t c = std::min<int64_t>((V + want - 1) / want, kMaxChunk);
  return (int)((c + 255) / 256 * 256);
}
int64_t chunks_of(int64_t T, int64_t V) {
  const int c = chunk_of(T, V);
  return (V + c - 1) / c;
}

// Threads of a workgroup.  Many short rows: a wave each, so that many selections
// run beside each other (16000 x 500 in fp32, 10 alternatives: 25 us against 91
// with 512 threads).  Long rows: 512 threads, four workgroups a CU with logits in
// fp32 and two in 16 bits, whose vectors take 92 registers (2048 x 151936 in bf16, 20
// alternatives: 123 us, 5.0 TB/s, against 178 with one wave).
int threads_of(int64_t T, int64_t V) { return T >= 1024 && V < 32768 ? 64 : 512; }

struct Call {
  int64_t ldl, rows;
  int V, top, chunk;
  const int64_t* tokens;
  float *logprob, *entropy;
  int64_t* top_ids;
  float* top_lp;
  void* ws;
  const float* scores;  // of beams: the rows' sums and keys are left in ws
};

template <typename T, int NT>
hipError_t launch_threads(const void* logits, const Call& c, hipStream_t s) {
  const int chunk = c.chunk, chunks = (c.V + chunk - 1) / chunk;
  const int batch = NT * VecOf<T>::N;  // group maxima are written for whole rounds of vectors
  const int groups = (std::min(chunk, c.V) + batch - 1) / batch * batch / kGroup;
  const int per_bucket = (groups + kBuckets - 1) / kBuckets;
  const int list = c.top > 0 ? c.top * std::max(per_bucket, kGroup) : 0;
  const size_t lds = c.top > 0 ? (size_t)groups * 4 + (size_t)list * 8 : 16;
  Sum* part = static_cast<Sum*>(c.ws);
  u64* keys = reinterpret_cast<u64*>(static_cast<char*>(c.ws) + ((size_t)c.rows * chunks * sizeof(Sum) + 255) / 256 * 256);
  const T* x = static_cast<const T*>(logits);
  logprobs_kernel<T, NT><<<dim3((unsigned)c.rows, chunks), NT, lds, s>>>(
      x, c.ldl, c.V, chunk, c.tokens, c.logprob, c.entropy, c.top, c.top_ids, c.top_lp,
      chunks > 1 || c.scores != nullptr ? part : nullptr, keys, groups, c.scores);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess || chunks == 1 || c.scores != nullptr) return e;
  logprobs_join_kernel<T><<<(unsigned)c.rows, 256, (size_t)std::max(chunks * c.top, 2) * 8, s>>>(
      x, c.ldl, c.V, chunks, c.tokens, c.logprob, c.entropy, c.top, c.top_ids, c.top_lp, part, keys);
  return hipGetLastError();
}

template <typename T>
hipError_t launch(const void* logits, const Call& c, hipStream_t s) {
  return threads_of(c.rows, c.V) == 64 ? launch_threads<T, 64>(logits, c, s) : launch_threads<T, 512>(logits, c, s);
}

// Places of a beam's list: its best candidates are among its `keep` best logits.
int beam_top(int64_t V, int keep) { return (int)std::min<int64_t>(V, keep); }

// Logits of a workgroup for beams.  They are joined in any case, so that rows are
// cut while there are at most 1024 workgroups, the four a CU that fp32 logits have
// room for; of 16-bit ones two fit (48 x 8 beams over 151936 in bf16, 16 kept: 47 us
// in two chunks a row, one and a half rounds of those, 60 in one, 63 in five), into
// chunks of 8192 or more (32 x 4 over 32000 in fp16: 17 us in three, 23 in seven), as
// long as a request has no more than 32 lists to join (16 x 4 over 151936: 19 us with
// 32, 26 with 64; 1 x 8: 20 with 32, 31 with 256).
int beam_chunk_of(int64_t rows, int beams, int64_t V) {
  const int64_t lists = std::max(1, 32 / beams);
  const int64_t want = std::max<int64_t>(1, std::min<int64_t>({1024 / std::max<int64_t>(rows, 1), V / 8192, lists, 64}));
  const int64_t c = std::min<int64_t>((V + want - 1) / want, kMaxChunk);
  return (int)((c + 255) / 256 * 256);
}

}  // namespace

size_t beam_select_ws_bytes(int64_t requests, int beams, int64_t V, int keep) {
  const int64_t rows = requests * beams, chunk = beam_chunk_of(rows, beams, V), c = (V + chunk - 1) / chunk;
  return ((size_t)rows * c * sizeof(Sum) + 255) / 256 * 256 + (size_t)rows * c * beam_top(V, keep) * 8;
}

// A few tokens of the histories for each thread.
int64_t beam_history_groups(int keep, int64_t length) {
  return std::max<int64_t>(1, std::min<int64_t>(64, (length + 1) * keep / 1024));
}

hipError_t launch_beam_select(const void* logits, int dtype, int64_t requests, int beams, int64_t V, int64_t ldl,
                              const float* scores, int keep, float* out_scores, int64_t* parents, int64_t* tokens,
                              const int64_t* history, int64_t ldh, int64_t length, int64_t* out_history, int64_t ldo, void* ws,
                              hipStream_t s) {
  const int64_t rows = requests * beams;
  const int top = beam_top(V, keep), chunk = beam_chunk_of(rows, beams, V), chunks = (int)((V + chunk - 1) / chunk);
  const Call c = {ldl, rows, (int)V, top, chunk, nullptr, nullptr, nullptr, nullptr, nullptr, ws, scores};
  const hipError_t e = dtype == 0 ? launch<float>(logits, c, s) : dtype == 1 ? launch<_Float16>(logits, c, s) : launch<__bf16>(logits, c, s);
  if (e != hipSuccess) return e;
  const Sum* part = static_cast<const Sum*>(ws);
  const u64* keys = reinterpret_cast<const u64*>(static_cast<const char*>(ws) + ((size_t)rows * chunks * sizeof(Sum) + 255) / 256 * 256);
  const unsigned copies = out_history != nullptr ? (unsigned)beam_history_groups(keep, length) : 1;
  const int room = beam_room(beams * chunks, top, keep);
  beam_join_kernel<<<dim3((unsigned)requests, copies), 256, (size_t)room * Candidates::kBytes, s>>>(
      scores, beams, chunks, top, keep, room, part, keys, out_scores, parents, tokens, history, ldh, length, out_history, ldo);
  return hipGetLastError();
}

int64_t token_logprobs_threads(int64_t T, int64_t V) { return T * threads_of(T, V); }

size_t token_logprobs_ws_bytes(int64_t T, int64_t V, int top) {
  const int64_t c = chunks_of(T, V);
  if (c <= 1) return 0;
  return ((size_t)T * c * sizeof(Sum) + 255) / 256 * 256 + (size_t)T * c * top * 8;
}

hipError_t launch_token_logprobs(const void* logits, int dtype, int64_t T, int64_t V, int64_t ldl,
                                 const int64_t* tokens, float* logprob, float* entropy, int top, int64_t* top_ids,
                                 float* top_lp, void* ws, hipStream_t s) {
  const Call c = {ldl, T, (int)V, top, chunk_of(T, V), tokens, logprob, entropy, top_ids, top_lp, ws, nullptr};
  switch (dtype) {
    case 0: return launch<float>(logits, c, s);
    case 1: return launch<_Float16>(logits, c, s);
    default: return launch<__bf16>(logits, c, s);
  }
}

}  // namespace ttq
