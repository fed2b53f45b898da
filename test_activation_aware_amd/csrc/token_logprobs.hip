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
template <typename T, int NT>
__global__ __launch_bounds__(NT) void logprobs_kernel(const T* __restrict__ logits, int64_t ldl, int V, int chunk,
                                                      const int64_t* __restrict__ tokens, float* __restrict__ logprob,
                                                      float* __restrict__ entropy, int top,
                                                      int64_t* __restrict__ top_ids, float* __restrict__ top_lp,
                                                      Sum* __restrict__ part, u64* __restrict__ part_keys,
                                                      int groups_max) {
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
  const bool whole = gridDim.y == 1;
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
// with 512 threads).  Long rows: 512 threads, four workgroups a CU (2048 x 151936
// in bf16, 20 alternatives: 123 us, 5.0 TB/s, against 178 with one wave).
int threads_of(int64_t T, int64_t V) { return T >= 1024 && V < 32768 ? 64 : 512; }

struct Call {
  int64_t ldl, rows;
  int V, top;
  const int64_t* tokens;
  float *logprob, *entropy;
  int64_t* top_ids;
  float* top_lp;
  void* ws;
};

template <typename T, int NT>
hipError_t launch_threads(const void* logits, const Call& c, hipStream_t s) {
  const int chunk = chunk_of(c.rows, c.V), chunks = (int)chunks_of(c.rows, c.V);
  const int batch = NT * VecOf<T>::N;  // group maxima are written for whole rounds of vectors
  const int groups = (std::min(chunk, c.V) + batch - 1) / batch * batch / kGroup;
  const int per_bucket = (groups + kBuckets - 1) / kBuckets;
  const int list = c.top > 0 ? c.top * std::max(per_bucket, kGroup) : 0;
  const size_t lds = c.top > 0 ? (size_t)groups * 4 + (size_t)list * 8 : 16;
  Sum* part = static_cast<Sum*>(c.ws);
  u64* keys = reinterpret_cast<u64*>(static_cast<char*>(c.ws) + ((size_t)c.rows * chunks * sizeof(Sum) + 255) / 256 * 256);
  const T* x = static_cast<const T*>(logits);
  logprobs_kernel<T, NT><<<dim3((unsigned)c.rows, chunks), NT, lds, s>>>(
      x, c.ldl, c.V, chunk, c.tokens, c.logprob, c.entropy, c.top, c.top_ids, c.top_lp, part, keys, groups);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess || chunks == 1) return e;
  logprobs_join_kernel<T><<<(unsigned)c.rows, 256, (size_t)std::max(chunks * c.top, 2) * 8, s>>>(
      x, c.ldl, c.V, chunks, c.tokens, c.logprob, c.entropy, c.top, c.top_ids, c.top_lp, part, keys);
  return hipGetLastError();
}

template <typename T>
hipError_t launch(const void* logits, const Call& c, hipStream_t s) {
  return threads_of(c.rows, c.V) == 64 ? launch_threads<T, 64>(logits, c, s) : launch_threads<T, 512>(logits, c, s);
}

}  // namespace

int64_t token_logprobs_threads(int64_t T, int64_t V) { return T * threads_of(T, V); }

size_t token_logprobs_ws_bytes(int64_t T, int64_t V, int top) {
  const int64_t c = chunks_of(T, V);
  if (c <= 1) return 0;
  return ((size_t)T * c * sizeof(Sum) + 255) / 256 * 256 + (size_t)T * c * top * 8;
}

hipError_t launch_token_logprobs(const void* logits, int dtype, int64_t T, int64_t V, int64_t ldl,
                                 const int64_t* tokens, float* logprob, float* entropy, int top, int64_t* top_ids,
                                 float* top_lp, void* ws, hipStream_t s) {
  const Call c = {ldl, T, (int)V, top, tokens, logprob, entropy, top_ids, top_lp, ws};
  switch (dtype) {
    case 0: return launch<float>(logits, c, s);
    case 1: return launch<_Float16>(logits, c, s);
    default: return launch<__bf16>(logits, c, s);
  }
}

}  // namespace ttq
