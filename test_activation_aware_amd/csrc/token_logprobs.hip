// Log probabilities of given tokens, the entropy of each row and its most
// likely alternatives, from logits x [T][V] in one read of them:
//   lse = log sum_v e^(x_v),  logprob = x_token - lse,
//   H = -sum_v p_v log p_v = log(sum e^(x - m)) - sum (x - m) e^(x - m) / sum e^(x - m)
// with a running maximum m; all sums in 32 bits, in units of log 2 relative
// to the maximum, so that a large common offset of the logits costs nothing.
//
// The alternatives need no sorting of the row.  While the row streams by, the
// maximum of each group of 32 consecutive logits goes to LDS (the vector's
// own maximum, which the softmax needs anyway, and two or three steps across
// neighbouring lanes).  In the order by (value, lowest index) the `top` best
// logits lie in the `top` best groups, since every better group holds a better
// logit.  A lower bound for the groups is the top-th best of the threads' best
// groups (each thread looks after every kThreads-th group); at most
// top * (groups per thread) groups reach it.  Ranks are counted, group against
// group, then logit against logit in the `top` groups, read again from the
// cache: every comparison is between distinct keys, so the result does not
// depend on any order of execution.  NaN ranks below everything.
//
// A row is split into chunks when there are too few rows to fill the GPU (and
// so that a chunk's groups fit LDS); a second kernel joins the chunks' sums
// and sorted lists.
#include "ttq_internal.h"

#include <type_traits>

namespace ttq {

namespace {

constexpr int kThreads = 256;
constexpr int kGroup = 32;          // logits whose maximum is kept
constexpr int kMaxChunk = 131072;   // logits of a workgroup: 16 KiB of group maxima
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
  float m, s, t;  // maximum (log 2 units), sum e, sum e d with d = x log2(e) - m
};
__device__ __forceinline__ Sum join(Sum a, Sum b) {
  Sum r;
  r.m = fmaxf(a.m, b.m);
  const float mu = r.m == -INFINITY ? 0.f : r.m;
  const float da = a.m == -INFINITY ? 0.f : a.m - mu, db = b.m == -INFINITY ? 0.f : b.m - mu;
  const float ea = __builtin_amdgcn_exp2f(da), eb = __builtin_amdgcn_exp2f(db);
  r.s = a.s * ea + b.s * eb;
  r.t = ea * (a.t + da * a.s) + eb * (b.t + db * b.s);
  return r;
}

// log p of a logit x of the row
__device__ __forceinline__ float logprob_of(const Sum& r, float x) {
  if (r.m == -INFINITY) return r.s != r.s ? r.s : -INFINITY;
  return (__builtin_fmaf(x, kLog2e, -r.m) - __builtin_log2f(r.s)) * kLn2;
}

// the row's logprob and entropy from its joined sums
__device__ __forceinline__ void finish(const Sum& r, float x_tok, bool has_tok, float* logprob, float* entropy) {
  const float l2 = __builtin_log2f(r.s);
  // a row of -inf alone: no distribution; its log probabilities are -inf, its entropy 0
  const bool none = r.m == -INFINITY;
  *logprob = has_tok ? logprob_of(r, x_tok) : 0.f;
  *entropy = none ? (r.s != r.s ? r.s : 0.f) : (l2 - r.t / r.s) * kLn2;
}

template <typename T>
__device__ __forceinline__ float load1(const T* p) {
  return (float)*p;
}

// One chunk of one row.  LDS: group maxima, then the list of candidate keys.
template <typename T>
__global__ __launch_bounds__(kThreads) void logprobs_kernel(const T* __restrict__ logits, int64_t ldl, int V,
                                                            int chunk, const int64_t* __restrict__ tokens,
                                                            float* __restrict__ logprob, float* __restrict__ entropy,
                                                            int top, int64_t* __restrict__ top_ids,
                                                            float* __restrict__ top_lp, Sum* __restrict__ part,
                                                            u64* __restrict__ part_keys, int groups_max) {
  extern __shared__ __attribute__((aligned(16))) char smem[];
  float* gmax = reinterpret_cast<float*>(smem);
  u64* list = reinterpret_cast<u64*>(smem + (size_t)groups_max * 4);
  __shared__ Sum wsum[kThreads / 64];
  __shared__ u64 best[kThreads];
  __shared__ u64 bound;
  __shared__ int count[2];
  __shared__ int sel[64];

  typedef typename VecOf<T>::type vec;
  constexpr int N = VecOf<T>::N, U = 4;
  const int tid = threadIdx.x;
  const int64_t row = blockIdx.x;
  const int c0 = blockIdx.y * chunk, len = min(chunk, V - c0);
  const T* x = logits + row * ldl + c0;

  Sum r = {-INFINITY, 0.f, 0.f};
  for (int b = tid * N; b - tid * N < len; b += kThreads * N * U) {
    float f[U][N];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int i = b + u * kThreads * N;
      if (i + N <= len) {
        const vec v = *reinterpret_cast<const vec*>(x + i);
#pragma unroll
        for (int e = 0; e < N; ++e) f[u][e] = (float)v[e];
      } else {
#pragma unroll
        for (int e = 0; e < N; ++e) f[u][e] = i + e < len ? load1(x + i + e) : -INFINITY;
      }
    }
    float bm = -INFINITY;
#pragma unroll
    for (int u = 0; u < U; ++u) {
      float vm = f[u][0];
#pragma unroll
      for (int e = 1; e < N; ++e) vm = fmaxf(vm, f[u][e]);
      bm = fmaxf(bm, vm);
      if (top > 0) {
        vm = dpp_max<0xB1>(vm);   // lane ^ 1
        vm = dpp_max<0x4E>(vm);   // lane ^ 2
        if constexpr (N == 4) vm = dpp_max<0x141>(vm);  // the other four of eight lanes
        const int i = b + u * kThreads * N;
        if (i % kGroup == 0 && i < len) gmax[i / kGroup] = vm;
      }
    }
    const float mn = fmaxf(r.m, bm * kLog2e);
    const float mu = mn == -INFINITY ? 0.f : mn;
    const float dm = r.m == -INFINITY ? 0.f : r.m - mu;
    const float al = __builtin_amdgcn_exp2f(dm);
    r.t = al * (r.t + dm * r.s);
    r.s *= al;
    r.m = mn;
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
      for (int e = 0; e < N; ++e) {
        const float d = __builtin_fmaf(f[u][e], kLog2e, -mu);
        const float p = __builtin_amdgcn_exp2f(d);
        r.s += p;
        r.t = __builtin_fmaf(p, fmaxf(d, -1e4f), r.t);  // -inf: p is 0, its term 0 too
      }
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
  for (int w = 1; w < kThreads / 64; ++w) r = join(r, wsum[w]);
  const bool whole = gridDim.y == 1;
  if (tid == 0) {
    if (whole) {
      const int64_t tok = tokens[row];
      const bool has = tok >= 0 && tok < V;
      finish(r, has ? load1(x + tok) : 0.f, has, logprob + row, entropy + row);
    } else {
      part[row * gridDim.y + blockIdx.y] = r;
    }
  }
  if (top <= 0) return;

  // the bound: the top-th best of the threads' best groups
  const int groups = (len + kGroup - 1) / kGroup;
  u64 mine = 0;
  for (int g = tid; g < groups; g += kThreads) {
    const u64 k = key_of(order_of(gmax[g]), (uint32_t)g);
    mine = k > mine ? k : mine;
  }
  best[tid] = mine;
  if (tid == 0) bound = 0;
  __syncthreads();
  {
    int rank = 0;
    for (int i = 0; i < kThreads; ++i) rank += best[i] > mine;
    if (mine != 0 && rank == top - 1) bound = mine;
  }
  __syncthreads();
  for (int g = tid; g < groups; g += kThreads) {
    const u64 k = key_of(order_of(gmax[g]), (uint32_t)g);
    if (k >= bound) list[atomicAdd(&count[0], 1)] = k;
  }
  __syncthreads();
  const int n1 = count[0];
  const int take = min(top, n1);
  for (int i = tid; i < n1; i += kThreads) {
    const u64 k = list[i];
    int rank = 0;
    for (int j = 0; j < n1; ++j) rank += list[j] > k;
    if (rank < take) sel[rank] = (int)~(uint32_t)k;
    if (rank == take - 1) bound = k;  // nothing below this group's maximum is among the best
  }
  __syncthreads();
  const uint32_t floor_order = n1 >= top ? (uint32_t)(bound >> 32) : 0u;
  for (int i = tid; i < take * kGroup; i += kThreads) {
    const int e = sel[i / kGroup] * kGroup + i % kGroup;
    if (e < len) {
      const uint32_t o = order_of(load1(x + e));
      if (o >= floor_order) list[atomicAdd(&count[1], 1)] = key_of(o, (uint32_t)(c0 + e));
    }
  }
  __syncthreads();
  const int n2 = count[1];
  for (int i = tid; i < n2; i += kThreads) {
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
    for (int i = n2 + tid; i < top; i += kThreads) part_keys[(row * gridDim.y + blockIdx.y) * top + i] = 0;
}

// Joins the chunks of a row: the sums in order, and the sorted lists, where a
// key's rank is the number of better keys in each list, found by bisection.
template <typename T>
__global__ __launch_bounds__(kThreads) void logprobs_join_kernel(const T* __restrict__ logits, int64_t ldl, int V,
                                                                 int chunks, const int64_t* __restrict__ tokens,
                                                                 float* __restrict__ logprob,
                                                                 float* __restrict__ entropy, int top,
                                                                 int64_t* __restrict__ top_ids,
                                                                 float* __restrict__ top_lp,
                                                                 const Sum* __restrict__ part,
                                                                 const u64* __restrict__ part_keys) {
  extern __shared__ __attribute__((aligned(16))) char smem[];
  u64* keys = reinterpret_cast<u64*>(smem);
  const int tid = threadIdx.x;
  const int64_t row = blockIdx.x;
  const int n = chunks * top;
  for (int i = tid; i < n; i += kThreads) keys[i] = part_keys[row * n + i];
  Sum r = part[row * chunks];
  for (int c = 1; c < chunks; ++c) r = join(r, part[row * chunks + c]);
  if (tid == 0) {
    const int64_t tok = tokens[row];
    const bool has = tok >= 0 && tok < V;
    finish(r, has ? load1(logits + row * ldl + tok) : 0.f, has, logprob + row, entropy + row);
  }
  __syncthreads();
  for (int i = tid; i < n; i += kThreads) {
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

// Logits of a workgroup.  One row fills a workgroup when there are enough of
// them (kFill: four workgroups for each of the 256 CUs); fewer rows are cut
// into chunks of at least 4096 logits, at most 64 of them.
constexpr int64_t kFill = 1024;
int chunk_of(int64_t T, int64_t V) {
  int64_t want = T > 0 ? (kFill + T - 1) / T : 1;
  if (want > 64) want = 64;
  int64_t c = (V + want - 1) / want;
  if (c < 4096) c = 4096;
  if (c > kMaxChunk) c = kMaxChunk;
  return (int)((c + 255) / 256 * 256);
}
int64_t chunks_of(int64_t T, int64_t V) {
  const int c = chunk_of(T, V);
  return (V + c - 1) / c;
}

template <typename T>
hipError_t launch(const void* logits, int64_t ldl, int64_t rows, int V, const int64_t* tokens, float* logprob,
                  float* entropy, int top, int64_t* top_ids, float* top_lp, void* ws, hipStream_t s) {
  const int chunk = chunk_of(rows, V), chunks = (int)chunks_of(rows, V);
  const int groups = (min(chunk, V) + kGroup - 1) / kGroup;
  const int per_thread = (groups + kThreads - 1) / kThreads;
  const int list = top > 0 ? top * max(per_thread, kGroup) : 0;
  const size_t lds = top > 0 ? (size_t)((groups + 3) & ~3) * 4 + (size_t)list * 8 : 16;
  Sum* part = static_cast<Sum*>(ws);
  u64* keys = reinterpret_cast<u64*>(static_cast<char*>(ws) + ((size_t)rows * chunks * sizeof(Sum) + 255) / 256 * 256);
  const T* x = static_cast<const T*>(logits);
  logprobs_kernel<T><<<dim3((unsigned)rows, chunks), kThreads, lds, s>>>(x, ldl, V, chunk, tokens, logprob, entropy,
                                                                         top, top_ids, top_lp, part, keys,
                                                                         (groups + 3) & ~3);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess || chunks == 1) return e;
  logprobs_join_kernel<T><<<(unsigned)rows, kThreads, (size_t)max(chunks * top, 2) * 8, s>>>(
      x, ldl, V, chunks, tokens, logprob, entropy, top, top_ids, top_lp, part, keys);
  return hipGetLastError();
}

}  // namespace

size_t token_logprobs_ws_bytes(int64_t T, int64_t V, int top) {
  const int64_t c = chunks_of(T, V);
  if (c <= 1) return 0;
  return ((size_t)T * c * sizeof(Sum) + 255) / 256 * 256 + (size_t)T * c * top * 8;
}

hipError_t launch_token_logprobs(const void* logits, int dtype, int64_t T, int64_t V, int64_t ldl,
                                 const int64_t* tokens, float* logprob, float* entropy, int top, int64_t* top_ids,
                                 float* top_lp, void* ws, hipStream_t s) {
  switch (dtype) {
    case 0: return launch<float>(logits, ldl, T, (int)V, tokens, logprob, entropy, top, top_ids, top_lp, ws, s);
    case 1: return launch<_Float16>(logits, ldl, T, (int)V, tokens, logprob, entropy, top, top_ids, top_lp, ws, s);
    default: return launch<__bf16>(logits, ldl, T, (int)V, tokens, logprob, entropy, top, top_ids, top_lp, ws, s);
  }
}

}  // namespace ttq
