// Log probabilities of given tokens, entropy and top alternatives of each row
// of logits, and the gradient of the first two.
//
// For a row x = scale * logits (V columns), in log2 units y = x log2(e):
//     m = max_j y_j,  s = sum_j 2^(y_j - m),  t = sum_j 2^(y_j - m) (y_j - m)
//     LSE = ln2 (m + log2 s)                      log p_j = x_j - LSE
//     H   = -sum_j p_j log p_j = ln2 (log2 s - t / s)
// One pass over the row: every thread keeps (m, s, t) of the columns it reads
// and moves its m when a 16-byte vector brings a larger value (s and t follow
// exactly: s' = a s, t' = a (t + s (m - m')), a = 2^(m - m')); the threads'
// triples merge the same way.  t is centred on m, so the entropy does not lose
// the digits that sum p x - LSE cancels.  Arguments below -256 are raised to
// -256: their weight is exactly 0 either way, and 0 * -inf never arises.
//
// y may leave fp32's range (rows masked with the type's lowest value), and a log
// probability x - LSE loses the digits that a large LSE has before the point.  So
// a row whose LSE comes out above 256, or not finite, is summed again from the
// differences x - m (row_sum), and its log probabilities are scale (x - m) - L.
//
// The forward reads a 16-bit logit with about as many instructions as its bytes
// take in DRAM time, so for 16-bit types a vector's maximum and its guard against
// -inf work on packed pairs (raised to -1e30, or fp16's lowest, where that times
// scale still has weight 0), and the fp32 arithmetic on pairs too: 4.5 issue slots
// a logit against 7.  8192 x 131072 bf16 logits with 8 alternatives take 320 us, 6.7 TB/s; 8 such rows 7.6 us, most of it the
// alternatives' chain of barriers (4.0 us without them).
//
// Top alternatives, also without sorting the row: the largest value of each
// group of four vectors is a by-product of the pass, kept in shared memory, and so is a
// thread's.  The K-th largest of the threads' maxima is a lower bound of the
// K-th largest value (any value that at least K of them reach will do, so the search
// stops at one that few more reach), so only the groups whose maximum reaches it are
// read again (about K of them), the values that reach it become
// candidates, and a candidate's place is the number of greater ones.  (Read again thread by
// thread, without the groups, a row cost 40 KB of DRAM traffic more.)  A value
// and its column make one 64-bit key (value's order above, column's complement
// below), so equal values go to the lowest column and the result does not
// depend on the order in which threads arrive.  Rows with more candidates than
// the list holds (thousands of equal values) take a second pass in which each
// warp keeps a sorted list.
#include <cooperative_groups.h>
#include <cuda_fp16.h>
#include <float.h>

#include "common.cuh"
#include "kernels.h"

namespace cg = cooperative_groups;

namespace skl {
namespace {

constexpr int kMaxCand = 512;      // candidate keys a block ranks
constexpr float kFloor = -256.0f;  // 2^-256 is 0 in fp32
constexpr int kUnroll = 4;         // 16-byte loads a thread has in flight
// The forward's threads on an SM: 40 registers each.  With 2048 and 32 the loop that reads spills (4096 x 131072 bf16, no
// alternatives: 167 against 161 us).
constexpr int kThreadsPerSm = 1536;

__device__ __forceinline__ float to_float(float x) { return x; }
__device__ __forceinline__ float to_float(__nv_bfloat16 x) { return __bfloat162float(x); }
__device__ __forceinline__ float to_float(__half x) { return __half2float(x); }
template <typename T>
__device__ __forceinline__ T from_float(float x);
template <>
__device__ __forceinline__ float from_float<float>(float x) {
  return x;
}
template <>
__device__ __forceinline__ __nv_bfloat16 from_float<__nv_bfloat16>(float x) {
  return __float2bfloat16_rn(x);
}
template <>
__device__ __forceinline__ __half from_float<__half>(float x) {
  return __float2half_rn(x);
}

template <typename T>
struct Vec {
  static constexpr int N = 16 / sizeof(T);
  union {
    uint4 u;
    uint32_t w[4];
    T e[N];
  };
};

__device__ __forceinline__ uint4 load_stream(const void* p) {
  uint4 v;
  asm volatile("ld.global.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "l"(p));
  return v;
}

__device__ __forceinline__ float max_nan(float a, float b) {
  float d;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(d) : "f"(a), "f"(b));
  return d;
}

// Unsigned order of fp32 values (-0 taken as +0), and back.
__device__ __forceinline__ uint32_t order_of(float x) {
  const uint32_t b = __float_as_uint(x + 0.0f);
  return b ^ ((uint32_t)((int32_t)b >> 31) | 0x80000000u);
}
__device__ __forceinline__ float value_of(uint32_t o) {
  return __uint_as_float(o & 0x80000000u ? o ^ 0x80000000u : ~o);
}
__device__ __forceinline__ uint64_t key_of(float x, uint32_t column) {
  return ((uint64_t)order_of(x) << 32) | (0xffffffffu - column);
}

struct Sums {
  float m, s, t;
};

// The sums of N lanes (of the warp's first N, which the others repeat), on all of them: one common maximum, then plain
// sums, equal on both sides of every exchange.
template <int N>
__device__ __forceinline__ void merge_lanes(Sums& a) {
  const float m = value_of(__reduce_max_sync(0xffffffffu, order_of(a.m)));
  const float d = max_nan(a.m - (m == kNegInf ? 0.f : m), kFloor), w = ex2(d);
  a.m = m;
  a.t = w * (a.t + a.s * d);
  a.s *= w;
#pragma unroll
  for (int o = N / 2; o; o >>= 1) {
    a.s += __shfl_xor_sync(0xffffffffu, a.s, o);
    a.t += __shfl_xor_sync(0xffffffffu, a.t, o);
  }
}

// A thread's sums while it reads: two of each, for the two halves of a pair.
struct Sums2 {
  float m;
  float2 s, t;
};

// Moves m up to y; the sums follow.
__device__ __forceinline__ void move_max(Sums2& a, float y) {
  if (y > a.m) {
    if (a.m != kNegInf) {
      const float d = max_nan(a.m - y, kFloor), w = ex2(d);
      a.t = make_float2(w * (a.t.x + a.s.x * d), w * (a.t.y + a.s.y * d));
      a.s = make_float2(a.s.x * w, a.s.y * w);
    }
    a.m = y;
  }
}

// Packed pairs of 16-bit logits.
template <typename T>
struct Pair;
template <>
struct Pair<__nv_bfloat16> {
  static constexpr float kLow = -1.0e30f;      // -inf is read as this ...
  static constexpr float kMinC = 1.0e-27f;     // ... where c = scale log2(e) is at least this: 2^(c kLow - m) is 0
  static constexpr uint32_t kLowBits = 0xf149f149u;  // bf16 of -1e30, twice
  static __device__ __forceinline__ uint32_t max2(uint32_t a, uint32_t b) {
    uint32_t d;
    asm("max.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
    return d;
  }
  static __device__ __forceinline__ uint32_t raise(uint32_t a) {  // NaN stays
    uint32_t d;
    asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(kLowBits));
    return d;
  }
  static __device__ __forceinline__ float2 unpack(uint32_t a) {
    return make_float2(__uint_as_float(a << 16), __uint_as_float(a & 0xffff0000u));
  }
};
template <>
struct Pair<__half> {
  static constexpr float kLow = -65504.0f;
  // Used where the vectors' maximum is above kLow / 2: what stands for -inf then lies at least 32752 * 0.02 = 655 binary
  // orders below the row's maximum, and its weight is 0.
  static constexpr float kMinC = 0.02f;
  static constexpr uint32_t kLowBits = 0xfbfffbffu;
  static __device__ __forceinline__ uint32_t max2(uint32_t a, uint32_t b) {
    uint32_t d;
    asm("max.f16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
    return d;
  }
  static __device__ __forceinline__ uint32_t raise(uint32_t a) {
    uint32_t d;
    asm("max.NaN.f16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(kLowBits));
    return d;
  }
  static __device__ __forceinline__ float2 unpack(uint32_t a) {
    return __half22float2(*reinterpret_cast<const __half2*>(&a));
  }
};

// NV 16-byte vectors of logits at once: one maximum, one look at whether m moves.  `packed`: c is large enough for the
// packed guard.  Vectors whose maximum itself lies near the guard's value take the other way.
template <typename T, int NV>
__device__ __forceinline__ void add_vectors(Sums2& a, float& top, const Vec<T> (&x)[NV], float c, bool packed) {
  float vm;
  bool pairs = false;
  if constexpr (sizeof(T) == 2) {
    uint32_t m = Pair<T>::max2(x[0].w[0], x[0].w[1]);
#pragma unroll
    for (int i = 2; i < 4 * NV; ++i) m = Pair<T>::max2(m, x[i / 4].w[i % 4]);
    const float2 m2 = Pair<T>::unpack(m);
    vm = fmaxf(m2.x, m2.y);
    pairs = packed && vm > Pair<T>::kLow * 0.5f;
  } else {
    vm = x[0].e[0];
#pragma unroll
    for (int i = 1; i < 4 * NV; ++i) vm = fmaxf(vm, x[i / 4].e[i % 4]);
  }
  top = fmaxf(top, vm);
  move_max(a, vm * c);
  if constexpr (sizeof(T) == 2) {
    if (pairs) {
      const float2 cc = make_float2(c, c), nm = make_float2(-a.m, -a.m);
#pragma unroll
      for (int i = 0; i < 4 * NV; ++i) {
        const float2 d = ffma2(Pair<T>::unpack(Pair<T>::raise(x[i / 4].w[i % 4])), cc, nm);
        const float2 e = make_float2(ex2(d.x), ex2(d.y));
        a.s = fadd2(a.s, e);
        a.t = ffma2(e, d, a.t);
      }
      return;
    }
  }
  const float z = a.m == kNegInf ? 0.f : -a.m;
#pragma unroll
  for (int i = 0; i < NV * Vec<T>::N; ++i) {
    const float d = max_nan(fmaf(to_float(x[i / Vec<T>::N].e[i % Vec<T>::N]), c, z), kFloor);
    const float e = ex2(d);
    a.s.x += e;
    a.t.x = fmaf(e, d, a.t.x);
  }
}

struct FwdArgs {
  const void* logits;
  long long stride;
  const long long* tokens;
  float *logp, *entropy, *lse, *top_logp;
  long long* top_index;
  int V, T, K, parts, log_parts;
  float scale;
};

// A row, cut for 16-byte loads: `head` columns up to the first 16-byte boundary, `nvec` vectors, then the tail.
struct Cut {
  int head, nvec, tail0;
};
template <typename T>
__device__ __forceinline__ Cut cut_row(const T* row, int V) {
  constexpr int N = Vec<T>::N;
  const int off = (int)(reinterpret_cast<uintptr_t>(row) & 15u) / (int)sizeof(T);
  Cut c;
  c.head = min(V, off ? N - off : 0);
  c.nvec = (V - c.head) / N;
  c.tail0 = c.head + c.nvec * N;
  return c;
}

// ---- a row from differences of logits
constexpr float kTrustedLse = 256.0f;  // up to here x - LSE is off by 1.5e-5 at most

// f over v of all threads, in a fixed order.
template <int NT, typename F>
__device__ __forceinline__ float block_all(float v, F f, float* shared) {
#pragma unroll
  for (int o = 16; o; o >>= 1) v = f(v, __shfl_xor_sync(0xffffffffu, v, o));
  __syncthreads();  // what was there before has been read
  if ((threadIdx.x & 31) == 0) shared[threadIdx.x >> 5] = v;
  __syncthreads();
  v = shared[0];
#pragma unroll
  for (int w = 1; w < NT / 32; ++w) v = f(v, shared[w]);
  return v;
}

// Every column of a row to f, several loads in flight.
template <typename T, int NT, typename F>
__device__ __forceinline__ void each_column(const T* row, int V, F f) {
  constexpr int N = Vec<T>::N;
  const Cut cut = cut_row(row, V);
  const uint4* vecs = reinterpret_cast<const uint4*>(row + cut.head);
  for (int v = threadIdx.x; v < cut.nvec; v += 2 * NT) {
    Vec<T> x[2];
    x[0].u = load_stream(vecs + v);
    const bool both = v + NT < cut.nvec;
    if (both) x[1].u = load_stream(vecs + v + NT);
#pragma unroll
    for (int i = 0; i < 2 * N; ++i)
      if (i < N || both) f(to_float(x[i / N].e[i % N]));
  }
  for (int j = threadIdx.x; j < V - cut.nvec * N; j += NT) f(to_float(row[j < cut.head ? j : j + cut.nvec * N]));
}

// The row's largest logit m, log2 of s = sum 2^d and t / s with t = sum 2^d d, d = c (x - m); s is 0 where every logit is
// -inf.  All threads of the block take part, and have read the row when it returns.
struct RowSum {
  float m, s, log2s, mean;
};
template <typename T, int NT>
__device__ __forceinline__ RowSum row_sum(const T* row, int V, float c, float* shared) {
  RowSum a;
  a.m = kNegInf;
  each_column<T, NT>(row, V, [&](float x) { a.m = fmaxf(a.m, x); });
  a.m = block_all<NT>(a.m, [](float x, float y) { return fmaxf(x, y); }, shared);
  const float m = a.m == kNegInf ? 0.f : a.m;
  float s = 0.f, t = 0.f;
  each_column<T, NT>(row, V, [&](float x) {
    const float d = max_nan((x - m) * c, kFloor), e = ex2(d);
    s += e;
    t = fmaf(e, d, t);
  });
  a.s = block_all<NT>(s, [](float x, float y) { return x + y; }, shared);
  t = block_all<NT>(t, [](float x, float y) { return x + y; }, shared);
  a.log2s = log2f(a.s);
  a.mean = t / a.s;
  return a;
}

constexpr int kGroups = 16;  // maxima that a thread keeps; group g of a long row goes with g mod 16

template <int NT>
struct FwdShared {
  float group_max[kGroups][NT];
  Sums warp_sums[NT / 32];
  uint32_t warp_lo[NT / 32], warp_hi[NT / 32];
  Sums part_sums[8];
  uint64_t cand[kMaxCand];
  uint64_t best[8 * 32];  // each part's top K, gathered in the first part's block
  unsigned short again[NT];
  int n_cand, n_again;
};

// Sorts nothing: the place of a key is the number of greater ones.  Keys are distinct.
template <int NT>
__device__ __forceinline__ void rank_keys(const uint64_t* keys, int n, int K, uint64_t* out) {
  for (int i = threadIdx.x; i < n; i += NT) {
    const uint64_t k = keys[i];
    int place = 0;
    for (int j = 0; j < n; ++j) place += keys[j] > k;
    if (place < K) out[place] = k;
  }
}

// The same for `lists` (at most eight) sorted lists of K keys, one after the other; 0 is no key.  A lane searches a list.
template <int NT>
__device__ __forceinline__ void rank_lists(const uint64_t* keys, int lists, int K, uint64_t* out) {
  const int q = threadIdx.x % 8;
  for (int i0 = 0; i0 < lists * K; i0 += NT / 8) {
    const int i = i0 + threadIdx.x / 8;
    const uint64_t k = i < lists * K ? keys[i] : 0;
    int place = 0, end = q < lists ? K : 0;
    while (place < end) {
      const int mid = (place + end) / 2;
      if (keys[q * K + mid] > k)
        place = mid + 1;
      else
        end = mid;
    }
#pragma unroll
    for (int o = 1; o < 8; o *= 2) place += __shfl_xor_sync(0xffffffffu, place, o);
    if (k && q == 0 && place < K) out[place] = k;
  }
}

// The block's K largest keys of columns [lo, hi), for any values: each warp reads a contiguous share in order and
// keeps its K best sorted over its lanes.
template <typename T, int NT>
__device__ void warp_lists(const T* row, int lo, int hi, int K, FwdShared<NT>& sh, uint64_t* out) {
  constexpr int NW = NT / 32;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int share = (hi - lo + NW - 1) / NW;
  const int w0 = lo + warp * share, w1 = min(hi, w0 + share);
  uint64_t mine = 0;
  for (int j0 = w0; j0 < w1; j0 += 32) {
    const int j = j0 + lane;
    const uint64_t key = j < w1 ? key_of(to_float(row[j]), (uint32_t)j) : 0;
    unsigned todo = __ballot_sync(0xffffffffu, key > __shfl_sync(0xffffffffu, mine, K - 1));
    while (todo) {
      const int src = __ffs(todo) - 1;
      todo &= todo - 1;
      const uint64_t k = __shfl_sync(0xffffffffu, key, src);
      const int place = __popc(__ballot_sync(0xffffffffu, mine > k));
      const uint64_t below = __shfl_up_sync(0xffffffffu, mine, 1);
      if (lane == place) mine = k;
      if (lane > place) mine = below;
    }
  }
  __syncthreads();  // every thread has left the candidate list of the first attempt
  if (lane < K) sh.cand[warp * K + lane] = mine;
  __syncthreads();
  // a share with fewer than K columns leaves zero keys: they rank behind every real one
  for (int i = threadIdx.x; i < NW * K; i += NT) {
    const uint64_t k = sh.cand[i];
    if (!k) continue;
    int place = 0;
    for (int j = 0; j < NW * K; ++j) place += sh.cand[j] > k;
    if (place < K) out[place] = k;
  }
}

// A row's outputs, from its sums or (FAR) from differences of logits; tok0, raw0: the thread's first given token and its logit.
template <typename T, int NT, bool FAR>
__device__ __forceinline__ void write_row(const FwdArgs& a, long long r, const T* row, FwdShared<NT>& sh, Sums all, long long tok0,
                                          float raw0) {
  const int tid = threadIdx.x;
  float log2s = log2f(all.s), mean = all.t / all.s;
  float lse = kLn2 * (all.m + log2s);
  float m = 0.f, L = lse;  // log p = scale (x - m) - L
  bool empty = false;      // every logit is -inf
  if (FAR) {
    const RowSum w = row_sum<T, NT>(row, a.V, a.scale * kLog2e, reinterpret_cast<float*>(sh.warp_sums));
    empty = w.s == 0.f;
    log2s = w.log2s;
    mean = w.mean;
    m = w.m;
    L = kLn2 * log2s;
    lse = empty ? kNegInf : fmaf(m, a.scale, L);
    if (isinf(lse) && !isinf(m)) lse = copysignf(FLT_MAX, lse);  // past fp32's range, but not a row of nothing
  }
  if (tid == 0) {
    a.lse[r] = lse;
    a.entropy[r] = empty ? 0.f : kLn2 * (log2s - mean);
  }
  auto log_prob = [&](float raw) { return empty ? kNegInf : fmaf(FAR ? raw - m : raw, a.scale, -L); };
  for (int t = tid; t < a.T; t += NT) {
    const long long tok = !FAR && t == tid ? tok0 : a.tokens[r * a.T + t];
    float out = 0.f;  // no token
    if (tok >= a.V) out = __uint_as_float(0x7fffffffu);
    else if (tok >= 0) out = log_prob(!FAR && t == tid ? raw0 : to_float(row[tok]));
    a.logp[r * a.T + t] = out;
  }
  if (a.K) {
    uint64_t* order = sh.best;
    if (a.parts > 1) {
      rank_lists<NT>(sh.best, a.parts, a.K, sh.cand);
      __syncthreads();
      order = sh.cand;
    }
    if (tid < a.K) {
      const uint64_t k = order[tid];
      a.top_index[r * a.K + tid] = (long long)(0xffffffffu - (uint32_t)k);
      a.top_logp[r * a.K + tid] = log_prob(value_of((uint32_t)(k >> 32)));
    }
  }
}

template <typename T, int NT>
__device__ __noinline__ void write_far_row(const FwdArgs& a, long long r, const T* row, FwdShared<NT>& sh) {
  write_row<T, NT, true>(a, r, row, sh, Sums{0.f, 1.f, 0.f}, -1, 0.f);
}

template <typename T, int NT>
__global__ void __launch_bounds__(NT, kThreadsPerSm / NT) logprobs_fwd_kernel(const __grid_constant__ FwdArgs a) {
  constexpr int N = Vec<T>::N;
  constexpr int NW = NT / 32;
  __shared__ FwdShared<NT> sh;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int part = (int)(blockIdx.x & (a.parts - 1u));
  const long long r = blockIdx.x >> a.log_parts;
  const T* row = static_cast<const T*>(a.logits) + r * a.stride;
  const Cut cut = cut_row(row, a.V);
  const int v0 = (int)((long long)cut.nvec * part >> a.log_parts), v1 = (int)((long long)cut.nvec * (part + 1) >> a.log_parts);
  const int nv = v1 - v0;
  const uint4* vecs = reinterpret_cast<const uint4*>(row + cut.head) + v0;
  const bool first = part == 0, last = part == a.parts - 1;
  const float c = a.scale * kLog2e;
  bool packed = false;
  if constexpr (sizeof(T) == 2) packed = c >= Pair<T>::kMinC && c <= 1.0e6f;
  if (tid == 0) sh.n_cand = sh.n_again = 0;
  if (a.parts > 1) cg::this_cluster().barrier_arrive();  // this block runs: its shared memory may be written

  Sums2 acc{kNegInf, make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
  float top = kNegInf;  // this thread's largest value among its vectors
  int v = tid, group = 0;
  auto keep = [&](float m) {  // a group's maximum
    top = fmaxf(top, m);
    if (a.K) {
      float& slot = sh.group_max[group % kGroups][tid];
      slot = group < kGroups ? m : fmaxf(slot, m);
    }
    ++group;
  };
  for (; v + (kUnroll - 1) * NT < nv; v += kUnroll * NT) {
    Vec<T> x[kUnroll];
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) x[u].u = load_stream(vecs + v + u * NT);
    float m = kNegInf;
    add_vectors<T, kUnroll>(acc, m, x, c, packed);
    keep(m);
  }
  if (v < nv) {  // the last group is shorter
    float m = kNegInf;
    for (; v < nv; v += NT) {
      Vec<T> x[1];
      x[0].u = load_stream(vecs + v);
      add_vectors<T, 1>(acc, m, x, c, packed);
    }
    keep(m);
  }
  // the columns outside the vectors: one a thread, and always candidates
  const uint32_t top_order = tid < nv ? order_of(top) : 0u;
  __syncthreads();  // the counters are zero
  for (int side = 0; side < 2; ++side) {
    const int j = side ? cut.tail0 + tid : tid;
    if (side ? last && j < a.V : first && j < cut.head) {
      const float f = to_float(row[j]);
      move_max(acc, f * c);
      const float d = max_nan(fmaf(f, c, acc.m == kNegInf ? 0.f : -acc.m), kFloor), e = ex2(d);
      acc.s.x += e;
      acc.t.x = fmaf(e, d, acc.t.x);
      if (a.K) sh.cand[atomicAdd(&sh.n_cand, 1)] = key_of(f, (uint32_t)j);  // at most 2 (N - 1) of them
    }
  }
  long long tok0 = -1;  // this thread's first given token and its logit, on their way meanwhile
  float raw0 = 0.f;
  if (first && tid < a.T) {
    tok0 = a.tokens[r * a.T + tid];
    if (tok0 >= 0 && tok0 < a.V) raw0 = to_float(row[tok0]);
  }
  Sums sums{acc.m, acc.s.x + acc.s.y, acc.t.x + acc.t.y};
  merge_lanes<32>(sums);
  const uint32_t prefix = top_order >> 16;  // 16 bits are enough for a lower bound
  const uint32_t warp_lo = __reduce_min_sync(0xffffffffu, prefix), warp_hi = __reduce_max_sync(0xffffffffu, prefix);
  if (lane == 0) {
    sh.warp_sums[warp] = sums;
    sh.warp_lo[warp] = warp_lo;
    sh.warp_hi[warp] = warp_hi;
  }

  const int k_here = min(a.K, cut.head * (int)first + nv * N + (a.V - cut.tail0) * (int)last);  // columns can be fewer
  uint64_t* best = sh.best;
  if (a.parts > 1) {
    cg::this_cluster().barrier_wait();
    best = cg::this_cluster().map_shared_rank(sh.best, 0);
    if (tid < a.K) best[part * a.K + tid] = 0;  // a part may hold fewer columns than K
  }
  if (a.K) {
    __syncthreads();
    uint32_t lo = sh.warp_lo[0], hi = sh.warp_hi[0];
    for (int w = 1; w < NW; ++w) {
      lo = min(lo, sh.warp_lo[w]);
      hi = max(hi, sh.warp_hi[w]);
    }
    // a prefix that at least K threads' maxima reach (0 when fewer threads hold vectors), and not many more; `lo` always
    // is one where K <= NT, which it is
    while (lo < hi) {
      const uint32_t mid = (lo + hi + 1) / 2;
      const int reach = __syncthreads_count(prefix >= mid);
      if (reach >= a.K) {
        lo = mid;
        if (reach <= a.K + 8) break;
      } else {
        hi = mid - 1;
      }
    }
    const uint32_t bound = lo << 16;
    if (top_order && top_order >= bound) sh.again[atomicAdd(&sh.n_again, 1)] = (unsigned short)tid;
    __syncthreads();
    for (int q = warp; q < sh.n_again; q += NW) {
      const int t = sh.again[q];
      // lane: group lane / 4 (then + 8) of the thread, vector lane % 4 of the group
      for (int slot = lane / kUnroll; slot < kGroups; slot += 32 / kUnroll) {
        const int base = t + (slot * kUnroll + lane % kUnroll) * NT;
        if (t + slot * kUnroll * NT >= nv || order_of(sh.group_max[slot][t]) < bound) continue;
        for (int w = base; w < nv; w += kGroups * kUnroll * NT) {
          Vec<T> x;
          x.u = __ldg(vecs + w);
#pragma unroll
          for (int i = 0; i < N; ++i) {
            const float f = to_float(x.e[i]);
            if (order_of(f) >= bound) {
              const int at = atomicAdd(&sh.n_cand, 1);
              if (at < kMaxCand) sh.cand[at] = key_of(f, (uint32_t)(cut.head + (v0 + w) * N + i));
            }
          }
        }
      }
    }
    __syncthreads();
    if (sh.n_cand <= kMaxCand)
      rank_keys<NT>(sh.cand, sh.n_cand, k_here, best + part * a.K);
    else
      warp_lists<T, NT>(row, first ? 0 : cut.head + v0 * N, last ? a.V : cut.head + v1 * N, k_here, sh,
                        best + part * a.K);
  }
  __syncthreads();
  if (warp == 0) {
    Sums all = sh.warp_sums[lane % NW];
    merge_lanes<NW>(all);
    Sums* to = sh.part_sums;
    if (a.parts > 1) to = cg::this_cluster().map_shared_rank(sh.part_sums, 0);
    if (lane == 0) to[part] = all;
  }
  if (a.parts > 1)
    cg::this_cluster().sync();
  else
    __syncthreads();
  if (part != 0) return;

  Sums all = lane % 8 < a.parts ? sh.part_sums[lane % 8] : Sums{kNegInf, 0.f, 0.f};
  merge_lanes<8>(all);
  if (fabsf(kLn2 * (all.m + log2f(all.s))) <= kTrustedLse)
    write_row<T, NT, false>(a, r, row, sh, all, tok0, raw0);
  else
    write_far_row<T, NT>(a, r, row, sh);
}

struct BwdArgs {
  const void* logits;
  long long stride, out_stride;
  const long long* tokens;
  const float *lse, *entropy, *g_logp, *g_entropy;
  void* out;
  int V, T, parts, log_parts;
  float scale;
};

// With A = sum of the row's g over its tokens, B = its g of the entropy, l_j = log p_j:
//     dx_j = sum_t g_t [j = token_t] - p_j (A + B (l_j + H)),   dlogits_j = scale dx_j
// The pass writes the second term; then the given tokens' columns, a handful, are written again with the sum of
// both in fp32, rounded once.  A token that is given twice adds twice: its first place takes the sum of all.
// FAR: l_j = scale (x_j - m) - L, of a row that is summed again; else x_j scale - LSE.  (A copy of its own, inline: a function
// call cost the ordinary rows 1 to 5%, m and L in their loop 2%.)
// Bound by DRAM: 4096 x 131072 bf16 324 us, 6.6 TB/s; 333 x 50021 fp16 with 16 tokens 13.8 us, 4.8 TB/s.  (With the first
// vectors' loads before the sums over the tokens the registers do not suffice: 332 us.)
template <typename T, int NT, bool FAR>
__device__ __forceinline__ void write_gradient(const BwdArgs& a, long long r, float* sum_g) {
  constexpr int N = Vec<T>::N;
  const int tid = threadIdx.x;
  const int part = (int)(blockIdx.x & (a.parts - 1u));
  const T* row = static_cast<const T*>(a.logits) + r * a.stride;
  T* out = static_cast<T*>(a.out) + r * a.out_stride;
  const long long* tokens = a.tokens + r * a.T;
  const float* g = a.g_logp + r * a.T;
  float m = 0.f, L = a.lse[r];
  const bool empty = L == kNegInf;  // every logit is -inf: nothing depends on them
  if (FAR) {
    const RowSum w = row_sum<T, NT>(row, a.V, a.scale * kLog2e, sum_g);
    m = w.m;
    L = kLn2 * w.log2s;
    __syncthreads();  // sum_g has been read
  }

  // A in a fixed order: thread t takes tokens t, t + NT, ...; lanes, then warps
  float A = 0.f;
  for (int t = tid; t < a.T; t += NT) {
    const long long tok = tokens[t];
    if (tok >= 0 && tok < a.V) A += g[t];
  }
#pragma unroll
  for (int o = 16; o; o >>= 1) A += __shfl_xor_sync(0xffffffffu, A, o);
  if ((tid & 31) == 0) sum_g[tid >> 5] = A;
  __syncthreads();
  A = 0.f;
#pragma unroll
  for (int w = 0; w < NT / 32; ++w) A += sum_g[w];
  if constexpr (!FAR) {
    if (fabsf(L) > kTrustedLse && !empty) {  // here and not sooner: the LSE's load runs beside the tokens'
      write_gradient<T, NT, true>(a, r, sum_g);
      return;
    }
  }
  const float B = a.g_entropy ? a.g_entropy[r] : 0.f;
  const float H = a.g_entropy ? a.entropy[r] : 0.f;
  // dlogits = p (a0 + a1 l2), l2 = log2 p
  const float a0 = -a.scale * (A + B * H), a1 = -a.scale * B * kLn2;
  auto grad = [&](float x) {
    const float l2 = max_nan(fmaf(FAR ? x - m : x, a.scale, -L) * kLog2e, kFloor);  // one rounding where x is near the LSE
    return empty ? 0.f : ex2(l2) * fmaf(a1, l2, a0);
  };

  // vectors where both rows have the same offset from a 16-byte boundary, else single columns
  const Cut cut = cut_row(row, a.V);
  const bool same = ((reinterpret_cast<uintptr_t>(row) ^ reinterpret_cast<uintptr_t>(out)) & 15u) == 0;
  int lo, hi;  // this block's columns
  if (same) {
    const int v0 = (int)((long long)cut.nvec * part >> a.log_parts), v1 = (int)((long long)cut.nvec * (part + 1) >> a.log_parts);
    lo = part == 0 ? 0 : cut.head + v0 * N;
    hi = part == a.parts - 1 ? a.V : cut.head + v1 * N;
    const uint4* in = reinterpret_cast<const uint4*>(row + cut.head);
    uint4* to = reinterpret_cast<uint4*>(out + cut.head);
    int v = v0 + tid;
    auto one = [&](uint4 u) {
      Vec<T> x;
      x.u = u;
#pragma unroll
      for (int i = 0; i < N; ++i) x.e[i] = from_float<T>(grad(to_float(x.e[i])));
      return x.u;
    };
    for (; v + (kUnroll - 1) * NT < v1; v += kUnroll * NT) {
      uint4 x[kUnroll];
#pragma unroll
      for (int u = 0; u < kUnroll; ++u) x[u] = load_stream(in + v + u * NT);
#pragma unroll
      for (int u = 0; u < kUnroll; ++u) to[v + u * NT] = one(x[u]);
    }
    for (; v < v1; v += NT) to[v] = one(load_stream(in + v));
    if (part == 0 && tid < cut.head) out[tid] = from_float<T>(grad(to_float(row[tid])));
    if (part == a.parts - 1 && cut.tail0 + tid < a.V)
      out[cut.tail0 + tid] = from_float<T>(grad(to_float(row[cut.tail0 + tid])));
  } else {
    lo = (int)((long long)a.V * part >> a.log_parts);
    hi = (int)((long long)a.V * (part + 1) >> a.log_parts);
    for (int j = lo + tid; j < hi; j += NT) out[j] = from_float<T>(grad(to_float(row[j])));
  }
  if (empty) return;
  __syncthreads();  // the block's columns are written
  for (int t = tid; t < a.T; t += NT) {
    const long long tok = tokens[t];
    if (tok < lo || tok >= hi) continue;
    float total = 0.f;
    bool leads = true;
    for (int u = 0; u < a.T; ++u)
      if (tokens[u] == tok) {
        leads = leads && u >= t;
        total += g[u];
      }
    if (leads) out[tok] = from_float<T>(fmaf(a.scale, total, grad(to_float(row[tok]))));
  }
}

template <typename T, int NT>
__global__ void __launch_bounds__(NT, 2048 / NT) logprobs_bwd_kernel(const __grid_constant__ BwdArgs a) {
  __shared__ float sum_g[NT / 32];
  write_gradient<T, NT, false>(a, blockIdx.x >> a.log_parts, sum_g);
}

// Blocks that share a row: as many (a power of two, at most 8, the portable cluster size) as keep the launch within
// two blocks for each SM, and no part below kMinPartBytes.
constexpr long long kMinPartBytes = 8192;
int log_parts_of(long long rows, long long row_bytes, int num_sms) {
  int n = 0;
  while (n < 3 && (rows << (n + 1)) <= 2ll * num_sms && (row_bytes >> (n + 1)) >= kMinPartBytes) ++n;
  return n;
}

// Threads of a block: 128 for short rows, where 512 would hold no vector.  The forward's longer rows: 512 where all blocks
// are resident at once, so that a row is read soon; fewer where they are not, since a block that ends then makes room in
// smaller pieces, and the blocks' searches for the alternatives overlap with more blocks' reading: 128 up to
// kFwdMidRowBytes, 256 above, where a thread of 128 would have too many groups.  In us with 512 / 256 / 128 threads:
// 8192 x 32000 bf16, 8 alternatives, 163 / 120 / 109; 5000 x 64000, 5: - / 118 / 110; 4096 x 131072, 8: 180 / 172 / 188;
// 333 x 50021 fp32, 16: 17.1 / 19.6 / -.  The gradient: 256 up to kBwdMidRowBytes (8192 x 32000 169 -> 164), 512 above
// (5000 x 64000 198 against 204).
constexpr long long kShortRowBytes = 8192, kFwdMidRowBytes = 144 * 1024, kBwdMidRowBytes = 96 * 1024;

template <typename T, int NT>
cudaError_t launch_fwd_nt(const FwdArgs& a, long long rows, cudaStream_t st) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(rows * a.parts));
  cfg.blockDim = dim3(NT);
  cfg.stream = st;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeClusterDimension;
  at[0].val.clusterDim.x = (unsigned)a.parts;
  at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
  cfg.attrs = at;
  cfg.numAttrs = a.parts > 1 ? 1 : 0;
  return cudaLaunchKernelEx(&cfg, logprobs_fwd_kernel<T, NT>, a);
}

template <typename T>
cudaError_t launch_fwd_t(FwdArgs a, long long rows, int num_sms, cudaStream_t st) {
  const long long bytes = (long long)a.V * sizeof(T);
  a.log_parts = log_parts_of(rows, bytes, num_sms);
  a.parts = 1 << a.log_parts;
  if (bytes <= kShortRowBytes) return launch_fwd_nt<T, 128>(a, rows, st);
  if (rows * a.parts > (long long)num_sms * (kThreadsPerSm / 512))
    return bytes <= kFwdMidRowBytes ? launch_fwd_nt<T, 128>(a, rows, st) : launch_fwd_nt<T, 256>(a, rows, st);
  return launch_fwd_nt<T, 512>(a, rows, st);
}

template <typename T>
cudaError_t launch_bwd_t(BwdArgs a, long long rows, int num_sms, cudaStream_t st) {
  const long long bytes = (long long)a.V * sizeof(T);
  // in place a row has one block, which has read it whole before it writes where it sums it again
  a.log_parts = a.out == a.logits ? 0 : log_parts_of(rows, bytes, num_sms);
  a.parts = 1 << a.log_parts;
  if (bytes <= kShortRowBytes)
    logprobs_bwd_kernel<T, 128><<<(unsigned)(rows * a.parts), 128, 0, st>>>(a);
  else if (bytes <= kBwdMidRowBytes)
    logprobs_bwd_kernel<T, 256><<<(unsigned)(rows * a.parts), 256, 0, st>>>(a);
  else
    logprobs_bwd_kernel<T, 512><<<(unsigned)(rows * a.parts), 512, 0, st>>>(a);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_logprobs_fwd(const LogprobsProblem& p, const void* logits, const long long* tokens, float* logp,
                                float* entropy, float* lse, float* top_logp, long long* top_index, int num_sms,
                                cudaStream_t st) {
  FwdArgs a{logits, p.stride, tokens, logp, entropy, lse, top_logp, top_index, p.V, p.T, p.K, 1, 0, p.scale};
  if (p.dtype == kTypeBf16) return launch_fwd_t<__nv_bfloat16>(a, p.rows, num_sms, st);
  if (p.dtype == kTypeFp16) return launch_fwd_t<__half>(a, p.rows, num_sms, st);
  return launch_fwd_t<float>(a, p.rows, num_sms, st);
}

cudaError_t launch_logprobs_bwd(const LogprobsProblem& p, const void* logits, const long long* tokens,
                                const float* lse, const float* entropy, const float* g_logp, const float* g_entropy,
                                void* dlogits, long long out_stride, int num_sms, cudaStream_t st) {
  BwdArgs a{logits, p.stride, out_stride, tokens, lse, entropy, g_logp, g_entropy, dlogits, p.V, p.T, 1, 0, p.scale};
  if (p.dtype == kTypeBf16) return launch_bwd_t<__nv_bfloat16>(a, p.rows, num_sms, st);
  if (p.dtype == kTypeFp16) return launch_bwd_t<__half>(a, p.rows, num_sms, st);
  return launch_bwd_t<float>(a, p.rows, num_sms, st);
}

}  // namespace skl
