// Rotary positions: pair i of a row at position p turns by the angle p f_i,
//     (x, y) -> A (x cos - y sin, y cos + x sin),
// the first `dim` of D channels in pairs, the others as they are.  The inverse, which is also the gradient's map, turns
// back: -sin for sin.
//
// The angle is kept as a fraction of a turn in 64 bits of fixed point: turns_i = 2^64 f_i / 2 pi, so p turns_i mod 2^64 is
// the angle mod a turn, for any 64-bit position, to p 2^-64 of a turn -- where p f_i in fp32 would be off by 0.06 at
// a position of a million.  The two highest bits, rounded, are the quadrant; the rest, at most an eighth of a turn, goes
// through the Taylor series of sin and cos, whose first left-out terms are below 2^-28 and 2^-32.
//
// A thread has one 16-byte vector of a row's pairs (HALF: one of either half) at one position, takes its sines and
// cosines once, and then goes through a share of the heads of q and k: 20 operations a pair for all of them.  Bound by
// HBM's rate for many rows, by the launch for few.
#include "common.cuh"
#include "kernels.h"

#include <cuda_fp16.h>

#include <algorithm>

namespace skl {
namespace {

constexpr int THREADS = 256;

template <typename T>
__device__ __forceinline__ float to_float(T x) {
  return static_cast<float>(x);
}
template <typename T>
__device__ __forceinline__ T from_float(float x);
template <>
__device__ __forceinline__ float from_float<float>(float x) {
  return x;
}
template <>
__device__ __forceinline__ __half from_float<__half>(float x) {
  return __float2half_rn(x);
}
template <>
__device__ __forceinline__ __nv_bfloat16 from_float<__nv_bfloat16>(float x) {
  return __float2bfloat16_rn(x);
}

// sin and cos of `turn` / 2^64 of a turn
__device__ __forceinline__ void sincos_of_turn(unsigned long long turn, float* sin_out, float* cos_out) {
  const unsigned long long to = turn + (1ull << 61);  // to the nearest quarter
  const unsigned quarter = (unsigned)(to >> 62);
  const long long rest = (long long)(turn - ((unsigned long long)quarter << 62));  // within 2^61
  const float x = (float)rest * (6.283185307179586f * 0x1p-64f), y = x * x;       // radians, |x| <= pi / 4
  float s = 1.f / 362880.f, c = -1.f / 3628800.f;
  s = fmaf(s, y, -1.f / 5040.f);
  s = fmaf(s, y, 1.f / 120.f);
  s = fmaf(s, y, -1.f / 6.f);
  s = fmaf(s * y, x, x);
  c = fmaf(c, y, 1.f / 40320.f);
  c = fmaf(c, y, -1.f / 720.f);
  c = fmaf(c, y, 1.f / 24.f);
  c = fmaf(c, y, -0.5f);
  c = fmaf(c, y, 1.f);
  const float a = quarter & 1 ? c : s, b = quarter & 1 ? s : c;
  *sin_out = quarter & 2 ? -a : a;
  *cos_out = (quarter + 1) & 2 ? -b : b;
}

// V elements a vector: 16 bytes, or one pair alone where sizes or addresses do not allow that
template <typename T, bool INTERLEAVED, int V>
__global__ void __launch_bounds__(THREADS) rotary_kernel(const RotaryProblem p) {
  constexpr int PAIRS = INTERLEAVED ? V / 2 : V, PARTS = INTERLEAVED ? 1 : 2;
  constexpr int AHEAD = 4;  // heads whose loads are in flight together
  struct alignas(V * sizeof(T) == 16 ? 16 : sizeof(T)) Vec {
    T x[V];
  };
  const unsigned item = blockIdx.x * THREADS + threadIdx.x;
  const unsigned token = p.by_slots.div(item), slot = item - token * p.by_slots.d;
  if (token >= p.tokens) return;
  const unsigned b = p.by_rows.div(token), n = token - b * p.by_rows.d;
  const bool turns = (int)slot < p.turning;
  const int heads = p.HQ + p.HK;
  const int first = blockIdx.y * p.heads_each, last = min(first + p.heads_each, heads);
  const int at = turns ? (int)slot * V : p.dim + ((int)slot - p.turning) * V;  // of the first part; the second half a `dim` on
  float c[PAIRS], s[PAIRS];
  if (turns) {
    long long pos = p.offset + n;
    if (p.positions) {
      const long long i = (long long)b * p.positions_stride + n;
      pos = p.positions_wide ? static_cast<const long long*>(p.positions)[i] : static_cast<const int*>(p.positions)[i];
    }
#pragma unroll
    for (int k = 0; k < PAIRS; ++k) {
      sincos_of_turn((unsigned long long)pos * p.turns[(INTERLEAVED ? at / 2 : at) + k], &s[k], &c[k]);
      c[k] *= p.amplitude;
      s[k] *= p.sin_sign;
    }
  }
  const long long in_q = (long long)b * p.q.b + (long long)n * p.q.n + at, in_k = (long long)b * p.k.b + (long long)n * p.k.n + at;
  const long long out_q = (long long)b * p.qo.b + (long long)n * p.qo.n + at, out_k = (long long)b * p.ko.b + (long long)n * p.ko.n + at;
  auto from = [&](int h) {
    return h < p.HQ ? static_cast<const T*>(p.q_in) + in_q + h * p.q.h : static_cast<const T*>(p.k_in) + in_k + (h - p.HQ) * p.k.h;
  };
  auto to = [&](int h) {
    return h < p.HQ ? static_cast<T*>(p.q_out) + out_q + h * p.qo.h : static_cast<T*>(p.k_out) + out_k + (h - p.HQ) * p.ko.h;
  };
  for (int h0 = first; h0 < last; h0 += AHEAD) {
    Vec v[AHEAD][PARTS];
#pragma unroll
    for (int i = 0; i < AHEAD; ++i) {
      if (h0 + i < last) {
        const T* src = from(h0 + i);
        v[i][0] = *reinterpret_cast<const Vec*>(src);
        if (PARTS == 2 && turns) v[i][PARTS - 1] = *reinterpret_cast<const Vec*>(src + p.dim / 2);
      }
    }
#pragma unroll
    for (int i = 0; i < AHEAD; ++i) {
      if (h0 + i < last) {
        T* dst = to(h0 + i);
        if (turns) {
#pragma unroll
          for (int k = 0; k < PAIRS; ++k) {
            T& first_of = INTERLEAVED ? v[i][0].x[(2 * k) % V] : v[i][0].x[k];
            T& second_of = INTERLEAVED ? v[i][0].x[(2 * k + 1) % V] : v[i][PARTS - 1].x[k];
            const float x = to_float(first_of), y = to_float(second_of);
            first_of = from_float<T>(fmaf(x, c[k], -(y * s[k])));
            second_of = from_float<T>(fmaf(y, c[k], x * s[k]));
          }
          if (PARTS == 2) *reinterpret_cast<Vec*>(dst + p.dim / 2) = v[i][PARTS - 1];
        }
        *reinterpret_cast<Vec*>(dst) = v[i][0];
      }
    }
  }
}

template <typename T>
cudaError_t launch_type(const RotaryProblem& p, cudaStream_t st) {
  constexpr int V = 16 / sizeof(T);
  const dim3 grid((unsigned)((p.items + THREADS - 1) / THREADS), (unsigned)((p.HQ + p.HK + p.heads_each - 1) / p.heads_each));
  if (p.interleaved && p.vectors) rotary_kernel<T, true, V><<<grid, THREADS, 0, st>>>(p);
  if (p.interleaved && !p.vectors) rotary_kernel<T, true, 2><<<grid, THREADS, 0, st>>>(p);
  if (!p.interleaved && p.vectors) rotary_kernel<T, false, V><<<grid, THREADS, 0, st>>>(p);
  if (!p.interleaved && !p.vectors) rotary_kernel<T, false, 1><<<grid, THREADS, 0, st>>>(p);
  return cudaGetLastError();
}

}  // namespace

bool rotary_plan(RotaryProblem* p, int num_sms) {
  const int V = p->dtype == kTypeFp32 ? 4 : 8;
  uintptr_t at = 0;
  long long sizes = (p->D - p->dim) | (p->interleaved ? p->dim : p->dim / 2);
  auto add = [&](const void* x, const RotaryStrides& r, int heads) {
    if (!heads) return;
    at |= reinterpret_cast<uintptr_t>(x);
    sizes |= (p->B > 1 ? r.b : 0) | (heads > 1 ? r.h : 0) | (p->N > 1 ? r.n : 0);
  };
  add(p->q_in, p->q, p->HQ);
  add(p->q_out, p->qo, p->HQ);
  add(p->k_in, p->k, p->HK);
  add(p->k_out, p->ko, p->HK);
  p->vectors = !(at & 15) && !(sizes & (V - 1));
  const int v = p->vectors ? V : p->interleaved ? 2 : 1;
  const bool in_place = p->q_in == p->q_out && p->k_in == p->k_out;  // what does not turn is there already
  p->turning = p->interleaved ? p->dim / v : p->dim / 2 / v;
  const int slots = p->turning + (in_place ? 0 : (p->D - p->dim) / v), heads = p->HQ + p->HK;
  p->items = (long long)p->tokens * slots;
  if (p->items > 0x7fffffffll - THREADS) return false;
  p->by_slots = FastDiv((unsigned)slots);
  p->by_rows = FastDiv((unsigned)p->N);
  // heads a thread: as many as leave threads for two thirds of what the SMs hold, between one and sixteen
  p->heads_each = (int)std::max(1ll, std::min<long long>({16, heads, p->items * heads / (num_sms * 1344ll)}));
  return true;
}

cudaError_t launch_rotary(const RotaryProblem& p, cudaStream_t st) {
  if (p.dtype == kTypeBf16) return launch_type<__nv_bfloat16>(p, st);
  if (p.dtype == kTypeFp16) return launch_type<__half>(p, st);
  return launch_type<float>(p, st);
}

}  // namespace skl
