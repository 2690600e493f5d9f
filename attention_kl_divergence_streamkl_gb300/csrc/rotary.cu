// Rotary positions: pair i of a row at position p turns by the angle p f_i,
//     (x, y) -> A (x cos - y sin, y cos + x sin),
// the first `dim` of D channels in pairs, the others as they are.  The inverse, which is also the gradient's map, turns
// back: -sin for sin.
//
// The angle is kept as a fraction of a turn in 64 bits of fixed point: turns_i = 2^64 f_i / 2 pi, so p turns_i mod 2^64 is
// the angle mod a turn, for any 64-bit position, to the |p| 2^-65 of a turn that rounding f_i to 2^-64 leaves -- where p f_i in
// fp32 would be off by 0.06 radians at a position of a million.  Sine and cosine are taken of the product's upper 32 bits, so of an
// angle that is less than 2^-32 of a turn too small.  The two highest bits, rounded, are the quadrant; the rest, at most an eighth
// of a turn, goes through the Taylor series of sin and cos, whose first left-out terms are below 2^-28 and 2^-32.
//
// A thread has one 16-byte vector of a row's pairs (HALF: one of either half) at one position, takes its sines and
// cosines once, and then goes through up to four heads of q and k, all of them loaded before the first angle is known.
// Bound by HBM's latency and rate for many rows, by the launch for few.  Measured: B2 H32 HK8 N4096 D128 bf16 29.5 us, 5.7
// TB/s of 6.8 (37 with eight heads a thread, two at a time, and 43 with values taken apart one by one); fp32 52.5 us, 6.4 TB/s.
// Without 16-byte granules one element (a pair, interleaved) is moved at a time: D80 with 20 that turn 56 us, 1.9 TB/s (36).
#include "common.cuh"
#include "kernels.h"

#include <cuda_fp16.h>

#include <algorithm>
#include <type_traits>

namespace skl {
namespace {

constexpr int THREADS = 128;
constexpr int kThreadsSm = 2048;

// Two neighbouring values of 2 bytes.
template <typename T>
__device__ __forceinline__ float2 unpack(uint32_t w) {
  if constexpr (sizeof(T) == 4) return make_float2(__uint_as_float(w), 0.f);
  if constexpr (std::is_same<T, __half>::value) return __half22float2(*reinterpret_cast<const __half2*>(&w));
  return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
}
template <typename T>
__device__ __forceinline__ uint32_t pack(float2 v) {
  if constexpr (std::is_same<T, __half>::value) {
    const __half2 h = __floats2half2_rn(v.x, v.y);
    return *reinterpret_cast<const uint32_t*>(&h);
  }
  return pack_bf16(v.x, v.y);
}
template <typename T>
__device__ __forceinline__ float one(T x) {
  return static_cast<float>(x);
}
template <typename T>
__device__ __forceinline__ T one_of(float x) {
  if constexpr (std::is_same<T, __half>::value) return __float2half_rn(x);
  if constexpr (std::is_same<T, __nv_bfloat16>::value) return __float2bfloat16_rn(x);
  if constexpr (std::is_same<T, float>::value) return x;
}

// sin and cos of `turn` / 2^64 of a turn.  The angle's highest 32 bits are enough: 2^-32 of a turn is 1.5e-9 radians, a twentieth of
// fp32's half step at 1.
__device__ __forceinline__ void sincos_of_turn(unsigned long long turn, float* sin_out, float* cos_out) {
  const unsigned t = (unsigned)(turn >> 32), quarter = (t + (1u << 29)) >> 30;  // the nearest
  const int rest = (int)(t - (quarter << 30));                                  // within 2^29
  const float x = (float)rest * (6.283185307179586f * 0x1p-32f), y = x * x;    // radians, |x| <= pi / 4
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

constexpr int HEADS = 4;  // of a thread at most
// V elements a vector: 16 bytes, or one pair alone where sizes or addresses do not allow that
template <typename T, bool INTERLEAVED, int V>
__global__ void __launch_bounds__(THREADS, INTERLEAVED ? 10 : 6) rotary_kernel(const RotaryProblem p) {
  constexpr int PAIRS = INTERLEAVED ? V / 2 : V, PARTS = INTERLEAVED ? 1 : 2;
  constexpr bool WIDE = sizeof(T) == 2 && V == 8;  // two values a register
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
  const long long in_q = (long long)b * p.q.b + (long long)n * p.q.n + at, in_k = (long long)b * p.k.b + (long long)n * p.k.n + at;
  const long long out_q = (long long)b * p.qo.b + (long long)n * p.qo.n + at, out_k = (long long)b * p.ko.b + (long long)n * p.ko.n + at;
  auto from = [&](int h) {
    return h < p.HQ ? static_cast<const T*>(p.q_in) + in_q + h * p.q.h : static_cast<const T*>(p.k_in) + in_k + (h - p.HQ) * p.k.h;
  };
  auto to = [&](int h) {
    return h < p.HQ ? static_cast<T*>(p.q_out) + out_q + h * p.qo.h : static_cast<T*>(p.k_out) + out_k + (h - p.HQ) * p.ko.h;
  };
  Vec v[HEADS][PARTS];  // on their way while the angles are formed
#pragma unroll
  for (int i = 0; i < HEADS; ++i) {
    if (first + i < last) {
      const T* src = from(first + i);
      v[i][0] = *reinterpret_cast<const Vec*>(src);
      if (PARTS == 2 && turns) v[i][PARTS - 1] = *reinterpret_cast<const Vec*>(src + p.dim / 2);
    }
  }
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
#pragma unroll
  for (int i = 0; i < HEADS; ++i) {
    if (first + i < last) {
      T* dst = to(first + i);
      if (turns) {
#pragma unroll
        for (int k = 0; k < PAIRS; k += WIDE && !INTERLEAVED ? 2 : 1) {
          if constexpr (WIDE && INTERLEAVED) {
            uint32_t& w = reinterpret_cast<uint32_t*>(&v[i][0])[k];
            const float2 z = unpack<T>(w);
            w = pack<T>(make_float2(fmaf(z.x, c[k], -(z.y * s[k])), fmaf(z.y, c[k], z.x * s[k])));
          } else if constexpr (WIDE) {
            uint32_t &w0 = reinterpret_cast<uint32_t*>(&v[i][0])[k / 2], &w1 = reinterpret_cast<uint32_t*>(&v[i][PARTS - 1])[k / 2];
            const float2 x = unpack<T>(w0), y = unpack<T>(w1);
            const float2 cc = make_float2(c[k], c[(k + 1) % PAIRS]), ss = make_float2(s[k], s[(k + 1) % PAIRS]);
            w0 = pack<T>(fsub2(fmul2(x, cc), fmul2(y, ss)));
            w1 = pack<T>(ffma2(x, ss, fmul2(y, cc)));
          } else {
            T& first_of = INTERLEAVED ? v[i][0].x[(2 * k) % V] : v[i][0].x[k];
            T& second_of = INTERLEAVED ? v[i][0].x[(2 * k + 1) % V] : v[i][PARTS - 1].x[k];
            const float x = one(first_of), y = one(second_of);
            first_of = one_of<T>(fmaf(x, c[k], -(y * s[k])));
            second_of = one_of<T>(fmaf(y, c[k], x * s[k]));
          }
        }
        if (PARTS == 2) *reinterpret_cast<Vec*>(dst + p.dim / 2) = v[i][PARTS - 1];
      }
      *reinterpret_cast<Vec*>(dst) = v[i][0];
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
  // heads a thread: as many as leave kThreadsSm threads an SM, between one and HEADS, and the same for all
  const long long each = std::max(1ll, std::min<long long>({HEADS, heads, p->items * heads / ((long long)num_sms * kThreadsSm)}));
  const int shares = (int)((heads + each - 1) / each);
  p->heads_each = (heads + shares - 1) / shares;
  return true;
}

cudaError_t launch_rotary(const RotaryProblem& p, cudaStream_t st) {
  if (p.dtype == kTypeBf16) return launch_type<__nv_bfloat16>(p, st);
  if (p.dtype == kTypeFp16) return launch_type<__half>(p, st);
  return launch_type<float>(p, st);
}

}  // namespace skl
