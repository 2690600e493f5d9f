// The attention kernels' problem description and the device helpers they share.
#pragma once

#include "common.cuh"
#include "kernels.h"
#include "tc.cuh"

namespace skl {

// The block owns the SM: all 512 TMEM columns, and registers that its warps pass to one another.  It asks for all of the
// shared memory that a block can have, so that no block of another stream's kernel runs beside it, however small.
constexpr int kWholeSmSmem = 227 * 1024;

// A sequence's length: the whole extent, or its entry of a device array, kept within the extent.
__device__ __forceinline__ int seq_len(const int* lens, int b, int n) { return lens ? min(max(lens[b], 0), n) : n; }

template <int R>
__device__ __forceinline__ void setmaxnreg_inc() {
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(R));
}
template <int R>
__device__ __forceinline__ void setmaxnreg_dec() {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(R));
}

// The barrier behind a block's set-up.  A vote on the sequence's lengths before it: their loads have been waited for, and none
// is in flight, when setmaxnreg deals the registers out anew.  (No length is negative, so the fence never runs; it keeps the
// vote.)
__device__ __forceinline__ void setup_barrier(int ql, int kl) {
  asm volatile(
      "{\n\t.reg .pred p, q;\n\tsetp.lt.s32 p, %0, 0;\n\tvote.sync.any.pred q, p, 0xffffffff;\n\t@q membar.cta;\n\t}" ::"r"(ql | kl)
      : "memory");
  __syncthreads();
}

__device__ __forceinline__ void st_shared_zero16(uint32_t addr) {
  asm volatile("st.shared.v4.u32 [%0], {%1, %1, %1, %1};" ::"r"(addr), "r"(0) : "memory");
}

__device__ __forceinline__ void st_shared16(uint32_t addr, uint4 v) {
  asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w) : "memory");
}

__device__ __forceinline__ uint4 ld_shared16(uint32_t addr) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(addr) : "memory");
  return v;
}

__device__ __forceinline__ void tmem_st32(uint32_t taddr, const uint32_t (&r)[32]) {
  tmem_st16(taddr, *reinterpret_cast<const uint32_t(*)[16]>(&r[0]));
  tmem_st16(taddr + 16, *reinterpret_cast<const uint32_t(*)[16]>(&r[16]));
}

__device__ __forceinline__ float2 from_bf16_pair(uint32_t v) {
  return make_float2(__uint_as_float(v << 16), __uint_as_float(v & 0xffff0000u));
}
// a += the pair, by additions that take a bf16.
__device__ __forceinline__ void add_bf16_pair(float2& a, uint32_t v) {
  asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %2;\n\tadd.f32.bf16 %0, l, %0;\n\tadd.f32.bf16 %1, h, %1;\n\t}"
      : "+f"(a.x), "+f"(a.y)
      : "r"(v));
}
// What rounding x to bf16 leaves.
__device__ __forceinline__ float bf16_rest(float x) { return x - __bfloat162float(__float2bfloat16_rn(x)); }

// ---- row values of the backward: -LSE / scale and -delta of a query row, each as three bf16 that add up to its 24
// bits, in 16 bytes.  128 rows of them are the 16-wide K step that adds the rows' values to a product.
constexpr float kNoRow = -1.0e30f;  // -LSE / scale of a row that sees no key: its P is exactly 0

__device__ __forceinline__ uint4 three_bf16(float x) {
  const float hi = __bfloat162float(__float2bfloat16_rn(x));
  const float mid = __bfloat162float(__float2bfloat16_rn(x - hi));
  return make_uint4(pack_bf16(hi, mid), pack_bf16(x - hi - mid, 0.f), 0u, 0u);
}
__device__ __forceinline__ float from_three_bf16(uint2 v) {
  return __uint_as_float(v.x << 16) + (__uint_as_float(v.x & 0xffff0000u) + __uint_as_float(v.y << 16));
}
__device__ __forceinline__ void bulk_load(uint32_t dst, const void* src, uint32_t bytes, uint32_t bar) {
  asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst),
               "l"(src), "r"(bytes), "r"(bar)
               : "memory");
}

// Descriptor of a K-major K step without swizzle: 8-row core matrices 128 bytes apart, the second half of K at `zero`.
__device__ __forceinline__ uint64_t sdesc_step(uint32_t addr, uint32_t zero) {
  return (uint64_t)((addr & 0x3FFFFu) >> 4) | ((uint64_t)(((zero - addr) >> 4) & 0x3FFFu) << 16) |
         ((uint64_t)(128u >> 4) << 32) | (1ull << 46);
}

// P = 2^(c (S - LSE / scale)) of 32 columns (0 for rows without keys and past the sequence), as fp32 over the logits and as
// bf16 pairs; the first `hidden` columns do not see the thread's key.  A copy of its own for the tiles without a mask: there
// the conversions run between the exponentials.
template <bool MASKED>
__device__ __forceinline__ void p32(uint32_t (&a)[32], uint32_t (&pk)[16], float2 cc, int hidden) {
#pragma unroll
  for (int i = 0; i < 32; i += 2) {
    const float2 x = fmul2(make_float2(__uint_as_float(a[i]), __uint_as_float(a[i + 1])), cc);
    float2 e = make_float2(ex2(x.x), ex2(x.y));
    if (MASKED) {
      e.x = i < hidden ? 0.f : e.x;
      e.y = i + 1 < hidden ? 0.f : e.y;
    }
    a[i] = __float_as_uint(e.x);
    a[i + 1] = __float_as_uint(e.y);
    pk[i / 2] = pack_bf16(e.x, e.y);
  }
}

// ---- parts: where a kind of block has fewer or longer tiles than the SMs can share evenly, a tile's stream is dealt out
// over `parts` blocks.  Each leaves its fp32 accumulators in the workspace, and the one that counts up to `parts` adds
// them all in the parts' order, so the sum does not depend on who that is.
struct TilePart {
  int tile, rank, parts;
  // The first of the stream's `n` elements that part `rank + next` takes.
  // (n is below 2^24, parts at most 8.)
  __device__ __forceinline__ int from(int n, int next = 0) const {
    if (parts == 1) return next ? n : 0;
    return (int)((unsigned)n * (unsigned)(rank + next) / (unsigned)parts);
  }
};
// Block x of a kind whose tiles [0, whole) are one block each and the later ones `by.d`.
__device__ __forceinline__ TilePart tile_part(unsigned x, unsigned whole, const FastDiv& by) {
  if (x < whole) return TilePart{(int)x, 0, 1};
  const unsigned t = by.div(x - whole);
  return TilePart{(int)(whole + t), (int)(x - whole - t * by.d), (int)by.d};
}
// A part is [COLS / 4][128 rows] float4: a warp, whose lanes are rows, writes and reads whole lines.
template <int COLS>
__device__ __forceinline__ void part_put(float4* tile, int rank, int r, int col, const uint32_t (&a)[32]) {
  float4* dst = tile + (size_t)rank * (COLS / 4 * 128) + col / 4 * 128 + r;
#pragma unroll
  for (int i = 0; i < 8; ++i)
    __stcg(dst + i * 128, make_float4(__uint_as_float(a[4 * i]), __uint_as_float(a[4 * i + 1]),
                                      __uint_as_float(a[4 * i + 2]), __uint_as_float(a[4 * i + 3])));
}
template <int COLS>
__device__ __forceinline__ void part_sum(const float4* tile, int parts, int r, int col, uint32_t (&a)[32]) {
  float s[32] = {};
#pragma unroll 1
  for (int q = 0; q < parts; ++q) {
    const float4* src = tile + (size_t)q * (COLS / 4 * 128) + col / 4 * 128 + r;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float4 v = __ldcg(src + i * 128);
      s[4 * i] += v.x;
      s[4 * i + 1] += v.y;
      s[4 * i + 2] += v.z;
      s[4 * i + 3] += v.w;
    }
  }
#pragma unroll
  for (int i = 0; i < 32; ++i) a[i] = __float_as_uint(s[i]);
}
// True on the block whose part is the last to be written; `threads` (the first of the block, by whole warps) call it once
// their writes are issued.  The counter is left at zero.
__device__ __forceinline__ bool part_last(unsigned* counter, int parts, int threads, volatile int* flag) {
  __threadfence();
  __syncwarp();
  named_bar_sync(2, threads);
  if (threadIdx.x == 0) {
    const unsigned before = atomicAdd(counter, 1u);
    if (before + 1 == (unsigned)parts) *counter = 0;
    *flag = before + 1 == (unsigned)parts;
    __threadfence();
  }
  __syncwarp();  // the barrier wants whole warps
  named_bar_sync(2, threads);
  return *flag;
}

// ---- a tile out: fp32 rows in registers -> bf16 in a swizzled tile in shared memory -> one TMA store.  Written from
// registers a thread's row would scatter over 32 lines to a store: 2000 cycles a 128 x 128 tile against 300.
__device__ __forceinline__ void tma_store_4d(const CUtensorMap* map, uint32_t src, int x, int y, int z, int w) {
  asm volatile("cp.async.bulk.tensor.4d.global.shared::cta.tile.bulk_group [%0, {%2, %3, %4, %5}], [%1];" ::"l"(
                   reinterpret_cast<uint64_t>(map)),
               "r"(src), "r"(x), "r"(y), "r"(z), "r"(w)
               : "memory");
}
__device__ __forceinline__ void bulk_commit() { asm volatile("cp.async.bulk.commit_group;" ::: "memory"); }
__device__ __forceinline__ void bulk_wait_read() { asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory"); }
// 32 columns from `col` of row r, `f` times, into the tile at `tile`.
__device__ __forceinline__ void stage_row32(uint32_t tile, int r, int col, const uint32_t (&a)[32], float f) {
#pragma unroll
  for (int v = 0; v < 4; ++v) {
    uint32_t w[4];
#pragma unroll
    for (int e = 0; e < 4; ++e)
      w[e] = pack_bf16(__uint_as_float(a[8 * v + 2 * e]) * f, __uint_as_float(a[8 * v + 2 * e + 1]) * f);
    st_shared16(sw128<128>(tile, r, col / 8 + v), make_uint4(w[0], w[1], w[2], w[3]));
  }
}
// Stores the tile (D / 64 halves of 128-byte rows); one thread, after a fence and a barrier of the writers.
template <int D>
__device__ __forceinline__ void store_tile(const CUtensorMap* map, uint32_t tile, int y, int z, int w) {
#pragma unroll
  for (int h = 0; h < D / 64; ++h) tma_store_4d(map, tile + h * 128 * 128, h * 64, y, z, w);
  bulk_commit();
  bulk_wait_read();
}

}  // namespace skl
