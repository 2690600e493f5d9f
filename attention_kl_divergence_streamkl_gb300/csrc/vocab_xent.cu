// Cross entropy over a vocabulary from hidden states, and its gradients, without the logits in memory:
//     z = scale h W^T,  loss_r = LSE_r - z_r,t,  LSE_r = log sum_v e^z_rv
//     d_rv = scale (g_r (p_rv - [v = t_r]) + g'_r p_rv),  p = e^(z - LSE),  dh = d W,  dW = d^T h
// for upstream gradients g of the losses and g' of the log-sum-exps.
//
// All three are matrix products of 2 R C V operations with something done to their tiles, so one product loop serves
// them: pairs of SMs (cta_group::2) work on 256 x 256 tiles, 64 of the summed index at a time.  Each block of a pair
// loads 128 rows of either operand, so a byte from L2 feeds twice the products that it would in a 128 x 256 tile of one
// SM; the accumulators, 256 of the 512 TMEM columns each, take turns, so that the tile's epilogue runs under the next
// tile's products.
//   warps 0-7  epilogue: warp w has the rows 32 (w % 4) and the column half w / 4; thread = row
//   warp 8     TMA producer of the block's own halves
//   warp 9     TMEM owner; in the even block the MMA issuer (one thread)
// Forward: a tile leaves each row's maximum and sum of 2^(z - max) over 128 columns, and the given token's logit where
// it has it; a second kernel joins them in a fixed order.
// Backward: the vocabulary goes by in pieces.  A piece's d (2 bytes, rows x columns) is written once by the first
// launch; the second reads it for both gradients: a piece's rows of dW are complete, the sum for dh goes on from piece
// to piece in fp32.  d is rounded to the inputs' type, as the other operand of the products that it enters is: half a
// step of each term.  In fp16 it is multiplied by a power of two that brings the largest upstream gradient in use to 2^14, for
// p's small values would be lost below 2^-24 otherwise.
// A row without a gradient has d = 0 whatever its logits are, but 0 * NaN would still reach dW through the product: the first
// launch notes rows without a gradient whose logits are not finite, and where there are any, dW is formed with a copy of the
// hidden states that has zeros there.
//
// Measured: forward of 8192 x 131072 x 4096 4.73 to 5.0 ms on different cards, 1.76 to 1.86 PFLOP/s, of 8 rows 178 to 195 us,
// 5.5 to 6 TB/s; gradients of 4096 x 131072 x 2048 3.75 to 4.0 ms, 1.65 to 1.76 PFLOP/s: what the power limit leaves a plain matrix
// product (1.71).  With few rows, pieces of W come from memory, and a chunk's products take 650 to 900 cycles where 606 are
// what the tensor core needs; a launch's first 4 us (the ring's first filling) and last 3.5 us (the last tile's epilogue) stand
// alone: gradients of 333 x 50021 x 1000 in fp16 135 us, floor 52.  Built and not kept: pieces of W brought to the L2 ahead of
// their loads, by TMA or by a warp of its own (forward of 8 x 131072 x 4096 186 -> 213 and 287 us: requests to the L2 are what
// it waits for), chunks of 128 in three stages (as fast), other orders of the summed index for each pair (slower).
#include "attn.cuh"
#include "pair.cuh"

#include <cuda_fp16.h>

#include <algorithm>

namespace skl {
namespace {

constexpr int BM = 128, BK = 64;         // rows of either operand in a block, and of the summed index, a stage
constexpr int TILE = 256;                // a pair's tile: TILE rows x up to TILE columns
constexpr int EPILOGUE_WARPS = 8, PRODUCER_WARP = 8, MMA_WARP = 9;
constexpr int THREADS = 10 * 32;
constexpr int STAGES = 5;
constexpr int HALF_STAGE = BM * BK * 2;  // one operand
constexpr uint32_t kTmemCols = 512;
constexpr int OFF_STAGE = 0, OFF_OUT = STAGES * 2 * HALF_STAGE;  // 8 KB for each epilogue warp
constexpr int OFF_BAR = OFF_OUT + EPILOGUE_WARPS * 8192;
constexpr int BAR_SLOT = 8 * (2 * STAGES + 4);  // full, empty; tile there [2], tile free [2]; TMEM slot, abort flag
static_assert(OFF_BAR + BAR_SLOT + 16 + 1024 <= kWholeSmSmem, "shared memory");

// The tensor core's own additions cut off what does not fit, so a sum loses with every one of its C / 16 steps: 5e-7 of a
// logit's terms for 32 of them, eight times that for 4096 channels in one go.  The forward, whose results are fp32, adds up
// so many chunks at a time and then goes on in registers.  (8192 x 131072 x 4096: 4727 us in one go, 4760 with 8 chunks.)
constexpr int kFlush = 8;

enum Kind { kForward, kGradLogits, kGradients };

// One matrix product: m_tiles x n_tiles tiles, each over `splits` ranges of the k_chunks 64-wide chunks.
struct Job {
  int m_tiles, n_tiles, splits, k_chunks;
  int width;         // columns of a tile, and of its two blocks' halves together
  int m_group;       // forward and d: that many tiles along m share what they read of the other operand
  int a_mn, b_mn;    // the operand lies with its rows (m or n), not the summed index, along the 128-byte lines
  int rows, cols;    // of the output
  int k;             // extent of the summed index
  int a_box, b_box;  // rows of memory in a load's box
  // what a tile's number is divided by: the tiles of a split, of a group, and its rows or (gradients) columns of tiles
  FastDiv by_split, by_group, by_m, by_last, by_n;
  __host__ __device__ long long tiles() const { return (long long)m_tiles * n_tiles * splits; }
};
Job make_job(int m_tiles, int n_tiles, int splits, int k_chunks, int width, int m_group, int a_mn, int b_mn, long long rows,
             long long cols, long long k) {
  Job j{m_tiles, n_tiles, splits, k_chunks, width, m_group, a_mn, b_mn, (int)rows, (int)cols, (int)k, 0, 0, {}, {}, {}, {}, {}};
  j.by_split = FastDiv((unsigned)((long long)m_tiles * n_tiles));
  j.by_n = FastDiv((unsigned)n_tiles);
  if (m_group) {
    j.by_group = FastDiv((unsigned)((long long)m_group * n_tiles));
    j.by_m = FastDiv((unsigned)m_group);
    j.by_last = FastDiv((unsigned)(m_tiles % m_group ? m_tiles % m_group : m_group));
  }
  return j;
}
struct Tile {
  int job, m, n, split, k0, k1;
  // chunks of an accumulator: kForward starts a new one every kFlush chunks, whose values are added outside the tensor core
  __device__ __forceinline__ int step(Kind kind) const { return kind == kForward ? kFlush : k1 - k0; }
};

struct XentParams {
  Job job[2];  // kGradients: dh, dW; else only the first
  // kGradients: pairs below `more` take one tile of the first job more; meanwhile the others take `early` each of the second
  int more, early;
  long long R;
  int V, v0;          // the vocabulary, and the first column of the piece
  float scale, c;     // c = scale log2(e)
  const long long* tokens;
  // forward
  float2* part;       // [2 tiles along V][part_rows]: maximum (log2 units), sum
  float* given;       // [R] the token's logit, before scale
  long long part_rows;
  // d
  const float *lse, *g, *g_lse;
  // fp16: the power of two on d and its inverse, else null
  const float* power;
  int* not_finite;    // d of the first piece: [rows / 32], 32 rows have such hidden states without a gradient
  const int* clean;   // gradients: dW reads the copy of the hidden states
  int accumulate;     // dh goes to the fp32 sums: 0 stored straight to the output, 1 written, 2 added
};

struct Maps {
  CUtensorMap a[2], b[2], out[2], out32, acc, clean;  // out32: d's last 32 columns of a tile
};

// The tiles of a pair, in its order.  One job: every pairs-th, the tiles along m first, in groups of m_group.
// Two: the pair's share of the first job's tiles, then of the second's, in rounds too, so that the tiles at work at a time
// are neighbours and read the same rows of d (a run of tiles to each pair read a piece of d from memory eight times,
// 1.17 GB for 16384 columns, 4096 rows and 2048 channels: gradients of 4096 x 131072 x 2048 4320 us, 3860 in rounds).
__device__ __forceinline__ Tile job_tile(const Job& j, int job, unsigned i) {
  Tile t;
  t.job = job;
  t.split = j.splits == 1 ? 0 : (int)j.by_split.div(i);
  unsigned x = i - (unsigned)t.split * j.by_split.d;
  if (j.m_group) {
    const unsigned group = j.by_group.div(x);
    x -= group * j.by_group.d;
    const FastDiv& here = (int)(group + 1) * j.m_group > j.m_tiles ? j.by_last : j.by_m;
    t.n = (int)here.div(x);
    t.m = (int)(group * j.by_m.d + (x - (unsigned)t.n * here.d));
  } else {
    t.m = (int)j.by_n.div(x);
    t.n = (int)(x - (unsigned)t.m * j.by_n.d);
  }
  t.k0 = 0;
  t.k1 = j.k_chunks;
  if (j.splits > 1) {  // (chunks below 2^24, splits at most 76: 32 bits)
    t.k0 = (int)((unsigned)j.k_chunks * (unsigned)t.split / (unsigned)j.splits);
    t.k1 = (int)((unsigned)j.k_chunks * (unsigned)(t.split + 1) / (unsigned)j.splits);
  }
  return t;
}
struct Walk {
  unsigned pair, pairs, n_first, n_all;
  unsigned early, others, index;  // of the second job: tiles before the common rounds, who has such, the number among them
  template <Kind KIND>
  __device__ __forceinline__ static Walk make(const XentParams& p, unsigned pair, unsigned pairs) {
    Walk w{};
    const unsigned a = (unsigned)p.job[0].tiles();
    w.pair = pair;
    w.pairs = pairs;
    w.n_first = w.n_all = pair < a ? (a - pair + pairs - 1) / pairs : 0;
    if (KIND == kGradients) {
      const unsigned more = (unsigned)p.more;
      w.others = pairs - more;
      w.index = pair - more;
      w.early = pair < more ? 0 : (unsigned)p.early;
      const unsigned common = (unsigned)p.job[1].tiles() - (unsigned)p.early * w.others;
      w.n_all += w.early + (pair < common ? (common - pair + pairs - 1) / pairs : 0);
    }
    return w;
  }
  __device__ __forceinline__ Tile tile(const XentParams& p, unsigned i) const {
    if (i < n_first) return job_tile(p.job[0], 0, pair + i * pairs);
    const unsigned k = i - n_first;
    if (k < early) return job_tile(p.job[1], 1, k * others + index);
    return job_tile(p.job[1], 1, (unsigned)p.early * others + (k - early) * pairs + pair);
  }
};

// What a block loads of its half of an operand for a chunk: `loads` boxes and their bytes.  Rows that do not exist are
// left out, by smaller boxes and fewer of them: TMA's zeros for them come at the price of loads, from one place of the L2
// for all (8 x 131072 x 4096: 298 us with whole boxes, 186 so).  What then lies in shared memory reaches only rows and
// columns of the tile that nobody reads.
struct Half {
  int loads;
  uint32_t bytes;
};
__device__ __forceinline__ Half half_of(int first, int extent, int mn, int box) {
  const int loads = mn ? min(max((extent - first + 63) / 64, 0), 2) : first < extent;
  return Half{loads, (uint32_t)(loads * box * 128)};
}

template <bool HALF>
__device__ __forceinline__ uint32_t pack16(float lo, float hi) {
  if (HALF) {
    const __half2 v = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&v);
  }
  return pack_bf16(lo, hi);
}

// Element `at` of 32 registers, or of 64: one select each, by the index's bits.
__device__ __forceinline__ float pick(const uint32_t (&s)[32], int at) {
  uint32_t t[16];
#pragma unroll
  for (int k = 0; k < 16; ++k) t[k] = at & 16 ? s[k + 16] : s[k];
#pragma unroll
  for (int half = 8; half; half /= 2) {
#pragma unroll
    for (int k = 0; k < half; ++k) t[k] = at & half ? t[k + half] : t[k];
  }
  return __uint_as_float(t[0]);
}
__device__ __forceinline__ float pick(const uint32_t (&s0)[32], const uint32_t (&s1)[32], int at) {
  uint32_t t[32];
#pragma unroll
  for (int k = 0; k < 32; ++k) t[k] = at & 32 ? s1[k] : s0[k];
  return pick(t, at);
}

// instruction descriptor of a pair's tile
template <bool HALF>
__device__ __forceinline__ uint32_t pair_idesc(bool a_mn, bool b_mn, int width) {
  const uint32_t type = HALF ? 0u : 1u;
  return (1u << 4) | (type << 7) | (type << 10) | ((a_mn ? 1u : 0u) << 15) | ((b_mn ? 1u : 0u) << 16) |
         ((uint32_t)(width >> 3) << 17) | ((uint32_t)(TILE >> 4) << 24);
}

template <Kind KIND, bool HALF>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(THREADS, 1)
    xent_kernel(const XentParams p, int* status, const __grid_constant__ Maps maps) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = align1024(smem_raw);
  const uint32_t sb = smem_u32(smem);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = cluster_rank();
  const Walk walk = Walk::make<KIND>(p, blockIdx.x >> 1, gridDim.x >> 1);

  const uint32_t bar = sb + OFF_BAR;
  const uint32_t full = bar, empty = full + 8 * STAGES, there = empty + 8 * STAGES, free_ = there + 16;
  const uint32_t slot = bar + BAR_SLOT;
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + OFF_BAR + BAR_SLOT + 4);

  if (warp == PRODUCER_WARP) {
    if (elect_one()) {
      for (int t = 0; t < (KIND == kGradients ? 2 : 1); ++t) {
        if (!p.job[t].m_tiles) continue;
        prefetch_tensormap(&maps.a[t]);
        prefetch_tensormap(&maps.b[t]);
      }
      for (int s = 0; s < STAGES; ++s) {
        mbar_init(full + 8 * s, 1);   // the even block's: the bytes of both
        mbar_init(empty + 8 * s, 1);  // both blocks', by one commit
      }
      for (int t = 0; t < 2; ++t) {
        mbar_init(there + 8 * t, 1);
        mbar_init(free_ + 8 * t, 2 * EPILOGUE_WARPS);  // the even block's: the epilogue warps of both
      }
      *abort_flag = 0;
      fence_mbar_init();
      fence_async_smem();
    }
    __syncwarp();
  }
  if (warp == MMA_WARP) {
    tmem_alloc_pair(slot, kTmemCols);
    tmem_relinquish_pair();
  }
  tc_fence_before();
  __syncthreads();
  cluster_sync();  // both blocks' barriers and TMEM are set up
  tc_fence_after();
  let_next_begin();
  if (KIND != kForward) wait_for_previous();
  whole_tmem(reinterpret_cast<volatile uint32_t*>(smem + OFF_BAR + BAR_SLOT), status);
  constexpr uint32_t tmem = 0;

  if (warp == PRODUCER_WARP) {
    if (elect_one()) {
      const uint32_t full_even = in_block(full, 0);
      const bool clean = KIND == kGradients && p.job[1].m_tiles && *p.clean;
      int s = 0;          // the stage that is filled next
      uint32_t lap = 0;   // how often the ring has been round
      bool ok = true;
      for (unsigned i = 0; ok && i < walk.n_all; ++i) {
        const Tile t = walk.tile(p, i);
        const Job& j = p.job[t.job];
        const CUtensorMap *ma = &maps.a[t.job], *mb = KIND == kGradients && t.job && clean ? &maps.clean : &maps.b[t.job];
        const int wide = j.width / 2, m0 = t.m * TILE + (int)rank * BM, n0 = t.n * j.width + (int)rank * wide;
        const Half a_half = half_of(m0, j.rows, j.a_mn, j.a_box), b_half = half_of(n0, j.cols, j.b_mn, j.b_box);
        // the bytes of both blocks
        const uint32_t bytes = half_of(t.m * TILE, j.rows, j.a_mn, j.a_box).bytes + half_of(t.m * TILE + BM, j.rows, j.a_mn, j.a_box).bytes +
                               half_of(t.n * j.width, j.cols, j.b_mn, j.b_box).bytes + half_of(t.n * j.width + wide, j.cols, j.b_mn, j.b_box).bytes;
        for (int k = t.k0; k < t.k1; ++k) {
          if (lap && !(ok = mbar_wait(empty + 8 * s, (lap - 1) & 1, status, abort_flag))) break;
          const uint32_t a = sb + OFF_STAGE + s * 2 * HALF_STAGE, b = a + HALF_STAGE, done = full_even + 8 * s;
          if (rank == 0) mbar_arrive_expect_tx(full + 8 * s, bytes);
          for (int h = 0; h < a_half.loads; ++h)
            tma_load_2d_pair(a + h * (HALF_STAGE / 2), ma, done, j.a_mn ? m0 + 64 * h : k * BK, j.a_mn ? k * BK : m0);
          for (int h = 0; h < b_half.loads; ++h)
            tma_load_2d_pair(b + h * (HALF_STAGE / 2), mb, done, j.b_mn ? n0 + 64 * h : k * BK, j.b_mn ? k * BK : n0);
          if (++s == STAGES) {
            s = 0;
            ++lap;
          }
        }
      }
      // the stages in flight have landed once the products that read them are done; after a wait that ran out, the even
      // block waits for the bytes of both
      for (int v = 0; v < STAGES; ++v) {
        if (v >= s && !lap) break;  // never filled
        const uint32_t parity = (v < s ? lap : lap - 1) & 1;
        if (ok)
          mbar_drain(empty + 8 * v, parity, status);
        else if (rank == 0)
          mbar_drain(full + 8 * v, parity, status);
      }
    }
    __syncwarp();
  } else if (warp == MMA_WARP) {
    if (rank == 0 && elect_one()) {
      int s = 0;
      uint32_t phase = 0, used = 0;  // used: accumulators begun
      bool ok = true;
      for (unsigned i = 0; ok && i < walk.n_all; ++i) {
        const Tile t = walk.tile(p, i);
        const Job& j = p.job[t.job];
        const uint32_t idesc = pair_idesc<HALF>(j.a_mn, j.b_mn, j.width);
        const uint32_t a_step = j.a_mn ? 2048 : 32, b_step = j.b_mn ? 2048 : 32;
        const uint32_t a_lbo = j.a_mn ? HALF_STAGE / 2 : 0, b_lbo = j.b_mn ? HALF_STAGE / 2 : 0;
        for (int k0 = t.k0; ok && k0 < t.k1; k0 += t.step(KIND), ++used) {
          const uint32_t buf = used & 1;
          if (used >= 2 && !(ok = mbar_wait(free_ + 8 * buf, (used / 2 - 1) & 1, status, abort_flag))) break;
          tc_fence_after();
          for (int k = k0; k < min(k0 + t.step(KIND), t.k1); ++k) {
            if (!(ok = mbar_wait(full + 8 * s, phase, status, abort_flag))) break;
            tc_fence_after();
            const uint32_t at = sb + OFF_STAGE + s * 2 * HALF_STAGE;
            const uint64_t ad = sdesc_sw128(at, a_lbo, 1024), bd = sdesc_sw128(at + HALF_STAGE, b_lbo, 1024);
            const int steps = min(BK / 16, (j.k - k * BK + 15) / 16);  // the last chunk may be short
#pragma unroll
            for (int ks = 0; ks < BK / 16; ++ks)
              if (ks < steps)
                mma_pair(tmem + TILE * buf, sdesc_add(ad, ks * a_step), sdesc_add(bd, ks * b_step), idesc, k > k0 || ks > 0);
            mma_commit_pair(empty + 8 * s);
            if (++s == STAGES) {
              s = 0;
              phase ^= 1;
            }
          }
          if (ok) mma_commit_pair(there + 8 * buf);
        }
      }
    }
    __syncwarp();
  } else {
    // -------------------------------------------------------------- epilogue
    const int quarter = warp & 3, half = warp >> 2;
    const uint32_t lanes = (uint32_t)(quarter * 32) << 16;
    // A warp's 32 rows leave through 8 KB, 128 columns of 2 bytes or 64 of 4, as two boxes under one fence (a fence
    // for each 64 columns: 4700 cycles a tile of dW where its sum is one chunk, 4100 so).
    const uint32_t stage = sb + OFF_OUT + warp * 8192;
    auto stage_free = [&]() {  // the stores before have read it
      if (elect_one()) bulk_wait_read();
      __syncwarp();
    };
    auto put = [&](int box, const uint32_t (&w)[32]) {  // the lane's row of a box, 128 bytes
#pragma unroll
      for (int k = 0; k < 8; ++k)
        st_shared16(stage + box * 4096 + lane * 128 + ((k ^ (lane & 7)) << 4), make_uint4(w[4 * k], w[4 * k + 1], w[4 * k + 2], w[4 * k + 3]));
    };
    const uint32_t free_even = in_block(free_, 0);
    const float power = HALF && KIND != kForward ? p.power[KIND == kGradients] : 1.f;
    uint32_t used = 0;  // accumulators taken
    for (unsigned i = 0; i < walk.n_all; ++i) {
      const Tile t = walk.tile(p, i);
      const uint32_t buf = used & 1, parity = used / 2 & 1;
      const int row0 = t.m * TILE + (int)rank * BM + quarter * 32;  // the warp's first row
      const int col0 = t.n * p.job[t.job].width + half * 128;       // and column
      const int here_cols = min(128, p.job[t.job].width - half * 128);  // of the tile's
      const int row = row0 + lane;
      const uint32_t ta = tmem + lanes + TILE * buf + 128 * half;
      if constexpr (KIND == kForward) {
        const bool real = row < p.R;
        const long long token = real ? p.tokens[row] : -1;
        uint32_t s0[32], s1[32], s2[32], s3[32];
        bool ok = true;
        for (int k0 = t.k0; k0 < t.k1; k0 += kFlush, ++used) {
          const uint32_t b = used & 1, from = tmem + lanes + TILE * b + 128 * half;
          if (!(ok = mbar_wait_warp(there + 8 * b, used / 2 & 1, status, abort_flag))) break;
          tc_fence_after();
          if (k0 == t.k0) {
            tmem_ld32(from, s0);
            tmem_ld32(from + 32, s1);
            tmem_ld32(from + 64, s2);
            tmem_ld32(from + 96, s3);
            tmem_ld_wait();
            reg_fence32(s0);
            reg_fence32(s1);
            reg_fence32(s2);
            reg_fence32(s3);
          } else {
#pragma unroll
            for (int q = 0; q < 8; ++q) {
              uint32_t x[16];
              tmem_ld16(from + 16 * q, x);
              tmem_ld_wait();
              reg_fence16(x);
              uint32_t* to = (q < 2 ? s0 : q < 4 ? s1 : q < 6 ? s2 : s3) + 16 * (q & 1);
#pragma unroll
              for (int k = 0; k < 16; k += 2) {
                const float2 y = fadd2(make_float2(__uint_as_float(to[k]), __uint_as_float(to[k + 1])),
                                       make_float2(__uint_as_float(x[k]), __uint_as_float(x[k + 1])));
                to[k] = __float_as_uint(y.x);
                to[k + 1] = __float_as_uint(y.y);
              }
            }
          }
          tc_fence_before();
          arrive_one_in(free_even + 8 * b);
        }
        if (!ok) break;
        const int seen = min(p.V - col0, here_cols);
        const long long at = token - col0;
        if (__any_sync(0xffffffffu, at >= 0 && at < min(128, seen))) {
          const float z = at & 64 ? pick(s2, s3, (int)at) : pick(s0, s1, (int)at);
          if (at >= 0 && at < min(128, seen)) p.given[row] = z;
        }
        if (seen < 128) {
#pragma unroll
          for (int k = 0; k < 32; ++k) {
            if (k >= seen) s0[k] = __float_as_uint(kNegInf);
            if (k + 32 >= seen) s1[k] = __float_as_uint(kNegInf);
            if (k + 64 >= seen) s2[k] = __float_as_uint(kNegInf);
            if (k + 96 >= seen) s3[k] = __float_as_uint(kNegInf);
          }
        }
        // Four chains of maxima and of sums, and the given token's logit by selects (a test of each of 128 for it held one tile in
        // two up): 4096 x 32000 x 256 88 -> 68 us, x 512 98 -> 81, 4096 x 50257 x 1024 244 -> 226; with less than 8 chunks a
        // tile the exponentials, 2048 cycles, and the way from tile to tile bound it.  (A quarter of them as polynomials: slower.)
        float top[4] = {kNegInf, kNegInf, kNegInf, kNegInf};
#pragma unroll
        for (int k = 0; k < 32; k += 2) {
          top[0] = fmax3(top[0], __uint_as_float(s0[k]), __uint_as_float(s0[k + 1]));
          top[1] = fmax3(top[1], __uint_as_float(s1[k]), __uint_as_float(s1[k + 1]));
          top[2] = fmax3(top[2], __uint_as_float(s2[k]), __uint_as_float(s2[k + 1]));
          top[3] = fmax3(top[3], __uint_as_float(s3[k]), __uint_as_float(s3[k + 1]));
        }
        const float mx = fmax3(fmaxf(top[0], top[1]), top[2], top[3]);
        const float m = mx * p.c;
        // (m, not mx: a logit near the type's lowest value is -inf in these units)
        const float2 cc = make_float2(p.c, p.c), nm = m == kNegInf ? make_float2(0.f, 0.f) : make_float2(-m, -m);
        float2 l0 = make_float2(0.f, 0.f), l1 = l0, l2 = l0, l3 = l0;
#pragma unroll
        for (int k = 0; k < 32; k += 2) {
          auto two = [&](const uint32_t (&s)[32]) { return ffma2(make_float2(__uint_as_float(s[k]), __uint_as_float(s[k + 1])), cc, nm); };
          const float2 x0 = two(s0), x1 = two(s1), x2 = two(s2), x3 = two(s3);
          l0 = fadd2(l0, make_float2(ex2(x0.x), ex2(x0.y)));
          l1 = fadd2(l1, make_float2(ex2(x1.x), ex2(x1.y)));
          l2 = fadd2(l2, make_float2(ex2(x2.x), ex2(x2.y)));
          l3 = fadd2(l3, make_float2(ex2(x3.x), ex2(x3.y)));
        }
        const float2 l = fadd2(fadd2(l0, l1), fadd2(l2, l3));
        if (real) p.part[(size_t)(2 * t.n + half) * p.part_rows + row] = make_float2(m, l.x + l.y);
      } else if constexpr (KIND == kGradLogits) {
        const bool real = row < p.R;
        long long at = -1;
        float lse2 = 0.f, a = 0.f, g = 0.f;
        if (real) {
          const long long token = p.tokens[row];
          lse2 = p.lse[row] * kLog2e;
          if (token >= 0 && token < p.V) {
            g = p.g[row] * p.scale * power;
            at = token - p.v0 - col0;
          }
          a = g + (p.g_lse ? p.g_lse[row] * p.scale * power : 0.f);
        }
        const bool none = g == 0.f && a == 0.f;
        const int seen = real ? min(p.job[0].cols - col0, here_cols) : 0;  // d is 0 past the piece; what is past the rows is not stored
        if (!mbar_wait_warp(there + 8 * buf, parity, status, abort_flag)) break;
        ++used;
        tc_fence_after();
#pragma unroll 1
        for (int q = 0; q < 2; ++q) {
          uint32_t s0[32], s1[32], w[32];
          tmem_ld32(ta + 64 * q, s0);
          tmem_ld32(ta + 64 * q + 32, s1);
          tmem_ld_wait();
          reg_fence32(s0);
          reg_fence32(s1);
          if (q == 1) {
            tc_fence_before();
            arrive_one_in(free_even + 8 * buf);
          }
          if (q == 0 && half == 0 && t.n == 0 && p.not_finite) {
            const bool bad = __any_sync(0xffffffffu, real && none && !(fabsf(__uint_as_float(s0[0])) <= 3.4e38f));
            if (row0 < p.R && elect_one()) p.not_finite[row0 / 32] = bad;
            __syncwarp();
          }
          const long long here = at - 64 * q;
          const bool given = __any_sync(0xffffffffu, here >= 0 && here < 64);
          const bool edge = __any_sync(0xffffffffu, seen < 64 * (q + 1));
          const float2 cc = make_float2(p.c, p.c), nl = make_float2(-lse2, -lse2), aa = make_float2(a, a);
          auto d_of = [&](int k) {
            const uint32_t* s = k < 32 ? s0 : s1;
            const float2 x = ffma2(make_float2(__uint_as_float(s[k & 31]), __uint_as_float(s[(k & 31) + 1])), cc, nl);
            return fmul2(make_float2(ex2(x.x), ex2(x.y)), aa);
          };
          if (!given && !edge) {  // most tiles
#pragma unroll
            for (int k = 0; k < 64; k += 2) {
              const float2 d = d_of(k);
              w[k / 2] = pack16<HALF>(d.x, d.y);
            }
          } else {
#pragma unroll
            for (int k = 0; k < 64; k += 2) {
              float2 d = d_of(k);
              if (here == k) d.x -= g;
              if (here == k + 1) d.y -= g;
              if (64 * q + k >= seen) d.x = 0.f;
              if (64 * q + k + 1 >= seen) d.y = 0.f;
              w[k / 2] = pack16<HALF>(d.x, d.y);
            }
          }
          if (__any_sync(0xffffffffu, none)) {  // no gradient is none, whatever the logits are
#pragma unroll
            for (int k = 0; k < 32; ++k) w[k] = none ? 0u : w[k];
          }
          if (q == 0) stage_free();
          if (64 * (q + 1) <= here_cols) {
            put(q, w);
          } else {  // 32 columns are left, rows of 64 bytes
#pragma unroll
            for (int k = 0; k < 4; ++k)
              st_shared16(stage + q * 4096 + lane * 64 + ((k ^ (lane >> 1 & 3)) << 4), make_uint4(w[4 * k], w[4 * k + 1], w[4 * k + 2], w[4 * k + 3]));
          }
        }
        fence_async_smem();
        __syncwarp();
        if (elect_one()) {
#pragma unroll
          for (int q = 0; q < 2; ++q) {
            const int left = here_cols - 64 * q, col = col0 + 64 * q;
            if (row0 >= p.R || col >= p.job[0].cols || left <= 0) continue;
            tma_store_2d(left >= 64 ? &maps.out[0] : &maps.out32, stage + 4096 * q, col, row0);
          }
          bulk_commit();
        }
        __syncwarp();
      } else {
        const Job& j = p.job[t.job];
        const bool sums = t.job == 0 && p.accumulate;
        if (!mbar_wait_warp(there + 8 * buf, parity, status, abort_flag)) break;
        ++used;
        tc_fence_after();
        const bool rows_there = row0 < j.rows;
        uint32_t s0[32], s1[32], s2[32], s3[32];
        tmem_ld32(ta, s0);
        tmem_ld32(ta + 32, s1);
        tmem_ld32(ta + 64, s2);
        tmem_ld32(ta + 96, s3);
        tmem_ld_wait();
        reg_fence32(s0);
        reg_fence32(s1);
        reg_fence32(s2);
        reg_fence32(s3);
        tc_fence_before();
        arrive_one_in(free_even + 8 * buf);
        if (sums) {
#pragma unroll
          for (int q = 0; q < 2; ++q) {
            stage_free();
            put(0, q ? s2 : s0);
            put(1, q ? s3 : s1);
            fence_async_smem();
            __syncwarp();
            if (elect_one()) {
#pragma unroll
              for (int h = 0; h < 2; ++h) {
                const int col = col0 + 64 * q + 32 * h;
                if (rows_there && col < j.cols) {
                  if (p.accumulate == 1)
                    tma_store_3d(&maps.acc, stage + 4096 * h, col, row0, t.split);
                  else
                    tma_add_3d(&maps.acc, stage + 4096 * h, col, row0, t.split);
                }
              }
              bulk_commit();
            }
            __syncwarp();
          }
        } else {
          stage_free();
#pragma unroll
          for (int q = 0; q < 2; ++q) {
            uint32_t w[32];
#pragma unroll
            for (int k = 0; k < 32; ++k) {
              const uint32_t* s = q ? (k < 16 ? s2 : s3) : (k < 16 ? s0 : s1);
              w[k] = pack16<HALF>(__uint_as_float(s[2 * (k & 15)]) * power, __uint_as_float(s[2 * (k & 15) + 1]) * power);
            }
            put(q, w);
          }
          fence_async_smem();
          __syncwarp();
          if (elect_one()) {
#pragma unroll
            for (int q = 0; q < 2; ++q)
              if (rows_there && col0 + 64 * q < j.cols)
                tma_store_2d(&maps.out[t.job], stage + 4096 * q, col0 + 64 * q, row0 + (t.job ? p.v0 : 0));
            bulk_commit();
          }
          __syncwarp();
        }
      }
    }
    if (KIND != kForward) {
      stage_free();  // the block's memory is read until then; the grid's end waits for the writes
    }
  }
  tc_fence_before();
  __syncthreads();
  cluster_sync();  // nothing of this block is read or arrived on any more
  if (warp == MMA_WARP) {
    tc_fence_after();
    tmem_dealloc_pair(tmem, kTmemCols);
  }
}

// Joins the tiles' maxima and sums.  A block has `each` rows (a power of two up to 32: neighbouring threads have
// neighbouring rows) and deals the parts of a row out over its other threads, whose loads go out four at a time.
constexpr int kJoinThreads = 512, kJoinAhead = 4;
__device__ __forceinline__ float2 join(float2 a, float2 b) {
  const float to = fmaxf(a.x, b.x);
  // (nothing but -inf on a side, and the sum's start, have a sum of 0 there; a NaN stays)
  const float l = (a.x == to ? a.y : a.y * ex2(a.x - to)) + (b.x == to ? b.y : b.y * ex2(b.x - to));
  return make_float2(to, l);
}
__global__ void __launch_bounds__(kJoinThreads)
    xent_join_kernel(long long R, int V, float c, int parts, int each, long long part_rows, const float2* __restrict__ part,
                     const float* __restrict__ given, const long long* __restrict__ tokens, float* __restrict__ loss,
                     float* __restrict__ lse) {
  __shared__ float2 sums[kJoinThreads];
  wait_for_previous();
  const int mine = threadIdx.x & (each - 1), share = threadIdx.x / each, shares = kJoinThreads / each;
  const long long row = (long long)blockIdx.x * each + mine;
  const bool real = row < R;
  float2 x = make_float2(kNegInf, 0.f);
  if (real)
    for (int i = share; i < parts; i += kJoinAhead * shares) {
      float2 y[kJoinAhead];
#pragma unroll
      for (int k = 0; k < kJoinAhead; ++k)
        y[k] = i + k * shares < parts ? part[(size_t)(i + k * shares) * part_rows + row] : make_float2(kNegInf, 0.f);
#pragma unroll
      for (int k = 0; k < kJoinAhead; ++k) x = join(x, y[k]);
    }
  sums[threadIdx.x] = x;
  for (int half = shares / 2; half; half /= 2) {
    __syncthreads();
    if (share < half) sums[threadIdx.x] = x = join(x, sums[threadIdx.x + half * each]);
  }
  if (share || !real) return;
  const float m = x.x, l = x.y, log_sum = logf(l);
  lse[row] = m == kNegInf && l == 0.f ? kNegInf : fmaf(m, kLn2, log_sum);
  const long long token = tokens[row];
  // The difference first, rounded once, as the sum's exponents are: a loss keeps its digits however far from 0 the logits lie.
  // (With c times the given logit rounded on its own, logits of 4096 cost 3e-4 of the loss.)
  loss[row] = token < 0 ? 0.f : token >= V ? __int_as_float(0x7fc00000) : fmaf(fmaf(-given[row], c, m), kLn2, log_sum);
}

// fp16: the power of two that brings the largest scale (|g| + |g'|) to [2^13, 2^14), and its inverse.  Of what d is made of: g
// only where the row has a token, and only finite values (one that is not leaves the other rows' digits alone).  One cluster, whose
// first block gathers the others' maxima (one block: 65536 rows, 64 channels, 512 words 340 us for the gradients, 329 so).
constexpr int kPowerBlocks = 8;
__global__ void __cluster_dims__(kPowerBlocks, 1, 1) __launch_bounds__(1024)
    xent_power_kernel(long long R, int V, float scale, const long long* __restrict__ tokens, const float* __restrict__ g,
                      const float* __restrict__ g_lse, float* __restrict__ power) {
  __shared__ float warp_max[32], block_max[kPowerBlocks];
  const uint32_t rank = cluster_rank();
  let_next_begin();
  cluster_sync();  // the first block is there
  float mx = 0.f;
  for (long long i = rank * 1024 + threadIdx.x; i < R; i += kPowerBlocks * 1024) {
    const long long token = tokens[i];
    const float of_loss = fabsf(g[i]), of_lse = g_lse ? fabsf(g_lse[i]) : 0.f;
    const float x = scale * ((token >= 0 && token < V ? of_loss : 0.f) + of_lse);
    if (x < __int_as_float(0x7f800000)) mx = fmaxf(mx, x);
  }
#pragma unroll
  for (int w = 16; w; w >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, w));
  if ((threadIdx.x & 31) == 0) warp_max[threadIdx.x >> 5] = mx;
  __syncthreads();
  if (threadIdx.x == 0) {
    for (int w = 1; w < 32; ++w) mx = fmaxf(mx, warp_max[w]);
    asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(in_block(smem_u32(&block_max[rank]), 0)), "f"(mx) : "memory");
  }
  __syncwarp();
  cluster_sync();
  if (rank || threadIdx.x) return;
  for (int r = 0; r < kPowerBlocks; ++r) mx = fmaxf(mx, block_max[r]);
  int e = 0;
  if (mx > 0.f) {
    frexpf(mx, &e);  // mx = f 2^e, f in [1/2, 1)
    e = min(max(14 - e, -100), 100);
  }
  power[0] = ldexpf(1.f, e);
  power[1] = ldexpf(1.f, -e);
}

// The copy of the hidden states with zeros in rows without a gradient, where one of these is not finite; 16 bytes a thread.
__global__ void __launch_bounds__(256)
    xent_clean_kernel(long long R, int V, int C, long long stride, const uint4* __restrict__ hidden, const long long* __restrict__ tokens,
                      const float* __restrict__ g, const float* __restrict__ g_lse, const int* __restrict__ not_finite,
                      int* __restrict__ clean, uint4* __restrict__ out) {
  let_next_begin();
  wait_for_previous();
  bool bad = false;
  for (long long i = threadIdx.x; i < (R + 31) / 32; i += 256) bad |= __ldcg(not_finite + i) != 0;
  bad = __syncthreads_or(bad);
  if (blockIdx.x == 0 && threadIdx.x == 0) *clean = bad;
  if (!bad) return;
  for (long long r = blockIdx.x; r < R; r += gridDim.x) {
    const long long token = tokens[r];
    const bool none = (token < 0 || token >= V || g[r] == 0.f) && (!g_lse || g_lse[r] == 0.f);
    for (int i = threadIdx.x; i < C / 8; i += 256)
      out[r * (C / 8) + i] = none ? make_uint4(0u, 0u, 0u, 0u) : hidden[r * (stride / 8) + i];
  }
}

// dh from the splits' fp32 sums, added in their order.
template <bool HALF>
__global__ void __launch_bounds__(256)
    xent_close_kernel(long long n, int splits, const float4* __restrict__ acc, const float* __restrict__ power,
                      uint2* __restrict__ out) {
  const long long i = (long long)blockIdx.x * 256 + threadIdx.x;  // four values
  wait_for_previous();
  if (i >= n) return;
  constexpr int AHEAD = 8;
  float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
  for (int k = 0; k < splits; k += AHEAD) {
    float4 v[AHEAD];
#pragma unroll
    for (int e = 0; e < AHEAD; ++e)
      if (k + e < splits) v[e] = __ldcg(acc + (k + e) * n + i);
#pragma unroll
    for (int e = 0; e < AHEAD; ++e) {
      if (k + e >= splits) break;
      s.x += v[e].x;
      s.y += v[e].y;
      s.z += v[e].z;
      s.w += v[e].w;
    }
  }
  const float f = HALF ? power[1] : 1.f;
  out[i] = make_uint2(pack16<HALF>(s.x * f, s.y * f), pack16<HALF>(s.z * f, s.w * f));
}

// What a tile takes, in the time of a chunk's products: its chunks and kMoreChunks for its epilogue, which the products
// share the shared memory with; a tile of dW, whose 128 KB go out to memory at a pair's share of its rate, kTileChunks at least.
constexpr int kTileChunks = 7, kMoreChunks = 4;

int tiles_of(long long n, int of) { return (int)((n + of - 1) / of); }
size_t up(size_t n, size_t to) { return (n + to - 1) / to * to; }

// Pairs of the device's SMs, no more than there are tiles.
int pairs_for(long long tiles, int num_sms) { return (int)std::max<long long>(1, std::min<long long>(tiles, num_sms / 2)); }

// Rows of h that stay in L2 beside the passing tiles of W: the tiles along m go by in groups of so many.
constexpr double kGroupBytes = 48e6;
int m_group(const XentProblem& p, int m_tiles) {
  return std::max(1, std::min(m_tiles, (int)(kGroupBytes / (2.0 * TILE * p.C))));
}

// Columns of the forward's and d's tiles: 256, or fewer where the last wave of pairs would have few tiles.  A chunk's products
// take as long as the tile is wide, its loads as long as both operands' rows; an epilogue kMoreChunks of the widest.  Narrower
// tiles only for a tenth (forward of 100 x 20000 x 4096: 62 us with 79 tiles of 256, 57.8 with 125 of 160; 64 x 32000 x 512, two
// waves either way: 21.0 with 256, 21.9 with 224).
int tile_width(int m_tiles, long long rows, long long cols, int k_chunks, int num_sms) {
  const int pairs = std::max(1, num_sms / 2);
  int best = TILE;
  double least = 0;
  for (int w = TILE; w >= 160; w -= 32) {
    const long long waves = (m_tiles * ((cols + w - 1) / w) + pairs - 1) / pairs;
    const double loads = (double)(std::min<long long>(rows, TILE) + w) / (2 * TILE);
    const double cost = waves * (k_chunks * std::max((double)w / TILE, loads) + kMoreChunks);
    if (w == TILE || cost < least * 0.9) {
      best = w;
      least = cost;
    }
  }
  return best;
}

template <Kind KIND, bool HALF>
cudaError_t launch(const XentParams& p, const Maps& maps, int pairs, int* status, cudaStream_t st, bool behind = false) {
  const auto kern = xent_kernel<KIND, HALF>;
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, kWholeSmSmem);
  if (e != cudaSuccess) return e;
  if (KIND != kForward && behind) return launch_behind(kern, (unsigned)(2 * pairs), THREADS, kWholeSmSmem, st, p, status, maps);
  kern<<<(unsigned)(2 * pairs), THREADS, kWholeSmSmem, st>>>(p, status, maps);
  return cudaGetLastError();
}

// A matrix [rows, cols] of 2-byte values: an operand whose lines run along the summed index (k_major) or along its rows.
// `box`: rows of a load, no more than there are (the summed index in whole steps of 16).
bool operand_map(CUtensorMap* map, const void* base, long long rows, long long cols, long long stride, bool k_major, int* box,
                 int most = BM) {
  *box = k_major ? (int)std::min<long long>(most, up(rows, 8)) : (int)std::min<long long>(BK, up(rows, 16));
  return encode_matrix_map(map, base, rows, cols, stride, *box, 64);
}

}  // namespace

// The vocabulary's pieces.  A piece's d lies in memory between the two launches: at most kPieceBytes of it, but at least
// kPieceColumns, so that the sums of dh, read and written once a piece (8 bytes for 6 V / pieces operations), stay below
// a few hundredths of the products' time.  Each launch ends with a wave that is not full, and no piece that is worth its
// launches stays in the L2.  Measured, us, gradients of 4096 x 131072 x 2048 and 8192 x 131072 x 4096: 64 MB 3956, 15694; 128 MB
// 3864, 15723; 256 MB 3756, 15331; 512 MB 3745, 15367; of 4096 x 65536 x 256 and 16384 x 50257 x 1024: 256 MB 407, 3440; 512 MB
// 369, 3145; 1 GB 369, 3117.
constexpr long long kLine = 64;  // rows of d begin on whole lines: a box's row is then one request to the L2, not two
constexpr long long kPieceBytes = 512ll << 20, kPieceColumns = 8192;
XentBwdPlan xent_bwd_plan(const XentProblem& p, bool want_dh, bool want_dw, int num_sms) {
  XentBwdPlan g{};
  const long long most = std::max(kPieceColumns, kPieceBytes / (2 * std::max(p.R, 1ll)));
  g.pieces = (int)((p.V + most - 1) / most);
  g.columns = (int)up((size_t)((p.V + g.pieces - 1) / g.pieces), TILE);
  g.pieces = (int)((p.V + g.columns - 1) / g.columns);
  // few tiles of dh: their long sums are split over blocks, until there is one for every pair or each is 16 chunks long
  g.splits = 1;
  if (want_dh) {
    const long long tiles = (long long)tiles_of(p.R, TILE) * tiles_of(p.C, TILE);
    const long long chunks = tiles_of(std::min<long long>(g.columns, p.V), BK);
    g.splits = (int)std::max(1ll, std::min((num_sms / 2) / tiles, chunks / 16));
  }
  g.direct = g.pieces == 1 && g.splits == 1;
  g.off_d = up(256 + (size_t)tiles_of(p.R, 32) * sizeof(int), 256);
  g.off_acc = g.off_d + up((size_t)p.R * std::min<long long>(g.columns, (long long)up(p.V, kLine)) * 2, 256);
  g.off_clean = g.off_acc + (want_dh && !g.direct ? up((size_t)g.splits * p.R * p.C * 4, 256) : 0);
  g.bytes = g.off_clean + (want_dw ? (size_t)p.R * p.C * 2 : 0);
  return g;
}

int xent_fwd_width(const XentProblem& p, int num_sms) {
  return tile_width(tiles_of(p.R, TILE), p.R, p.V, tiles_of(p.C, BK), num_sms);
}

size_t xent_fwd_workspace(const XentProblem& p, int num_sms) {
  return up((size_t)p.R * 4, 256) + (size_t)2 * tiles_of(p.V, xent_fwd_width(p, num_sms)) * up(p.R, 32) * sizeof(float2);
}

cudaError_t launch_xent_fwd(const XentProblem& p, const void* hidden, const void* weight, const long long* tokens, float* loss,
                            float* lse, void* workspace, int num_sms, int* status, cudaStream_t st) {
  Maps maps{};
  XentParams k{};
  const int width = xent_fwd_width(p, num_sms), m_tiles = tiles_of(p.R, TILE), n_tiles = tiles_of(p.V, width);
  k.job[0] = make_job(m_tiles, n_tiles, 1, tiles_of(p.C, BK), width, m_group(p, m_tiles), 0, 0, p.R, p.V, p.C);
  if (!operand_map(&maps.a[0], hidden, p.R, p.C, p.hidden_stride, true, &k.job[0].a_box) ||
      !operand_map(&maps.b[0], weight, p.V, p.C, p.weight_stride, true, &k.job[0].b_box, width / 2))
    return cudaErrorInvalidValue;
  k.R = p.R;
  k.V = (int)p.V;
  k.scale = p.scale;
  k.c = p.scale * kLog2e;
  k.tokens = tokens;
  k.given = static_cast<float*>(workspace);
  k.part_rows = (long long)up(p.R, 32);
  k.part = reinterpret_cast<float2*>(static_cast<uint8_t*>(workspace) + up((size_t)p.R * 4, 256));
  const int pairs = pairs_for(k.job[0].tiles(), num_sms);
  cudaError_t e = p.half ? launch<kForward, true>(k, maps, pairs, status, st) : launch<kForward, false>(k, maps, pairs, status, st);
  if (e != cudaSuccess) return e;
  int each = 32;
  while (each > 1 && each / 2 >= p.R) each /= 2;
  return launch_behind(xent_join_kernel, (unsigned)tiles_of(p.R, each), kJoinThreads, 0, st, p.R, (int)p.V, k.c, 2 * n_tiles, each,
                       k.part_rows, k.part, k.given, tokens, loss, lse);
}

cudaError_t launch_xent_bwd(const XentProblem& p, const XentBwdPlan& g, const XentBwdIn& in, void* dhidden, void* dweight,
                            void* workspace, int num_sms, int* status, cudaStream_t st) {
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  float* power = reinterpret_cast<float*>(ws);
  uint8_t* d = ws + g.off_d;
  float* acc = reinterpret_cast<float*>(ws + g.off_acc);
  int *clean = reinterpret_cast<int*>(ws + 128), *not_finite = reinterpret_cast<int*>(ws + 256);
  cudaError_t e = cudaSuccess;
  if (p.half) {
    xent_power_kernel<<<kPowerBlocks, 1024, 0, st>>>(p.R, (int)p.V, p.scale, in.tokens, in.g, in.g_lse, power);
    if ((e = cudaGetLastError()) != cudaSuccess) return e;
  }
  const int m_tiles = tiles_of(p.R, TILE), c_tiles = tiles_of(p.C, TILE);
  for (int piece = 0; piece < g.pieces; ++piece) {
    const long long v0 = (long long)piece * g.columns, cols = std::min<long long>(g.columns, p.V - v0);
    const long long stride = (long long)up(cols, kLine);
    const uint8_t* w = static_cast<const uint8_t*>(in.weight) + v0 * p.weight_stride * 2;
    XentParams k{};
    k.R = p.R;
    k.V = (int)p.V;
    k.v0 = (int)v0;
    k.scale = p.scale;
    k.c = p.scale * kLog2e;
    k.tokens = in.tokens;
    k.lse = in.lse;
    k.g = in.g;
    k.g_lse = in.g_lse;
    k.power = p.half ? power : nullptr;
    k.not_finite = dweight && piece == 0 ? not_finite : nullptr;
    k.clean = clean;
    {
      Maps maps{};
      const int width = tile_width(m_tiles, p.R, cols, tiles_of(p.C, BK), num_sms);
      k.job[0] = make_job(m_tiles, tiles_of(cols, width), 1, tiles_of(p.C, BK), width, m_group(p, m_tiles), 0, 0, p.R, cols, p.C);
      if (!operand_map(&maps.a[0], in.hidden, p.R, p.C, p.hidden_stride, true, &k.job[0].a_box) ||
          !operand_map(&maps.b[0], w, cols, p.C, p.weight_stride, true, &k.job[0].b_box, width / 2) ||
          !encode_matrix_map(&maps.out[0], d, p.R, cols, stride, 32, 64) || !encode_matrix_map(&maps.out32, d, p.R, cols, stride, 32, 32))
        return cudaErrorInvalidValue;
      const int pairs = pairs_for(k.job[0].tiles(), num_sms);
      e = p.half ? launch<kGradLogits, true>(k, maps, pairs, status, st, true)
                 : launch<kGradLogits, false>(k, maps, pairs, status, st, piece > 0);
      if (e != cudaSuccess) return e;
    }
    if (dweight && piece == 0) {
      e = launch_behind(xent_clean_kernel, (unsigned)std::min<long long>(p.R, 2ll * num_sms), 256, 0, st, p.R, (int)p.V, p.C,
                        p.hidden_stride, static_cast<const uint4*>(in.hidden), in.tokens, in.g, in.g_lse, not_finite, clean,
                        reinterpret_cast<uint4*>(ws + g.off_clean));
      if (e != cudaSuccess) return e;
    }
    Maps maps{};
    k.job[0] = k.job[1] = Job{};
    if (dhidden) {
      // (a last, short piece adds to the first sums only)
      k.job[0] = make_job(m_tiles, c_tiles, std::min(g.splits, tiles_of(cols, BK)), tiles_of(cols, BK), TILE, 0, 0, 1, p.R, p.C, cols);
      if (!operand_map(&maps.a[0], d, p.R, cols, stride, true, &k.job[0].a_box) ||
          !operand_map(&maps.b[0], w, cols, p.C, p.weight_stride, false, &k.job[0].b_box) ||
          !encode_matrix_map(&maps.out[0], dhidden, p.R, p.C, p.C, 32, 64) ||
          (!g.direct && !encode_rows_f32_map(&maps.acc, acc, p.C, (int)p.R, g.splits, 32, 32)))
        return cudaErrorInvalidValue;
      k.accumulate = g.direct ? 0 : piece == 0 ? 1 : 2;
    }
    if (dweight) {
      k.job[1] = make_job(tiles_of(cols, TILE), c_tiles, 1, tiles_of(p.R, BK), TILE, 0, 1, 1, cols, p.C, p.R);
      if (!operand_map(&maps.a[1], d, p.R, cols, stride, false, &k.job[1].a_box) ||
          !operand_map(&maps.b[1], in.hidden, p.R, p.C, p.hidden_stride, false, &k.job[1].b_box) ||
          !operand_map(&maps.clean, ws + g.off_clean, p.R, p.C, p.C, false, &k.job[1].b_box) ||
          !encode_matrix_map(&maps.out[1], dweight, p.V, p.C, p.C, 32, 64))
        return cudaErrorInvalidValue;
    }
    const long long a = k.job[0].tiles(), b = k.job[1].tiles();
    const int pairs = pairs_for(a + b, num_sms);
    // while some pairs have one more tile of dh, the others take so many of dW
    k.more = (int)(a % pairs);
    const double la = k.job[0].splits ? (double)k.job[0].k_chunks / k.job[0].splits + kMoreChunks : 0;
    const double lb = std::max(k.job[1].k_chunks + kMoreChunks, kTileChunks);
    k.early = k.more ? (int)std::min(la / lb + 0.5, (double)(b / (pairs - k.more))) : 0;
    e = p.half ? launch<kGradients, true>(k, maps, pairs, status, st, true)
               : launch<kGradients, false>(k, maps, pairs, status, st, true);
    if (e != cudaSuccess) return e;
  }
  if (dhidden && !g.direct) {
    const long long n = p.R * p.C / 4;
    const unsigned blocks = (unsigned)((n + 255) / 256);
    e = launch_behind(p.half ? xent_close_kernel<true> : xent_close_kernel<false>, blocks, 256, 0, st, n, g.splits,
                      reinterpret_cast<float4*>(acc), power, static_cast<uint2*>(dhidden));
  }
  return e;
}

}  // namespace skl
