// Attention backward: dQ, dK, dV from Q, K, V, O, dO and the saved log-sum-exp,
// on the 5th-generation tensor cores.
//
// The probabilities are rebuilt tile by tile, P = exp(S - LSE), and with
// dP = dO V^T, delta_i = dO_i . O_i - dLSE_i (which is sum_j P_ij dP_ij, the
// softmax's coupling, less the gradient of the LSE itself):
//     dS = P (dP - delta),  dQ = scale dS K,  dK = scale dS^T Q,  dV = P^T dO
// Two kinds of block, each output written by one block, so no atomics and the
// same bits on every run:
//   dK/dV block  128 keys stationary; streams the query tiles of every query
//                head that reads them: four products a tile pair
//   dQ block     128 queries stationary; streams the key tiles: three products
// (attn_bwd_fused.cu visits each tile pair once, for five, and adds dQ up in
// L2).  Both kinds run in one launch, the kind with the longer blocks first: the
// shorter ones fill the SMs that the longer ones leave.  Tiles whose streams are
// long for the number of SMs are dealt out over several blocks (attn_bwd_plan).
//
// A small kernel first writes, per query row, -LSE / scale and -delta, each as
// three bf16 that add up to its 24 bits, in 16 bytes and 128-row padded: a
// tile's 128 rows are one bulk copy and lie in shared memory as the 16-wide
// K step that adds the row's value to a product (the other operand's step is
// ones).  Rows that see no key, and rows past a sequence's length, get -1e30
// and 0: their P is exactly 0.
//
// Measured at D 128, five products counted: 8 heads, N8192, non-causal 570 to 595
// us, 1150 to 1200 TFLOP/s, with the recomputed two 1620 to 1690, which is near what
// the power limit leaves a plain matrix product (1750); B2 H32 HK8 N4096 causal 625
// to 680 us.  Built and
// not kept: Q and dO of the dQ block as operands in TMEM (64 KB less
// shared-memory traffic a tile pair, and 3% slower).
#include "attn.cuh"

namespace skl {
namespace {

constexpr int BT = 128;  // keys and queries of a tile
constexpr int DS_WARPS = 16;
constexpr int PRODUCER_WARP = 16, MMA_WARP = 17, PATCH_WARP = 18;
constexpr int THREADS = 20 * 32;
constexpr int kRegsDs = 104, kRegsOther = 64;  // 512 * 104 + 128 * 64 = 640 * 96 registers at launch
constexpr uint32_t kTmemCols = 512;

struct BwdMaps {  // of the inputs, and of the outputs
  CUtensorMap q, k, v, go, dq, dk, dv;
};

// ---------------------------------------------------------------------------
// Row values: -LSE / scale and -delta, delta = dO . O - dLSE.  A row takes D / 8
// lanes of 16 bytes; bound by the read of O and dO (262144 rows of D 128: 27 us,
// 5.1 TB/s).  Three blocks to an SM where all rows are exact, which want the
// registers: B4 H16 N64 D64 10.0 us for the whole backward, 11.3 with four.
//
// O is rounded to bf16, so dO . O is off by up to 2^-8 sum_d |dO_d O_d|, while what it is subtracted from differs from it by
// no more than the spread of dO . v over the row's keys: the error of dS grows with the part that the values have in
// common, and where the weights lie on few keys it does not average out.  Error of dQ against 64 bits, in times of its last
// rounding's: 1.5 for values and logits of ordinary spread; 2 to 3 with a common vector of the values' size, 4 to 10 with one
// of three times it, 13 to 31 of ten times; 2.5 with logits four times as wide.  With what the forward's rounding left (REST)
// delta is exact to 16 bits, and all of these are 1.4 to 1.6.  Without it, for rows of at most 32 keys (the first rows under a
// causal mask) and where no sequence has more than 64, delta is computed as sum_j P_ij dP_ij: 16 such rows are one or two
// warps', whose S and dP are warp-wide products with the head's first keys in shared memory.  (Latency: B4 H12 N1001/777
// causal D128 44.4 us for the whole backward, 42.5 with the rest instead; 45.7 with a key to a group of lanes.  B4 H16 N64
// D64 10.0, 8.3 with dO . O.)
// Sum of the products of 8 bf16 pairs.
__device__ __forceinline__ float dot8(uint4 x, uint4 y, float sum) {
  const uint32_t xs[4] = {x.x, x.y, x.z, x.w}, ys[4] = {y.x, y.y, y.z, y.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    sum = fmaf(__uint_as_float(xs[i] << 16), __uint_as_float(ys[i] << 16), sum);
    sum = fmaf(__uint_as_float(xs[i] & 0xffff0000u), __uint_as_float(ys[i] & 0xffff0000u), sum);
  }
  return sum;
}

// 16 bytes of a row to shared memory, on their own (cp.async); zeros where it is not `there`.
__device__ __forceinline__ void copy_row(void* to, const void* from, bool there) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(smem_u32(to)), "l"(from), "r"(there ? 16 : 0) : "memory");
}
// Brings 16 bytes to the L1 cache: a load that nobody waits for.
__device__ __forceinline__ void touch(const void* p) {
  uint32_t a, b, c, d;
  asm volatile("ld.global.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(a), "=r"(b), "=r"(c), "=r"(d) : "l"(p));
}

// The totals of N values over LANES lanes: on return lane l holds in v[0] the total of value lane_index<N>(l).
template <int N>
__device__ __forceinline__ int lane_index(int lane) {
  int i = 0;
#pragma unroll
  for (int o = 1; o < N; o *= 2) i = 2 * i + ((lane & o) != 0);
  return i;
}
template <int LANES, int N>
__device__ __forceinline__ void lane_totals(float (&v)[N], int lane) {
  static_assert(N <= LANES, "a lane for each value");
#pragma unroll
  for (int o = 1, n = N / 2; n; o *= 2, n /= 2)
#pragma unroll
    for (int i = 0; i < n; ++i) {
      const bool upper = lane & o;
      const float other = __shfl_xor_sync(0xffffffffu, upper ? v[i] : v[i + n], o);
      v[i] = (upper ? v[i + n] : v[i]) + other;
    }
#pragma unroll
  for (int o = N; o < LANES; o *= 2) v[0] += __shfl_xor_sync(0xffffffffu, v[0], o);
}

constexpr int kRowsEach = 4;  // rows of a thread, all loaded before the first is used; a quarter of the head apart, so
                              // that the rows that see few keys, which lie together, spread over many blocks
// kRowsShort: no sequence has more than kShortKeys keys, and all rows are exact; kRowsLong: rows of at most kExactKeys (more would
// cost the launches of long sequences, which have few such rows, shared memory and registers).
constexpr int kExactKeys = 32, kShortKeys = 64;
enum RowsKind { kRowsLong, kRowsShort, kRowsRest };

template <int D, RowsKind KIND>
__global__ void __launch_bounds__(256, KIND == kRowsShort ? 3 : 4)
    attn_rows_kernel(const AttnProblem p, const AttnBwdIn in, uint4* __restrict__ row_s, uint4* __restrict__ row_d,
                     float4* __restrict__ acc, unsigned* __restrict__ counters, unsigned n_counters, int padded) {
  constexpr int LANES = D / 8, ROWS = 256 / LANES, KEYS = KIND == kRowsShort ? kShortKeys : kExactKeys;
  constexpr bool REST = KIND == kRowsRest;
  static_assert(BT % (ROWS * kRowsEach) == 0, "a block's rows are one head's");
  for (unsigned i = blockIdx.x * 256 + threadIdx.x; i < n_counters; i += gridDim.x * 256) counters[i] = 0;
  const int step = padded / kRowsEach;
  const unsigned per_head = (unsigned)step / ROWS;
  const int bh = (int)(blockIdx.x / per_head);
  const int b = bh / p.H, h = bh % p.H;
  const int n0 = (int)(blockIdx.x % per_head) * ROWS + threadIdx.x / LANES;  // rows n0, n0 + step, ...
  const int lane = threadIdx.x % LANES;
  const int ql = seq_len(p.q_lens, b, p.NQ), kl = seq_len(p.k_lens, b, p.NK);
  auto seen = [&](int n) { return n < ql ? (p.causal ? min(kl, n + kl - ql + 1) : kl) : 0; };  // keys a row sees, or <= 0
  const long long r0 = (long long)bh * padded + n0;  // row of [B H][padded]
  const auto* o = static_cast<const __nv_bfloat16*>(in.o) + b * p.os_b + h * p.os_h + lane * 8;
  const auto* go = static_cast<const __nv_bfloat16*>(in.go) + b * p.os_b + h * p.os_h + lane * 8;
  const float* lse = in.lse + (long long)bh * p.NQ;
  const float* dlse = in.dlse ? in.dlse + (long long)bh * p.NQ : nullptr;
  const uint4 none = make_uint4(0u, 0u, 0u, 0u);
  // The head's first keys, which all rows of few keys see, for a block that has any: on their way beside the rows.  Rows of 64
  // bytes more, so that two of them fill the banks.
  constexpr int LD = LANES + 4;
  __shared__ uint4 first_k[REST ? 1 : KEYS * LD], first_v[REST ? 1 : KEYS * LD];
  bool few = false;
  if constexpr (!REST) {
#pragma unroll
    for (int u = 0; u < kRowsEach; ++u) {  // of the group's rows the first to see a key sees the fewest
      const int from = (int)(blockIdx.x % per_head) * ROWS + u * step, to = min(from + ROWS, ql) - 1;
      const int first = p.causal ? max(from, ql - kl) : from;
      few = few || (first <= to && kl > 0 && seen(first) <= KEYS);
    }
  }
  uint4 x[kRowsEach], y[kRowsEach];
#pragma unroll
  for (int u = 0; u < kRowsEach; ++u) {
    const int n = n0 + u * step, keys = seen(n);
    x[u] = y[u] = none;
    if (keys > 0) {
      if (!REST && keys <= KEYS)
        touch(static_cast<const __nv_bfloat16*>(in.q) + b * p.qs_b + h * p.qs_h + n * p.qs_n + lane * 8);
      x[u] = *reinterpret_cast<const uint4*>(o + n * p.os_n);
      y[u] = *reinterpret_cast<const uint4*>(go + n * p.os_n);
    }
  }
  if (few) {
    const auto* k = static_cast<const __nv_bfloat16*>(in.k) + b * p.ks_b + h / p.G * p.ks_h + lane * 8;
    const auto* v = static_cast<const __nv_bfloat16*>(in.v) + b * p.vs_b + h / p.G * p.vs_h + lane * 8;
#pragma unroll
    for (int i = 0; i < KEYS / ROWS; ++i) {
      const int j = i * ROWS + threadIdx.x / LANES;
      copy_row(&first_k[j * LD + lane], k + (j < kl ? j : 0) * p.ks_n, j < kl);
      copy_row(&first_v[j * LD + lane], v + (j < kl ? j : 0) * p.vs_n, j < kl);
    }
  }
  // lanes 0 to 3 write the values of a row each
  const int own = lane_index<kRowsEach>(lane), n_own = n0 + own * step;
  const bool sees_own = lane < kRowsEach && seen(n_own) > 0;
  const float l_own = sees_own ? lse[n_own] : kNegInf, g_own = sees_own && dlse ? dlse[n_own] : 0.f;
  if (acc) {  // the fused kernel's accumulator starts at zero
#pragma unroll
    for (int u = 0; u < kRowsEach; ++u) {
      acc[(r0 + u * step) * (D / 4) + lane] = make_float4(0.f, 0.f, 0.f, 0.f);
      acc[(r0 + u * step) * (D / 4) + LANES + lane] = make_float4(0.f, 0.f, 0.f, 0.f);
    }
  }
  float sums[kRowsEach];
#pragma unroll
  for (int u = 0; u < kRowsEach; ++u) sums[u] = dot8(x[u], y[u], 0.f);
  if constexpr (REST) {
    const auto* rest = static_cast<const __nv_bfloat16*>(in.o_rest) + b * p.os_b + h * p.os_h + lane * 8;
#pragma unroll
    for (int u = 0; u < kRowsEach; ++u) {
      const int n = n0 + u * step;
      x[u] = seen(n) > 0 ? *reinterpret_cast<const uint4*>(rest + n * p.os_n) : none;
    }
#pragma unroll
    for (int u = 0; u < kRowsEach; ++u) sums[u] += dot8(x[u], y[u], 0.f);
  }
  lane_totals<LANES>(sums, lane);
  if (lane < kRowsEach) {
    row_s[r0 + own * step] = three_bf16(l_own == kNegInf ? kNoRow : -l_own * (1.f / p.scale));
    row_d[r0 + own * step] = three_bf16(l_own == kNegInf ? 0.f : g_own - sums[0]);
  }
  if constexpr (REST) return;
  if (!few) return;
  asm volatile("cp.async.wait_all;" ::: "memory");
  __syncthreads();
  // 16 neighbouring rows to SHARE warps, which take 16 keys in turn.  A thread has rows quad and quad + 8, and of each 32
  // columns the 8 from 8 sub on, as two steps' pairs of both operands: which columns stand at which place of a step does not
  // matter to the sum, so both come in 16 bytes.
  constexpr int TILES = ROWS * kRowsEach / 16, SHARE = 8 / TILES;
  __shared__ float shares[8][16];
  const int warp = threadIdx.x >> 5, tile = warp / SHARE, quad = (threadIdx.x & 31) >> 2, sub = threadIdx.x & 3;
  const int row0 = (int)(blockIdx.x % per_head) * ROWS + tile / (ROWS / 16) * step + tile % (ROWS / 16) * 16 + quad;
  int keys[2];
  float nl[2], sum[2] = {0.f, 0.f};
  const uint4 *q[2], *g[2];  // the rows' queries and gradients
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int n = row0 + 8 * i, sees = seen(n);
    keys[i] = sees > 0 && sees <= KEYS ? sees : 0;
    const float lr = keys[i] ? lse[n] : 0.f;
    nl[i] = -lr * kLog2e;
    if (lr == kNegInf) keys[i] = 0;  // written above
    const long long qn = b * p.qs_b + h * p.qs_h + n * p.qs_n, on = b * p.os_b + h * p.os_h + n * p.os_n;
    q[i] = reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(in.q) + qn) + sub;
    g[i] = reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(in.go) + on) + sub;
  }
  const int most = __reduce_max_sync(0xffffffffu, max(keys[0], keys[1]));
  for (int j0 = warp % SHARE * 16; j0 < most; j0 += SHARE * 16) {
    float s[2][4] = {}, dp[2][4] = {};
#pragma unroll 2
    for (int c = 0; c < D / 32; ++c) {
      const uint4 q0 = keys[0] ? q[0][4 * c] : none, q1 = keys[1] ? q[1][4 * c] : none;
      const uint4 g0 = keys[0] ? g[0][4 * c] : none, g1 = keys[1] ? g[1][4 * c] : none;
      const uint32_t qa[2][4] = {{q0.x, q1.x, q0.y, q1.y}, {q0.z, q1.z, q0.w, q1.w}};
      const uint32_t ga[2][4] = {{g0.x, g1.x, g0.y, g1.y}, {g0.z, g1.z, g0.w, g1.w}};
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const uint4 kb = first_k[(j0 + i * 8 + quad) * LD + 4 * c + sub], vb = first_v[(j0 + i * 8 + quad) * LD + 4 * c + sub];
        mma16816(s[i], qa[0], kb.x, kb.y);
        mma16816(dp[i], ga[0], vb.x, vb.y);
        mma16816(s[i], qa[1], kb.z, kb.w);
        mma16816(dp[i], ga[1], vb.z, vb.w);
      }
    }
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
      for (int e = 0; e < 4; ++e)
        if (j0 + i * 8 + 2 * sub + (e & 1) < keys[e >> 1])
          sum[e >> 1] = fmaf(ex2(fmaf(s[i][e], p.c, nl[e >> 1])), dp[i][e], sum[e >> 1]);
  }
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    sum[i] += __shfl_xor_sync(0xffffffffu, sum[i], 1);
    sum[i] += __shfl_xor_sync(0xffffffffu, sum[i], 2);
    if (SHARE > 1 && sub == 0) shares[warp][quad + 8 * i] = sum[i];
  }
  if (SHARE > 1) __syncthreads();
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    if (!keys[i] || sub != 0 || warp % SHARE != 0) continue;
#pragma unroll
    for (int w = 1; w < SHARE; ++w) sum[i] += shares[warp + w][quad + 8 * i];
    row_d[(long long)bh * padded + row0 + 8 * i] = three_bf16((dlse ? dlse[row0 + 8 * i] : 0.f) - sum[i]);
  }
}

// ---------------------------------------------------------------------------
// dK/dV block.  The logits are computed transposed, so the TMEM lanes are keys
// and the columns queries: S^T = K Q^T and dP^T = V dO^T (both operands K-major
// in shared memory).  P^T and dS^T (bf16 pairs) overwrite their logits and are
// the A operands of dV += P^T dO and dK += dS^T Q, which read dO and Q
// MN-major from the tiles that are there already: neither P nor dS passes
// through shared memory.  The queries' LSE and delta belong to columns here; a
// ninth K step of each product adds them (64 cycles), where reading them from
// shared memory, 16 bytes to a lane, kept the load pipe busy for 1024 cycles a
// tile pair.
//   TMEM: S^T/P^T [0,128), dP^T/dS^T [128,256), dV [256, 256+D), dK [384, 384+D)
//   warps 0-15  thread = key, group g = warp / 4 takes queries [32g, 32g+32); its
//               pairs go to the first 16 of its own 32 columns
//   warp 16     TMA producer: K, V once; Q(u) and dO(u) with their rows' values
//   warp 17     TMEM owner and MMA issuer: dV(u), S(u+1), dK(u), dP(u+1): while the
//               warps turn S(u+1) into P, the pipe runs dK(u) and dP(u+1), and
//               while they form dS(u+1) it runs dV(u+1) and S(u+2)
//   warp 18     clears the rows of Q and dO tiles past a sequence's length
namespace kv {
constexpr int SLOTS = 2;
constexpr uint32_t kColS = 0, kColP = 128, kColV = 256, kColK = 384;
template <int D>
struct Smem {
  static constexpr int TILE = BT * D * 2;
  static constexpr int OFF_K = 0, OFF_V = TILE;
  static constexpr int OFF_Q = 2 * TILE;                 // Q slots
  static constexpr int OFF_O = OFF_Q + SLOTS * TILE;     // dO slots
  // K steps without swizzle: 128 rows of 16 bytes are 16 core matrices of 8 rows for k = 0 .. 7; k = 8 .. 15 is ZERO
  static constexpr int STEP = 128 * 16;
  static constexpr int OFF_RS = OFF_O + SLOTS * TILE;    // -LSE / scale of the Q slots
  static constexpr int OFF_RD = OFF_RS + SLOTS * STEP;   // -delta of the dO slots
  static constexpr int OFF_ONES = OFF_RD + SLOTS * STEP; // 1, 1, 1, 0, ...
  static constexpr int OFF_ZERO = OFF_ONES + STEP;
  static constexpr int OFF_BAR = OFF_ZERO + STEP;
  // kv_full, q_full[2], q_empty[2], o_full[2], o_empty[2], s_full, dp_full, p_full, ds_full, g_done, to_patch, patched
  static constexpr int BAR_SLOT = 8 * 16;
  static constexpr int BYTES = OFF_BAR + BAR_SLOT + 16 + 1024;
};
static_assert(Smem<128>::BYTES <= kWholeSmSmem, "shared memory");
}  // namespace kv

template <int D>
__device__ __forceinline__ void kv_block(const AttnProblem& p, const uint4* __restrict__ row_s,
                                         const uint4* __restrict__ row_d, int padded, int* status, const BwdMaps& maps,
                                         const AttnBwdPlan& plan, const unsigned blk, float4* __restrict__ part_acc,
                                         unsigned* __restrict__ counters) {
  using L = kv::Smem<D>;
  using kv::SLOTS;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = align1024(smem_raw);
  const uint32_t sb = smem_u32(smem);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  // heads in order (the blocks in flight share one key head's query tiles in L2); within a head the first key
  // tiles, which see the most queries under a causal mask, first.  A small grid: the first key tiles of all heads first
  const TilePart part = tile_part(blk, plan.kv_whole, plan.by_kv_parts);
  const int x = (int)plan.by_kv_tile.div(part.tile), y = part.tile - x * (int)plan.by_kv_tile.d;
  const int bhk = plan.longest_first ? y : x, k0 = (plan.longest_first ? x : y) * BT;
  const int b = (int)plan.by_key_heads.div(bhk), hk = bhk - b * p.HK;
  const int ql = seq_len(p.q_lens, b, p.NQ), kl = seq_len(p.k_lens, b, p.NK);
  const int off = kl - ql;
  const int q_begin = p.causal ? max(0, k0 - off) / BT * BT : 0;
  const int n_qt = (k0 < kl && q_begin < ql) ? (ql - q_begin + BT - 1) / BT : 0;
  // tile u: head u / n_qt of the group, query tile u % n_qt; this block takes the tiles [u0, u0 + n)
  const int u0 = part.from(p.G * n_qt), n = part.from(p.G * n_qt, 1) - u0;
  const int head0 = u0 > 0 ? u0 / n_qt : 0, qt0 = u0 - head0 * n_qt;  // of the first
  const bool ragged = n > 0 && ql < p.NQ && (ql & (BT - 1));  // the last query tile has rows past the sequence

  const uint32_t bar = sb + L::OFF_BAR;
  const uint32_t kv_full = bar, q_full = bar + 8, q_empty = bar + 24, o_full = bar + 40, o_empty = bar + 56,
                 s_full = bar + 72, dp_full = bar + 80, p_full = bar + 88, ds_full = bar + 96, g_done = bar + 104,
                 to_patch = bar + 112, patched = bar + 120, slot = bar + L::BAR_SLOT;
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + L::OFF_BAR + L::BAR_SLOT + 4);
  volatile int* part_flag = abort_flag + 1;
  auto load_q = [&](int u, int hq, int q0) {
    const int s = u % SLOTS;
    mbar_arrive_expect_tx(q_full + 8 * s, L::TILE + L::STEP);
#pragma unroll
    for (int h = 0; h < D / 64; ++h)
      tma_load_4d(sb + L::OFF_Q + s * L::TILE + h * BT * 128, &maps.q, q_full + 8 * s, h * 64, q0, hq, b);
    bulk_load(sb + L::OFF_RS + s * L::STEP, row_s + ((long long)b * p.H + hq) * padded + q0, L::STEP, q_full + 8 * s);
  };
  auto load_o = [&](int u, int hq, int q0) {
    const int s = u % SLOTS;
    mbar_arrive_expect_tx(o_full + 8 * s, L::TILE + L::STEP);
#pragma unroll
    for (int h = 0; h < D / 64; ++h)
      tma_load_4d(sb + L::OFF_O + s * L::TILE + h * BT * 128, &maps.go, o_full + 8 * s, h * 64, q0, hq, b);
    bulk_load(sb + L::OFF_RD + s * L::STEP, row_d + ((long long)b * p.H + hq) * padded + q0, L::STEP, o_full + 8 * s);
  };
  if (warp == PRODUCER_WARP) {
    if (elect_one()) {
      mbar_init(kv_full, 1);
      for (int s = 0; s < SLOTS; ++s) {
        mbar_init(q_full + 8 * s, 1);
        mbar_init(q_empty + 8 * s, 1);
        mbar_init(o_full + 8 * s, 1);
        mbar_init(o_empty + 8 * s, 1);
      }
      mbar_init(s_full, 1);
      mbar_init(dp_full, 1);
      mbar_init(p_full, DS_WARPS);
      mbar_init(ds_full, DS_WARPS);
      mbar_init(g_done, 1);
      mbar_init(to_patch, 1);
      mbar_init(patched, 1);
      *abort_flag = 0;
      fence_mbar_init();
      fence_async_smem();  // the copies' proxy sees the barriers too
    }
    __syncwarp();  // the warp's other lanes wait for the one that sets the barriers up
  }
  if (threadIdx.x < 128) {
    st_shared16(sb + L::OFF_ONES + threadIdx.x * 16, make_uint4(0x3f803f80u, 0x00003f80u, 0u, 0u));
    st_shared16(sb + L::OFF_ZERO + threadIdx.x * 16, make_uint4(0u, 0u, 0u, 0u));
    fence_async_smem();
  }
  if (warp == MMA_WARP) {
    tmem_alloc(slot, kTmemCols);
    tmem_relinquish();
  }
  tc_fence_before();
  setup_barrier(ql, kl);
  tc_fence_after();
  whole_tmem(reinterpret_cast<volatile uint32_t*>(smem + L::OFF_BAR + L::BAR_SLOT), status);
  constexpr uint32_t tmem = 0;

  if (warp >= DS_WARPS) {
    setmaxnreg_dec<kRegsOther>();
    if (warp == PRODUCER_WARP) {
      if (n > 0 && elect_one()) {
        mbar_arrive_expect_tx(kv_full, 2 * L::TILE);
#pragma unroll
        for (int h = 0; h < D / 64; ++h) tma_load_4d(sb + L::OFF_K + h * BT * 128, &maps.k, kv_full, h * 64, k0, hk, b);
        load_q(0, hk * p.G + head0, q_begin + qt0 * BT);
#pragma unroll
        for (int h = 0; h < D / 64; ++h) tma_load_4d(sb + L::OFF_V + h * BT * 128, &maps.v, kv_full, h * 64, k0, hk, b);
        load_o(0, hk * p.G + head0, q_begin + qt0 * BT);
        int issued_q = 1, issued_o = 1, hq = hk * p.G + head0, qt = qt0;
        for (int u = 1; u < n; ++u) {
          const int s = u % SLOTS;
          if (++qt == n_qt) {
            qt = 0;
            ++hq;
          }
          if (u >= SLOTS && !mbar_wait(q_empty + 8 * s, ((u / SLOTS) - 1) & 1, status, abort_flag)) break;
          load_q(u, hq, q_begin + qt * BT);
          issued_q = u + 1;
          if (u >= SLOTS && !mbar_wait(o_empty + 8 * s, ((u / SLOTS) - 1) & 1, status, abort_flag)) break;
          load_o(u, hq, q_begin + qt * BT);
          issued_o = u + 1;
        }
        mbar_drain(kv_full, 0, status);
        for (int u = max(0, issued_q - SLOTS); u < issued_q; ++u)
          mbar_drain(q_full + 8 * (u % SLOTS), (u / SLOTS) & 1, status);
        for (int u = max(0, issued_o - SLOTS); u < issued_o; ++u)
          mbar_drain(o_full + 8 * (u % SLOTS), (u / SLOTS) & 1, status);
      }
      __syncwarp();
    } else if (warp == PATCH_WARP) {
      // for each head's last tile: its Q, then its dO, when the MMA thread has seen them land
      if (ragged) {
        const int first = n_qt - 1 - qt0;  // the first of this block's tiles that is a head's last
        for (int e = 0; first + e / 2 * n_qt < n; ++e) {
          if (!mbar_wait_warp(to_patch, e & 1, status, abort_flag)) break;
          const int s = (first + e / 2 * n_qt) % SLOTS, from = ql & (BT - 1);
          const uint32_t tile = sb + ((e & 1) ? L::OFF_O : L::OFF_Q) + s * L::TILE;
          for (int i = lane; i < (BT - from) * (D / 8); i += 32)
            st_shared_zero16(sw128<BT>(tile, from + i / (D / 8), i % (D / 8)));
          fence_async_smem();
          __syncwarp();
          arrive_one(patched);
        }
      }
      __syncwarp();
    } else if (warp == MMA_WARP) {
      if (n > 0 && elect_one()) {
        constexpr uint32_t id_s = idesc_bf16(BT, BT, false, false);
        constexpr uint32_t id_g = idesc_bf16(BT, D, false, true);
        const uint64_t kd = sdesc_sw128(sb + L::OFF_K, 0, 1024), vd = sdesc_sw128(sb + L::OFF_V, 0, 1024);
        const uint64_t ones = sdesc_step(sb + L::OFF_ONES, sb + L::OFF_ZERO);
        int patches = 0;
        auto patch = [&](int u) {  // the head's last tile: wait until its rows past the sequence are cleared
          if (!ragged || (qt0 + u + 1) % n_qt) return true;
          mbar_arrive(to_patch);
          return mbar_wait(patched, patches++ & 1, status, abort_flag);
        };
        auto issue_s = [&](int u) {  // S^T(u) = K Q^T - LSE / scale
          const int s = u % SLOTS;
          if (!mbar_wait(q_full + 8 * s, (u / SLOTS) & 1, status, abort_flag) || !patch(u)) return false;
          tc_fence_after();
          const uint64_t qd = sdesc_sw128(sb + L::OFF_Q + s * L::TILE, 0, 1024);
#pragma unroll
          for (int ks = 0; ks < D / 16; ++ks) {
            const uint32_t o = (ks >> 2) * (BT * 128) + (ks & 3) * 32;
            mma_ss(tmem + kv::kColS, sdesc_add(kd, o), sdesc_add(qd, o), id_s, ks > 0);
          }
          mma_ss(tmem + kv::kColS, ones, sdesc_step(sb + L::OFF_RS + s * L::STEP, sb + L::OFF_ZERO), id_s, true);
          mma_commit(s_full);
          return true;
        };
        auto issue_dp = [&](int u) {  // dP^T(u) = V dO^T - delta
          const int s = u % SLOTS;
          if (!mbar_wait(o_full + 8 * s, (u / SLOTS) & 1, status, abort_flag) || !patch(u)) return false;
          tc_fence_after();
          const uint64_t od = sdesc_sw128(sb + L::OFF_O + s * L::TILE, 0, 1024);
#pragma unroll
          for (int ks = 0; ks < D / 16; ++ks) {
            const uint32_t o = (ks >> 2) * (BT * 128) + (ks & 3) * 32;
            mma_ss(tmem + kv::kColP, sdesc_add(vd, o), sdesc_add(od, o), id_s, ks > 0);
          }
          mma_ss(tmem + kv::kColP, ones, sdesc_step(sb + L::OFF_RD + s * L::STEP, sb + L::OFF_ZERO), id_s, true);
          mma_commit(dp_full);
          return true;
        };
        // G += A B: A = pairs in TMEM (16 queries = 8 columns; a group's 32 queries lie in 32 columns' first 16)
        auto issue_g = [&](uint32_t g_col, uint32_t a_col, uint32_t tile, bool first) {
          const uint64_t bd = sdesc_sw128(tile, BT * 128, 1024);
#pragma unroll
          for (int ks = 0; ks < BT / 16; ++ks)
            mma_ts(tmem + g_col, tmem + a_col + 32 * (ks >> 1) + 8 * (ks & 1), sdesc_add(bd, ks * 2048), id_g,
                   !first || ks > 0);
        };
        bool ok = mbar_wait(kv_full, 0, status, abort_flag) && issue_s(0) && issue_dp(0);
        for (int u = 0; ok && u < n; ++u) {
          const int s = u % SLOTS;
          if (!mbar_wait(p_full, u & 1, status, abort_flag)) break;
          tc_fence_after();
          issue_g(kv::kColV, kv::kColS, sb + L::OFF_O + s * L::TILE, u == 0);  // dV += P^T dO
          mma_commit(o_empty + 8 * s);
          if (u + 1 < n && !(ok = issue_s(u + 1))) break;
          if (!mbar_wait(ds_full, u & 1, status, abort_flag)) break;
          tc_fence_after();
          issue_g(kv::kColK, kv::kColP, sb + L::OFF_Q + s * L::TILE, u == 0);  // dK += dS^T Q
          mma_commit(q_empty + 8 * s);
          if (u + 1 < n) ok = issue_dp(u + 1);
        }
        mma_commit(g_done);
        mbar_drain(g_done, 0, status);
      }
      __syncwarp();
    }
  } else {
    setmaxnreg_inc<kRegsDs>();
    const int grp = warp >> 2, wq = warp & 3;
    const int r = wq * 32 + lane;
    const int key = k0 + r;
    const float c = p.c;
    const float2 cc = make_float2(c, c);
    const uint32_t lanes = (uint32_t)(wq * 32) << 16;
    const uint32_t ts = tmem + lanes + kv::kColS + 32 * grp, tp = tmem + lanes + kv::kColP + 32 * grp;
    bool ok = true;
    const int q_last = q_begin + (n_qt - 1) * BT + 32 * grp;
    int q0 = q_begin + qt0 * BT + 32 * grp;  // first query of this warp's columns
    for (int u = 0; u < n; ++u) {
      ok = mbar_wait_warp(s_full, u & 1, status, abort_flag);
      __syncwarp();
      if (!ok) break;
      tc_fence_after();
      uint32_t a[32], pk[16];
      tmem_ld32(ts, a);
      tmem_ld_wait();
      reg_fence32(a);
      const int hidden = key >= kl ? 32 : p.causal ? key - off - q0 : 0;  // the first columns that do not see this key
      if (__any_sync(0xffffffffu, hidden > 0))
        p32<true>(a, pk, cc, hidden);
      else
        p32<false>(a, pk, cc, 0);
      tmem_st16(ts, pk);
      tmem_st_wait();
      tc_fence_before();
      __syncwarp();
      arrive_one(p_full);
      ok = mbar_wait_warp(dp_full, u & 1, status, abort_flag);
      __syncwarp();
      if (!ok) break;
      tc_fence_after();
      uint32_t d[32];
      tmem_ld32(tp, d);
      tmem_ld_wait();
      reg_fence32(d);
#pragma unroll
      for (int i = 0; i < 32; i += 2) {
        const float2 e = fmul2(make_float2(__uint_as_float(a[i]), __uint_as_float(a[i + 1])),
                               make_float2(__uint_as_float(d[i]), __uint_as_float(d[i + 1])));
        pk[i / 2] = pack_bf16(e.x, e.y);
      }
      tmem_st16(tp, pk);
      tmem_st_wait();
      tc_fence_before();
      __syncwarp();
      arrive_one(ds_full);
      q0 = q0 == q_last ? q_last - (n_qt - 1) * BT : q0 + BT;
    }
    // ---- out: thread = key row, group g writes d columns [32g, 32g + 32) of both
    bool got = ok;
    if (n > 0 && ok) {
      got = mbar_wait_warp(g_done, 0, status, abort_flag);
      __syncwarp();
    }
    // dV through the first Q slot, dK through the first dO slot: every product that read them is done.  A part's
    // accumulators of both are one tile of 2 D columns
    float4* mine = part_acc + (size_t)(part.tile - plan.kv_whole) * part.parts * (2 * D / 4 * BT);
    const bool cols = grp * 32 < D;
    bool last = true;
    if (part.parts > 1) {
      if (got && cols) {
        tc_fence_after();
#pragma unroll
        for (int which = 0; which < 2; ++which) {
          uint32_t g[32] = {};
          __syncwarp();
          if (n > 0) {
            tmem_ld32(tmem + lanes + (which ? kv::kColK : kv::kColV) + 32 * grp, g);
            tmem_ld_wait();
            reg_fence32(g);
          }
          part_put<2 * D>(mine, part.rank, r, which * D + 32 * grp, g);
        }
      }
      last = part_last(counters + (part.tile - plan.kv_whole), part.parts, DS_WARPS * 32, part_flag);
    }
    if (got && last && cols) {
      tc_fence_after();
#pragma unroll
      for (int which = 0; which < 2; ++which) {
        uint32_t g[32] = {};
        __syncwarp();  // rows differ in what they do below; the load wants the whole warp
        if (part.parts > 1) {
          part_sum<2 * D>(mine, part.parts, r, which * D + 32 * grp, g);
        } else if (n > 0) {
          tmem_ld32(tmem + lanes + (which ? kv::kColK : kv::kColV) + 32 * grp, g);
          tmem_ld_wait();
          reg_fence32(g);
        }
        if (key >= kl) {
#pragma unroll
          for (int i = 0; i < 32; ++i) g[i] = 0u;
        }
        stage_row32(sb + (which ? L::OFF_O : L::OFF_Q), r, 32 * grp, g, which ? p.scale : 1.f);
      }
      fence_async_smem();
    }
    // every warp comes here; one that gave up makes none of them store
    if (!named_bar_any(1, DS_WARPS * 32, !got) && last && warp == 0) {
      if (elect_one()) {
        store_tile<D>(&maps.dv, sb + L::OFF_Q, k0, hk, b);
        store_tile<D>(&maps.dk, sb + L::OFF_O, k0, hk, b);
      }
      __syncwarp();
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == MMA_WARP) {
    tc_fence_after();
    tmem_dealloc(tmem, kTmemCols);
  }
}

// ---------------------------------------------------------------------------
// dQ block.  The TMEM lanes are queries: a thread owns a row and holds its LSE
// and delta.  S = Q K^T and dP = dO V^T are copied into registers and released
// at once, before anything is computed, so the next tile's products run meanwhile; dS (bf16 pairs)
// goes to a double buffer in TMEM, the A operand of dQ += dS K.
//   TMEM: S [0,128), dP [128,256), dS [256,320) and [320,384), dQ [384, 384+D)
//   warps 0-15  thread = query, group g = warp / 4 takes keys [32g, 32g+32)
//   warp 16     TMA producer: Q, dO once; K (held until dQ's product) through three
//               slots, V through two
//   warp 17     TMEM owner and MMA issuer: S(j), dP(j), then dQ(j-1)
//   warp 18     clears the rows of the K tile past a sequence's key length
namespace qq {
constexpr int K_SLOTS = 3, V_SLOTS = 2;
constexpr uint32_t kColS = 0, kColP = 128, kColDS = 256, kColG = 384;
template <int D>
struct Smem {
  static constexpr int TILE = BT * D * 2;
  static constexpr int OFF_Q = 0, OFF_O = TILE;
  static constexpr int OFF_K = 2 * TILE;
  static constexpr int OFF_V = OFF_K + K_SLOTS * TILE;
  static constexpr int OFF_BAR = OFF_V + V_SLOTS * TILE;
  // x_full, k_full[3], k_empty[3], v_full[2], v_empty[2], s_full, s_free, ds_full[2], ds_free[2], g_done, to_patch,
  // patched
  static constexpr int BAR_SLOT = 8 * 20;
  static constexpr int BYTES = OFF_BAR + BAR_SLOT + 16 + 1024;
};
static_assert(Smem<128>::BYTES <= kWholeSmSmem, "shared memory");
}  // namespace qq

// dS of 32 columns: a, d = S, dP; `seen` of them are visible.
template <bool MASKED>
__device__ __forceinline__ void ds32(const uint32_t (&a)[32], const uint32_t (&d)[32], uint32_t (&pk)[16], float c,
                                     float nlse, float delta, int seen) {
  const float2 cc = make_float2(c, c), nl = make_float2(nlse, nlse), dl = make_float2(delta, delta);
#pragma unroll
  for (int i = 0; i < 32; i += 2) {
    const float2 x = ffma2(make_float2(__uint_as_float(a[i]), __uint_as_float(a[i + 1])), cc, nl);
    float2 e = fmul2(make_float2(ex2(x.x), ex2(x.y)),
                     fsub2(make_float2(__uint_as_float(d[i]), __uint_as_float(d[i + 1])), dl));
    if (MASKED) {
      e.x = i < seen ? e.x : 0.f;
      e.y = i + 1 < seen ? e.y : 0.f;
    }
    pk[i / 2] = pack_bf16(e.x, e.y);
  }
}

template <int D>
__device__ __forceinline__ void q_block(const AttnProblem& p, const uint4* __restrict__ row_s,
                                        const uint4* __restrict__ row_d, int padded, int* status, const BwdMaps& maps,
                                        const AttnBwdPlan& plan, const unsigned blk, float4* __restrict__ part_acc,
                                        unsigned* __restrict__ counters) {
  using L = qq::Smem<D>;
  using qq::K_SLOTS;
  using qq::V_SLOTS;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = align1024(smem_raw);
  const uint32_t sb = smem_u32(smem);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int n_qt = (p.NQ + BT - 1) / BT;
  const TilePart part = tile_part(blk, plan.q_whole, plan.by_q_parts);
  const int x = (int)plan.by_q_tile.div(part.tile), y = part.tile - x * (int)plan.by_q_tile.d;
  const int bh = plan.longest_first ? y : x;
  const int b = (int)plan.by_heads.div(bh), h = bh - b * p.H, hk = (int)plan.by_group.div(h);
  const int q0 = (n_qt - 1 - (plan.longest_first ? x : y)) * BT;  // the last query tiles, which see the most keys, first
  const int ql = seq_len(p.q_lens, b, p.NQ), kl = seq_len(p.k_lens, b, p.NK);
  const int off = kl - ql;
  const int last = min(q0 + BT, ql) - 1;
  const int end = q0 < ql ? (p.causal ? min(kl, last + off + 1) : kl) : 0;
  const int tiles = end > 0 ? (end + BT - 1) / BT : 0;
  const int j0 = part.from(tiles), n = part.from(tiles, 1) - j0;  // this block takes the key tiles [j0, j0 + n)
  const int patch_j = (kl < p.NK && (kl & (BT - 1))) ? kl / BT - j0 : -1;  // the K tile with rows past the sequence

  const uint32_t bar = sb + L::OFF_BAR;
  const uint32_t x_full = bar, k_full = bar + 8, k_empty = bar + 32, v_full = bar + 56, v_empty = bar + 72,
                 s_full = bar + 88, s_free = bar + 96, ds_full = bar + 104, ds_free = bar + 120, g_done = bar + 136,
                 to_patch = bar + 144, patched = bar + 152, slot = bar + L::BAR_SLOT;
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + L::OFF_BAR + L::BAR_SLOT + 4);
  volatile int* part_flag = abort_flag + 1;
  auto load_k = [&](int j) {
    const int s = j % K_SLOTS;
    mbar_arrive_expect_tx(k_full + 8 * s, L::TILE);
#pragma unroll
    for (int d = 0; d < D / 64; ++d)
      tma_load_4d(sb + L::OFF_K + s * L::TILE + d * BT * 128, &maps.k, k_full + 8 * s, d * 64, (j0 + j) * BT, hk, b);
  };
  auto load_v = [&](int j) {
    const int s = j % V_SLOTS;
    mbar_arrive_expect_tx(v_full + 8 * s, L::TILE);
#pragma unroll
    for (int d = 0; d < D / 64; ++d)
      tma_load_4d(sb + L::OFF_V + s * L::TILE + d * BT * 128, &maps.v, v_full + 8 * s, d * 64, (j0 + j) * BT, hk, b);
  };
  if (warp == PRODUCER_WARP) {
    if (elect_one()) {
      mbar_init(x_full, 1);
      for (int s = 0; s < K_SLOTS; ++s) {
        mbar_init(k_full + 8 * s, 1);
        mbar_init(k_empty + 8 * s, 1);
      }
      for (int s = 0; s < 2; ++s) {
        mbar_init(v_full + 8 * s, 1);
        mbar_init(v_empty + 8 * s, 1);
        mbar_init(ds_full + 8 * s, DS_WARPS);
        mbar_init(ds_free + 8 * s, 1);
      }
      mbar_init(s_full, 1);
      mbar_init(s_free, DS_WARPS);
      mbar_init(g_done, 1);
      mbar_init(to_patch, 1);
      mbar_init(patched, 1);
      *abort_flag = 0;
      fence_mbar_init();
      fence_async_smem();  // the copies' proxy sees the barriers too
    }
    __syncwarp();  // the warp's other lanes wait for the one that sets the barriers up
  }
  if (warp == MMA_WARP) {
    tmem_alloc(slot, kTmemCols);
    tmem_relinquish();
  }
  tc_fence_before();
  setup_barrier(ql, kl);
  tc_fence_after();
  whole_tmem(reinterpret_cast<volatile uint32_t*>(smem + L::OFF_BAR + L::BAR_SLOT), status);
  constexpr uint32_t tmem = 0;

  if (warp >= DS_WARPS) {
    setmaxnreg_dec<kRegsOther>();
    if (warp == PRODUCER_WARP) {
      if (n > 0 && elect_one()) {
        mbar_arrive_expect_tx(x_full, 2 * L::TILE);
#pragma unroll
        for (int d = 0; d < D / 64; ++d) tma_load_4d(sb + L::OFF_Q + d * BT * 128, &maps.q, x_full, d * 64, q0, h, b);
        load_k(0);
#pragma unroll
        for (int d = 0; d < D / 64; ++d) tma_load_4d(sb + L::OFF_O + d * BT * 128, &maps.go, x_full, d * 64, q0, h, b);
        load_v(0);
        int issued_k = 1, issued_v = 1;
        for (int j = 1; j < n; ++j) {
          const int sk = j % K_SLOTS, sv = j % V_SLOTS;
          if (j >= K_SLOTS && !mbar_wait(k_empty + 8 * sk, ((j / K_SLOTS) - 1) & 1, status, abort_flag)) break;
          load_k(j);
          issued_k = j + 1;
          if (j >= V_SLOTS && !mbar_wait(v_empty + 8 * sv, ((j / V_SLOTS) - 1) & 1, status, abort_flag)) break;
          load_v(j);
          issued_v = j + 1;
        }
        mbar_drain(x_full, 0, status);
        for (int j = max(0, issued_k - K_SLOTS); j < issued_k; ++j)
          mbar_drain(k_full + 8 * (j % K_SLOTS), (j / K_SLOTS) & 1, status);
        for (int j = max(0, issued_v - V_SLOTS); j < issued_v; ++j)
          mbar_drain(v_full + 8 * (j % V_SLOTS), (j / V_SLOTS) & 1, status);
      }
      __syncwarp();
    } else if (warp == PATCH_WARP) {
      if (patch_j >= 0 && patch_j < n && mbar_wait_warp(to_patch, 0, status, abort_flag)) {
        const int from = kl & (BT - 1);
        for (int i = lane; i < (BT - from) * (D / 8); i += 32)
          st_shared_zero16(sw128<BT>(sb + L::OFF_K + (patch_j % K_SLOTS) * L::TILE, from + i / (D / 8), i % (D / 8)));
        fence_async_smem();
        __syncwarp();
        arrive_one(patched);
      }
      __syncwarp();
    } else if (warp == MMA_WARP) {
      if (n > 0 && elect_one()) {
        constexpr uint32_t id_s = idesc_bf16(BT, BT, false, false);
        constexpr uint32_t id_g = idesc_bf16(BT, D, false, true);
        const uint64_t qd = sdesc_sw128(sb + L::OFF_Q, 0, 1024), od = sdesc_sw128(sb + L::OFF_O, 0, 1024);
        bool ok = mbar_wait(x_full, 0, status, abort_flag);
        for (int j = 0; ok && j <= n; ++j) {
          if (j < n) {
            const int sk = j % K_SLOTS, sv = j % V_SLOTS;
            if (!mbar_wait(k_full + 8 * sk, (j / K_SLOTS) & 1, status, abort_flag)) break;
            if (j == patch_j) {
              mbar_arrive(to_patch);
              if (!mbar_wait(patched, 0, status, abort_flag)) break;
            }
            if (!mbar_wait(v_full + 8 * sv, (j / V_SLOTS) & 1, status, abort_flag)) break;
            if (j >= 1 && !mbar_wait(s_free, (j - 1) & 1, status, abort_flag)) break;
            tc_fence_after();
            const uint64_t kd = sdesc_sw128(sb + L::OFF_K + sk * L::TILE, 0, 1024);
            const uint64_t vd = sdesc_sw128(sb + L::OFF_V + sv * L::TILE, 0, 1024);
#pragma unroll
            for (int ks = 0; ks < D / 16; ++ks) {
              const uint32_t o = (ks >> 2) * (BT * 128) + (ks & 3) * 32;
              mma_ss(tmem + qq::kColS, sdesc_add(qd, o), sdesc_add(kd, o), id_s, ks > 0);
            }
#pragma unroll
            for (int ks = 0; ks < D / 16; ++ks) {
              const uint32_t o = (ks >> 2) * (BT * 128) + (ks & 3) * 32;
              mma_ss(tmem + qq::kColP, sdesc_add(od, o), sdesc_add(vd, o), id_s, ks > 0);
            }
            mma_commit(s_full);
            mma_commit(v_empty + 8 * sv);
          }
          if (j >= 1) {
            const int jj = j - 1, bf = jj & 1;
            if (!mbar_wait(ds_full + 8 * bf, (jj >> 1) & 1, status, abort_flag)) break;
            tc_fence_after();
            const uint64_t kd = sdesc_sw128(sb + L::OFF_K + (jj % K_SLOTS) * L::TILE, BT * 128, 1024);
#pragma unroll
            for (int ks = 0; ks < BT / 16; ++ks)
              mma_ts(tmem + qq::kColG, tmem + qq::kColDS + 64 * bf + 8 * ks, sdesc_add(kd, ks * 2048), id_g,
                     jj > 0 || ks > 0);
            mma_commit(k_empty + 8 * (jj % K_SLOTS));
            mma_commit(ds_free + 8 * bf);
          }
        }
        mma_commit(g_done);
        mbar_drain(g_done, 0, status);
      }
      __syncwarp();
    }
  } else {
    setmaxnreg_inc<kRegsDs>();
    const int grp = warp >> 2, wq = warp & 3;
    const int r = wq * 32 + lane;
    const int q = q0 + r;
    const float c = p.c;
    // the padding's rows are there too: -1e30 and 0
    const float nl = c * from_three_bf16(*reinterpret_cast<const uint2*>(row_s + (size_t)bh * padded + q));
    const float dl = -from_three_bf16(*reinterpret_cast<const uint2*>(row_d + (size_t)bh * padded + q));
    const int row_end = q < ql ? (p.causal ? min(kl, q + off + 1) : kl) : 0;  // keys this row sees
    const uint32_t lanes = (uint32_t)(wq * 32) << 16;
    const uint32_t tcol = tmem + lanes + grp * 32;
    bool ok = true;
    for (int j = 0; j < n; ++j) {
      const int bf = j & 1;
      ok = mbar_wait_warp(s_full, j & 1, status, abort_flag);
      __syncwarp();
      if (!ok) break;
      tc_fence_after();
      const int seen = row_end - ((j0 + j) * BT + grp * 32);
      const bool masked = __any_sync(0xffffffffu, seen < 32);
      uint32_t a[32], d[32], pk[16];
      tmem_ld32(tcol + qq::kColS, a);
      tmem_ld32(tcol + qq::kColP, d);
      tmem_ld_wait();
      reg_fence32(a);
      reg_fence32(d);
      tc_fence_before();
      __syncwarp();
      arrive_one(s_free);
      if (masked)
        ds32<true>(a, d, pk, c, nl, dl, seen);
      else
        ds32<false>(a, d, pk, c, nl, dl, 32);
      if (j >= 2) {  // this dS buffer's last product is done
        ok = mbar_wait_warp(ds_free + 8 * bf, ((j >> 1) - 1) & 1, status, abort_flag);
        __syncwarp();
        if (!ok) break;
      }
      tc_fence_after();
      tmem_st16(tmem + lanes + qq::kColDS + 64 * bf + 16 * grp, pk);
      tmem_st_wait();
      tc_fence_before();
      __syncwarp();
      arrive_one(ds_full + 8 * bf);
    }
    bool got = ok;
    if (n > 0 && ok) {
      got = mbar_wait_warp(g_done, 0, status, abort_flag);
      __syncwarp();
    }
    const bool cols = grp * 32 < D;
    uint32_t g[32] = {};
    if (got && cols && n > 0) {
      tc_fence_after();
      tmem_ld32(tmem + lanes + qq::kColG + grp * 32, g);
      tmem_ld_wait();
      reg_fence32(g);
    }
    bool last = true;
    if (part.parts > 1) {
      float4* mine = part_acc + (size_t)(part.tile - plan.q_whole) * part.parts * (D / 4 * BT);
      if (cols) part_put<D>(mine, part.rank, r, grp * 32, g);
      last = part_last(counters + (part.tile - plan.q_whole), part.parts, DS_WARPS * 32, part_flag);
      if (last && cols) part_sum<D>(mine, part.parts, r, grp * 32, g);
    }
    if (got && last && cols) {
      if (row_end <= 0) {
#pragma unroll
        for (int i = 0; i < 32; ++i) g[i] = 0u;
      }
      stage_row32(sb + L::OFF_K, r, 32 * grp, g, p.scale);  // through the first K slot: its products are done
      fence_async_smem();
    }
    // every warp comes here; one that gave up makes none of them store
    if (!named_bar_any(1, DS_WARPS * 32, !got) && last && warp == 0) {
      if (elect_one()) store_tile<D>(&maps.dq, sb + L::OFF_K, q0, h, b);
      __syncwarp();
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == MMA_WARP) {
    tc_fence_after();
    tmem_dealloc(tmem, kTmemCols);
  }
}

template <int D>
__global__ void __launch_bounds__(THREADS, 1)
    attn_bwd_kernel(const AttnProblem p, const uint4* __restrict__ row_s, const uint4* __restrict__ row_d, int padded,
                    int* status, const __grid_constant__ BwdMaps maps, const AttnBwdPlan plan,
                    float4* __restrict__ kv_parts, unsigned* __restrict__ kv_counters, float4* __restrict__ q_parts,
                    unsigned* __restrict__ q_counters) {
  const unsigned x = blockIdx.x, first = plan.q_first ? plan.q_blocks : plan.kv_blocks;
  const bool is_q = plan.q_first ? x < first : x >= first;
  const unsigned blk = x < first ? x : x - first;
  if (is_q)
    q_block<D>(p, row_s, row_d, padded, status, maps, plan, blk, q_parts, q_counters);
  else
    kv_block<D>(p, row_s, row_d, padded, status, maps, plan, blk, kv_parts, kv_counters);
}

// Zeros for `rows` rows of each of B H heads (a backward without queries or without keys).
__global__ void attn_zero_rows_kernel(__nv_bfloat16* dst, int H, int rows, int D, long long sb, long long sh,
                                      long long sn) {
  const long long r = blockIdx.x;
  dst[r / rows / H * sb + r / rows % H * sh + r % rows * sn + threadIdx.x] = __float2bfloat16_rn(0.f);
}

template <int D>
cudaError_t launch_d(const AttnProblem& p, const AttnBwdPlan& plan, const AttnBwdIn& in, void* dq, void* dk, void* dv,
                     void* workspace, int* status, cudaStream_t st) {
  const AttnBwdScratch w = attn_bwd_scratch(p, plan, workspace);
  const long long rows = (long long)p.B * p.H * w.padded;
  auto *row_s = static_cast<uint4*>(w.row_s), *row_d = static_cast<uint4*>(w.row_d);
  constexpr int per_block = 256 / (D / 8) * kRowsEach;
  const auto rows_kern = in.o_rest            ? attn_rows_kernel<D, kRowsRest>
                         : p.NK <= kShortKeys ? attn_rows_kernel<D, kRowsShort>
                                              : attn_rows_kernel<D, kRowsLong>;
  rows_kern<<<(unsigned)(rows / per_block), 256, 0, st>>>(p, in, row_s, row_d, reinterpret_cast<float4*>(w.acc),
                                                         w.kv_counters, w.n_counters, w.padded);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  if (plan.fused) return launch_attn_bwd_fused(p, plan, in, dq, dk, dv, w, status, st);
  BwdMaps m;
  auto q_map = [&](CUtensorMap* map, const void* x, long long sn, long long sh, long long sb) {
    return encode_tile_map(map, x, p.D, p.NQ, p.H, p.B, sn, sh, sb, BT);
  };
  auto k_map = [&](CUtensorMap* map, const void* x, long long sn, long long sh, long long sb) {
    return encode_tile_map(map, x, p.D, p.NK, p.HK, p.B, sn, sh, sb, BT);
  };
  if (!q_map(&m.q, in.q, p.qs_n, p.qs_h, p.qs_b) || !k_map(&m.k, in.k, p.ks_n, p.ks_h, p.ks_b) ||
      !k_map(&m.v, in.v, p.vs_n, p.vs_h, p.vs_b) || !q_map(&m.go, in.go, p.os_n, p.os_h, p.os_b) ||
      !q_map(&m.dq, dq, p.qs_n, p.qs_h, p.qs_b) || !k_map(&m.dk, dk, p.ks_n, p.ks_h, p.ks_b) ||
      !k_map(&m.dv, dv, p.vs_n, p.vs_h, p.vs_b))
    return cudaErrorInvalidValue;
  constexpr int smem = kWholeSmSmem;
  auto kern = attn_bwd_kernel<D>;
  if ((e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem)) != cudaSuccess) return e;
  kern<<<plan.q_blocks + plan.kv_blocks, THREADS, smem, st>>>(
      p, row_s, row_d, w.padded, status, m, plan, static_cast<float4*>(w.kv_parts), w.kv_counters,
      static_cast<float4*>(w.q_parts), w.q_counters);
  return cudaGetLastError();
}

}  // namespace

bool attn_bwd_has_fused(const AttnProblem& p) { return p.D == 64; }

// The plan.  Lengths are in products of a tile pair: a dK/dV block does four for each query tile of its G heads, a dQ
// block three for each key tile, a fused one five; setting a block up, filling its pipeline and storing its tile take as
// long as about kBlockCost more.
//   separate  of the ways to deal both kinds' tiles out over 1 to 8 parts each, one whose larger of the longest block and
//             the SMs' share of all is clearly smallest; a part's trip through the workspace costs kPartCost more.
//             Measured, us without and with parts: B1 H4 HK1 N4096 D128 causal 176 / 59, B1 H16 HK4 N2048 D64 causal 80 /
//             51, B1 H8 HK1 N512 D128 51 / 27, B1 H16 HK4 N4096 D128 causal 184 / 177; where the rule leaves them whole
//             (measured on an earlier build): B1 H32 HK8 N2048 D128 causal 119 / 133, B1 H32 N_Q128 N_K64K D128 866 / 910.
//   fused     the tiles of the last, incomplete wave are dealt out so that it fills the SMs (non-causal: a causal grid's
//             short blocks fill the end by themselves).
// In a grid of few waves the order of lengths counts for more than the L2 (whose reuse a head-major order is for).
constexpr int kBlockCost = 12, kPartCost = 4;
constexpr int kMaxParts = 8;
constexpr int kMinPartTiles = 4;
constexpr int kSmallGrid = 6;

AttnBwdPlan attn_bwd_plan(const AttnProblem& p, int mode, int num_sms) {
  const int nq = (p.NQ + BT - 1) / BT, nk = (p.NK + BT - 1) / BT;
  AttnBwdPlan g{};
  g.kv_tiles = (unsigned)((long long)p.B * p.HK * nk);
  g.q_tiles = (unsigned)((long long)p.B * p.H * nq);
  g.kv_parts = g.q_parts = 1;
  if (nq == 0 || nk == 0) return g;
  const long long stream = (long long)p.G * nq;  // tiles a dK/dV block streams
  // STREAMKL_BWD_AUTO, 0: fused where it exists and its blocks fill the SMs
  g.fused = attn_bwd_has_fused(p) && (mode == 1 || (mode == 0 && g.kv_tiles >= (unsigned)num_sms));
  if (g.fused) {
    g.q_tiles = 0;
    const unsigned tail = g.kv_tiles % num_sms;
    g.kv_whole = g.kv_tiles;
    if (tail && (!p.causal || g.kv_tiles < (unsigned)num_sms)) {
      long long parts = num_sms / tail;
      if (parts > kMaxParts) parts = kMaxParts;
      if (parts > stream / kMinPartTiles) parts = stream / kMinPartTiles;
      if (parts > 1) {
        g.kv_whole = g.kv_tiles - tail;
        g.kv_parts = (int)parts;
      }
    }
  } else {
    const double mean = p.causal ? 0.5 : 1.0;
    double best = 0;
    int best_kv = 1, best_q = 1;
    for (int a = 1; a <= kMaxParts; ++a) {
      if (a > 1 && stream / a < kMinPartTiles) break;
      for (int b = 1; b <= kMaxParts; ++b) {
        if (b > 1 && nk / b < kMinPartTiles) break;
        const double kv = 4.0 * stream / a, q = 3.0 * nk / b;
        const double kv_cost = kBlockCost + (a > 1 ? kPartCost : 0), q_cost = kBlockCost + (b > 1 ? kPartCost : 0);
        const double longest = kv + kv_cost > q + q_cost ? kv + kv_cost : q + q_cost;
        const double all = (g.kv_tiles * a * (mean * kv + kv_cost) + g.q_tiles * b * (mean * q + q_cost)) / num_sms;
        const double cost = longest > all ? longest : all;
        if (best == 0 || cost < best * 0.85) {  // more parts only for a clear gain
          best = cost;
          best_kv = a;
          best_q = b;
        }
      }
    }
    g.kv_parts = best_kv;
    g.q_parts = best_q;
    g.kv_whole = best_kv > 1 ? 0 : g.kv_tiles;
    g.q_whole = best_q > 1 ? 0 : g.q_tiles;
  }
  g.kv_blocks = g.kv_whole + (g.kv_tiles - g.kv_whole) * g.kv_parts;
  g.q_blocks = g.q_whole + (g.q_tiles - g.q_whole) * g.q_parts;
  g.longest_first = (long long)g.kv_blocks + g.q_blocks <= (long long)kSmallGrid * num_sms;
  g.q_first = 3.0 * nk / g.q_parts > 4.0 * stream / g.kv_parts;
  g.by_kv_parts = FastDiv((unsigned)g.kv_parts);
  g.by_q_parts = FastDiv((unsigned)g.q_parts);
  g.by_kv_tile = FastDiv((unsigned)(g.longest_first ? p.B * p.HK : nk));
  g.by_q_tile = FastDiv((unsigned)(g.longest_first ? p.B * p.H : nq));
  g.by_key_heads = FastDiv((unsigned)p.HK);
  g.by_heads = FastDiv((unsigned)p.H);
  g.by_group = FastDiv((unsigned)p.G);
  return g;
}

AttnBwdScratch attn_bwd_scratch(const AttnProblem& p, const AttnBwdPlan& plan, void* workspace) {
  AttnBwdScratch w{};
  w.padded = (p.NQ + BT - 1) / BT * BT;
  if (p.NQ == 0 || p.NK == 0) return w;
  const size_t rows = (size_t)p.B * p.H * w.padded;
  const size_t kv_split = plan.kv_tiles - plan.kv_whole, q_split = plan.q_tiles - plan.q_whole;
  auto take = [&](size_t bytes) {
    void* at = static_cast<char*>(workspace) + w.bytes;
    w.bytes += (bytes + 15) / 16 * 16;
    return at;
  };
  w.row_s = take(rows * 16);
  w.row_d = take(rows * 16);
  if (plan.fused) w.acc = static_cast<float*>(take(rows * p.D * sizeof(float)));
  w.kv_parts = take(kv_split * plan.kv_parts * 2 * p.D * BT * sizeof(float));
  w.q_parts = take(q_split * plan.q_parts * p.D * BT * sizeof(float));
  w.n_counters = (unsigned)(kv_split + q_split);
  w.kv_counters = static_cast<unsigned*>(take(w.n_counters * sizeof(unsigned)));
  w.q_counters = w.kv_counters + kv_split;
  return w;
}

cudaError_t launch_attn_bwd(const AttnProblem& p, const AttnBwdPlan& plan, const AttnBwdIn& in, void* dq, void* dk,
                            void* dv, void* workspace, int* status, cudaStream_t st) {
  if (p.NQ == 0 || p.NK == 0) {
    auto* q = static_cast<__nv_bfloat16*>(dq);
    auto* k = static_cast<__nv_bfloat16*>(dk);
    auto* v = static_cast<__nv_bfloat16*>(dv);
    if (p.NQ > 0)
      attn_zero_rows_kernel<<<(unsigned)((long long)p.B * p.H * p.NQ), p.D, 0, st>>>(q, p.H, p.NQ, p.D, p.qs_b, p.qs_h,
                                                                                    p.qs_n);
    if (p.NK > 0) {
      const unsigned n = (unsigned)((long long)p.B * p.HK * p.NK);
      attn_zero_rows_kernel<<<n, p.D, 0, st>>>(k, p.HK, p.NK, p.D, p.ks_b, p.ks_h, p.ks_n);
      attn_zero_rows_kernel<<<n, p.D, 0, st>>>(v, p.HK, p.NK, p.D, p.vs_b, p.vs_h, p.vs_n);
    }
    return cudaGetLastError();
  }
  if (p.D == 64) return launch_d<64>(p, plan, in, dq, dk, dv, workspace, status, st);
  return launch_d<128>(p, plan, in, dq, dk, dv, workspace, status, st);
}

}  // namespace skl
