// Attention backward, fused, for D = 64: every tile pair is visited once and
// gives its share of dK, dV and dQ -- five products a tile pair where the separate
// blocks (attn_bwd.cu, which states the mathematics) need seven, and one exp
// instead of two.  Its price: a block owns 128 keys, so dQ is added up over the
// blocks of a head, in fp32 by bulk reductions into an accumulator that lies in L2
// while a head is worked on.  The order of those additions is not fixed: the last
// bits of dQ can differ between runs (dK and dV do not).
//
//   S^T = K Q^T - LSE / scale, dP^T = V dO^T - delta   (lanes = keys; a K step more adds the rows' values)
//   P^T = 2^(c S^T) as bf16 pairs over its logits in TMEM:  dV += P^T dO
//   dS^T = P^T dP^T as bf16 pairs over dP in TMEM:          dK += dS^T Q
//          and in shared memory [key][query]:               dQ = dS K (MN-major A)
// TMEM: S/P [0,128), dP/dS [128,256), dV, dK, dQ 64 columns each from 256 on, and K and V as bf16 pairs in the last 64,
// the A operands of S and dP: read from shared memory with the other operands they brought a tile pair's traffic there to
// 350 KB (8 heads, N8192, non-causal: 403 us against 388).  What bounds a tile pair, about 2500 cycles, are the 260 KB that
// are left, 2000 cycles at 128 bytes a clock; the products alone take 1550.  The traffic comes in two halves, between the
// two barriers of the P and dS warps; dQ is computed before dP, and so staged and reduced while the first half's products
// leave room (32 heads, 8 key heads, N8192, non-causal: 1190 to 1220 us, 1140 TFLOP/s of five products; the other way round 1290).
//   warps 0-15   thread = key, group g = warp / 4 takes queries [32g, 32g + 32)
//   warps 16-19  dQ: TMEM -> registers -> a ring of staging chunks a warp -> bulk reductions
//   warp 20      TMA producer: K, V once; Q(u) and dO(u) with their rows' values
//   warp 21      TMEM owner and MMA issuer: dV(u), S(u+1), dK(u), dQ(u), dP(u+1)
//   warp 22      clears rows past a sequence's lengths in K, V, Q and dO tiles
// At D = 128 the same kernel (built, measured, not kept) has 532 KB of shared-memory traffic a tile pair, dQ's staging
// and reductions 128 KB of it: 4450 cycles against 4460 for the separate blocks' two visits (B2 H32 HK8 N4096 causal
// 0.69 against 0.68 ms).  At D = 64: 8 heads, N8192, non-causal 0.31 against 0.43 ms; with red.add from registers instead of
// staging and bulk reductions 0.39.
#include "attn.cuh"

namespace skl {
namespace {

constexpr int BT = 128;
constexpr int D = 64;
constexpr int DS_WARPS = 16, DQ_WARPS = 4;
constexpr int PRODUCER_WARP = 20, MMA_WARP = 21, PATCH_WARP = 22;
constexpr int THREADS = 24 * 32;
// 512 * 80 + 128 * 88 + 128 * 72 = 768 * 80 registers at launch; the P and dS warps keep their 80 (an inc to the count that a
// warp has already is not described)
constexpr int kRegsDq = 88, kRegsOther = 72;
constexpr uint32_t kTmemCols = 512;

struct Maps {
  CUtensorMap q, k, v, go, dk, dv, acc;  // acc: fp32 [B H][padded rows][D], boxes of a staging chunk
};

constexpr uint32_t kS = 0, kP = 128, kV = 256, kK = 320, kQ = 384, kTK = 448, kTV = 480;  // TMEM columns
constexpr int SLOTS = 2;                                                                 // of Q and of dO tiles
// A dQ warp's staging ring: chunks of 32 rows x 32 columns.  What is on its way to L2 bounds the reductions' rate (24
// bytes a clock with a latency of 1000 to 1500).
constexpr int RING = 4, CHUNK_BYTES = 32 * 32 * 4;

struct Smem {
  static constexpr int TILE = BT * D * 2;
  static constexpr int OFF_K = 0, OFF_V = TILE, OFF_Q = 2 * TILE;
  static constexpr int OFF_O = OFF_Q + SLOTS * TILE;
  static constexpr int OFF_DS = OFF_O + SLOTS * TILE;      // [128 keys][128 queries] bf16, two halves
  static constexpr int OFF_STAGE = OFF_DS + BT * BT * 2;   // the dQ warps' rings
  static constexpr int STEP = 128 * 16;                    // rows' values of a tile
  static constexpr int OFF_RS = OFF_STAGE + DQ_WARPS * RING * CHUNK_BYTES;
  static constexpr int OFF_RD = OFF_RS + SLOTS * STEP;
  static constexpr int OFF_ONES = OFF_RD + SLOTS * STEP;
  static constexpr int OFF_ZERO = OFF_ONES + STEP;
  static constexpr int OFF_BAR = OFF_ZERO + STEP;
  // kv_full, kv_patched, q_full[2], q_empty[2], o_full[2], o_empty[2], s_full, dp_full, p_full, ds_full, dq_full,
  // dq_free, g_done, to_patch, patched, kv_tmem; TMEM slot, abort flag, part flag
  static constexpr int BAR_SLOT = 8 * 20;
  static constexpr int BYTES = OFF_BAR + BAR_SLOT + 16;
};
static_assert(Smem::BYTES <= kWholeSmSmem, "shared memory");

__device__ __forceinline__ void reduce_add_3d(const CUtensorMap* map, uint32_t src, int x, int y, int z) {
  asm volatile("cp.reduce.async.bulk.tensor.3d.global.shared::cta.add.tile.bulk_group [%0, {%2, %3, %4}], [%1];" ::"l"(
                   reinterpret_cast<uint64_t>(map)),
               "r"(src), "r"(x), "r"(y), "r"(z)
               : "memory");
}

__global__ void __launch_bounds__(THREADS, 1)
    attn_bwd_fused_kernel(const AttnProblem p, const uint4* __restrict__ row_s, const uint4* __restrict__ row_d, int padded,
                          int* status, const __grid_constant__ Maps maps, const AttnBwdPlan plan, float4* __restrict__ part_acc,
                          unsigned* __restrict__ counters) {
  using L = Smem;
  extern __shared__ __align__(1024) uint8_t smem[];  // the swizzled tiles' alignment; nothing lies before it
  const uint32_t sb = smem_u32(smem);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  // heads in order (the blocks in flight share one key head's query tiles and dQ rows in L2); within a head the first
  // key tiles, which see the most queries under a causal mask, first.  A small grid: the first key tiles of all heads
  const TilePart part = tile_part(blockIdx.x, plan.kv_whole, plan.by_kv_parts);
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
  const bool ragged_q = n > 0 && ql < p.NQ && (ql & (BT - 1));  // the last query tile has rows past the sequence
  const bool ragged_k = n > 0 && kl < p.NK && kl - k0 < BT;     // so has this key tile

  const uint32_t bar = sb + L::OFF_BAR;
  const uint32_t kv_full = bar, kv_patched = bar + 8, q_full = bar + 16, q_empty = bar + 32, o_full = bar + 48,
                 o_empty = bar + 64, s_full = bar + 80, dp_full = bar + 88, p_full = bar + 96, ds_full = bar + 104,
                 dq_full = bar + 112, dq_free = bar + 120, g_done = bar + 128, to_patch = bar + 136, patched = bar + 144,
                 kv_tmem = bar + 152, slot = bar + L::BAR_SLOT;
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + L::OFF_BAR + L::BAR_SLOT + 4);
  volatile int* part_flag = abort_flag + 1;
  if (warp == PRODUCER_WARP) {
    if (elect_one()) {
      mbar_init(kv_full, 1);
      mbar_init(kv_patched, 1);
      for (int s = 0; s < 2; ++s) {
        mbar_init(q_full + 8 * s, 1);
        mbar_init(q_empty + 8 * s, 1);
        mbar_init(o_full + 8 * s, 1);
        mbar_init(o_empty + 8 * s, 1);
      }
      mbar_init(s_full, 1);
      mbar_init(dp_full, 1);
      mbar_init(p_full, DS_WARPS);
      mbar_init(ds_full, DS_WARPS);
      mbar_init(dq_full, 1);
      mbar_init(dq_free, DQ_WARPS);
      mbar_init(g_done, 1);
      mbar_init(to_patch, 1);
      mbar_init(patched, 1);
      mbar_init(kv_tmem, 8);
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

  if (warp >= PRODUCER_WARP) {
    setmaxnreg_dec<kRegsOther>();
    if (warp == PRODUCER_WARP) {
      if (n > 0 && elect_one()) {
        mbar_arrive_expect_tx(kv_full, 2 * L::TILE);
#pragma unroll
        for (int h = 0; h < D / 64; ++h) {
          tma_load_4d(sb + L::OFF_K + h * BT * 128, &maps.k, kv_full, h * 64, k0, hk, b);
          tma_load_4d(sb + L::OFF_V + h * BT * 128, &maps.v, kv_full, h * 64, k0, hk, b);
        }
        int issued_q = 0, issued_o = 0, hq = hk * p.G + head0, qt = qt0;
        for (int u = 0; u < n; ++u) {
          const int s = u % SLOTS, q0 = q_begin + qt * BT;
          const long long row = ((long long)b * p.H + hq) * padded + q0;
          if (u >= SLOTS && !mbar_wait(q_empty + 8 * s, ((u / SLOTS) - 1) & 1, status, abort_flag)) break;
          mbar_arrive_expect_tx(q_full + 8 * s, L::TILE + L::STEP);
#pragma unroll
          for (int h = 0; h < D / 64; ++h)
            tma_load_4d(sb + L::OFF_Q + s * L::TILE + h * BT * 128, &maps.q, q_full + 8 * s, h * 64, q0, hq, b);
          bulk_load(sb + L::OFF_RS + s * L::STEP, row_s + row, L::STEP, q_full + 8 * s);
          issued_q = u + 1;
          if (u >= SLOTS && !mbar_wait(o_empty + 8 * s, ((u / SLOTS) - 1) & 1, status, abort_flag)) break;
          mbar_arrive_expect_tx(o_full + 8 * s, L::TILE + L::STEP);
#pragma unroll
          for (int h = 0; h < D / 64; ++h)
            tma_load_4d(sb + L::OFF_O + s * L::TILE + h * BT * 128, &maps.go, o_full + 8 * s, h * 64, q0, hq, b);
          bulk_load(sb + L::OFF_RD + s * L::STEP, row_d + row, L::STEP, o_full + 8 * s);
          issued_o = u + 1;
          if (++qt == n_qt) {
            qt = 0;
            ++hq;
          }
        }
        mbar_drain(kv_full, 0, status);
        for (int u = max(0, issued_q - SLOTS); u < issued_q; ++u) mbar_drain(q_full + 8 * (u % SLOTS), (u / SLOTS) & 1, status);
        for (int u = max(0, issued_o - SLOTS); u < issued_o; ++u) mbar_drain(o_full + 8 * (u % SLOTS), (u / SLOTS) & 1, status);
      }
      __syncwarp();
    } else if (warp == PATCH_WARP) {
      auto clear = [&](uint32_t tile, int from) {
        for (int i = lane; i < (BT - from) * (D / 8); i += 32)
          st_shared_zero16(sw128<BT>(tile, from + i / (D / 8), i % (D / 8)));
      };
      bool ok = true;
      if (ragged_k) {
        ok = mbar_wait_warp(kv_full, 0, status, abort_flag);
        if (ok) {
          clear(sb + L::OFF_K, kl - k0);
          clear(sb + L::OFF_V, kl - k0);
          fence_async_smem();
          __syncwarp();
          arrive_one(kv_patched);
        }
      }
      // for each head's last tile: its Q, then its dO, when the MMA thread has seen them land
      const int first = n_qt - 1 - qt0;  // the first of this block's tiles that is a head's last
      for (int e = 0; ok && ragged_q && first + e / 2 * n_qt < n; ++e) {
        if (!(ok = mbar_wait_warp(to_patch, e & 1, status, abort_flag))) break;
        const int u = first + e / 2 * n_qt;
        clear(sb + ((e & 1) ? L::OFF_O + u % SLOTS * L::TILE : L::OFF_Q + u % SLOTS * L::TILE), ql & (BT - 1));
        fence_async_smem();
        __syncwarp();
        arrive_one(patched);
      }
      __syncwarp();
    } else if (warp == MMA_WARP) {
      if (n > 0 && elect_one()) {
        constexpr uint32_t id_s = idesc_bf16(BT, BT, false, false);
        constexpr uint32_t id_g = idesc_bf16(BT, D, false, true);
        constexpr uint32_t id_q = idesc_bf16(BT, D, true, true);
        const uint64_t kmn = sdesc_sw128(sb + L::OFF_K, BT * 128, 1024);
        const uint64_t dsmn = sdesc_sw128(sb + L::OFF_DS, BT * 128, 1024);
        const uint64_t ones = sdesc_step(sb + L::OFF_ONES, sb + L::OFF_ZERO);
        int patches = 0;
        auto patch = [&](int u) {  // the head's last tile: wait until its rows past the sequence are cleared
          if (!ragged_q || (qt0 + u + 1) % n_qt) return true;
          mbar_arrive(to_patch);
          return mbar_wait(patched, patches++ & 1, status, abort_flag);
        };
        auto issue_s = [&](int u) {  // S^T(u)
          const int s = u % SLOTS;
          if (!mbar_wait(q_full + 8 * s, (u / SLOTS) & 1, status, abort_flag) || !patch(u)) return false;
          tc_fence_after();
          const uint64_t qd = sdesc_sw128(sb + L::OFF_Q + s * L::TILE, 0, 1024);
#pragma unroll
          for (int ks = 0; ks < D / 16; ++ks) {
            const uint32_t o = (ks >> 2) * (BT * 128) + (ks & 3) * 32;
            mma_ts(tmem + kS, tmem + kTK + 8 * ks, sdesc_add(qd, o), id_s, ks > 0);
          }
          mma_ss(tmem + kS, ones, sdesc_step(sb + L::OFF_RS + s * L::STEP, sb + L::OFF_ZERO), id_s, true);
          mma_commit(s_full);
          return true;
        };
        auto issue_dp = [&](int u) {  // dP^T(u)
          const int s = u % SLOTS;
          if (!mbar_wait(o_full + 8 * s, (u / SLOTS) & 1, status, abort_flag) || !patch(u)) return false;
          tc_fence_after();
          const uint64_t od = sdesc_sw128(sb + L::OFF_O + s * L::TILE, 0, 1024);
#pragma unroll
          for (int ks = 0; ks < D / 16; ++ks) {
            const uint32_t o = (ks >> 2) * (BT * 128) + (ks & 3) * 32;
            mma_ts(tmem + kP, tmem + kTV + 8 * ks, sdesc_add(od, o), id_s, ks > 0);
          }
          mma_ss(tmem + kP, ones, sdesc_step(sb + L::OFF_RD + s * L::STEP, sb + L::OFF_ZERO), id_s, true);
          mma_commit(dp_full);
          return true;
        };
        bool ok = mbar_wait(kv_full, 0, status, abort_flag) &&
                  (!ragged_k || mbar_wait(kv_patched, 0, status, abort_flag)) &&
                  mbar_wait(kv_tmem, 0, status, abort_flag) && issue_s(0) && issue_dp(0);
        for (int u = 0; ok && u < n; ++u) {
          const int s = u % SLOTS;
          if (!mbar_wait(p_full, u & 1, status, abort_flag)) break;
          tc_fence_after();
          const uint64_t omn = sdesc_sw128(sb + L::OFF_O + s * L::TILE, BT * 128, 1024);
#pragma unroll
          for (int ks = 0; ks < BT / 16; ++ks)  // dV += P^T dO; a group's 32 queries lie in 32 columns' first 16
            mma_ts(tmem + kV, tmem + kS + 32 * (ks >> 1) + 8 * (ks & 1), sdesc_add(omn, ks * 2048), id_g, u > 0 || ks > 0);
          mma_commit(o_empty + 8 * s);
          if (u + 1 < n && !(ok = issue_s(u + 1))) break;
          if (!mbar_wait(ds_full, u & 1, status, abort_flag)) break;
          tc_fence_after();
          const uint64_t qmn = sdesc_sw128(sb + L::OFF_Q + s * L::TILE, BT * 128, 1024);
#pragma unroll
          for (int ks = 0; ks < BT / 16; ++ks)  // dK += dS^T Q
            mma_ts(tmem + kK, tmem + kP + 32 * (ks >> 1) + 8 * (ks & 1), sdesc_add(qmn, ks * 2048), id_g, u > 0 || ks > 0);
          mma_commit(q_empty + 8 * s);
          if (u >= 1 && !mbar_wait(dq_free, (u - 1) & 1, status, abort_flag)) break;
          tc_fence_after();
#pragma unroll
          for (int ks = 0; ks < BT / 16; ++ks)  // dQ = dS K
            mma_ss(tmem + kQ, sdesc_add(dsmn, ks * 2048), sdesc_add(kmn, ks * 2048), id_q, ks > 0);
          mma_commit(dq_full);
          // last, when dK has read dS from dP's columns; dQ before it, so that its way out is over before dV and S run
          if (u + 1 < n && !issue_dp(u + 1)) break;
        }
        mma_commit(g_done);
        mbar_drain(g_done, 0, status);
      }
      __syncwarp();
    }
  } else if (warp >= DS_WARPS) {
    setmaxnreg_inc<kRegsDq>();
    // ---------------------------------------------------------------- dQ out
    const int wq = warp & 3;
    const uint32_t tq = tmem + ((uint32_t)(wq * 32) << 16) + kQ;
    const uint32_t ring = sb + L::OFF_STAGE + (warp - DS_WARPS) * RING * CHUNK_BYTES;
    int at = 0;                          // ring position
    int hq = hk * p.G + head0, q0 = q_begin + qt0 * BT;
    for (int u = 0; u < n; ++u) {
      const bool ok = mbar_wait_warp(dq_full, u & 1, status, abort_flag);
      __syncwarp();
      if (!ok) break;
      tc_fence_after();
      uint32_t a[D / 32][32];
#pragma unroll
      for (int c = 0; c < D / 32; ++c) tmem_ld32(tq + 32 * c, a[c]);
      tmem_ld_wait();
#pragma unroll
      for (int c = 0; c < D / 32; ++c) reg_fence32(a[c]);
      tc_fence_before();
      __syncwarp();
      arrive_one(dq_free);
#pragma unroll
      for (int c = 0; c < D / 32; ++c) {
        // the reduction that last used this chunk has read it
        if (elect_one()) asm volatile("cp.async.bulk.wait_group.read %0;" ::"n"(RING - 1) : "memory");
        __syncwarp();
        const uint32_t stage = ring + at * CHUNK_BYTES;
        at = (at + 1) % RING;
#pragma unroll
        for (int i = 0; i < 8; ++i)
          st_shared16(stage + lane * 128 + ((i ^ (lane & 7)) << 4),
                      make_uint4(a[c][4 * i], a[c][4 * i + 1], a[c][4 * i + 2], a[c][4 * i + 3]));
        fence_async_smem();
        __syncwarp();
        if (elect_one()) {  // the same lane every time: bulk groups are a thread's own
          reduce_add_3d(&maps.acc, stage, 32 * c, q0 + 32 * wq, b * p.H + hq);
          bulk_commit();
        }
        __syncwarp();
      }
      q0 += BT;
      if (q0 == q_begin + n_qt * BT) {
        q0 = q_begin;
        ++hq;
      }
    }
    if (elect_one()) asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");
    __syncwarp();
  } else {
    // ---------------------------------------------------------------- P and dS
    const int grp = warp >> 2, wq = warp & 3;
    const int r = wq * 32 + lane;
    const int key = k0 + r;
    const float2 cc = make_float2(p.c, p.c);
    const uint32_t lanes = (uint32_t)(wq * 32) << 16;
    const uint32_t ts = tmem + lanes + kS + 32 * grp, tp = tmem + lanes + kP + 32 * grp;
    bool ok = true;
    if (n > 0 && grp < 2) {  // K (group 0) and V (group 1) into TMEM: lane = key, a column two of its elements
      ok = mbar_wait_warp(kv_full, 0, status, abort_flag) &&
           (!ragged_k || mbar_wait_warp(kv_patched, 0, status, abort_flag));
      __syncwarp();
      if (ok) {
        uint32_t w[32];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const uint4 x = ld_shared16(sw128<BT>(sb + (grp ? L::OFF_V : L::OFF_K), r, i));
          w[4 * i] = x.x;
          w[4 * i + 1] = x.y;
          w[4 * i + 2] = x.z;
          w[4 * i + 3] = x.w;
        }
        tc_fence_after();
        tmem_st32(tmem + lanes + (grp ? kTV : kTK), w);
        tmem_st_wait();
        tc_fence_before();
        __syncwarp();
        arrive_one(kv_tmem);
      }
    }
    const int q_last = q_begin + (n_qt - 1) * BT + 32 * grp;
    int q0 = q_begin + qt0 * BT + 32 * grp;  // first query of this warp's columns
    for (int u = 0; ok && u < n; ++u) {
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
      ok = mbar_wait_warp(dp_full, u & 1, status, abort_flag);  // dQ(u-1), issued before dP(u), has read dS too
      __syncwarp();
      if (!ok) break;
      tc_fence_after();
      uint32_t d[32];
      tmem_ld32(tp, d);
      tmem_ld_wait();
      reg_fence32(d);
#pragma unroll
      for (int v = 0; v < 4; ++v) {
#pragma unroll
        for (int i = 8 * v; i < 8 * v + 8; i += 2) {
          const float2 x = fmul2(make_float2(__uint_as_float(a[i]), __uint_as_float(a[i + 1])),
                                 make_float2(__uint_as_float(d[i]), __uint_as_float(d[i + 1])));
          pk[i / 2] = pack_bf16(x.x, x.y);
        }
        st_shared16(sw128<BT>(sb + L::OFF_DS, r, grp * 4 + v),
                    make_uint4(pk[4 * v], pk[4 * v + 1], pk[4 * v + 2], pk[4 * v + 3]));
      }
      tmem_st16(tp, pk);
      tmem_st_wait();
      tc_fence_before();
      fence_async_smem();
      __syncwarp();
      arrive_one(ds_full);
      q0 = q0 == q_last ? q_last - (n_qt - 1) * BT : q0 + BT;
    }
    // ---- dV (groups 0, 1) through the first Q slot, dK (2, 3) through the second: every product that read them is done
    bool got = ok;
    if (n > 0 && ok) {
      got = mbar_wait_warp(g_done, 0, status, abort_flag);
      __syncwarp();
    }
    const int which = grp / 2, col = (grp & 1) * 32;
    uint32_t g[32];
    if (got && n > 0) {
      tc_fence_after();
      tmem_ld32(tmem + lanes + (which ? kK : kV) + col, g);
      tmem_ld_wait();
      reg_fence32(g);
    }
    if (n == 0 || key >= kl) {
#pragma unroll
      for (int i = 0; i < 32; ++i) g[i] = 0u;
    }
    bool last = true;
    if (part.parts > 1) {
      // both tensors' accumulators of a part are one tile of 2 D columns
      float4* mine = part_acc + (size_t)(part.tile - plan.kv_whole) * part.parts * (2 * D / 4 * BT);
      part_put<2 * D>(mine, part.rank, r, which * D + col, g);
      last = part_last(counters + (part.tile - plan.kv_whole), part.parts, DS_WARPS * 32, part_flag);
      if (last) part_sum<2 * D>(mine, part.parts, r, which * D + col, g);
    }
    if (got && last) stage_row32(sb + L::OFF_Q + which * L::TILE, r, col, g, which ? p.scale : 1.f);
    fence_async_smem();
    // every warp comes here; one that gave up makes none of them store
    if (!named_bar_any(1, DS_WARPS * 32, !got) && last && warp == 0) {
      if (elect_one()) {
        store_tile<D>(&maps.dv, sb + L::OFF_Q, k0, hk, b);
        store_tile<D>(&maps.dk, sb + L::OFF_Q + L::TILE, k0, hk, b);
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

// dQ = scale acc, as bf16 with q's strides; a thread takes 8 columns.
__global__ void __launch_bounds__(256) attn_dq_out_kernel(const AttnProblem p, const float* __restrict__ acc, int padded,
                                                          __nv_bfloat16* __restrict__ dq) {
  constexpr int LANES = D / 8;
  const long long i = (long long)blockIdx.x * 256 + threadIdx.x;
  const long long row = i / LANES;
  if (row >= p.rows) return;
  const int lane = (int)(i % LANES);
  const long long bh = row / p.NQ, n = row % p.NQ;
  const float4* src = reinterpret_cast<const float4*>(acc + (bh * padded + n) * D + lane * 8);
  const float4 x = src[0], y = src[1];
  const float f = p.scale;
  *reinterpret_cast<uint4*>(dq + bh / p.H * p.qs_b + bh % p.H * p.qs_h + n * p.qs_n + lane * 8) =
      make_uint4(pack_bf16(x.x * f, x.y * f), pack_bf16(x.z * f, x.w * f), pack_bf16(y.x * f, y.y * f),
                 pack_bf16(y.z * f, y.w * f));
}

}  // namespace

cudaError_t launch_attn_bwd_fused(const AttnProblem& p, const AttnBwdPlan& plan, const AttnBwdIn& in, void* dq, void* dk,
                                  void* dv, const AttnBwdScratch& w, int* status, cudaStream_t st) {
  Maps m;
  if (!encode_tile_map(&m.q, in.q, D, p.NQ, p.H, p.B, p.qs_n, p.qs_h, p.qs_b, BT) ||
      !encode_tile_map(&m.k, in.k, D, p.NK, p.HK, p.B, p.ks_n, p.ks_h, p.ks_b, BT) ||
      !encode_tile_map(&m.v, in.v, D, p.NK, p.HK, p.B, p.vs_n, p.vs_h, p.vs_b, BT) ||
      !encode_tile_map(&m.go, in.go, D, p.NQ, p.H, p.B, p.os_n, p.os_h, p.os_b, BT) ||
      !encode_tile_map(&m.dk, dk, D, p.NK, p.HK, p.B, p.ks_n, p.ks_h, p.ks_b, BT) ||
      !encode_tile_map(&m.dv, dv, D, p.NK, p.HK, p.B, p.vs_n, p.vs_h, p.vs_b, BT) ||
      !encode_rows_f32_map(&m.acc, w.acc, D, w.padded, p.B * p.H, 32, 32))
    return cudaErrorInvalidValue;
  constexpr int smem = kWholeSmSmem;
  cudaError_t e = cudaFuncSetAttribute(attn_bwd_fused_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) return e;
  attn_bwd_fused_kernel<<<plan.kv_blocks, THREADS, smem, st>>>(p, static_cast<const uint4*>(w.row_s),
                                                              static_cast<const uint4*>(w.row_d), w.padded, status, m, plan,
                                                              static_cast<float4*>(w.kv_parts), w.kv_counters);
  if ((e = cudaGetLastError()) != cudaSuccess) return e;
  attn_dq_out_kernel<<<(unsigned)((p.rows * (D / 8) + 255) / 256), 256, 0, st>>>(p, w.acc, w.padded,
                                                                               static_cast<__nv_bfloat16*>(dq));
  return cudaGetLastError();
}

}  // namespace skl
