// Attention forward: O = softmax(scale Q K^T) V and the rows' log-sum-exp, on
// the 5th-generation tensor cores.
//
// One pass over the keys with a running maximum m and sum l per query row, in
// log2 units x = c (q . k), c = scale log2(e):
//     p_j = 2^(x_j - m),  l += sum_j p_j,  O += sum_j bf16(p_j) v_j
//     when m moves to m': l *= 2^(m - m'), O *= 2^(m - m')
//     at the end O / l and LSE = ln2 (m + log2 l)
// m is a reference, not the exact maximum: once a row has one, a tile is summed
// against it without taking its own maximum, and only where a row's sum would
// pass 2^16 is m moved to the tile's maximum and O, which stays in TMEM, scaled.
// That is exact because p, l and O share m and bf16 has fp32's exponent range;
// rounding p to bf16 costs half a bf16 step of each weight, as the product's
// other operand v has; l sums the unrounded p.  O holds up to 2^16 |v| a tile before
// the division, so values up to 2^88 give finite sums at any length (2^23 tiles);
// 2^16 is seldom passed, a higher limit would narrow the values' range.
//
// A block owns two tiles of 128 rows and streams 128-key tiles of K and V, so
// each K and V tile loaded from L2 serves 256 rows:
//   warps 0-3, 4-7  softmax of tile A and of tile B; thread = row (TMEM lane)
//   warp 8          TMA producer: Q_A, Q_B, then K(j), V(j), K(j+1), ... through a ring
//   warp 9          TMEM owner and MMA issuer (one thread)
//   warp 10         clears rows of the V tile that lie past a sequence's key length
// TMEM at D 128: S_A [0,128), S_B [128,256), O_A [256,384), O_B [384,512); P (bf16
// pairs) overwrites the first 64 columns of its own S and is the A operand of
// O += P V.  The pipe runs S_A(j+1) behind P V_A(j), then P V_B(j), S_B(j+1):
// while one tile's softmax works, the other tile's two products run.
// At D 64 there is room for three S buffers, [0,384), O_A and O_B behind them: the
// pairs (A,0), (B,0), (A,1), ... take them in turn and S runs three pairs ahead, so
// no softmax waits for its next S (one query over 64K keys, B8 H32 HK8: 301 -> 226
// us when it was built, 218 now; N8192 full, 32 heads: 510 -> 498).
//
// Measured: D 128, 32 heads, 8 key heads, N16384 causal 1270 to 1480 us on different
// cards, 1490 to 1730 TFLOP/s, near what the power limit leaves a plain matrix
// product (1750); 8 heads, N8192 full 174 to 188 us, 1460 to 1580 (two waves for 256
// blocks of 152 SMs).  One query over 131072 keys, B8 H32 HK8: 670 us, 6.4 TB/s.  At
// D 64 the softmax and the one thread that issues the products bound it: N8192 full,
// 32 heads, 537 us, 1020 TFLOP/s (498 before the arrivals came from an elected lane).
//
// For a backward pass (o_rest) the forward also leaves O - bf16(O), as bf16: delta
// = dO . O is subtracted from dP, and O's rounding would stand against no more than
// the spread of dO . v over the keys.  O is then divided by the sum of the rounded
// weights: an error of theirs moves O by its share of v - O, not of v.  (Cost, the
// second sum and the second store: B2 H32 N4096 causal D128 232 -> 263 us, N16384
// 1338 -> 1460, N8192 32 heads D64 586 -> 614.)
//
// Few query rows: where all query heads of a key head fit in one tile (G N_Q <=
// 128) they are packed into it, row g N_Q + n, so that K and V are read once for
// the whole group.  Few tiles: the keys are split over blocks, each writes its
// (m, l, O) in fp32 and a second kernel merges them.
#include "attn.cuh"

namespace skl {
namespace {

constexpr int BM = 128, BN = 128;
constexpr int SOFTMAX_WARPS = 8;
constexpr int PRODUCER_WARP = 8, MMA_WARP = 9, PATCH_WARP = 10;
constexpr int THREADS = 12 * 32;
constexpr int kRegsSoftmax = 200, kRegsOther = 104;  // 256 * 200 + 128 * 104 = 384 * 168 at launch
constexpr uint32_t kTmemCols = 512;
constexpr int kFreshTiles = 16;  // see attn_fwd_kernel's FRESH
constexpr float kSumLimit = 65536.0f;  // 2^16

template <int D>
struct Smem {
  static constexpr int SLOTS = D == 64 ? 8 : 5;  // ring of K and V tiles
  static constexpr int S_BUFS = D == 64 ? 3 : 2;
  static constexpr int TILE = 128 * D * 2;
  static constexpr int OFF_Q = 0;  // Q_A, Q_B
  static constexpr int OFF_KV = 2 * TILE;
  static constexpr int OFF_BAR = OFF_KV + SLOTS * TILE;
  // q_full[2], kv_full[SLOTS], kv_empty[SLOTS], s_full[S_BUFS], p_ready[S_BUFS], o_done[S_BUFS], to_patch, patched; TMEM
  // slot, abort flag
  static constexpr int BAR_SLOT = 8 * (4 + 2 * SLOTS + 3 * S_BUFS);
  static constexpr int BYTES = OFF_BAR + BAR_SLOT + 16 + 1024;
};
static_assert(Smem<64>::BYTES <= kWholeSmSmem && Smem<128>::BYTES <= kWholeSmSmem, "shared memory");

// Sum of 2^(c s - m) over a row's 128 columns; the bf16 pairs of the terms go to pk, with REST their sum to `rounded`
// (MIXED: by additions that take a bf16; which is faster depends on what bounds the loop, N8192 32 heads D64 641 -> 614 us,
// N16384 causal D128 1472 -> 1517).
template <bool REST, bool MIXED>
__device__ __forceinline__ float row_exps(const uint32_t (&s0)[32], const uint32_t (&s1)[32], const uint32_t (&s2)[32],
                                          const uint32_t (&s3)[32], float c, float m, uint32_t (&pk)[64], float& rounded) {
  const float2 cc = make_float2(c, c), nm = make_float2(-m, -m);
  float2 l0 = make_float2(0.f, 0.f), l1 = l0, r0 = l0, r1 = l0;
#pragma unroll
  for (int h = 0; h < 4; ++h) {
    const uint32_t* s = h == 0 ? s0 : h == 1 ? s1 : h == 2 ? s2 : s3;
#pragma unroll
    for (int i = 0; i < 32; i += 4) {
      const float2 x0 = ffma2(make_float2(__uint_as_float(s[i]), __uint_as_float(s[i + 1])), cc, nm);
      const float2 x1 = ffma2(make_float2(__uint_as_float(s[i + 2]), __uint_as_float(s[i + 3])), cc, nm);
      const float2 p0 = make_float2(ex2(x0.x), ex2(x0.y)), p1 = make_float2(ex2(x1.x), ex2(x1.y));
      l0 = fadd2(l0, p0);
      l1 = fadd2(l1, p1);
      pk[h * 16 + i / 2] = pack_bf16(p0.x, p0.y);
      pk[h * 16 + i / 2 + 1] = pack_bf16(p1.x, p1.y);
      if (REST) {
        if (MIXED) {
          add_bf16_pair(r0, pk[h * 16 + i / 2]);
          add_bf16_pair(r1, pk[h * 16 + i / 2 + 1]);
        } else {
          r0 = fadd2(r0, from_bf16_pair(pk[h * 16 + i / 2]));
          r1 = fadd2(r1, from_bf16_pair(pk[h * 16 + i / 2 + 1]));
        }
      }
    }
  }
  if (REST) {
    r0 = fadd2(r0, r1);
    rounded = r0.x + r0.y;
  }
  l0 = fadd2(l0, l1);
  return l0.x + l0.y;
}

// FRESH: a warp whose rows have no reference yet takes the tile's maximum without summing first, which saves 0.5 us of a
// block's first tile; in the loop of a long stream the test costs more (D 64: N1024 causal 24.5 -> 23.4 us, one token and
// 129 keys 7.3 -> 6.8; N8192 518 -> 542).
// REST: the part of O that its rounding leaves is stored too.
template <int D, bool FRESH, bool REST>
__global__ void __launch_bounds__(THREADS, 1)
    attn_fwd_kernel(const AttnProblem p, float* __restrict__ out_lse,
                    float* __restrict__ part_o, float2* __restrict__ part_ml, int* status,
                    const __grid_constant__ CUtensorMap mq, const __grid_constant__ CUtensorMap mk,
                    const __grid_constant__ CUtensorMap mv, const __grid_constant__ CUtensorMap mo,
                    const __grid_constant__ CUtensorMap mrest) {
  using L = Smem<D>;
  constexpr int SLOTS = L::SLOTS, S_BUFS = L::S_BUFS;
  constexpr uint32_t kColO = 128 * S_BUFS;  // O_B follows O_A; S buffer i at 128 i
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = align1024(smem_raw);
  const uint32_t sb = smem_u32(smem);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  // item: (batch, head or key head, pair of query tiles), the longest causal ones first; then the key split, whose
  // tiles are dealt out evenly
  unsigned item = blockIdx.x;
  const int tiles_all = (p.NK + BN - 1) / BN;
  int split = 0, kt0 = 0, kt1 = tiles_all;
  if (p.splits > 1) {
    item = p.by_splits.div(blockIdx.x);
    split = (int)(blockIdx.x - item * (unsigned)p.splits);
    const unsigned each = p.by_splits.div((unsigned)tiles_all), more = (unsigned)tiles_all - each * (unsigned)p.splits;
    kt0 = (int)(split * each + min((unsigned)split, more));
    kt1 = kt0 + (int)(each + ((unsigned)split < more));
  }
  const unsigned x = p.by_items.div(item), y = item - x * p.by_items.d;
  const int qt = p.q_items - 1 - (int)(p.longest_first ? x : y), bh = (int)(p.longest_first ? y : x);
  const int heads = p.packed ? p.HK : p.H;
  const int b = (int)p.by_heads.div(bh), hx = bh - b * heads;  // hx: key head when packed, else query head
  const int hk = p.packed ? hx : (int)p.by_group.div(hx);
  const int ql = seq_len(p.q_lens, b, p.NQ), kl = seq_len(p.k_lens, b, p.NK);
  const int off = kl - ql;
  const int q0 = qt * 2 * BM;
  // key tiles of query tile t within this split
  auto key_tiles = [&](int t) {
    int last;  // last query of the tile
    if (p.packed) {
      if (t) return 0;
      last = ql - 1;
    } else {
      const int first = q0 + t * BM;
      if (first >= ql) return 0;
      last = min(first + BM, ql) - 1;
    }
    const int end = p.causal ? min(kl, last + off + 1) : kl;
    if (last < 0 || end <= 0) return 0;
    return max(0, min(kt1, (end + BN - 1) / BN) - kt0);
  };
  const int nA = key_tiles(0), nB = key_tiles(1);
  const int n = max(nA, nB);
  // A pair's three barriers (S there, P there, its product done) go with its S buffer: nobody can be two uses behind or
  // ahead of one, as the phases' parities require.
  // The tile pairs in the order in which they are worked on: A0, B0, A1, B1, ... and then what is left of the longer tile.
  const int both = min(nA, nB);
  auto pair_of = [&](int t, int i) { return i < both ? 2 * i + t : both + i; };
  auto buf_of = [&](int t, int i) { return S_BUFS == 2 ? t : pair_of(t, i) % 3; };       // its S buffer,
  auto use_of = [&](int t, int i) { return S_BUFS == 2 ? i : pair_of(t, i) / 3; };       // and how often it was used before
  const bool has_b = !p.packed && q0 + BM < p.NQ;
  // the V tile that a sequence ends inside: its rows past the end may hold anything, and 0 * NaN is NaN
  const int patch_i = (kl < p.NK && (kl & (BN - 1))) ? (kl / BN) - kt0 : -1;

  const uint32_t bar = sb + L::OFF_BAR;
  const uint32_t q_full = bar, kv_full = bar + 16, kv_empty = kv_full + 8 * SLOTS, s_full = kv_empty + 8 * SLOTS,
                 p_ready = s_full + 8 * S_BUFS, o_done = p_ready + 8 * S_BUFS, to_patch = o_done + 8 * S_BUFS, patched = to_patch + 8;
  const uint32_t slot = bar + L::BAR_SLOT;
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + L::OFF_BAR + L::BAR_SLOT + 4);

  const uint32_t q_bytes = (p.packed ? (uint32_t)(p.G * p.NQ) : (uint32_t)BM) * D * 2;
  auto load_kv = [&](int u) {  // K(0), V(0), K(1), ...
    const int s = u % SLOTS;
    mbar_arrive_expect_tx(kv_full + 8 * s, L::TILE);
#pragma unroll
    for (int h = 0; h < D / 64; ++h)
      tma_load_4d(sb + L::OFF_KV + s * L::TILE + h * BN * 128, (u & 1) ? &mv : &mk, kv_full + 8 * s, h * 64,
                  (kt0 + (u >> 1)) * BN, hk, b);
  };
  if (warp == PRODUCER_WARP) {
    if (elect_one()) {
      for (int t = 0; t < 2; ++t) {
        mbar_init(q_full + 8 * t, 1);
      }
      for (int s = 0; s < S_BUFS; ++s) {
        mbar_init(s_full + 8 * s, 1);
        mbar_init(p_ready + 8 * s, SOFTMAX_WARPS / 2);
        mbar_init(o_done + 8 * s, 1);
      }
      for (int s = 0; s < SLOTS; ++s) {
        mbar_init(kv_full + 8 * s, 1);
        mbar_init(kv_empty + 8 * s, 1);
      }
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

  if (warp >= SOFTMAX_WARPS) {
    setmaxnreg_dec<kRegsOther>();
    if (warp == PRODUCER_WARP) {
      if (n > 0 && elect_one()) {
        for (int t = 0; t < 2; ++t) {
          if ((t ? nB : nA) == 0) continue;
          mbar_arrive_expect_tx(q_full + 8 * t, q_bytes);
#pragma unroll
          for (int h = 0; h < D / 64; ++h)
            tma_load_4d(sb + L::OFF_Q + t * L::TILE + h * BM * 128, &mq, q_full + 8 * t, h * 64,
                        p.packed ? 0 : q0 + t * BM, p.packed ? hk * p.G : hx, b);
          if (t == 0 || nA == 0) load_kv(0);
        }
        for (int u = 1; u < min(SLOTS, 2 * n); ++u) load_kv(u);
        int issued = min(SLOTS, 2 * n);
        for (int u = SLOTS; u < 2 * n; ++u) {
          if (!mbar_wait(kv_empty + 8 * (u % SLOTS), ((u / SLOTS) - 1) & 1, status, abort_flag)) break;
          load_kv(u);
          issued = u + 1;
        }
        // copies that may still be landing
        if (nA > 0) mbar_drain(q_full, 0, status);
        if (nB > 0) mbar_drain(q_full + 8, 0, status);
        for (int u = max(0, issued - SLOTS); u < issued; ++u)
          mbar_drain(kv_full + 8 * (u % SLOTS), (u / SLOTS) & 1, status);
      }
      __syncwarp();
    } else if (warp == PATCH_WARP) {
      if (patch_i >= 0 && patch_i < n) {
        // the MMA thread, which follows the ring's phases, says when the tile is there
        const int s = (2 * patch_i + 1) % SLOTS;
        if (mbar_wait_warp(to_patch, 0, status, abort_flag)) {
          const int from = kl & (BN - 1);
          for (int i = lane; i < (BN - from) * (D / 8); i += 32) {
            const int r = from + i / (D / 8);
            st_shared_zero16(sw128<BN>(sb + L::OFF_KV + s * L::TILE, r, i % (D / 8)));
          }
          fence_async_smem();
          __syncwarp();
          arrive_one(patched);
        }
      }
      __syncwarp();
    } else if (warp == MMA_WARP) {
      if (n > 0 && elect_one()) {
        constexpr uint32_t id_s = idesc_bf16(BM, BN, false, false);
        constexpr uint32_t id_o = idesc_bf16(BM, D, false, true);
        const int nt[2] = {nA, nB};
        bool ok = true;
        auto issue_s = [&](int t, int i) {  // S_t(i) = Q_t K(i)^T
          const int u = 2 * i, s = u % SLOTS, buf = buf_of(t, i);
          if (i == 0 && !mbar_wait(q_full + 8 * t, 0, status, abort_flag)) return false;
          if (!mbar_wait(kv_full + 8 * s, (u / SLOTS) & 1, status, abort_flag)) return false;
          tc_fence_after();
          const uint64_t qd = sdesc_sw128(sb + L::OFF_Q + t * L::TILE, 0, 1024);
          const uint64_t kd = sdesc_sw128(sb + L::OFF_KV + s * L::TILE, 0, 1024);
#pragma unroll
          for (int ks = 0; ks < D / 16; ++ks) {
            const uint32_t o = (ks >> 2) * (128 * 128) + (ks & 3) * 32;
            mma_ss(tmem + 128 * buf, sdesc_add(qd, o), sdesc_add(kd, o), id_s, ks > 0);
          }
          mma_commit(s_full + 8 * buf);
          if (t == 1 || i >= nB) mma_commit(kv_empty + 8 * s);  // K(i) is read by no later tile
          return true;
        };
        auto issue_o = [&](int t, int i) {  // O_t += P_t(i) V(i)
          const int u = 2 * i + 1, s = u % SLOTS;
          if (!mbar_wait(kv_full + 8 * s, (u / SLOTS) & 1, status, abort_flag)) return false;
          if (i == patch_i) {
            if (t == 0 || i >= nA) mbar_arrive(to_patch);  // the first of the tiles that read it
            if (!mbar_wait(patched, 0, status, abort_flag)) return false;
          }
          const int buf = buf_of(t, i);
          if (!mbar_wait(p_ready + 8 * buf, use_of(t, i) & 1, status, abort_flag)) return false;
          tc_fence_after();
          const uint64_t vd = sdesc_sw128(sb + L::OFF_KV + s * L::TILE, BN * 128, 1024);
#pragma unroll
          for (int ks = 0; ks < BN / 16; ++ks)
            mma_ts(tmem + kColO + D * t, tmem + 128 * buf + 8 * ks, sdesc_add(vd, ks * 2048), id_o, i > 0 || ks > 0);
          if (t == 1 || i >= nB) mma_commit(kv_empty + 8 * s);
          mma_commit(o_done + 8 * buf);  // last: the block leaves once it has arrived
          return true;
        };
        // tile A has the key tiles [0, nA), tile B [0, nB); B is the last to read a tile both have, and where
        // only A reads it (i >= nB) A is.  Where only B reads it (i >= nA) the same rule holds.
        if constexpr (S_BUFS == 3) {
          // S runs three tile pairs ahead: its buffer is free when the product three pairs before has been issued
          const int all = nA + nB, longer = nA > nB ? 0 : 1;
          auto tile_of = [&](int k) { return k < 2 * both ? k & 1 : longer; };
          auto key_of = [&](int k) { return k < 2 * both ? k >> 1 : k - both; };
          for (int k = 0; ok && k < min(3, all); ++k) ok = issue_s(tile_of(k), key_of(k));
          for (int k = 0; ok && k < all; ++k) {
            ok = issue_o(tile_of(k), key_of(k));
            if (ok && k + 3 < all) ok = issue_s(tile_of(k + 3), key_of(k + 3));
          }
        } else {
          for (int t = 0; ok && t < 2; ++t)
            if (nt[t] > 0) ok = issue_s(t, 0);
          for (int i = 0; ok && i < n; ++i) {
            for (int t = 0; ok && t < 2; ++t) {
              if (i < nt[t]) ok = issue_o(t, i);
              if (ok && i + 1 < nt[t]) ok = issue_s(t, i + 1);
            }
          }
        }
        if (ok)
          for (int t = 0; t < 2; ++t)
            if (nt[t] > 0) mbar_drain(o_done + 8 * buf_of(t, nt[t] - 1), use_of(t, nt[t] - 1) & 1, status);
      }
      __syncwarp();
    }
  } else {
    setmaxnreg_inc<kRegsSoftmax>();
    // -------------------------------------------------------------- softmax
    const int t = warp >> 2, wq = warp & 3;
    const int r = wq * 32 + lane;
    const int nt = t ? nB : nA;
    const int g = p.packed ? r / p.NQ : 0;
    const int qn = p.packed ? r - g * p.NQ : q0 + t * BM + r;  // query position of this row
    const int h = p.packed ? hk * p.G + g : hx;
    const bool real = p.packed ? (t == 0 && g < p.G) : (qn < p.NQ);
    const int row_end = (real && qn < ql) ? (p.causal ? min(kl, qn + off + 1) : kl) : 0;  // keys this row sees
    const uint32_t lanes = (uint32_t)(wq * 32) << 16;
    const uint32_t to = tmem + lanes + kColO + D * t;
    const float c = p.c;
    float m = kNegInf, l = 0.f, lr = 0.f;  // lr (REST): the sum of the rounded weights
    bool ok = true, started = false;  // started: some row of the warp has a reference
    for (int i = 0; i < nt; ++i) {
      const int buf = buf_of(t, i);
      const uint32_t ts = tmem + lanes + 128 * buf;
      ok = mbar_wait_warp(s_full + 8 * buf, use_of(t, i) & 1, status, abort_flag);
      __syncwarp();
      if (!ok) break;
      tc_fence_after();
      const int seen = row_end - (kt0 + i) * BN;  // columns this row sees: [0, seen)
      const bool masked = __any_sync(0xffffffffu, seen < BN);
      uint32_t s0[32], s1[32], s2[32], s3[32], pk[64];
      auto load_s = [&]() {
        tmem_ld32(ts, s0);
        tmem_ld32(ts + 32, s1);
        tmem_ld32(ts + 64, s2);
        tmem_ld32(ts + 96, s3);
        tmem_ld_wait();
        reg_fence32(s0);
        reg_fence32(s1);
        reg_fence32(s2);
        reg_fence32(s3);
        if (masked) {
#pragma unroll
          for (int k = 0; k < 32; ++k) {
            if (k >= seen) s0[k] = __float_as_uint(kNegInf);
            if (k + 32 >= seen) s1[k] = __float_as_uint(kNegInf);
            if (k + 64 >= seen) s2[k] = __float_as_uint(kNegInf);
            if (k + 96 >= seen) s3[k] = __float_as_uint(kNegInf);
          }
        }
      };
      // move: a row without a reference that sees keys here, or whose terms grew too large (inf and NaN included)
      float sum = 0.f, rounded = 0.f;
      bool move = m == kNegInf && seen > 0;
      if (!FRESH || started || !__any_sync(0xffffffffu, move)) {
        load_s();
        sum = row_exps<REST, D == 64>(s0, s1, s2, s3, c, m == kNegInf ? 0.f : m, pk, rounded);
        move = m == kNegInf ? seen > 0 : !(sum < kSumLimit);
      }
      if (__any_sync(0xffffffffu, move)) {
        load_s();
        float mx = kNegInf;
#pragma unroll
        for (int k = 0; k < 32; ++k) {
          mx = fmax3(mx, __uint_as_float(s0[k]), __uint_as_float(s1[k]));
          mx = fmax3(mx, __uint_as_float(s2[k]), __uint_as_float(s3[k]));
        }
        const float m2 = move ? fmaxf(m, mx * c) : m;
        const float w = m == kNegInf ? 0.f : ex2(m - m2);
        m = m2;
        l *= w;
        if (REST) lr *= w;
        if (FRESH) started = __any_sync(0xffffffffu, m != kNegInf);
        sum = row_exps<REST, D == 64>(s0, s1, s2, s3, c, m == kNegInf ? 0.f : m, pk, rounded);
        if (i > 0) {
          ok = mbar_wait_warp(o_done + 8 * buf_of(t, i - 1), use_of(t, i - 1) & 1, status, abort_flag);
          __syncwarp();
          if (!ok) break;
          tc_fence_after();
#pragma unroll 1
          for (int d = 0; d < D; d += 32) {
            __syncwarp();
            tmem_ld32(to + d, s0);
            tmem_ld_wait();
            reg_fence32(s0);
#pragma unroll
            for (int k = 0; k < 32; ++k) s0[k] = __float_as_uint(__uint_as_float(s0[k]) * w);
            tmem_st32(to + d, s0);
          }
        }
      }
      l += sum;
      if (REST) lr += rounded;
      __syncwarp();
#pragma unroll
      for (int q = 0; q < 4; ++q) tmem_st16(ts + 16 * q, *reinterpret_cast<const uint32_t(*)[16]>(&pk[16 * q]));
      tmem_st_wait();
      tc_fence_before();
      __syncwarp();
      arrive_one(p_ready + 8 * buf);
    }
    if (nt > 0 && ok) {
      ok = mbar_wait_warp(o_done + 8 * buf_of(t, nt - 1), use_of(t, nt - 1) & 1, status, abort_flag);
      __syncwarp();
    }
    if (t == 0 || has_b) {
      const size_t row = ((size_t)b * p.H + h) * p.NQ + qn;
      const bool nan = l != l;
      // a row that sees no key: zeros.  The splits' partials are weighed by their l, so theirs are O l / lr
      const float f = nan ? l : l > 0.f ? (REST && p.splits > 1 ? l : 1.f) / (REST ? lr : l) : 0.f;
      if (ok) {
        tc_fence_after();
        if (real && p.splits > 1)
          part_ml[(size_t)split * p.rows + row] = make_float2(m, l);
        else if (real)
          out_lse[row] = (l > 0.f || nan) ? (m + log2f(l)) * kLn2 : kNegInf;
#pragma unroll 1
        for (int d = 0; d < D; d += 32) {
          uint32_t o[32];
          __syncwarp();  // rows differ in what they do above; the load wants the whole warp
          if (nt > 0) {
            tmem_ld32(to + d, o);
            tmem_ld_wait();
            reg_fence32(o);
          }
          if (!(l > 0.f) && !nan) {
#pragma unroll
            for (int k = 0; k < 32; ++k) o[k] = 0;
          }
          if (p.splits == 1) {
            stage_row32(sb + L::OFF_Q + t * L::TILE, r, d, o, f);  // Q's products are done
          } else {
            // through the warp's share of the Q tile: eight lanes write a row's 128 bytes (a lane that writes its own row
            // scatters every store over 32 lines: 6400 cycles a 128 x 128 tile)
            const uint32_t stage = sb + L::OFF_Q + t * L::TILE + wq * 4096;
            if (REST) {
#pragma unroll
              for (int k = 0; k < 32; ++k) o[k] = __float_as_uint(__uint_as_float(o[k]) * f);
            }
            __syncwarp();
#pragma unroll
            for (int k = 0; k < 8; ++k)
              st_shared16(stage + lane * 128 + ((k ^ (lane & 7)) << 4),
                          make_uint4(o[4 * k], o[4 * k + 1], o[4 * k + 2], o[4 * k + 3]));
            __syncwarp();
            const long long mine = real ? (long long)row : -1;
#pragma unroll
            for (int k = 0; k < 8; ++k) {
              const int y = 4 * k + (lane >> 3);
              const long long to_row = __shfl_sync(0xffffffffu, mine, y);
              const uint4 v = ld_shared16(stage + y * 128 + (((lane ^ y) & 7) << 4));
              if (to_row >= 0)
                reinterpret_cast<uint4*>(part_o + ((size_t)split * p.rows + to_row) * D + d)[lane & 7] = v;
            }
          }
        }
        fence_async_smem();
      }
      // every warp of the tile comes here; one that gave up makes none of them store
      const bool store = !named_bar_any(1 + t, SOFTMAX_WARPS / 2 * 32, !ok) && p.splits == 1;
      if (store && wq == 0) {
        if (elect_one())
          store_tile<D>(&mo, sb + L::OFF_Q + t * L::TILE, p.packed ? 0 : q0 + t * BM, p.packed ? hk * p.G : hx, b);
        __syncwarp();
      }
      if (REST && store) {  // the rest through the same tile, once the copy has read it
        named_bar_sync(1 + t, SOFTMAX_WARPS / 2 * 32);
#pragma unroll 1
        for (int d = 0; d < D; d += 32) {
          uint32_t o[32];
          __syncwarp();
          if (nt > 0) {
            tmem_ld32(to + d, o);
            tmem_ld_wait();
            reg_fence32(o);
          }
#pragma unroll
          for (int k = 0; k < 32; ++k) {
            const float x = l > 0.f || nan ? __uint_as_float(o[k]) * f : 0.f;
            o[k] = __float_as_uint(bf16_rest(x));
          }
          stage_row32(sb + L::OFF_Q + t * L::TILE, r, d, o, 1.f);
        }
        fence_async_smem();
        named_bar_sync(1 + t, SOFTMAX_WARPS / 2 * 32);
        if (wq == 0) {
          if (elect_one())
            store_tile<D>(&mrest, sb + L::OFF_Q + t * L::TILE, p.packed ? 0 : q0 + t * BM, p.packed ? hk * p.G : hx, b);
          __syncwarp();
        }
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == MMA_WARP) {
    tc_fence_after();
    tmem_dealloc(tmem, kTmemCols);
  }
}

// Merges the splits' (m, l, O), a block to a row: the weights with a thread to a split, then O with a warp to every eighth
// split, whose first loads are on their way before the weights are known.  Bound by the two trips to L2 (a warp to a row
// with one split after the other took 16 us for 19 splits, this 4).
constexpr int kMergeWarps = 8, kMergeAhead = 2;
constexpr int kMaxSplits = 1024;  // the plan makes at most four blocks an SM
template <int D>
__global__ void __launch_bounds__(kMergeWarps * 32)
    attn_merge_kernel(const AttnProblem p, const float* __restrict__ part_o, const float2* __restrict__ part_ml,
                      __nv_bfloat16* __restrict__ out, float* __restrict__ out_lse) {
  constexpr int W = D / 32;  // columns of a lane
  struct alignas(W * 4) Cols {
    float x[W];
  };
  __shared__ float weight[kMaxSplits], warp_m[kMergeWarps], warp_l[kMergeWarps];
  __shared__ Cols sums[kMergeWarps][32];
  const long long row = blockIdx.x;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  auto load = [&](int s) { return *(reinterpret_cast<const Cols*>(part_o + ((size_t)s * p.rows + row) * D) + lane); };
  Cols first[kMergeAhead];
#pragma unroll
  for (int k = 0; k < kMergeAhead; ++k)
    if (warp + k * kMergeWarps < p.splits) first[k] = load(warp + k * kMergeWarps);
  float m = kNegInf;
  for (int s = threadIdx.x; s < p.splits; s += kMergeWarps * 32) m = fmaxf(m, part_ml[(size_t)s * p.rows + row].x);
#pragma unroll
  for (int w = 16; w; w >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, w));
  if (lane == 0) warp_m[warp] = m;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < kMergeWarps; ++w) m = fmaxf(m, warp_m[w]);
  float l = 0.f;
  for (int s = threadIdx.x; s < p.splits; s += kMergeWarps * 32) {
    const float2 ml = part_ml[(size_t)s * p.rows + row];
    const bool none = ml.x == kNegInf && ml.y == 0.f;  // this split has no key for the row
    const float w = none ? 0.f : ml.x == m ? 1.f : ex2(ml.x - m);
    weight[s] = w;
    l += none ? 0.f : w * ml.y;
  }
#pragma unroll
  for (int w = 16; w; w >>= 1) l += __shfl_xor_sync(0xffffffffu, l, w);
  if (lane == 0) warp_l[warp] = l;
  __syncthreads();
  l = 0.f;
#pragma unroll
  for (int w = 0; w < kMergeWarps; ++w) l += warp_l[w];
  Cols o{};
  auto add = [&](int s, const Cols& x) {
#pragma unroll
    for (int i = 0; i < W; ++i) o.x[i] = fmaf(weight[s], x.x[i], o.x[i]);
  };
#pragma unroll
  for (int k = 0; k < kMergeAhead; ++k)
    if (warp + k * kMergeWarps < p.splits) add(warp + k * kMergeWarps, first[k]);
  for (int s = warp + kMergeAhead * kMergeWarps; s < p.splits; s += kMergeWarps) add(s, load(s));
  sums[warp][lane] = o;
  __syncthreads();
  const bool none = l == 0.f;
  if (threadIdx.x == 0) out_lse[row] = none ? kNegInf : (m + log2f(l)) * kLn2;
  if (warp != 0) return;
#pragma unroll
  for (int w = 1; w < kMergeWarps; ++w) {
    const Cols x = sums[w][lane];
#pragma unroll
    for (int i = 0; i < W; ++i) o.x[i] += x.x[i];
  }
  const float inv = none ? 0.f : 1.f / l;
  const long long bh = row / p.NQ;
  const long long at = (bh / p.H) * p.os_b + (bh % p.H) * p.os_h + (row % p.NQ) * p.os_n + lane * W;
#pragma unroll
  for (int k = 0; k < W; k += 2) *reinterpret_cast<uint32_t*>(out + at + k) = pack_bf16(o.x[k] * inv, o.x[k + 1] * inv);
  if (p.o_rest) {
    auto* rest = static_cast<__nv_bfloat16*>(p.o_rest);
#pragma unroll
    for (int k = 0; k < W; k += 2)
      *reinterpret_cast<uint32_t*>(rest + at + k) = pack_bf16(bf16_rest(o.x[k] * inv), bf16_rest(o.x[k + 1] * inv));
  }
}

template <int D>
cudaError_t launch_d(const AttnProblem& p, const void* q, const void* k, const void* v, void* o, float* lse,
                     void* workspace, int* status, cudaStream_t st) {
  CUtensorMap mq, mk, mv, mo, mrest{};
  if (!encode_tile_map(&mq, q, p.D, p.NQ, p.H, p.B, p.qs_n, p.qs_h, p.qs_b, p.packed ? p.NQ : BM, p.packed ? p.G : 1) ||
      !encode_tile_map(&mk, k, p.D, p.NK, p.HK, p.B, p.ks_n, p.ks_h, p.ks_b, BN) ||
      !encode_tile_map(&mv, v, p.D, p.NK, p.HK, p.B, p.vs_n, p.vs_h, p.vs_b, BN) ||
      !encode_tile_map(&mo, o, p.D, p.NQ, p.H, p.B, p.os_n, p.os_h, p.os_b, p.packed ? p.NQ : BM, p.packed ? p.G : 1) ||
      (p.o_rest && !encode_tile_map(&mrest, p.o_rest, p.D, p.NQ, p.H, p.B, p.os_n, p.os_h, p.os_b, p.packed ? p.NQ : BM,
                                    p.packed ? p.G : 1)))
    return cudaErrorInvalidValue;
  constexpr int smem = kWholeSmSmem;
  const bool fresh = D == 64 && ((p.NK + BN - 1) / BN + p.splits - 1) / p.splits <= kFreshTiles;
  const auto kern = p.o_rest ? (fresh ? attn_fwd_kernel<D, D == 64, true> : attn_fwd_kernel<D, false, true>)
                             : (fresh ? attn_fwd_kernel<D, D == 64, false> : attn_fwd_kernel<D, false, false>);
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) return e;
  float* part_o = static_cast<float*>(workspace);
  float2* part_ml = p.splits > 1 ? reinterpret_cast<float2*>(part_o + (size_t)p.splits * p.rows * D) : nullptr;
  auto* out = static_cast<__nv_bfloat16*>(o);
  const long long blocks = attn_fwd_items(p) * p.splits;
  kern<<<(unsigned)blocks, THREADS, smem, st>>>(p, lse, part_o, part_ml, status, mq, mk, mv, mo, mrest);
  if ((e = cudaGetLastError()) != cudaSuccess || p.splits == 1) return e;
  attn_merge_kernel<D><<<(unsigned)p.rows, kMergeWarps * 32, 0, st>>>(p, part_o, part_ml, out, lse);
  return cudaGetLastError();
}

// No keys at all: O = 0, LSE = -inf.
__global__ void attn_no_keys_kernel(const AttnProblem p, __nv_bfloat16* out, float* lse) {
  const long long row = blockIdx.x;
  const long long bh = row / p.NQ;
  const long long at = (bh / p.H) * p.os_b + (bh % p.H) * p.os_h + (row % p.NQ) * p.os_n + threadIdx.x;
  out[at] = __float2bfloat16_rn(0.f);
  if (p.o_rest) static_cast<__nv_bfloat16*>(p.o_rest)[at] = __float2bfloat16_rn(0.f);
  if (threadIdx.x == 0) lse[row] = kNegInf;
}

}  // namespace

long long attn_fwd_items(const AttnProblem& p) {
  return (long long)p.B * (p.packed ? p.HK : p.H) * p.q_items;
}

// In times of a key tile (1.5 us where a block has one tile of rows, and its K and V are new): setting a block up and
// storing its tile take kBlockCost, the second launch with the partials' round trip through L2 kMergeCost.  Measured, one
// query and 8 heads of D 128, us by key tiles of a block: 4096 keys 14.6 with 4, 11.6 with 2, 10.7 with 1; 512 keys 11.0 with
// all 4 and no merge.  A split's partials cost another tile time for each kMergedPerTile values (B1 H8 N512 D128 causal, 4096
// rows, 11.7 whole, 15.2 with 4 splits).
constexpr double kBlockCost = 3.0, kMergeCost = 2.5, kMergedPerTile = 1.5e6;
constexpr int kSmallGrid = 6;
void attn_fwd_plan(AttnProblem* p, int num_sms) {
  p->packed = (long long)p->G * p->NQ <= BM;
  p->q_items = p->packed ? 1 : (p->NQ + 2 * BM - 1) / (2 * BM);
  p->rows = (long long)p->B * p->H * p->NQ;
  const long long items = attn_fwd_items(*p);
  const int tiles = (p->NK + BN - 1) / BN;
  // the split count that needs the fewest tile times: waves of blocks; more splits only for a gain
  int best = 1;
  double cost = (double)((items + num_sms - 1) / num_sms) * (tiles + kBlockCost);
  for (int s = 2; s <= tiles && s <= kMaxSplits && items * s <= 4ll * num_sms; ++s) {
    const double c = (double)((items * s + num_sms - 1) / num_sms) * ((tiles + s - 1) / s + kBlockCost) + kMergeCost +
                     (double)p->rows * s * p->D / kMergedPerTile;
    if (c < cost) {
      cost = c;
      best = s;
    }
  }
  p->splits = best;
  // in a grid of few waves the order of lengths counts for more than the L2 (whose reuse a head-major order is for)
  p->longest_first = items * best <= kSmallGrid * num_sms;
  const unsigned heads = p->packed ? p->HK : p->H;
  p->by_splits = FastDiv((unsigned)p->splits);
  p->by_items = FastDiv(p->longest_first ? p->B * heads : (unsigned)p->q_items);
  p->by_heads = FastDiv(heads);
  p->by_group = FastDiv((unsigned)p->G);
}

size_t attn_fwd_workspace(const AttnProblem& p) {
  return p.splits > 1 ? (size_t)p.splits * p.rows * (p.D + 2) * sizeof(float) : 0;
}

cudaError_t launch_attn_fwd(const AttnProblem& p, const void* q, const void* k, const void* v, void* o, float* lse,
                            void* workspace, int* status, cudaStream_t st) {
  if (p.NK == 0) {
    attn_no_keys_kernel<<<(unsigned)p.rows, p.D, 0, st>>>(p, static_cast<__nv_bfloat16*>(o), lse);
    return cudaGetLastError();
  }
  if (p.D == 64) return launch_d<64>(p, q, k, v, o, lse, workspace, status, st);
  return launch_d<128>(p, q, k, v, o, lse, workspace, status, st);
}

}  // namespace skl
