/*
 * libstreamkl — fused attention KL divergence for one GB300 GPU (sm_103a).
 *
 * For every (batch b, head h, query row i) the library computes
 *
 *     S_t = scale * Q_t K_t^T,  P_t = row-softmax(S_t)   (t = 1 teacher, t = 2 student)
 *     KL_i = sum_j P1_ij (log P1_ij - log P2_ij)           i.e. KL(P1 || P2)
 *     LSE_t,i = log sum_j exp(S_t,ij)
 *
 * over the keys j that the (optional) causal mask keeps, without ever writing
 * an N_Q x N_K matrix to memory.  The forward is the one-pass online
 * formulation with five running scalars per row (m1, m2, l1, l2, acc) and the
 * closing identity KL = acc/l1 + LSE2 - LSE1 (StreamKL technical summary,
 * gist.science/ja/paper/2606.20005, section 手法 1 "online formulation").  The
 * backward rebuilds P_t = exp(S_t - LSE_t) tile by tile from Q, K and the saved
 * LSE (section 手法 2 "recompute strategy") in the two settings named there.
 *
 * Conventions shared by every entry point
 * ---------------------------------------
 * - Q_t are [B, H, N_Q, D] and K_t are [B, H, N_K, D], bf16, DEVICE
 *   pointers, 16-byte aligned, contiguous unless the shape's strides say
 *   otherwise (see streamkl_shape).  D is 64 or 128.
 * - Row outputs and inputs (KL, LSE1, LSE2, g) are fp32 [B, H, N_Q], device.
 * - Gradient outputs are bf16 in the layout of the tensor they belong to.
 * - scale <= 0 selects 1/sqrt(D).  causal != 0 keeps key j for row i iff
 *   j <= i + N_K - N_Q (bottom-right alignment); causal with N_Q > N_K is
 *   rejected so that no row is left without keys.
 * - The caller owns every buffer; the library allocates no device memory.
 *   Scratch memory is passed in as a workspace whose size is queried first.
 *   The one exception is streamkl_fwd_splitk_noalloc, whose scratch is a
 *   fixed static device array inside the library.
 * - `stream` is a cudaStream_t (NULL = the legacy default stream).  Calls are
 *   asynchronous on it.  Argument errors are returned synchronously before
 *   anything is launched.  Launch failures return STREAMKL_ERR_CUDA.
 * - Device-side waits are bounded.  A wait that runs out sets a device status
 *   word instead of hanging; streamkl_check_device_status() reads it.
 * - No C++ exception crosses this interface.
 */
#ifndef STREAMKL_H
#define STREAMKL_H

#include <stddef.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
  STREAMKL_OK = 0,
  STREAMKL_ERR_INVALID = 1,     /* bad shape, null/misaligned pointer, causal with N_Q > N_K */
  STREAMKL_ERR_UNSUPPORTED = 2, /* valid but not handled (e.g. D not in {64,128}, Split-K N_Q > 16) */
  STREAMKL_ERR_WORKSPACE = 3,   /* workspace pointer missing, misaligned or too small */
  STREAMKL_ERR_CUDA = 4,        /* a CUDA runtime/driver call failed (launch, memset, tensor map) */
  STREAMKL_ERR_TIMEOUT = 5,     /* a bounded device-side wait ran out (reported by check_device_status) */
  STREAMKL_ERR_SCRATCH_LIMIT = 6 /* needs more than the fixed scratch of streamkl_fwd_splitk_noalloc */
} streamkl_status;

/*
 * Problem shape.  scale <= 0 means 1/sqrt(D).
 *
 * q_stride_* and k_stride_* are ELEMENT strides along b, h and n of the
 * logical [B, H, N, D] views of Q1/Q2 and of K1/K2 (D itself is contiguous).
 * All three zero selects the contiguous [B, H, N, D] layout; otherwise each is
 * positive and a multiple of 8 (16 bytes), n's stride is at least D, and both
 * tensors of a pair (Q1 and Q2, K1 and K2) share the strides.  A [B, N, H, D]
 * tensor, as many attention implementations store it, is passed without a
 * copy as strides (N*H*D, D, H*D).  Gradient outputs (dQ, dK) are written
 * with the strides of the input they belong to, so those strides must not
 * make two rows overlap (inputs are only read and may overlap); row-shaped
 * tensors (KL, LSE, g) stay contiguous [B, H, N_Q].
 */
typedef struct {
  int B, H, NQ, NK, D;
  float scale;
  int causal;
  long long q_stride_b, q_stride_h, q_stride_n;
  long long k_stride_b, k_stride_h, k_stride_n;
} streamkl_shape;

/* Backward path selection (the adaptive rule of section 手法 2 "kernel fusion"). */
typedef enum {
  STREAMKL_BWD_AUTO = 0,     /* the rule of streamkl_bwd_select */
  STREAMKL_BWD_FUSED = 1,    /* one pass over each QK tile pair, dQ on chip, dK by atomics into fp32 */
  STREAMKL_BWD_SEPARATE = 2, /* a Q-stationary dQ kernel and a K-stationary dK kernel */
  STREAMKL_BWD_DQ_ONLY = 3,  /* separate path, dQ kernel only (dK pointer may be NULL) */
  STREAMKL_BWD_DK_ONLY = 4   /* separate path, dK kernel only (dQ pointer may be NULL) */
} streamkl_bwd_mode;

/* Largest N_Q the Split-K forward takes. */
#define STREAMKL_SPLITK_MAX_NQ 16

/*
 * Forward: KL, LSE1, LSE2 [B,H,N_Q] fp32 from bf16 Q1, K1, Q2, K2.
 * (technical summary, 手法 1 "online formulation": five running scalars,
 *  KL = acc/l1 + LSE2 - LSE1, whole key tiles past the causal boundary skipped.)
 * One CTA owns a tile of query rows and streams every key tile it needs.
 */
streamkl_status streamkl_fwd(const void* q1, const void* k1, const void* q2, const void* k2,
                             streamkl_shape s, float* kl, float* lse1, float* lse2, void* stream);

/*
 * Split-K forward for few query rows (decode, N_Q <= STREAMKL_SPLITK_MAX_NQ).
 * (technical summary, 手法 3 "Split-K variant": the key dimension is divided
 *  over thread blocks so that a small N_Q still fills the SMs.)
 * Each of `num_splits` blocks per (b, h) reduces a contiguous key range to the
 * five partial scalars per row; a second kernel merges them.  num_splits = 0
 * picks a count that fills the GPU.  Workspace: fp32 [B,H,N_Q,splits,5], size
 * from streamkl_fwd_splitk_workspace(), 16-byte aligned, contents ignored.
 */
streamkl_status streamkl_fwd_splitk_workspace(streamkl_shape s, int num_splits, size_t* bytes);
streamkl_status streamkl_fwd_splitk(const void* q1, const void* k1, const void* q2, const void* k2,
                                    streamkl_shape s, int num_splits, void* workspace,
                                    size_t workspace_bytes, float* kl, float* lse1, float* lse2,
                                    void* stream);
/*
 * The split count num_splits = 0 resolves to, for a GPU with `num_sms` SMs
 * (num_sms <= 0: the current device).  It minimises waves x (tiles per block
 * + a fixed per-block cost); with num_sms > 0 it is a pure host computation.
 */
streamkl_status streamkl_fwd_splitk_plan(streamkl_shape s, int num_sms, int* num_splits);

/*
 * Split-K forward that allocates nothing and takes no workspace.  The paper
 * has no counterpart of this entry point; it exists for callers that cannot
 * call cudaMalloc or hand out scratch memory -- code that runs inside a host
 * application or serving runtime owning all device memory, or a decode loop
 * whose memory budget is fixed before it starts.  The caller still passes the
 * inputs and outputs.
 *
 * The per-split partial states live in one static device array of
 * STREAMKL_NOALLOC_SCRATCH_BYTES built into the library; every GPU that loads
 * the library keeps it until the process exits.  A problem whose partials
 * (B*H*N_Q*splits*5 floats) do not fit returns STREAMKL_ERR_SCRATCH_LIMIT with
 * nothing launched.  All calls share that array and it keeps the last call's
 * contents: a call that completes writes every partial it then reads, so
 * nothing needs clearing.  If one of its bounded waits runs out, a partial
 * block stops without writing and the merge reads what an earlier call left
 * there, so the outputs are valid only when streamkl_check_device_status
 * returns STREAMKL_OK afterwards.  Calls that overlap on the GPU -- on
 * different streams, or from different host threads -- race on the array
 * and must be serialised by the caller.
 * The first call on a device looks up the array's device address with that
 * device current (once per device); make that first call before any stream
 * capture.  Results equal streamkl_fwd_splitk's for the same num_splits.
 */
#define STREAMKL_NOALLOC_SCRATCH_BYTES (4u << 20)
streamkl_status streamkl_fwd_splitk_noalloc(const void* q1, const void* k1, const void* q2, const void* k2,
                                            streamkl_shape s, int num_splits, float* kl, float* lse1,
                                            float* lse2, void* stream);

/*
 * Key shards (context parallelism): the keys of a long sequence split into
 * contiguous ranges, e.g. one per GPU, every range seen by every query row.
 * (technical summary, 手法 3 "Split-K variant": a key range reduces to five
 *  scalars per row and ranges merge exactly; the pages split over thread
 *  blocks, here the same algebra splits over devices.)
 *
 * In each of these calls s.NK is the shard's key count and K1, K2 point at the
 * shard's rows (any strides the shape allows, so a row slice of a larger
 * [B, H, N, D] tensor is passed as is), which are the keys at global positions
 * [key_offset, key_offset + s.NK) of a sequence of nk_total keys.  The causal
 * frontier is the global one: row i keeps global key j iff
 * j <= i + nk_total - N_Q; rows that see none of the shard's keys are allowed.
 * Requires 0 <= key_offset, key_offset + s.NK <= nk_total, and, when causal,
 * N_Q <= nk_total.
 *
 * streamkl_fwd_partials: the five scalars of every row over the shard's keys,
 *   fp32 [B, H, N_Q, 5] = (m1, m2, l1, l2, acc): m_t the reference maximum of
 *   scale * log2(e) * q_t.k_t, l_t = sum 2^(that - m_t), acc = sum of
 *   2^(...1 - m1) (q1.k1 - q2.k2) (unscaled).  A row with no visible key gets
 *   (-inf, -inf, 0, 0, 0).
 * streamkl_merge_partials: KL, LSE1, LSE2 [B, H, N_Q] from num_parts such
 *   partial sets stored one after the other, [num_parts][B, H, N_Q, 5] (what
 *   an all-gather of every shard's partials produces).  Only B, H, N_Q, D and
 *   the scale of s are used.  Every row must see a key in some part.
 * streamkl_bwd_keyshard: the backward (setting 1 or 2, as streamkl_bwd_s1 /
 *   streamkl_bwd_s2) over the shard's keys, given the merged LSE1, LSE2, KL of
 *   the whole sequence: the shard's dK rows (bf16, K's layout, complete since
 *   every query row is here) and this shard's unscaled contribution to dQ,
 *   fp32 [B, H, N_Q, D] contiguous, 16-byte aligned, overwritten.  Summing the
 *   dq_partial of all shards (an all-reduce) gives the full unscaled dQ.
 *   Workspace (16-byte aligned) from streamkl_bwd_keyshard_workspace: the fused
 *   path's fp32 dK rows of one key range.
 * streamkl_dq_from_partial: bf16 dQ = scale * dq_partial, written with the Q
 *   strides of s (the full problem's shape).
 */
streamkl_status streamkl_fwd_partials(const void* q1, const void* k1, const void* q2, const void* k2,
                                      streamkl_shape s, long long key_offset, long long nk_total, float* partials,
                                      void* stream);
streamkl_status streamkl_merge_partials(const float* partials, int num_parts, streamkl_shape s, float* kl,
                                        float* lse1, float* lse2, void* stream);
streamkl_status streamkl_bwd_keyshard_workspace(streamkl_shape s, long long key_offset, long long nk_total,
                                                size_t* bytes);
streamkl_status streamkl_bwd_keyshard(int setting, const void* q1, const void* k1, const void* q2, const void* k2,
                                      streamkl_shape s, long long key_offset, long long nk_total, const float* lse1,
                                      const float* lse2, const float* kl, const float* g, float* dq_partial,
                                      void* dk, void* workspace, size_t workspace_bytes, void* stream);
streamkl_status streamkl_dq_from_partial(const float* dq_partial, streamkl_shape s, void* dq, void* stream);

/*
 * Backward workspace for the current device (0 bytes for the separate path).
 * The fused path adds dK partials (TMA bulk fp32 reductions) into an
 * accumulator that the library zeroes; they stay cheap while the rows being
 * accumulated sit in L2.  Its blocks run head by head, so the live rows are one head's keys times
 * the heads a wave of blocks spans.  When all N_K keys fit that way, one
 * launch covers them and the workspace is the fp32 [B,H,N_K,D] dK accumulator
 * (dQ stays on chip).  Otherwise the keys are split into ranges whose live rows
 * fit in half the L2, each range one launch, and the workspace is the fp32
 * [B,H,range,D] dK rows of one range followed by an fp32 [B,H,N_Q,D] dQ
 * accumulator.  streamkl_bwd_fused_plan gives the same figures for any L2
 * size.  The environment variable STREAMKL_FUSED_KEY_TILES, a positive count of
 * 128-key tiles, fixes the range length instead (for testing and tuning).
 */
streamkl_status streamkl_bwd_workspace(streamkl_shape s, int bwd_mode, size_t* bytes);
/*
 * Which path AUTO takes (pure host rule, no device; 0 for an invalid shape or
 * num_sms <= 0): the fused path (over key ranges when N_K is long; see
 * streamkl_bwd_fused_plan), except the separate kernels when a head has at
 * most eight 128-row query tiles and the fused path would either need more
 * than one key range or launch fewer blocks (B*H*query tiles) than num_sms --
 * a key tile is then reused by few query tiles, the separate kernels' extra
 * recompute costs less than the fused path's dK atomics and per-range dQ round
 * trips, and the separate dK grid's many short blocks fill the SMs its few
 * long dQ blocks leave free (the two grids run as one launch).  This is the
 * "separate kernels under contention" rule of section 手法 2 "kernel fusion",
 * with the thresholds measured on GB300.
 */
int streamkl_bwd_select(streamkl_shape s, size_t l2_bytes, int num_sms);
/*
 * The fused path's plan on a device with `l2_bytes` of L2 and `num_sms` SMs
 * (pure host rule, no device): the number of key ranges (launches) and the
 * workspace bytes, as described at streamkl_bwd_workspace.
 */
streamkl_status streamkl_bwd_fused_plan(streamkl_shape s, size_t l2_bytes, int num_sms, int* key_ranges,
                                        size_t* workspace_bytes);

/*
 * Setting 1: P1 held fixed, Q2/K2 optimised (standard distillation).
 * (technical summary, 手法 2 "recompute strategy", setting 1.)
 * Rebuilds P_t = exp(S_t - LSE_t); dS2 = g_i (P2 - P1); writes
 * dQ2 = scale dS2 K2 and dK2 = scale dS2^T Q2 (bf16).  g is dLoss/dKL_i, fp32
 * [B,H,N_Q] (a mean over rows is g = 1/N_Q).  lse1/lse2 are the forward's.
 */
streamkl_status streamkl_bwd_s1(const void* q1, const void* k1, const void* q2, const void* k2,
                                streamkl_shape s, const float* lse1, const float* lse2,
                                const float* g, void* dq2, void* dk2, int bwd_mode,
                                void* workspace, size_t workspace_bytes, void* stream);

/*
 * Setting 2: P2 held fixed, Q1/K1 optimised.
 * (technical summary, 手法 2, setting 2; 手法 3 "numerical stability": the log
 *  ratio comes from logits and stored LSEs, never from log of probabilities.)
 * r = (S1 - LSE1) - (S2 - LSE2); dS1 = g_i P1 (r - KL_i); writes
 * dQ1 = scale dS1 K1 and dK1 = scale dS1^T Q1 (bf16).  kl is the forward's.
 */
streamkl_status streamkl_bwd_s2(const void* q1, const void* k1, const void* q2, const void* k2,
                                streamkl_shape s, const float* lse1, const float* lse2,
                                const float* kl, const float* g, void* dq1, void* dk1, int bwd_mode,
                                void* workspace, size_t workspace_bytes, void* stream);

/*
 * The mutual case: Q1, K1, Q2, K2 all optimised (both distributions train).
 * (technical summary, 手法 2 "recompute strategy", settings 1 and 2.)
 * P2 does not depend on Q1/K1 nor P1 on Q2/K2, so the gradients of
 * L = sum_i g_i KL_i are setting 2's (dQ1, dK1) and setting 1's (dQ2, dK2).
 * bwd_mode:
 *   STREAMKL_BWD_SEPARATE  the mutual kernels: S1 and S2 of each tile pair are
 *                          rebuilt once and both dS tiles formed from them
 *                          (dQ blocks and dK blocks in one launch, no atomics,
 *                          no workspace); dS1 and dS2 are bit-identical to the
 *                          single settings', and so are the four outputs to
 *                          those of streamkl_bwd_s2 / streamkl_bwd_s1 with
 *                          STREAMKL_BWD_SEPARATE.
 *   STREAMKL_BWD_FUSED     one fused pass per setting (setting 1, then setting
 *                          2), sharing the workspace of streamkl_bwd_workspace.
 *   STREAMKL_BWD_AUTO      as streamkl_bwd_mutual_select decides.
 * Arguments are those of streamkl_bwd_s2 (kl is required) with four bf16
 * outputs, each [B,H,N,D] with the strides of its input (dq1: q1's strides,
 * dk2: k2's, ...), all four non-NULL and 16-byte aligned.  Work runs on
 * `stream`.  With N_Q = 0 both dK are written as zeros.  Errors:
 * STREAMKL_ERR_INVALID for a bad shape, pointer or mode (DQ_ONLY / DK_ONLY are
 * refused), STREAMKL_ERR_WORKSPACE when the fused passes are chosen and the
 * workspace is missing or smaller than streamkl_bwd_mutual_workspace's,
 * STREAMKL_ERR_UNSUPPORTED for D not in {64, 128}; nothing is launched then.
 */
streamkl_status streamkl_bwd_mutual(const void* q1, const void* k1, const void* q2, const void* k2,
                                    streamkl_shape s, const float* lse1, const float* lse2,
                                    const float* kl, const float* g, void* dq1, void* dk1,
                                    void* dq2, void* dk2, int bwd_mode, void* workspace,
                                    size_t workspace_bytes, void* stream);
/*
 * AUTO's choice for the mutual case (pure host rule; the arguments match
 * streamkl_bwd_select's): STREAMKL_BWD_SEPARATE (the mutual kernels) when a
 * head has at most 64 query tiles of 128 rows, else STREAMKL_BWD_FUSED (a
 * fused pass per setting) -- the threshold measured on GB300.  0 for an
 * invalid shape or num_sms <= 0.
 */
int streamkl_bwd_mutual_select(streamkl_shape s, size_t l2_bytes, int num_sms);
/* Workspace bytes streamkl_bwd_mutual needs in `bwd_mode` on the current device (0 for the mutual kernels). */
streamkl_status streamkl_bwd_mutual_workspace(streamkl_shape s, int bwd_mode, size_t* bytes);

/*
 * Attention: O = softmax(scale Q K^T) V with the rows' log-sum-exp, and its
 * backward -- what a model whose attention is distilled runs beside the loss
 * (its LSE is the loss's LSE_t for the same Q and K).
 *
 * Q [B, H, N_Q, D]; K, V [B, HK, N_K, D] with H a multiple of HK (query head h
 * reads key head h / (H / HK)); O like Q; bf16, D 64 or 128.  LSE fp32
 * [B, H, N_Q].  Strides as in streamkl_shape, each tensor its own (three zeros:
 * contiguous); O's must not make rows overlap.
 * q_lens, k_lens: device int32 [B], or NULL for whole sequences: sequence b has
 * the first q_lens[b] of N_Q queries and k_lens[b] of N_K keys (values are kept
 * within 0 .. N).  What lies past them is not used, whatever it holds, NaN
 * included.  causal keeps key j for query i iff j <= i + k_len - q_len.
 * A row that sees no key -- past its sequence, causal with more queries than
 * keys, no keys at all -- has O = 0 and LSE = -inf.  Values |v| up to 2^88 give finite
 * results at any length (sums are fp32, before their division).
 * Workspace: fp32 partials of the key splits that few query tiles get, 0 bytes
 * where the query tiles fill the SMs; streamkl_attn_fwd_plan gives the choice for any SM count (a
 * pure host rule): packed != 0 when all query heads of a key head share one
 * 128-row tile, and the number of key splits.
 */
typedef struct {
  int B, H, HK, NQ, NK, D;
  float scale;
  int causal;
  const int* q_lens;
  const int* k_lens;
  long long q_stride_b, q_stride_h, q_stride_n;
  long long k_stride_b, k_stride_h, k_stride_n;
  long long v_stride_b, v_stride_h, v_stride_n;
  long long o_stride_b, o_stride_h, o_stride_n;
  void* o_rest; /* NULL, or bf16 like O: see below */
} streamkl_attn_shape;
streamkl_status streamkl_attn_fwd_workspace(streamkl_attn_shape s, size_t* bytes);
streamkl_status streamkl_attn_fwd_plan(streamkl_attn_shape s, int num_sms, int* packed, int* splits);
streamkl_status streamkl_attn_fwd(const void* q, const void* k, const void* v, streamkl_attn_shape s, void* o,
                                  float* lse, void* workspace, size_t workspace_bytes, void* stream);

/*
 * Attention backward: with P = exp(scale Q K^T - LSE) rebuilt from the saved LSE,
 * dP = dO V^T, delta_i = dO_i . O_i - dLSE_i and dS = P (dP - delta):
 *     dQ = scale dS K,  dK = scale dS^T Q,  dV = P^T dO  (dK, dV summed over the
 *     query heads that share a key head)
 * s.o_rest (NULL, or [B, H, N_Q, D] bf16 with o's strides): the forward writes what
 * rounding O to bf16 left to it and divides by the sum of its rounded weights, the
 * backward reads it.  Without it delta carries O's rounding, and dQ, dK an error that
 * grows with the part that the values have in common (zero mean 1.5 times, a
 * common vector of three times their size 4 to 9 times that of the last
 * rounding); with it 1.4 to 1.6 times.  Rows of at most 32 keys need it not, nor any
 * where N_K is at most 64: their delta is formed from P and dP.
 * o, lse: the forward's; go = dLoss/dO with o's strides; dlse = dLoss/dLSE, fp32
 * [B, H, N_Q], or NULL.  dq, dk, dv: bf16 with the strides of q, k, v (which must
 * not make rows overlap).  Lengths and causal as in the forward; gradients of
 * what lies past a sequence are 0, and go, dlse are not used there.
 * bwd_mode:
 *   STREAMKL_BWD_SEPARATE  dQ blocks and dK/dV blocks in one launch; what several
 *                          blocks add up is added in a fixed order: the same bits on
 *                          every run.  Workspace: 32 bytes per query row (N_Q
 *                          rounded up to 128), and the fp32 accumulators of tiles
 *                          that are dealt out over several blocks.
 *   STREAMKL_BWD_FUSED     D = 64 only (else STREAMKL_ERR_UNSUPPORTED): one visit of
 *                          each tile pair; dQ is added up in fp32 by reductions in
 *                          L2, in no fixed order, so its last bits can differ between
 *                          runs (dK and dV do not).  Workspace: 4 D bytes more per row.
 *   STREAMKL_BWD_AUTO      fused for D = 64 where the key tiles alone fill the SMs,
 *                          else separate.
 * streamkl_attn_bwd_plan gives the path, the parts that dK/dV tiles and dQ tiles are
 * dealt out over (1: one block each; the fused path deals out only its last wave)
 * and the workspace for any SM count (num_sms <= 0: the current device); with
 * num_sms > 0 it is a pure host rule.
 */
streamkl_status streamkl_attn_bwd_plan(streamkl_attn_shape s, int num_sms, int bwd_mode, int* path, int* kv_parts,
                                       int* q_parts, size_t* workspace_bytes);
streamkl_status streamkl_attn_bwd_workspace(streamkl_attn_shape s, int bwd_mode, size_t* bytes);
streamkl_status streamkl_attn_bwd(const void* q, const void* k, const void* v, const void* o, const float* lse,
                                  const void* go, const float* dlse, streamkl_attn_shape s, void* dq, void* dk,
                                  void* dv, int bwd_mode, void* workspace, size_t workspace_bytes, void* stream);

/*
 * Differential attention: the difference of two softmax maps over the same keys and
 * values, with a learned weight,
 *     O = softmax(scale Q1 K^T) V - lam softmax(scale Q2 K^T) V,
 * and its backward, dlam included.
 *
 * s.maps describes both maps as streamkl_attn_fwd does its attention: H counts the query
 *   heads of both, heads 2 i and 2 i + 1 of q are the maps of difference i, and H / 2 is a
 *   multiple of HK; lengths, causal, scale and strides as there.  lse [B, H, N_Q] has both
 *   maps' log-sum-exps.
 * lam: fp32, element b lam_stride_b + i lam_stride_h + n lam_stride_n for difference i of row n
 *   (strides may be 0: one weight for all).
 * d, the difference: bf16 [B, H / 2, N_Q, D], strides d_stride_* (three zeros: contiguous).  It is
 *   formed in fp32 and rounded once.  Rows that see no key are 0; lam is not used there.
 * maps and s.maps.o_rest: NULL for the difference alone; both for a backward: each map's own
 *   result and what its rounding left, bf16 [B, H, N_Q, D] with the strides o_stride_*.
 * Backward: go = dLoss/dd with d's strides, dlse (or NULL) fp32 [B, H, N_Q]; maps and o_rest are
 *   required.  dq, dk, dv as in streamkl_attn_bwd; dlam fp32 [B, H / 2, N_Q] contiguous, a value
 *   for every row whatever lam's strides are, as exact as the second map's two parts: each term dO O2 to 2^-16 of
 *   itself.  |lam| is part of the second map's weights, which enter the products rounded to bf16 as the
 *   first's do; with dlse, where |lam| is below 1/64, it multiplies dO instead, rounded to bf16.
 *   bwd_mode as in streamkl_attn_bwd.
 * Workspaces as in streamkl_attn_fwd and streamkl_attn_bwd; the backward's also has the maps' gradients,
 *   2 D bytes per query row of both.  streamkl_diff_attn_fwd_plan: packed, splits and the workspace for any SM count
 *   (num_sms <= 0: the current device; with num_sms > 0 a pure host rule).
 */
typedef struct {
  streamkl_attn_shape maps;
  const float* lam;
  long long lam_stride_b, lam_stride_h, lam_stride_n;
  long long d_stride_b, d_stride_h, d_stride_n;
} streamkl_diff_attn_shape;
streamkl_status streamkl_diff_attn_fwd_plan(streamkl_diff_attn_shape s, int num_sms, int* packed, int* splits,
                                            size_t* workspace_bytes);
streamkl_status streamkl_diff_attn_fwd_workspace(streamkl_diff_attn_shape s, size_t* bytes);
streamkl_status streamkl_diff_attn_fwd(const void* q, const void* k, const void* v, streamkl_diff_attn_shape s, void* d,
                                       void* maps, float* lse, void* workspace, size_t workspace_bytes, void* stream);
streamkl_status streamkl_diff_attn_bwd_workspace(streamkl_diff_attn_shape s, int bwd_mode, size_t* bytes);
streamkl_status streamkl_diff_attn_bwd(const void* q, const void* k, const void* v, const void* maps, const float* lse,
                                       const void* go, const float* dlse, streamkl_diff_attn_shape s, void* dq, void* dk,
                                       void* dv, float* dlam, int bwd_mode, void* workspace, size_t workspace_bytes,
                                       void* stream);

/*
 * Log probabilities of given tokens, with entropy and top alternatives: the
 * output-layer companion of the attention loss (a student scored on the data's
 * tokens, or on its teacher's most likely ones).
 *
 * logits: [rows, vocab] of `dtype`, rows `row_stride` elements apart, aligned to
 *   an element.  x = scale * logits, scale > 0 (an inverse temperature).
 * tokens: [rows, num_tokens] 64-bit.  logp[r, t] = x[r, token] - LSE_r.  A
 *   negative token is no token: its logp is 0 and it has no gradient.  A token
 *   >= vocab gives NaN and has no gradient; nothing is read for it.
 * entropy, lse: [rows], H = -sum p log p and log sum e^x.
 * top_logp, top_index: [rows, top_k], the largest logits in descending order,
 *   equal ones from the lowest column up (-0 equals +0), with their log
 *   probabilities.  top_k <= STREAMKL_LOGPROBS_MAX_TOP_K and <= vocab; 0 for none
 *   (both may be NULL then, as tokens and logp with num_tokens = 0).
 * A logit of -inf has probability 0.  A row of nothing but -inf has LSE -inf,
 * entropy 0, log probabilities -inf and a zero gradient.  A +inf or NaN logit
 * makes its row's values NaN (alternatives are then any columns of the row).
 * Finite logits are finite numbers, the type's lowest value too: a row masked
 * whole with it is uniform.  An LSE past fp32's range is given as its end.  A row
 * whose |LSE| is above 256 is read twice more, for log probabilities that do
 * not lose the digits which the LSE has before the point.
 *
 * streamkl_logprobs_bwd writes dlogits [rows, vocab] (rows `out_stride` elements
 * apart, `dtype`) for upstream gradients g_logp [rows, num_tokens] and, unless
 * NULL, g_entropy [rows] (entropy is read only then); lse and entropy are the
 * forward's.  A token given twice in a row adds twice.  The alternatives have no
 * gradient: to train on some, give them as tokens.  dlogits may be the logits
 * themselves, with the same stride, only where num_tokens is 0 (a row is then one
 * block's work).  A given token is compared with the row's others: num_tokens is
 * meant for alternatives, tens or hundreds, its square is the cost.
 * Sums are fp32.  Results do not depend on the order in which blocks run.
 */
typedef enum { STREAMKL_BF16 = 0, STREAMKL_FP16 = 1, STREAMKL_FP32 = 2 } streamkl_dtype;
#define STREAMKL_LOGPROBS_MAX_TOP_K 32
streamkl_status streamkl_logprobs_fwd(const void* logits, int dtype, long long rows, long long vocab,
                                      long long row_stride, const long long* tokens, int num_tokens, float scale,
                                      int top_k, float* logp, float* entropy, float* lse, float* top_logp,
                                      long long* top_index, void* stream);
streamkl_status streamkl_logprobs_bwd(const void* logits, int dtype, long long rows, long long vocab,
                                      long long row_stride, const long long* tokens, int num_tokens, float scale,
                                      const float* lse, const float* entropy, const float* g_logp,
                                      const float* g_entropy, void* dlogits, long long out_stride, void* stream);

/*
 * Cross entropy over a vocabulary, from the hidden states, without the logits in
 * memory: the output layer's loss and its gradients where the logits themselves are
 * not wanted (with them in memory, streamkl_logprobs_fwd's logp is -loss).
 *
 * hidden [rows, channels], weight [vocab, channels]: both of `dtype` (bf16 or fp16),
 *   rows hidden_stride and weight_stride elements apart, 16-byte aligned; channels and
 *   strides multiples of 8.  z = scale hidden weight^T, scale > 0.
 * tokens [rows], 64-bit.  loss_r = LSE_r - z[r, token], lse_r = LSE_r, fp32 [rows].  A
 *   negative token is no token: its loss is 0 and has no gradient (lse does).  A token
 *   >= vocab gives NaN and has no gradient.
 * A +inf or NaN logit makes its row's values NaN, -inf has probability 0; |z| above 2.3e38, 2^128 in
 *   units of log 2, counts as infinite.
 *
 * streamkl_vocab_xent_bwd: for upstream gradients g_loss [rows] and, unless NULL, g_lse
 *   [rows] of the two outputs, and the forward's lse:
 *     d = scale (g_loss (p - [v = token]) + g_lse p),  p = exp(z - lse)
 *     dhidden = d weight [rows, channels],  dweight = d^T hidden [vocab, channels]
 *   contiguous, of `dtype`, overlapping nothing; one of them may be NULL where it is not wanted (with no rows
 *   dhidden is empty and may be NULL too; dweight is 0).  d enters the
 *   products rounded to `dtype`, in fp16 times one power of two for all rows, which brings the largest finite
 *   scale (|g_loss| + |g_lse|) to [2^13, 2^14), g_loss counted where the row has a token: entries of d below 2^-38 of
 *   the largest row's gradient are lost then.  p is formed from lse as it is stored: far from 0 the roundings of
 *   lse, and of z and lse in units of log 2, move it by up to 8 max(|z|, |lse|) 2^-24 of itself.  Sums are fp32,
 *   dhidden and dweight are rounded once.  What
 *   several blocks add up is added in a fixed order: the same bits on every run.  A row whose
 *   gradients are 0 has dhidden 0 and no part in dweight, whatever its hidden states are, NaN
 *   included; the weight has to be finite.
 * Workspaces (16-byte aligned): forward, 16 bytes per row and tile of 160 to 256 columns; backward, a piece
 *   of d, fp32 sums of dhidden and, for dweight, room for a copy of hidden:
 *   streamkl_vocab_xent_bwd_plan gives the number of the vocabulary's pieces, the splits of
 *   dhidden's sums and the bytes, streamkl_vocab_xent_fwd_plan the forward's tile and bytes,
 *   for any SM count (num_sms <= 0: the current device; with num_sms > 0 a pure host rule).
 */
typedef struct {
  long long rows, vocab;
  int channels, dtype;
  float scale;
  long long hidden_stride, weight_stride;
} streamkl_xent_shape;
streamkl_status streamkl_vocab_xent_fwd_plan(streamkl_xent_shape s, int num_sms, int* tile_width, size_t* bytes);
streamkl_status streamkl_vocab_xent_fwd_workspace(streamkl_xent_shape s, size_t* bytes);
streamkl_status streamkl_vocab_xent_fwd(const void* hidden, const void* weight, const long long* tokens, streamkl_xent_shape s,
                                        float* loss, float* lse, void* workspace, size_t workspace_bytes, void* stream);
streamkl_status streamkl_vocab_xent_bwd_plan(streamkl_xent_shape s, int num_sms, int want_dhidden, int want_dweight, int* pieces,
                                             int* splits, size_t* bytes);
streamkl_status streamkl_vocab_xent_bwd_workspace(streamkl_xent_shape s, int want_dhidden, int want_dweight, size_t* bytes);
streamkl_status streamkl_vocab_xent_bwd(const void* hidden, const void* weight, const long long* tokens, const float* lse,
                                        const float* g_loss, const float* g_lse, streamkl_xent_shape s, void* dhidden,
                                        void* dweight, void* workspace, size_t workspace_bytes, void* stream);

/*
 * Rotary positions: what turns the queries and keys before an attention, or before
 * the attention loss, in one launch for both.
 *
 * q [B, HQ, N, D], k [B, HK, N, D] of `dtype` (HQ or HK may be 0, and that pointer NULL then),
 *   D even, channels contiguous, element strides along b, h, n as given, any alignment to an
 *   element (16-byte granules are faster).  The first `dim` channels (even) turn, the others are
 *   copied.  Pair i is the channels i and dim / 2 + i, with `interleaved` 2 i and 2 i + 1.
 * A row at position p: (x, y) -> amplitude (x cos a - y sin a, y cos a + x sin a), a = p turns[i]
 *   2^-64 of a turn: turns [dim / 2], device, 2^64 f_i / 2 pi mod 2^64 for a frequency of f_i radians
 *   a position.  For any 64-bit p, negative ones too, the angle is within 2^-32 turns (1.5e-9 radians) of p turns[i], whose
 *   own rounding is |p| 2^-65 turns.
 *   Arithmetic is fp32, results are rounded once.
 * positions: device, 32-bit or 64-bit integers (positions_bytes), sequence b's N of them from element
 *   b positions_stride on (stride 0: the same for all); NULL: row n is at offset + n.
 * inverse != 0 turns back (-a), with the same amplitude: the gradient's map.
 * Outputs: strides of their own, rows that do not overlap; q_out may be q and k_out k, with the same
 *   strides.  Otherwise no output may overlap an input or the other output.
 */
typedef struct {
  int B, HQ, HK, N, D, dim;
  int dtype, interleaved;
  float amplitude;
  long long offset;
  const void* positions;
  int positions_bytes;
  long long positions_stride;
  long long q_stride_b, q_stride_h, q_stride_n;
  long long k_stride_b, k_stride_h, k_stride_n;
  long long q_out_stride_b, q_out_stride_h, q_out_stride_n;
  long long k_out_stride_b, k_out_stride_h, k_out_stride_n;
} streamkl_rotary_shape;
streamkl_status streamkl_rotary(const void* q, const void* k, streamkl_rotary_shape s, const unsigned long long* turns,
                                void* q_out, void* k_out, int inverse, void* stream);

/* Text for a status code (static storage). */
const char* streamkl_status_string(streamkl_status st);

/*
 * Synchronises `stream`, then reads and clears the device status word of the
 * current device.  Returns STREAMKL_ERR_TIMEOUT if a bounded wait ran out since
 * the last check (or a block that owns its SM's tensor memory was given it from
 * another column than the first, which is recorded the same way),
 * STREAMKL_ERR_CUDA if the sync failed, else STREAMKL_OK.
 *
 * The status word is one flag per device for the whole process, shared by
 * every caller, stream and thread that uses the library: a timeout on any
 * stream sets it, and the first check afterwards -- from whichever thread --
 * reports and clears it.  Callers that share a device and each want to see
 * their own timeouts must serialise their checks (or agree on one checker).
 */
streamkl_status streamkl_check_device_status(void* stream);

/*
 * Test hook for the timeout path: launches one block that waits on a barrier
 * nobody arrives at, giving up after `timeout_us` microseconds (clamped to
 * [1, 1000000]) and recording STREAMKL_ERR_TIMEOUT in the status word.
 */
streamkl_status streamkl_debug_wait_timeout(int timeout_us, void* stream);

/* Library version, major*10000 + minor*100 + patch. */
int streamkl_version(void);

#ifdef __cplusplus
}
#endif

#endif /* STREAMKL_H */
