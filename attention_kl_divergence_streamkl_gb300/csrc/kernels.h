// Internal interface between the C-ABI layer (api.cu) and the kernel files.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <stdint.h>

namespace skl {

// A validated problem.  Logits are handled in log2 units: c = scale * log2(e).
struct Problem {
  int B, H, NQ, NK, D;
  int BH;
  int causal;
  int off;      // NK - NQ: row i keeps key j iff j <= i + off (causal)
  float scale;  // softmax scale applied to Q K^T
  float c;      // scale * log2(e)
  // element strides of Q1/Q2 (and dQ) and of K1/K2 (and dK) along b, h, n; d is contiguous
  long long qs_b, qs_h, qs_n, ks_b, ks_h, ks_n;
};

// Element offset of row n of head (b, h) = bh in a tensor with strides (sb, sh, sn).
__host__ __device__ inline long long row_offset(int bh, int H, long long n, long long sb, long long sh, long long sn) {
  return (long long)(bh / H) * sb + (long long)(bh % H) * sh + n * sn;
}

// Builds a 4-D TMA map {d, n, h, b} over a bf16 [B, H, N, D] view with the given
// element strides (d contiguous), a {64, box_rows, box_heads, 1} box and the 128-byte
// swizzle.  Returns false if the driver rejects it.
bool encode_tile_map(CUtensorMap* map, const void* base, int D, int N, int H, int B, long long sn, long long sh,
                     long long sb, int box_rows, int box_heads = 1);
// A 3-D TMA map {d, row, bh} over an fp32 [BH][rows][D] accumulator, a {D, box_rows, 1} box, no swizzle
// (for bulk reductions into it).
// With box_cols 32 the box is {32, box_rows, 1} with the swizzle of its 128-byte rows.
bool encode_rows_f32_map(CUtensorMap* map, float* base, int D, int rows, int BH, int box_rows, int box_cols = 0);
// A 2-D TMA map {col, row} over a matrix of 2-byte values whose rows lie `stride` elements apart, a {box_cols, box_rows} box
// of 64 or 32 columns with the swizzle of its 128- or 64-byte rows.
bool encode_matrix_map(CUtensorMap* map, const void* base, long long rows, long long cols, long long stride, int box_rows,
                       int box_cols);
// The maps of Q1/Q2 and K1/K2 of a problem.
inline bool encode_q_map(CUtensorMap* map, const void* base, const Problem& p, int box_rows) {
  return encode_tile_map(map, base, p.D, p.NQ, p.H, p.B, p.qs_n, p.qs_h, p.qs_b, box_rows);
}
inline bool encode_k_map(CUtensorMap* map, const void* base, const Problem& p, int box_rows) {
  return encode_tile_map(map, base, p.D, p.NK, p.H, p.B, p.ks_n, p.ks_h, p.ks_b, box_rows);
}

// ---- forward (one CTA per 128-row query tile) -------------------------------
cudaError_t launch_fwd(const Problem& p, const void* q1, const void* k1, const void* q2, const void* k2,
                       float* kl, float* lse1, float* lse2, int* status, cudaStream_t st);
// The same forward over one key shard (p.off already shifted by the shard's
// first key): the five scalars of every row, fp32 [B*H*N_Q][5] (m1, m2 in log2
// units, l1, l2, acc unscaled), instead of KL and LSE.
cudaError_t launch_fwd_partials(const Problem& p, const void* q1, const void* k1, const void* q2, const void* k2,
                                float* partials, int* status, cudaStream_t st);
// Merges `parts` partial sets laid out [part][B*H*N_Q][5] into KL, LSE1, LSE2.
cudaError_t launch_merge_partials(const Problem& p, int parts, const float* partials, float* kl, float* lse1,
                                  float* lse2, cudaStream_t st);

// ---- Split-K forward ---------------------------------------------------------
constexpr int kSplitKTile = 64;        // keys per pipeline stage
constexpr int kSplitKCtasPerSm = 2;    // resident blocks per SM the planner assumes
int splitk_key_tiles(const Problem& p);
int splitk_plan(int BH, int key_tiles, int num_sms);
cudaError_t launch_splitk(const Problem& p, const void* q1, const void* k1, const void* q2, const void* k2,
                          int splits, float* partials, float* kl, float* lse1, float* lse2, int* status,
                          cudaStream_t st);
// Device address (current device) of the fixed scratch of the allocation-free entry point.
cudaError_t splitk_noalloc_scratch(float** out);

// ---- backward ------------------------------------------------------------------
struct BwdIn {
  const void *q1, *k1, *q2, *k2;
  const float *lse1, *lse2, *kl, *g;
};
// setting 1: dq/dk are dQ2/dK2; setting 2: dQ1/dK1.  The separate path skips a NULL output; with both
// outputs its dQ and dK grids run as one launch.
cudaError_t launch_bwd_separate(const Problem& p, int setting, const BwdIn& in, void* dq, void* dk, int* status,
                                cudaStream_t st);
// Fused backward over key ranges of range_tiles 128-key tiles (all keys when
// range_tiles >= the tile count).  workspace: the fp32 dK rows of one range
// ([B*H][min(128 range_tiles, N_K)][D]), then, with more than one range, the
// fp32 dQ accumulator ([B*H][N_Q][D]).
// With dq_f32 non-null, dQ is not written to dq: the unscaled fp32 sum over
// this launch's keys goes to dq_f32 ([B*H][N_Q][D], zeroed first), and the
// workspace holds only the dK rows of one range.
cudaError_t launch_bwd_fused(const Problem& p, int setting, const BwdIn& in, void* dq, void* dk, float* workspace,
                             int range_tiles, int* status, cudaStream_t st, float* dq_f32 = nullptr);
// Both settings' gradients in one recompute (the mutual case): dQ1, dK1 (setting 2) and dQ2, dK2
// (setting 1), each written with its input's strides; the dQ and the dK blocks in one launch, no workspace.
cudaError_t launch_bwd_mutual(const Problem& p, const BwdIn& in, void* dq1, void* dk1, void* dq2, void* dk2,
                              int* status, cudaStream_t st);
// dK = 0 for every key row of every head, written with K's strides (a backward with no query rows).
cudaError_t launch_zero_k_rows(const Problem& p, void* dk, cudaStream_t st);
// out row n of head bh = bf16(scale * acc[bh][n]) for n < N_Q, with Q's strides.
cudaError_t launch_rows_to_bf16(const Problem& p, const float* acc, void* out, cudaStream_t st);
// First 128-query tile whose rows see key k0.
int fused_first_qtile(const Problem& p, long long k0);

// ---- attention -----------------------------------------------------------------------
// Division of n < 2^31 by a number that the host knows, by multiplication (Granlund and Montgomery): with s = ceil(log2 d)
// and mul = floor(2^32 (2^s - d) / d) + 1, n / d = (mulhi(n, mul) + n) >> s.
struct FastDiv {
  unsigned d = 1, mul = 1, shift = 0;
  FastDiv() = default;
  explicit FastDiv(unsigned by) : d(by), shift(0) {
    while ((1ull << shift) < by) ++shift;
    mul = (unsigned)((((1ull << shift) - by) << 32) / by + 1);
  }
#ifdef __CUDACC__
  __device__ __forceinline__ unsigned div(unsigned n) const { return (__umulhi(n, mul) + n) >> shift; }
#endif
};

struct AttnProblem {
  int B, H, HK, G, NQ, NK, D;  // G = H / HK query heads to a key head
  int causal;                  // row i keeps key j iff j <= i + k_len - q_len
  float scale, c;              // c = scale * log2(e)
  const int *q_lens, *k_lens;  // device, [B], or null: every sequence has N_Q queries, N_K keys
  // element strides along b, h, n of q (and dq), k (dk), v (dv), o (and do)
  long long qs_b, qs_h, qs_n, ks_b, ks_h, ks_n, vs_b, vs_h, vs_n, os_b, os_h, os_n;
  long long gs_b, gs_h, gs_n;  // of do, in the backward's products
  // a difference of two maps: heads 2 i and 2 i + 1 of q, o, lse and their gradients are its maps
  int diff;
  const float* lam;            // the second map's weight, fp32 by (b, pair of heads, n) with strides that may be 0
  long long ls_b, ls_h, ls_n;
  long long cs_b, cs_h, cs_n;  // strides of the difference, [B, H / 2, N_Q, D], and of its gradient
  long long rows;              // B H N_Q
  void* o_rest;                // null, or what rounding O to bf16 left, with O's strides: the forward writes it
  // forward plan (attn_fwd_plan)
  int packed;   // the query heads of a key head share one tile
  int q_items;  // blocks along the queries, per (batch, head)
  int splits;   // blocks along the keys
  int longest_first;  // the last query tiles of all heads first, not head by head
  FastDiv by_splits, by_items, by_heads, by_group;  // by_items: what an item's number is first divided by
};
void attn_fwd_plan(AttnProblem* p, int num_sms);
long long attn_fwd_items(const AttnProblem& p);
size_t attn_fwd_workspace(const AttnProblem& p);  // bytes, 0 without splits
// diff: the difference's result, where p.diff (o, each map's own, is then null unless p.o_rest is wanted too)
cudaError_t launch_attn_fwd(const AttnProblem& p, const void* q, const void* k, const void* v, void* o, float* lse,
                            void* workspace, int* status, cudaStream_t st, void* diff = nullptr);

struct AttnBwdIn {
  const void *q, *k, *v, *o, *go;  // go = dO, with o's strides
  const void* o_rest;              // null, or the forward's
  const float *lse, *dlse;         // dlse may be null
  const void* ddiff;               // a difference's gradient (go is then null), and where that of its weights goes
  float* dlam;
};
// How a backward runs on a device (a pure rule of sizes).  Tiles [0, whole) of a kind are one block each, the later ones
// `parts` blocks.  Fused: one visit of each tile pair by the kv blocks, dQ added up in an fp32 accumulator.
struct AttnBwdPlan {
  bool fused;
  unsigned kv_tiles, kv_whole, kv_blocks;
  unsigned q_tiles, q_whole, q_blocks;  // dQ blocks; none when fused
  int kv_parts, q_parts;
  int q_first;        // which kind comes first in the grid
  int longest_first;  // the longest tiles of all heads first, not head by head
  // of a block's number by parts, of a tile's by what it is first divided by, of a (batch, head) by heads, of a head by G
  FastDiv by_kv_parts, by_q_parts, by_kv_tile, by_q_tile, by_key_heads, by_heads, by_group;
};
// Where things lie in the workspace.
struct AttnBwdScratch {
  int padded;             // N_Q rounded up to 128
  void *row_s, *row_d;    // 16 bytes per row of [B H][padded]
  float* acc;             // fused: [B H][padded][D]
  void *kv_parts, *q_parts;
  unsigned *kv_counters, *q_counters;
  unsigned n_counters;    // of both, one after the other
  void* go;               // a difference: what reaches each map, bf16 [B, H, N_Q, D]
  size_t bytes;
};
bool attn_bwd_has_fused(const AttnProblem& p);
AttnBwdPlan attn_bwd_plan(const AttnProblem& p, int mode, int num_sms);  // mode: streamkl_bwd_mode
AttnBwdScratch attn_bwd_scratch(const AttnProblem& p, const AttnBwdPlan& plan, void* workspace);
cudaError_t launch_attn_bwd(const AttnProblem& p, const AttnBwdPlan& plan, const AttnBwdIn& in, void* dq, void* dk,
                            void* dv, void* workspace, int* status, cudaStream_t st);
cudaError_t launch_attn_bwd_fused(const AttnProblem& p, const AttnBwdPlan& plan, const AttnBwdIn& in, void* dq, void* dk,
                                  void* dv, const AttnBwdScratch& w, int* status, cudaStream_t st);

// ---- log probabilities of given tokens ---------------------------------------------
constexpr int kTypeBf16 = 0, kTypeFp16 = 1, kTypeFp32 = 2;  // streamkl_dtype
struct LogprobsProblem {
  long long rows, stride;  // stride: elements between rows of the logits
  int V, T, K, dtype;
  float scale;
};
cudaError_t launch_logprobs_fwd(const LogprobsProblem& p, const void* logits, const long long* tokens, float* logp,
                                float* entropy, float* lse, float* top_logp, long long* top_index, int num_sms,
                                cudaStream_t st);
cudaError_t launch_logprobs_bwd(const LogprobsProblem& p, const void* logits, const long long* tokens,
                                const float* lse, const float* entropy, const float* g_logp, const float* g_entropy,
                                void* dlogits, long long out_stride, int num_sms, cudaStream_t st);

// ---- cross entropy over a vocabulary, from hidden states -----------------------------
struct XentProblem {
  long long R, V;  // rows of hidden states, the vocabulary
  int C;           // channels
  int half;        // fp16, else bf16
  long long hidden_stride, weight_stride;
  float scale;
};
int xent_fwd_width(const XentProblem& p, int num_sms);  // columns of a tile
size_t xent_fwd_workspace(const XentProblem& p, int num_sms);
cudaError_t launch_xent_fwd(const XentProblem& p, const void* hidden, const void* weight, const long long* tokens, float* loss,
                            float* lse, void* workspace, int num_sms, int* status, cudaStream_t st);
struct XentBwdPlan {
  int pieces, splits;   // of the vocabulary; of dh's sums over a piece
  long long columns;    // of a piece
  bool direct;          // dh needs no sums between launches
  size_t off_d, off_acc, off_clean, bytes;
};
XentBwdPlan xent_bwd_plan(const XentProblem& p, bool want_dh, bool want_dw, int num_sms);
struct XentBwdIn {
  const void *hidden, *weight;
  const long long* tokens;
  const float *lse, *g, *g_lse;  // g_lse may be null
};
// dhidden, dweight: null where it is not wanted
cudaError_t launch_xent_bwd(const XentProblem& p, const XentBwdPlan& plan, const XentBwdIn& in, void* dhidden, void* dweight,
                            void* workspace, int num_sms, int* status, cudaStream_t st);

// ---- rotary positions ----------------------------------------------------------------
struct RotaryStrides {
  long long b, h, n;  // elements; channels are contiguous
};
struct RotaryProblem {
  int B, HQ, HK, N, D, dim;  // the first dim channels turn
  unsigned tokens;           // B N
  int dtype, interleaved;
  float amplitude, sin_sign;  // cos is multiplied by amplitude, sin by sin_sign: amplitude, or -amplitude for the inverse
  long long offset;           // position of row 0 where positions is null
  const void* positions;      // 64-bit, or 32-bit unless positions_wide
  long long positions_stride;
  int positions_wide;
  const unsigned long long* turns;  // [dim / 2], 2^-64 of a turn a position
  const void *q_in, *k_in;
  void *q_out, *k_out;
  RotaryStrides q, k, qo, ko;
  // plan
  int vectors;     // 16-byte loads
  int turning;     // slots of a row that turn
  int heads_each;  // heads that a thread goes through
  long long items;
  FastDiv by_slots, by_rows;
};
bool rotary_plan(RotaryProblem* p, int num_sms);  // false: too large for one launch
cudaError_t launch_rotary(const RotaryProblem& p, cudaStream_t st);

// ---- test hook ------------------------------------------------------------------
cudaError_t launch_wait_timeout_probe(int timeout_us, int* status, cudaStream_t st);

}  // namespace skl
