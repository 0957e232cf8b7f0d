// Internal launch functions of liblmhead (host side). Each returns a
// cudaError_t from the launch; arguments have been validated by api.cu.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <stdint.h>

namespace lmhead {

typedef uint16_t bf16_t;

// Largest k_tile handled by the fused score + tile top-k kernels.
constexpr int kFusedMaxKTile = 32;
// Largest selection budget of the radix select (global C or k_tile).
constexpr int kSelectMaxK = 4096;

// K1: u = bf16(B h), fp32 accumulation. Tensor cores (cluster split over d)
// up to d = kProjTcMaxD, CUDA cores beyond. Also zeroes `zero_ints` ints at
// `zero_ptr` (tickets of the fused kernels that follow), if non-null.
constexpr int kProjTcMaxD = 5120;
cudaError_t launch_project_u(const bf16_t* B, const bf16_t* h, int d, int r, int M, bf16_t* u,
                             int* zero_ptr, int zero_ints, cudaStream_t s);

// K4 (CUDA cores): fused tile scores + per-tile top-k_tile, no score writeback.
// For M <= kLocalGemvMaxM and tiles of 32..256 rows dividing 256 (k_tile <= 8,
// r = 256 or 512) it runs the warp-per-row GEMV kernel (measured faster than
// the tensor-core kernel up to four hidden vectors; at five to eight the
// GEMV's registers leave too few warps per SM).
constexpr int kLocalGemvMaxM = 4;  // compiled up to; gemv_max_m() is the limit in use
int gemv_max_m();
bool local_topk_gemv_supported(int M, int r, int T, int k_tile);
// The GEMV score writeback (below): one or two hidden vectors.
bool scores_gemv_supported(int M, int r);
// The same GEMV kernel writing every score to S (M x n fp32 by position)
// instead of selecting: the global path's writeback for one or two hidden
// vectors at r = 256 or 512. hist0 != nullptr: it also adds the counts of the
// scores' top kSelectHistBits order bits of hidden vector m into
// hist0 + m * hist0_stride (kSelectHistBins ints; the multi-CTA selection's
// first histogram).
cudaError_t launch_scores_gemv(const bf16_t* A, const bf16_t* u, int64_t n, int r, int M, float* S,
                               cudaStream_t s, int* hist0 = nullptr, int hist0_stride = 0);
// ready: the gather's ready counters (GEMV kernel only; may be nullptr).
cudaError_t launch_local_topk_fma(const bf16_t* A, const bf16_t* u, const int32_t* token_ids,
                                  int64_t n, int r, int M, int T, int k_tile, int32_t* out_ids,
                                  float* out_scores, cudaStream_t s, int* ready = nullptr);

// K4 (tensor cores): tcgen05 MMA with TMA-staged A chunks, persistent CTAs.
constexpr int kLocalTcMaxR = 512;
constexpr int kLocalTcMaxCtas = 256;
bool local_topk_tc_supported(int r, int T, int k_tile);
// workspace bytes for the split-tile partial lists; tile tickets are counted separately
size_t local_topk_tc_scratch_bytes(int64_t n, int M, int T);
int local_topk_tc_tickets(int64_t n, int M, int T);
// ready: the gather's ready counters (tiles of a multiple of 128 rows only;
// may be nullptr).
cudaError_t launch_local_topk_tc(const bf16_t* A, const bf16_t* u, const int32_t* token_ids,
                                 int64_t n, int r, int M, int T, int k_tile, int32_t* out_ids,
                                 float* out_scores, void* partials, int* tile_tickets, int* err,
                                 cudaStream_t s, int* ready = nullptr);

// K3: per row m, per segment of `seg_len` positions, exact top-k of S by
// (score desc, vocabulary id asc). k <= kSelectMaxK.
cudaError_t launch_segment_topk(const float* S, const int32_t* token_ids, int64_t n, int M,
                                int64_t seg_len, int k, int32_t* out_ids, float* out_scores,
                                int* err, cudaStream_t s);

// Overlap of the gather with the fused scoring kernel (local mode): the
// scoring kernel counts, per block of kReadyTiles consecutive tiles, the
// hidden rows whose ids of the block's tiles it has written (ready[b] reaches
// tiles_in_block * M when block b is complete); the gather waits on those
// counters instead of on the scoring kernel's completion. The counters, and
// after them one stop word that the scoring kernel sets if it aborts, live in
// the workspace's ticket area, zeroed by the projection kernel every call.
constexpr int kReadyTiles = 16;
__host__ __device__ inline int ready_blocks(int64_t tiles) {
  return (int)((tiles + kReadyTiles - 1) / kReadyTiles);
}
inline int ready_words(int64_t tiles) { return ready_blocks(tiles) + 1; }  // counters + stop

// K3 for long rows and few of them (global Top-k, several CTAs per row):
// `zero` holds row_select_multi_ints(M) ints that are zero on entry (the
// projection kernel zeroes them), `scratch` row_select_multi_bytes(M, k)
// bytes (no initial value). Same result and order as launch_segment_topk with
// one segment per row. The first histogram of row m (kSelectHistBins counts of
// the scores' top kSelectHistBits order bits, float_key(score) >> 20) is at
// zero + row_select_multi_hist0(m); hist0_filled: the score writeback has
// counted it already.
constexpr int kSelectHistBits = 12;
constexpr int kSelectHistBins = 1 << kSelectHistBits;
bool row_select_multi(int64_t n, int M, int k);
int row_select_multi_ints(int M);
int row_select_multi_hist0(int m);
size_t row_select_multi_bytes(int M, int k);
cudaError_t launch_row_select_multi(const float* S, const int32_t* token_ids, int64_t n, int M,
                                    int k, int32_t* out_ids, float* out_scores, int* zero,
                                    void* scratch, bool hist0_filled, cudaStream_t s);

// K5 (+K6 fused when q != nullptr): L[m,j] = W[ids[m,j]] . h[m]; q = softmax.
// `tickets` (M ints, zero on entry, left zero on exit) enable the fusion.
// span > 0: warps take the candidates in blocks of `span` columns (all rows
// of a block together) instead of row by row; see the kernel.
// ready != nullptr: wait on the scoring kernel's ready counters (tiles of
// k_tile columns, `tiles` in all) instead of on its completion.
// row_of_id != nullptr: W holds n_rows rows, the row of vocabulary id i being
// row_of_id[i] (a vocabulary shard; ids outside it are bad ids).
cudaError_t launch_gather_logits(const bf16_t* W, const bf16_t* h, const int32_t* ids, int64_t n,
                                 int d, int M, int K, float* logits, float* q, float inv_temp,
                                 int* tickets, int* err, cudaStream_t s, int span = 0,
                                 const int* ready = nullptr, int k_tile = 0, int64_t tiles = 0,
                                 const int32_t* row_of_id = nullptr, int64_t n_rows = 0);

// Vocabulary shards: per row of L (M x K), stats[m] = (max_j L/T, sum_j
// exp(L/T - max)); and q of one shard's candidates from all G shards' stats
// (G x M x 2, any order): q = exp(L/T - Mx) / Z, Mx = max of the maxima,
// Z = sum_g sum_g exp(max_g - Mx).
cudaError_t launch_row_stats(const float* L, int M, int K, float inv_temp, float* stats,
                             cudaStream_t s);
cudaError_t launch_shard_softmax(const float* all_stats, int G, const float* L, int M, int K,
                                 float inv_temp, float* q, cudaStream_t s);

// K6 standalone: row softmax of an M x K matrix (any K).
cudaError_t launch_row_softmax(const float* L, int M, int64_t K, float inv_temp, float* q,
                               cudaStream_t s);

// Tensor-core row products (rows_tc.cu): out[m * ldo + j] = X[j] . Y[m] for
// every row j of X (n x kdim) and hidden vector m of Y (M x kdim); any M
// (blocks of kRowsTcMaxN). Used for the dense and pruned heads and the
// global path's score writeback.
constexpr int kRowsTcMaxN = 256;
cudaError_t launch_rows_dense_tc(const bf16_t* X, int64_t n, int kdim, const bf16_t* Y, int M,
                                 float* out, int64_t ldo, int* err, cudaStream_t s);

// Cluster-level route: ids[m, j*group + t] = groups[m, j]*group + t (M x G*group).
cudaError_t launch_expand_groups(const int32_t* groups, int M, int G, int group, int64_t ngroups,
                                 int32_t* ids, int* err, cudaStream_t s);

// K8: per row, the k_sel (<= kDraftMaxK) largest q (ties: smaller id) with
// value parent * q, and optionally a Gumbel-max draw from q (uniforms M x K).
constexpr int kDraftMaxK = 16;
cudaError_t launch_draft_select(const float* q, const int32_t* ids, int M, int K, int k_sel,
                                const float* parent_value, const float* uniforms, int32_t* top_ids,
                                float* top_q, float* top_value, int32_t* sample_id,
                                float* sample_q, cudaStream_t s);
// K9: chain verification of B chains of Kd drafted tokens against dense
// target rows p (B x (Kd + 1) x n), candidate lists B x Kd x K.
cudaError_t launch_verify_chain(const float* p, int64_t n, int B, int Kd, const int32_t* x,
                                const int32_t* cand_ids, const float* cand_q, int K, const float* r,
                                const float* u, int32_t* out_tokens, int32_t* out_count, int* err,
                                cudaStream_t s);

// ---- serving operators around the head
// Block tables and slot maps of a step's new tokens (paged.cu).
cudaError_t launch_page_plan(const int32_t* lens, const int32_t* fresh, int S, int32_t* table,
                             int width, const int32_t* free_pages, int free_cap,
                             const int32_t* free_count, int page, int T, int32_t* slots,
                             int32_t* positions, int32_t* cu, int32_t* granted,
                             int32_t* free_left, int* err, cudaStream_t s);

struct CacheStrides {
  int64_t page, token, head;  // bytes
};
// Validated arguments of lmhead_chunk_attention; strides in bytes.
struct AttnArgs {
  int dtype;  // lmhead_dtype
  const void *q, *k, *v;
  int64_t q_tok, q_head, k_tok, k_head, v_tok, v_head;
  void *k_cache, *v_cache;
  CacheStrides ks, vs;
  int64_t pages;
  int page_shift;  // log2 of the page size
  const int32_t *table, *lens, *cu, *granted, *slots;  // granted: or nullptr
  int width, S, T, heads, kv_heads, dim, window;
  const uint64_t* tree;
  float scale;
  void* out;
  float* lse;
};
// The new tokens' K and V to their slots, if given, and the attention of the
// chunk over the pages (attention.cu); scratch holds attention_scratch_bytes(...)
// bytes.
size_t attention_scratch_bytes(int S, int T, int heads, int kv_heads, int dim);
cudaError_t launch_attention(const AttnArgs& a, void* scratch, int* err, cudaStream_t s);

// 4-bit rows with group scales (q4.cu): out[m * ldo + j] = row_j . h[m] over
// rows 0..n-1, or over rows ids[m * K + j] when ids != nullptr.
struct Q4Args {
  int dtype;
  const uint8_t* codes;
  const void *scales, *mins, *h;
  const int32_t* ids;
  int64_t n;
  int d, group, M, K;
  float* out;
};
cudaError_t launch_q4(const Q4Args& a, int* err, cudaStream_t s);

// Beam selection and the reordering of the beams' states (beams.cu).
constexpr int kBeamMaxK = 32;
constexpr int kBeamMaxBeams = 256;
struct BeamArgs {
  int dtype;  // lmhead_dtype
  const void* logits;
  int64_t row_stride, n;  // elements
  const float* scores;
  const int32_t* ids;
  const uint8_t* finished;
  int S, beams, k, eos;
  int32_t *parent, *token;
  float* out_score;
};
size_t beam_scratch_bytes(int S, int beams, int64_t n, int k);
cudaError_t launch_beam_select(const BeamArgs& a, void* scratch, cudaStream_t s);
constexpr int kReorderMax = 8;
struct ReorderArgs {
  const void* src[kReorderMax];
  void* dst[kReorderMax];
  int64_t bytes[kReorderMax];  // of one row
  int count, S, beams, k;
  const int32_t* parent;
};
cudaError_t launch_beam_reorder(const ReorderArgs& a, int* err, cudaStream_t s);

// ---- operators of a step over the paged cache
// Most tokens of a request where kernels walk over them in blocks: places behind the
// last block stay within 32 bits.
constexpr int kMaxTokens = INT32_MAX - 65535;

// Rotary positions (rotary.cu); strides in elements, k may be nullptr.
struct RotaryArgs {
  int dtype;  // lmhead_dtype
  const void *q, *k;
  void *qo, *ko;
  int64_t q_tok, q_head, k_tok, k_head, qo_tok, qo_head, ko_tok, ko_head;
  const int32_t* pos;
  const int64_t* turns;
  int T, heads, kv_heads, dim, rot;  // kv_heads 0 without k
  bool interleaved, backward;
  float magnitude;
};
cudaError_t launch_rotary(const RotaryArgs& a, cudaStream_t s);

// Draft trees against the target's probabilities (tree.cu).
constexpr int kTreeMaxNodes = 64;
struct TreeArgs {
  const float* p;  // T x n
  int64_t n;
  const int32_t *tokens, *parent, *cu, *granted;
  const float *r, *u;
  const int32_t* cand_ids;  // T x K, or nullptr
  const float* cand_q;
  int S, T, K, depth;
  int32_t *out_tokens, *out_path, *out_accepted;
};
cudaError_t launch_verify_tree(const TreeArgs& a, int* err, cudaStream_t s);

// Sums of attention weights a cached token (weights.cu); strides in bytes.
struct WeightArgs {
  int dtype;
  const void* q;
  int64_t q_tok, q_head;
  const void* k_cache;
  CacheStrides ks;
  int64_t pages;
  int page_shift;
  const int32_t *table, *lens, *cu, *granted;
  int width, S, T, heads, kv_heads, dim, window;
  const uint64_t* tree;
  const float* lse;
  float scale, decay;
  void* weights;
  CacheStrides ws;
};
size_t weights_scratch_bytes();
cudaError_t launch_cache_weights(const WeightArgs& a, void* scratch, int* err, cudaStream_t s);

// Tokens that stay, rows moved together and pages given back (keep.cu).
struct SelectArgs {
  const void* weights;
  CacheStrides ws;
  int64_t pages;
  int page, width, S, kv_heads, budget, sinks, recent;
  const int32_t *table, *lens;
  int32_t* kept;
};
cudaError_t launch_cache_select(const SelectArgs& a, int* err, cudaStream_t s);
constexpr int kKeepMax = 8;
struct KeepTensor {
  void* base;
  CacheStrides st;
  int row;                 // bytes of a token and head
  int vec, slice, slices;  // set by the launch
};
struct KeepArgs {
  KeepTensor t[kKeepMax];
  int count;
  int64_t pages;
  int page, width, S, kv_heads, n;
  bool per_head;
  const int32_t *table, *kept, *first;
  int32_t* new_lens;
};
cudaError_t launch_cache_keep(KeepArgs a, int* err, cudaStream_t s);
struct ReleaseArgs {
  const int32_t *lens, *new_lens, *cu, *granted, *table;
  int S, width, page, free_cap;
  int32_t* free_pages;
  const int32_t* free_count;
  int32_t* free_left;
};
cudaError_t launch_page_release(const ReleaseArgs& a, int* err, cudaStream_t s);

int* device_error_word();  // this device's error word (nullptr on failure)
// Budget (SM cycles) of the tensor-core kernels' role waits; tc::kWaitCycles
// unless lmhead_debug_set_wait_cycles changed it.
long long role_wait_cycles();

// TMA map of a rows x cols bf16 row-major matrix: box_rows x box_cols
// (box_cols * 2 == 128 bytes), 128-byte swizzle, zero fill out of bounds.
bool make_bf16_map(CUtensorMap* map, const void* base, uint64_t rows, uint64_t cols,
                   uint32_t box_rows, uint32_t box_cols);
// TMA map of a paged cache (16-bit elements, one head's box of box_tokens rows of
// 64): dimensions (dim, heads, tokens, pages) when head_first, else (dim, tokens,
// heads, pages).
bool make_cache_map(CUtensorMap* map, const void* base, bool bf16, int dim, int page_tokens,
                    int heads, int64_t pages, const CacheStrides& st, int box_tokens,
                    bool head_first);
// TMA map of tokens x heads x dim (16-bit elements, strides in bytes): boxes of 64
// elements of box_heads heads of box_tokens tokens.
bool make_rows_map(CUtensorMap* map, const void* base, bool bf16, int dim, int heads, int64_t tokens,
                   int64_t head_stride, int64_t token_stride, int box_heads, int box_tokens);
int sm_count();  // SMs of the current device (cached)

}  // namespace lmhead
