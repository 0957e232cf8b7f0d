// C entry points of the serving operators (include/lmhead.h): host-side
// validation and launches.
#include <math.h>
#include <stdint.h>

#include "common.cuh"
#include "kernels.h"
#include "lmhead.h"

using namespace lmhead;

namespace {

constexpr int kMaxRows = 1 << 20;
constexpr int kMaxRequests = 1 << 16;  // of one attention call
constexpr int kMaxDim = 65536;

inline bool aligned(const void* p, uintptr_t a) {
  return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0;
}
// Do two ranges of bytes have one in common?
inline bool meet(const void* a, int64_t a_bytes, const void* b, int64_t b_bytes) {
  const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
  return x < y + (uintptr_t)b_bytes && y < x + (uintptr_t)a_bytes;
}
inline int status(cudaError_t e) { return e == cudaSuccess ? LMHEAD_OK : LMHEAD_ERR_CUDA; }

// Strides of a tensor read 16 bytes at a time: non-negative multiples of 8
// elements, small enough that byte offsets stay far from 2^63.
inline bool stride_ok(int64_t s) { return s >= 0 && s % 8 == 0 && s < (1ll << 38); }

int check_attention(int heads, int kv_heads, int dim, int S, int T) {
  if (S < 1 || S > kMaxRequests || T < 1 || kv_heads < 1 || heads < kv_heads || heads % kv_heads ||
      heads > 65535 || heads / kv_heads > 128)
    return LMHEAD_ERR_SHAPE;
  if ((int64_t)T * heads > INT32_MAX) return LMHEAD_ERR_SHAPE;
  if (dim != 64 && dim != 128) return LMHEAD_ERR_UNSUPPORTED;
  return LMHEAD_OK;
}

int check_q4(int dtype, int64_t n, int d, int group, int M) {
  if (dtype != LMHEAD_BF16 && dtype != LMHEAD_FP16) return LMHEAD_ERR_UNSUPPORTED;
  if (group != 32 && group != 64 && group != 128) return LMHEAD_ERR_UNSUPPORTED;
  if (n < 1 || n > INT32_MAX || d < group || d % group || d > kMaxDim || M < 1 || M > 65535)
    return LMHEAD_ERR_SHAPE;
  return LMHEAD_OK;
}

int q4(int dtype, const void* codes, const void* scales, const void* mins, const void* h,
       const int32_t* ids, int64_t n, int d, int group, int M, int K, float* out,
       lmhead_stream stream) {
  if (!aligned(codes, 16) || !aligned(scales, 2) || !aligned(mins, 2) || !aligned(h, 16))
    return LMHEAD_ERR_ALIGN;
  Q4Args a = {};
  a.dtype = dtype;
  a.codes = static_cast<const uint8_t*>(codes);
  a.scales = scales;
  a.mins = mins;
  a.h = h;
  a.ids = ids;
  a.n = n;
  a.d = d;
  a.group = group;
  a.M = M;
  a.K = K;
  a.out = out;
  return status(launch_q4(a, device_error_word(), (cudaStream_t)stream));
}

int check_beams(int S, int beams, int64_t n, int k) {
  if (S < 1 || beams < 1 || n < 1 || k < 1) return LMHEAD_ERR_SHAPE;
  if (k > kBeamMaxK || beams > kBeamMaxBeams) return LMHEAD_ERR_UNSUPPORTED;
  if ((int64_t)S * beams > 65535 || n > (1ll << 30) || beams * n > INT32_MAX)
    return LMHEAD_ERR_SHAPE;
  return LMHEAD_OK;
}

}  // namespace

extern "C" {

int lmhead_page_plan(const int32_t* lens, const int32_t* new_lens, int S, int32_t* table,
                     int width, const int32_t* free_pages, int free_cap,
                     const int32_t* free_count, int page_size, int max_tokens,
                     int32_t* out_slots, int32_t* out_positions, int32_t* out_cu,
                     int32_t* out_granted, int32_t* out_free_left, lmhead_stream stream) {
  // (an empty list of free pages may have no address)
  if (!lens || !new_lens || !table || (!free_pages && free_cap != 0) || !free_count || !out_slots ||
      !out_positions || !out_cu || !out_granted || !out_free_left)
    return LMHEAD_ERR_NULL;
  if (S < 1 || S > kMaxRows || width < 1 || free_cap < 0 || page_size < 1 || page_size > 65536 ||
      max_tokens < 1 || (int64_t)S * width > INT32_MAX)
    return LMHEAD_ERR_SHAPE;
  if (out_free_left == free_count) return LMHEAD_ERR_SHAPE;
  return status(launch_page_plan(lens, new_lens, S, table, width, free_pages, free_cap, free_count,
                                 page_size, max_tokens, out_slots, out_positions, out_cu,
                                 out_granted, out_free_left, device_error_word(),
                                 (cudaStream_t)stream));
}

size_t lmhead_chunk_attention_workspace_size(int S, int T, int heads, int kv_heads, int dim) {
  if (check_attention(heads, kv_heads, dim, S, T) != LMHEAD_OK) return 0;
  return attention_scratch_bytes(S, T, heads, kv_heads, dim);
}

int lmhead_chunk_attention(int dtype, const void* q, int64_t q_tok, int64_t q_head, const void* k,
                           int64_t k_tok, int64_t k_head, const void* v, int64_t v_tok,
                           int64_t v_head, void* k_cache, int64_t kc_page, int64_t kc_token,
                           int64_t kc_head, void* v_cache, int64_t vc_page, int64_t vc_token,
                           int64_t vc_head, int64_t pages, int page_size, const int32_t* table,
                           int width, const int32_t* lens, const int32_t* cu,
                           const int32_t* slots, const uint64_t* tree, int S, int T, int heads,
                           int kv_heads, int dim, int window, float scale, void* out,
                           float* out_lse, void* workspace, size_t workspace_bytes,
                           lmhead_stream stream) {
  return lmhead_chunk_attention_granted(
      dtype, q, q_tok, q_head, k, k_tok, k_head, v, v_tok, v_head, k_cache, kc_page, kc_token,
      kc_head, v_cache, vc_page, vc_token, vc_head, pages, page_size, table, width, lens, cu,
      nullptr, slots, tree, S, T, heads, kv_heads, dim, window, scale, out, out_lse, workspace,
      workspace_bytes, stream);
}

int lmhead_chunk_attention_granted(
    int dtype, const void* q, int64_t q_tok, int64_t q_head, const void* k, int64_t k_tok,
    int64_t k_head, const void* v, int64_t v_tok, int64_t v_head, void* k_cache, int64_t kc_page,
    int64_t kc_token, int64_t kc_head, void* v_cache, int64_t vc_page, int64_t vc_token,
    int64_t vc_head, int64_t pages, int page_size, const int32_t* table, int width,
    const int32_t* lens, const int32_t* cu, const int32_t* granted, const int32_t* slots,
    const uint64_t* tree, int S, int T, int heads, int kv_heads, int dim, int window, float scale,
    void* out, float* out_lse, void* workspace, size_t workspace_bytes, lmhead_stream stream) {
  if (!q || !k_cache || !v_cache || !table || !lens || !cu || !out) return LMHEAD_ERR_NULL;
  if ((k == nullptr) != (v == nullptr) || (k && !slots)) return LMHEAD_ERR_NULL;
  if (dtype != LMHEAD_BF16 && dtype != LMHEAD_FP16) return LMHEAD_ERR_UNSUPPORTED;
  const int st = check_attention(heads, kv_heads, dim, S, T);
  if (st != LMHEAD_OK) return st;
  if (width < 1 || (int64_t)S * width > INT32_MAX || pages < 1 || window < 0 || !(scale > 0.f) ||
      !isfinite(scale))
    return LMHEAD_ERR_SHAPE;
  int shift = 4;
  while (shift < 8 && (1 << shift) != page_size) ++shift;
  if ((1 << shift) != page_size) return LMHEAD_ERR_UNSUPPORTED;
  if (pages > (INT32_MAX >> shift) || width > (INT32_MAX >> shift)) return LMHEAD_ERR_SHAPE;
  if (tree && window) return LMHEAD_ERR_UNSUPPORTED;
  const int64_t strides[] = {q_tok, q_head, kc_page, kc_token, kc_head, vc_page, vc_token, vc_head};
  for (int64_t x : strides)
    if (!stride_ok(x)) return LMHEAD_ERR_SHAPE;
  if (kc_token < dim || vc_token < dim || kc_page < dim || vc_page < dim ||
      (kv_heads > 1 && (kc_head < dim || vc_head < dim)))
    return LMHEAD_ERR_SHAPE;
  if (k && (!stride_ok(k_tok) || !stride_ok(k_head) || !stride_ok(v_tok) || !stride_ok(v_head)))
    return LMHEAD_ERR_SHAPE;
  if (!aligned(q, 16) || !aligned(k, 16) || !aligned(v, 16) || !aligned(k_cache, 16) ||
      !aligned(v_cache, 16) || !aligned(out, 16) || !aligned(tree, 8))
    return LMHEAD_ERR_ALIGN;
  if (!workspace || !aligned(workspace, 256) ||
      workspace_bytes < attention_scratch_bytes(S, T, heads, kv_heads, dim))
    return LMHEAD_ERR_WORKSPACE;
  AttnArgs a = {};
  a.dtype = dtype;
  a.q = q;
  a.k = k;
  a.v = v;
  a.q_tok = q_tok * 2;
  a.q_head = q_head * 2;
  a.k_tok = k_tok * 2;
  a.k_head = k_head * 2;
  a.v_tok = v_tok * 2;
  a.v_head = v_head * 2;
  a.k_cache = k_cache;
  a.v_cache = v_cache;
  a.ks = {kc_page * 2, kc_token * 2, kc_head * 2};
  a.vs = {vc_page * 2, vc_token * 2, vc_head * 2};
  a.pages = pages;
  a.page_shift = shift;
  a.table = table;
  a.lens = lens;
  a.cu = cu;
  a.granted = granted;
  a.slots = slots;
  a.width = width;
  a.S = S;
  a.T = T;
  a.heads = heads;
  a.kv_heads = kv_heads;
  a.dim = dim;
  a.window = window;
  a.tree = tree;
  a.scale = scale;
  a.out = out;
  a.lse = out_lse;
  // the stride of a single head means nothing
  if (kv_heads == 1) a.ks.head = a.ks.token, a.vs.head = a.vs.token;
  return status(launch_attention(a, workspace, device_error_word(), (cudaStream_t)stream));
}

int lmhead_q4_head(int dtype, const void* codes, const void* scales, const void* mins,
                   const void* h, int64_t n, int d, int group, int M, float* out_logits,
                   lmhead_stream stream) {
  if (!codes || !scales || !h || !out_logits) return LMHEAD_ERR_NULL;
  const int st = check_q4(dtype, n, d, group, M);
  if (st != LMHEAD_OK) return st;
  return q4(dtype, codes, scales, mins, h, nullptr, n, d, group, M, 0, out_logits, stream);
}

int lmhead_q4_gather_logits(int dtype, const void* codes, const void* scales, const void* mins,
                            const void* h, const int32_t* ids, int64_t n, int d, int group, int M,
                            int K, float* out_logits, lmhead_stream stream) {
  if (!codes || !scales || !h || !ids || !out_logits) return LMHEAD_ERR_NULL;
  const int st = check_q4(dtype, n, d, group, M);
  if (st != LMHEAD_OK) return st;
  if (K < 1 || (int64_t)M * K > INT32_MAX) return LMHEAD_ERR_SHAPE;
  return q4(dtype, codes, scales, mins, h, ids, n, d, group, M, K, out_logits, stream);
}

size_t lmhead_beam_workspace_size(int S, int beams, int64_t n, int k) {
  if (check_beams(S, beams, n, k) != LMHEAD_OK) return 0;
  return beam_scratch_bytes(S, beams, n, k);
}

int lmhead_beam_select(int dtype, const void* logits, int64_t row_stride, const float* scores,
                       const int32_t* ids, const void* finished, int S, int beams, int64_t n,
                       int k, int eos, int32_t* out_parent, int32_t* out_token, float* out_score,
                       void* workspace, size_t workspace_bytes, lmhead_stream stream) {
  if (!logits || !scores || !out_parent || !out_token || !out_score) return LMHEAD_ERR_NULL;
  if (dtype != LMHEAD_BF16 && dtype != LMHEAD_FP16 && dtype != LMHEAD_FP32)
    return LMHEAD_ERR_UNSUPPORTED;
  const int st = check_beams(S, beams, n, k);
  if (st != LMHEAD_OK) return st;
  if (row_stride < n || row_stride > (1ll << 40)) return LMHEAD_ERR_SHAPE;
  if (!aligned(logits, dtype == LMHEAD_FP32 ? 4 : 2)) return LMHEAD_ERR_ALIGN;
  if (!workspace || !aligned(workspace, 256) ||
      workspace_bytes < beam_scratch_bytes(S, beams, n, k))
    return LMHEAD_ERR_WORKSPACE;
  BeamArgs a = {};
  a.dtype = dtype;
  a.logits = logits;
  a.row_stride = row_stride;
  a.n = n;
  a.scores = scores;
  a.ids = ids;
  a.finished = static_cast<const uint8_t*>(finished);
  a.S = S;
  a.beams = beams;
  a.k = k;
  a.eos = eos;
  a.parent = out_parent;
  a.token = out_token;
  a.out_score = out_score;
  return status(launch_beam_select(a, workspace, (cudaStream_t)stream));
}

int lmhead_beam_reorder(const int32_t* parent, int S, int beams, int k, int count,
                        const void* const* src, void* const* dst, const int64_t* row_bytes,
                        lmhead_stream stream) {
  if (!parent || !src || !dst || !row_bytes) return LMHEAD_ERR_NULL;
  if (S < 1 || beams < 1 || k < 1 || (int64_t)S * k > INT32_MAX || (int64_t)S * beams > INT32_MAX)
    return LMHEAD_ERR_SHAPE;
  if (count < 1 || count > kReorderMax) return LMHEAD_ERR_UNSUPPORTED;
  ReorderArgs a = {};
  for (int i = 0; i < count; ++i) {
    if (!src[i] || !dst[i]) return LMHEAD_ERR_NULL;
    if (row_bytes[i] < 1 || row_bytes[i] > (1ll << 29)) return LMHEAD_ERR_SHAPE;
    a.src[i] = src[i];
    a.dst[i] = dst[i];
    a.bytes[i] = row_bytes[i];
  }
  // what one CTA writes is read by no other: moving rows within one buffer, as any
  // destination that meets a source, the parents or another destination, is refused
  const int64_t from = (int64_t)S * beams, to = (int64_t)S * k;
  for (int i = 0; i < count; ++i) {
    if (meet(dst[i], to * row_bytes[i], parent, to * 4)) return LMHEAD_ERR_SHAPE;
    for (int j = 0; j < count; ++j)
      if (meet(dst[i], to * row_bytes[i], src[j], from * row_bytes[j]) ||
          (i != j && meet(dst[i], to * row_bytes[i], dst[j], to * row_bytes[j])))
        return LMHEAD_ERR_SHAPE;
  }
  a.count = count;
  a.S = S;
  a.beams = beams;
  a.k = k;
  a.parent = parent;
  return status(launch_beam_reorder(a, device_error_word(), (cudaStream_t)stream));
}

}  // extern "C"
