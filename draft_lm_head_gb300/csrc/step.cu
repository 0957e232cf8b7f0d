// C entry points of the operators of a step over the paged cache
// (include/lmhead.h): host-side validation and launches.
#include <math.h>
#include <stdint.h>

#include "common.cuh"
#include "kernels.h"
#include "lmhead.h"

using namespace lmhead;

namespace {

constexpr int kMaxRows = 1 << 20;
constexpr int kMaxRequests = 1 << 16;  // of one call over a cache's rows

inline bool aligned(const void* p, uintptr_t a) {
  return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0;
}
// Do two ranges of bytes have one in common?
inline bool meet(const void* a, int64_t a_bytes, const void* b, int64_t b_bytes) {
  const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
  return x < y + (uintptr_t)b_bytes && y < x + (uintptr_t)a_bytes;
}
inline int status(cudaError_t e) { return e == cudaSuccess ? LMHEAD_OK : LMHEAD_ERR_CUDA; }
// Strides small enough that byte offsets stay far from 2^63.
inline bool stride_ok(int64_t s) { return s >= 0 && s < (1ll << 38); }
inline bool sixteen(int64_t s) { return s % 8 == 0; }  // 16-bit elements

// Sizes of a table of pages.
int check_table(int S, int width, int64_t pages, int page_size) {
  if (S < 1 || S > kMaxRequests || width < 1 || (int64_t)S * width > INT32_MAX || pages < 1 ||
      pages > INT32_MAX || page_size < 1 || page_size > 65536 ||
      (int64_t)width * page_size > INT32_MAX)
    return LMHEAD_ERR_SHAPE;
  return LMHEAD_OK;
}

}  // namespace

extern "C" {

int lmhead_rotary(int dtype, const void* q, int64_t q_tok, int64_t q_head, const void* k,
                  int64_t k_tok, int64_t k_head, const int32_t* positions, const int64_t* turns,
                  int T, int heads, int kv_heads, int dim, int rot, int interleaved, int backward,
                  float magnitude, void* out_q, int64_t oq_tok, int64_t oq_head, void* out_k,
                  int64_t ok_tok, int64_t ok_head, lmhead_stream stream) {
  if (!q || !positions || !turns || !out_q || (k == nullptr) != (out_k == nullptr))
    return LMHEAD_ERR_NULL;
  if (dtype != LMHEAD_BF16 && dtype != LMHEAD_FP16 && dtype != LMHEAD_FP32)
    return LMHEAD_ERR_UNSUPPORTED;
  if (T < 1 || heads < 1 || heads > 65535 || (k && (kv_heads < 1 || kv_heads > 65535)) || dim < 2 ||
      dim > 65536 || rot < 2 || rot > dim || rot % 2 || !isfinite(magnitude))
    return LMHEAD_ERR_SHAPE;
  if ((int64_t)T * (heads + (k ? kv_heads : 0)) > INT32_MAX) return LMHEAD_ERR_SHAPE;
  const int64_t strides[] = {q_tok, q_head, oq_tok, oq_head, k_tok, k_head, ok_tok, ok_head};
  for (int i = 0; i < (k ? 8 : 4); ++i)
    if (!stride_ok(strides[i])) return LMHEAD_ERR_SHAPE;
  auto span = [&](int64_t tok, int64_t head, int h) {  // elements from the first to the last
    return (T - 1) * tok + (h - 1) * head + dim;
  };
  for (int i = 0; i < (k ? 8 : 4); ++i)
    if (strides[i] > (1ll << 58) / (i % 2 == 0 ? T : 65535)) return LMHEAD_ERR_SHAPE;
  // a place of the results is written once: tokens lie apart by all of their heads,
  // or heads by all of their tokens
  auto apart = [&](int64_t tok, int64_t head, int h) {
    return (T == 1 || tok >= dim) && (h == 1 || head >= dim) &&
           (T == 1 || h == 1 || tok >= (h - 1) * head + dim || head >= (T - 1) * tok + dim);
  };
  if (!apart(oq_tok, oq_head, heads) || (k && !apart(ok_tok, ok_head, kv_heads)))
    return LMHEAD_ERR_SHAPE;
  const int size = dtype == LMHEAD_FP32 ? 4 : 2;
  // in place, or to somewhere else: no thread may write what another is to read
  auto same_or_apart = [&](const void* in, int64_t tok, int64_t head, const void* out, int64_t otok,
                           int64_t ohead, int h) {
    if (in == out) return (T == 1 || tok == otok) && (h == 1 || head == ohead);
    return !meet(in, span(tok, head, h) * size, out, span(otok, ohead, h) * size);
  };
  if (!same_or_apart(q, q_tok, q_head, out_q, oq_tok, oq_head, heads)) return LMHEAD_ERR_SHAPE;
  if (k && !same_or_apart(k, k_tok, k_head, out_k, ok_tok, ok_head, kv_heads)) return LMHEAD_ERR_SHAPE;
  // q and k may lie in one tensor, their places among one another's, but share none
  auto clear = [&](const void* x, int64_t x_tok, int64_t x_head, int x_h, const void* y, int64_t y_tok,
                   int64_t y_head, int y_h) {
    if (!meet(x, span(x_tok, x_head, x_h) * size, y, span(y_tok, y_head, y_h) * size)) return true;
    const int64_t bytes = (int64_t)(reinterpret_cast<uintptr_t>(y) - reinterpret_cast<uintptr_t>(x));
    if (bytes % size != 0) return false;
    // blocks of x_n and y_n elements, repeated every `step`, y's begin `bytes` behind x's
    auto between = [&](int64_t x_n, int64_t y_n, int64_t step) {
      int64_t d = bytes / size % step;
      if (d < 0) d += step;
      return x_n <= d && d + y_n <= step;
    };
    return (T > 1 && x_tok == y_tok &&
            between((x_h - 1) * x_head + dim, (y_h - 1) * y_head + dim, x_tok)) ||
           (x_h > 1 && y_h > 1 && x_head == y_head &&
            between((T - 1) * x_tok + dim, (T - 1) * y_tok + dim, x_head));
  };
  if (k && (!clear(out_q, oq_tok, oq_head, heads, out_k, ok_tok, ok_head, kv_heads) ||
            !clear(out_q, oq_tok, oq_head, heads, k, k_tok, k_head, kv_heads) ||
            !clear(out_k, ok_tok, ok_head, kv_heads, q, q_tok, q_head, heads)))
    return LMHEAD_ERR_SHAPE;
  if (!aligned(q, size) || !aligned(k, size) || !aligned(out_q, size) || !aligned(out_k, size) ||
      !aligned(turns, 8))
    return LMHEAD_ERR_ALIGN;
  RotaryArgs a = {};
  a.dtype = dtype;
  a.q = q;
  a.k = k;
  a.qo = out_q;
  a.ko = out_k;
  a.q_tok = q_tok;
  a.q_head = q_head;
  a.qo_tok = oq_tok;
  a.qo_head = oq_head;
  if (k) {
    a.k_tok = k_tok;
    a.k_head = k_head;
    a.ko_tok = ok_tok;
    a.ko_head = ok_head;
    a.kv_heads = kv_heads;
  }
  a.pos = positions;
  a.turns = turns;
  a.T = T;
  a.heads = heads;
  a.dim = dim;
  a.rot = rot;
  a.interleaved = interleaved != 0;
  a.backward = backward != 0;
  a.magnitude = magnitude;
  return status(launch_rotary(a, (cudaStream_t)stream));
}

int lmhead_verify_tree(const float* p, int64_t n, const int32_t* tokens, const int32_t* parent,
                       const int32_t* cu, const int32_t* granted, const float* r, const float* u,
                       const int32_t* cand_ids, const float* cand_q, int K, int S, int T, int depth,
                       int32_t* out_tokens, int32_t* out_path, int32_t* out_accepted,
                       lmhead_stream stream) {
  if (!p || !tokens || !parent || !cu || !r || !u || !out_tokens || !out_path || !out_accepted ||
      (cand_ids == nullptr) != (cand_q == nullptr))
    return LMHEAD_ERR_NULL;
  if (n < 1 || n > INT32_MAX || S < 1 || S > kMaxRequests || T < 1 || depth < 0 ||
      depth >= kTreeMaxNodes || (cand_ids && K < 1))
    return LMHEAD_ERR_SHAPE;
  const int64_t out_bytes = 4ll * S * (depth + 1);
  if (cand_ids && K > kSelectMaxK) return LMHEAD_ERR_UNSUPPORTED;
  if (meet(out_tokens, out_bytes, out_path, out_bytes) || meet(out_tokens, out_bytes, out_accepted, 4ll * S) ||
      meet(out_path, out_bytes, out_accepted, 4ll * S))
    return LMHEAD_ERR_SHAPE;
  TreeArgs a = {};
  a.p = p;
  a.n = n;
  a.tokens = tokens;
  a.parent = parent;
  a.cu = cu;
  a.granted = granted;
  a.r = r;
  a.u = u;
  a.cand_ids = cand_ids;
  a.cand_q = cand_q;
  a.S = S;
  a.T = T;
  a.K = cand_ids ? K : 0;
  a.depth = depth;
  a.out_tokens = out_tokens;
  a.out_path = out_path;
  a.out_accepted = out_accepted;
  return status(launch_verify_tree(a, device_error_word(), (cudaStream_t)stream));
}

int lmhead_cache_keep(int count, void* const* base, const int64_t* page_stride,
                      const int64_t* token_stride, const int64_t* head_stride,
                      const int64_t* row_bytes, int64_t pages, int page_size, int kv_heads,
                      const int32_t* table, int width, const int32_t* kept, int n, int per_head,
                      const int32_t* first, int S, int32_t* out_new_lens, lmhead_stream stream) {
  if (!base || !page_stride || !token_stride || !head_stride || !row_bytes || !table || !kept ||
      !out_new_lens)
    return LMHEAD_ERR_NULL;
  if (count < 1 || count > kKeepMax) return LMHEAD_ERR_UNSUPPORTED;
  const int st = check_table(S, width, pages, page_size);
  if (st != LMHEAD_OK) return st;
  if (kv_heads < 1 || kv_heads > 65535 || n < 1 || n > (1 << 30) ||
      (int64_t)S * n > INT32_MAX)
    return LMHEAD_ERR_SHAPE;
  if (first && meet(first, 4ll * S, out_new_lens, 4ll * S)) return LMHEAD_ERR_SHAPE;
  KeepArgs a = {};
  for (int i = 0; i < count; ++i) {
    if (!base[i]) return LMHEAD_ERR_NULL;
    const int64_t row = row_bytes[i];
    if (row < 1 || row > (1 << 20) || !stride_ok(page_stride[i]) || !stride_ok(token_stride[i]) ||
        !stride_ok(head_stride[i]))
      return LMHEAD_ERR_SHAPE;
    // rows of different places do not meet
    if ((page_size > 1 && token_stride[i] < row) || (pages > 1 && page_stride[i] < row) ||
        (kv_heads > 1 && head_stride[i] < row))
      return LMHEAD_ERR_SHAPE;
    for (int j = 0; j < i; ++j) {  // bytes that would be moved twice
      if (base[j] == base[i]) return LMHEAD_ERR_SHAPE;
      if ((pages == 1 || page_stride[j] == page_stride[i]) &&
          (page_size == 1 || token_stride[j] == token_stride[i]) &&
          (kv_heads == 1 || head_stride[j] == head_stride[i]) &&
          meet(base[j], row_bytes[j], base[i], row))
        return LMHEAD_ERR_SHAPE;  // parts of one row
    }
    a.t[i].base = base[i];
    a.t[i].st = {page_stride[i], token_stride[i], head_stride[i]};
    a.t[i].row = (int)row;
  }
  a.count = count;
  a.pages = pages;
  a.page = page_size;
  a.width = width;
  a.S = S;
  a.kv_heads = kv_heads;
  a.n = n;
  a.per_head = per_head != 0;
  a.table = table;
  a.kept = kept;
  a.first = first;
  a.new_lens = out_new_lens;
  return status(launch_cache_keep(a, device_error_word(), (cudaStream_t)stream));
}

int lmhead_page_release(const int32_t* lens, const int32_t* new_lens, const int32_t* cu,
                        const int32_t* granted, int S, const int32_t* table, int width,
                        int32_t* free_pages, int free_cap, const int32_t* free_count,
                        int page_size, int32_t* out_free_left, lmhead_stream stream) {
  if (!lens || !new_lens || !table || (!free_pages && free_cap != 0) || !free_count || !out_free_left)
    return LMHEAD_ERR_NULL;
  if (S < 1 || S > kMaxRows || width < 1 || free_cap < 0 || page_size < 1 || page_size > 65536 ||
      (int64_t)S * width > INT32_MAX || (int64_t)width * page_size > INT32_MAX)
    return LMHEAD_ERR_SHAPE;
  if (out_free_left == free_count) return LMHEAD_ERR_SHAPE;
  // pages are written behind the free ones while tables are read
  if (free_cap > 0 && meet(free_pages, (int64_t)free_cap * 4, table, (int64_t)S * width * 4))
    return LMHEAD_ERR_SHAPE;
  ReleaseArgs a = {};
  a.lens = lens;
  a.new_lens = new_lens;
  a.cu = cu;
  a.granted = granted;
  a.table = table;
  a.S = S;
  a.width = width;
  a.page = page_size;
  a.free_cap = free_cap;
  a.free_pages = free_pages;
  a.free_count = free_count;
  a.free_left = out_free_left;
  return status(launch_page_release(a, device_error_word(), (cudaStream_t)stream));
}

size_t lmhead_cache_weights_workspace_size(int S) {
  return S < 1 || S > kMaxRequests ? 0 : weights_scratch_bytes();
}

int lmhead_cache_weights(int dtype, const void* q, int64_t q_tok, int64_t q_head,
                         const void* k_cache, int64_t kc_page, int64_t kc_token, int64_t kc_head,
                         int64_t pages, int page_size, const int32_t* table, int width,
                         const int32_t* lens, const int32_t* cu, const int32_t* granted,
                         const uint64_t* tree, const float* lse, int S, int T, int heads,
                         int kv_heads, int dim, int window, float scale, float decay,
                         float* weights, int64_t w_page, int64_t w_token, int64_t w_head,
                         void* workspace, size_t workspace_bytes, lmhead_stream stream) {
  if (!q || !k_cache || !table || !lens || !cu || !lse || !weights) return LMHEAD_ERR_NULL;
  if (dtype != LMHEAD_BF16 && dtype != LMHEAD_FP16) return LMHEAD_ERR_UNSUPPORTED;
  if (T < 1 || kv_heads < 1 || heads < kv_heads || heads % kv_heads || heads > 65535 ||
      heads / kv_heads > 128 || (int64_t)T * heads > INT32_MAX)
    return LMHEAD_ERR_SHAPE;
  if (dim != 64 && dim != 128) return LMHEAD_ERR_UNSUPPORTED;
  int shift = 4;
  while (shift < 8 && (1 << shift) != page_size) ++shift;
  if ((1 << shift) != page_size) return LMHEAD_ERR_UNSUPPORTED;
  const int st = check_table(S, width, pages, page_size);
  if (st != LMHEAD_OK) return st;
  if (window < 0 || !(scale > 0.f) || !isfinite(scale) || !(decay >= 0.f) || !isfinite(decay))
    return LMHEAD_ERR_SHAPE;
  if (tree && window) return LMHEAD_ERR_UNSUPPORTED;
  const int64_t strides[] = {q_tok, q_head, kc_page, kc_token, kc_head};
  for (int64_t x : strides)
    if (!stride_ok(x) || !sixteen(x)) return LMHEAD_ERR_SHAPE;
  // rows that meet are no tensor of their own (the stride of a dimension of one means nothing)
  if ((T > 1 && q_tok < dim) || (heads > 1 && q_head < dim) || kc_token < dim || kc_page < dim ||
      (kv_heads > 1 && kc_head < dim))
    return LMHEAD_ERR_SHAPE;
  if (!stride_ok(w_page) || !stride_ok(w_token) || !stride_ok(w_head) || w_token < 1 ||
      (pages > 1 && w_page < 1) || (kv_heads > 1 && w_head < 1))
    return LMHEAD_ERR_SHAPE;
  if (!aligned(q, 16) || !aligned(k_cache, 16) || !aligned(tree, 8) || !aligned(weights, 4))
    return LMHEAD_ERR_ALIGN;
  if (!workspace || !aligned(workspace, 256) || workspace_bytes < weights_scratch_bytes())
    return LMHEAD_ERR_WORKSPACE;
  WeightArgs a = {};
  a.dtype = dtype;
  a.q = q;
  a.q_tok = q_tok * 2;
  a.q_head = q_head * 2;
  a.k_cache = k_cache;
  a.ks = {kc_page * 2, kc_token * 2, kc_head * 2};
  a.pages = pages;
  a.page_shift = shift;
  a.table = table;
  a.lens = lens;
  a.cu = cu;
  a.granted = granted;
  a.width = width;
  a.S = S;
  a.T = T;
  a.heads = heads;
  a.kv_heads = kv_heads;
  a.dim = dim;
  a.window = window;
  a.tree = tree;
  a.lse = lse;
  a.scale = scale;
  a.decay = decay;
  a.weights = weights;
  a.ws = {w_page * 4, w_token * 4, w_head * 4};
  if (kv_heads == 1) a.ks.head = a.ks.token;
  return status(launch_cache_weights(a, workspace, device_error_word(), (cudaStream_t)stream));
}

int lmhead_cache_select(const float* weights, int64_t w_page, int64_t w_token, int64_t w_head,
                        int64_t pages, int page_size, int kv_heads, const int32_t* table, int width,
                        const int32_t* lens, int S, int budget, int sinks, int recent,
                        int32_t* out_kept, lmhead_stream stream) {
  if (!weights || !table || !lens || !out_kept) return LMHEAD_ERR_NULL;
  const int st = check_table(S, width, pages, page_size);
  if (st != LMHEAD_OK) return st;
  if (kv_heads < 1 || kv_heads > 65535 || budget < 1 || sinks < 0 || recent < 0 ||
      sinks > budget || recent > budget - sinks || (int64_t)S * kv_heads * budget > INT32_MAX)
    return LMHEAD_ERR_SHAPE;
  if (!stride_ok(w_page) || !stride_ok(w_token) || !stride_ok(w_head)) return LMHEAD_ERR_SHAPE;
  if (!aligned(weights, 4)) return LMHEAD_ERR_ALIGN;
  SelectArgs a = {};
  a.weights = weights;
  a.ws = {w_page * 4, w_token * 4, w_head * 4};
  a.pages = pages;
  a.page = page_size;
  a.width = width;
  a.S = S;
  a.kv_heads = kv_heads;
  a.budget = budget;
  a.sinks = sinks;
  a.recent = recent;
  a.table = table;
  a.lens = lens;
  a.kept = out_kept;
  return status(launch_cache_select(a, device_error_word(), (cudaStream_t)stream));
}

}  // extern "C"
