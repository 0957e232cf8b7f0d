// Attention of a chunk of new tokens over a paged K/V cache.
//
// For token i of request s (len_s tokens cached before the chunk) and head a:
//   o = sum_j p_j v_j,  p = softmax_j(scale * q . k_j),  lse = log sum exp,
// over the keys the mask leaves: j <= len + i (and j > len + i - window), or
// the cached ones and those whose bit is set in the token's tree word. A row
// left with no key gives o = 0 and lse = -inf.
//
// Both products run on the tensor cores: the rows of one K/V head (tokens x
// the G = heads / kv_heads query heads that share it) are packed into tiles of
// 128, so that a decoding step of G heads reads its K and V once, and a block
// of 128 keys is one 128 x 128 product of scores and one 128 x dim product of
// values. Two launches:
//   prepare   writes the chunk's K and V to the cache, and (one CTA) cuts the
//             work into items (a request's one or two row tiles x a K/V head)
//             and shares their key blocks out evenly over the CTAs, wherever
//             an item's end falls;
//   attend    one CTA per SM, warp-specialised; walks over its range of
//             blocks: a TMA warp streams pages into a ring of shared memory, a
//             warp issues the MMAs, two warpgroups (a row per thread) turn
//             scores into weights. With two row tiles each warpgroup has its
//             own and both use every block; with one tile they take blocks in
//             turn and join at the end, so the tensor cores work on one while
//             the other is exponentiated. Of an item that was cut between
//             CTAs each leaves its piece in the scratch, and the warp that
//             brings the last one of its rows joins them, in the order of the
//             pieces.
// Bound: few rows, by reading K and V once; many rows, by the tensor cores.
// Measured (whole call, both launches, other inputs each time): 32 requests of
// 4000-8000 cached tokens and one new each, 32 heads over 8, dim 128: 132-135 us for
// 801 MB (5.9-6.1 TB/s); two chunks of 2048 tokens over 6144 cached: 345-348 us for
// 0.48 TFLOP (1.39 PFLOP/s; 325-331 us where one set of inputs is replayed). The
// latter is bound by the hand-overs between the roles: without the exponentials it
// takes as long, with an eighth of the softmax 4 % less, without loads 1 % less,
// with an eighth of the MMAs still three quarters of the time.
// The softmax runs in the base-2 domain with a running reference instead of
// the running maximum: a row's first block with a key sets it, and it moves only
// when weights pass 2^9 or so, which their sum shows; a block's maximum is not
// even looked for before (it cost a fifth of a block's time). Scores, sums,
// references and accumulators are fp32; the weights are rounded once, to the
// tensors' 16 bits, as the tensor cores take them beside V (the row's sum keeps them
// in fp32): against 64 bits 2.3e-3 of the outputs' size for bf16 and 2.9e-4 for
// fp16, where rounding the output alone leaves 1.7e-3 and 2.1e-4.
#include <cuda_fp16.h>

#include "common.cuh"
#include "kernels.h"
#include "tc_util.cuh"

namespace lmhead {
namespace {

constexpr int kRows = 128;  // rows of a tile
constexpr int kKeys = 128;  // keys of a block
constexpr int kItemCost = 1;
// Two softmax warpgroups and one of which two warps work (TMA, MMAs). The
// block is launched with 168 registers a thread and splits them 216 + 216 + 72.
constexpr int kThreads = 384;
constexpr int kRegsMore = 216, kRegsLess = 72;
constexpr int kPrepThreads = 256;
constexpr float kNegInf = -__builtin_huge_valf();
constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;

// What becomes of a request's rows: kFillZero those of one that was refused (its
// pages were never taken, so there is nothing to read), kFillNan those of one
// whose lengths the table has no room for.
enum Fate { kAttend, kFillZero, kFillNan };

// An item: up to two row tiles of one request, for every K/V head alike. One of
// rows that are only filled has no key blocks.
struct Item {
  int s, tok0, ntok, len;        // request, its first token (of all), tokens, cached before
  int i0, kb0, nblk, ntile;      // first token in the request, key blocks, row tiles
  int kend, kbeg, prefix, fate;  // keys [kbeg, kend) are loaded; units before it
};
static_assert(sizeof(Item) == 48, "three 16-byte loads");

struct Header {
  long long units;  // of all heads
  int items, per_head, parts;
  int fill;  // kFillSome: items among them that are only filled; kFillAll: no
             // plan could be made, every row is
};
enum Fill { kFillNone, kFillSome, kFillAll };

// Work units of an item: one per row tile and block, and kItemCost for what an
// item costs besides. Unit x of an item is at block ceil((x - kItemCost) / ntile).
__host__ __device__ inline int item_units(int nblk, int ntile) { return nblk * ntile + kItemCost; }
__device__ __forceinline__ int block_at(int x, int nblk, int ntile) {
  const int y = x - kItemCost;
  return y <= 0 ? 0 : min(nblk, (y + ntile - 1) / ntile);
}

struct Scratch {
  Header* head;
  int4* start;    // per CTA: item, K/V head, units of the item before its range
  float2* ml;     // per CTA and piece (place 2 c: of an item begun earlier, 2 c + 1: of
                  // one that goes on later), 256 rows: reference (base 2) and sum
  float* o;       // per CTA and piece, 256 rows x dim, not normalised
  Item* items;
  int* done;      // per item, K/V head and warp's rows (below): blocks done
};

struct ScratchSize {
  size_t start, ml, o, items, done, total;
};

__host__ inline ScratchSize scratch_size(int parts, int64_t items, int kv_heads, int dim) {
  ScratchSize z;
  size_t at = 256;
  auto take = [&](size_t bytes) {
    const size_t was = at;
    at = (at + bytes + 255) / 256 * 256;
    return was;
  };
  z.start = take((size_t)parts * sizeof(int4));
  z.ml = take((size_t)parts * 2 * 256 * sizeof(float2));
  z.o = take((size_t)parts * 2 * 256 * dim * sizeof(float));
  z.items = take((size_t)items * sizeof(Item));
  z.done = take((size_t)items * kv_heads * 8 * sizeof(int));
  z.total = at;
  return z;
}

inline int64_t most_items(int S, int T, int group) { return (int64_t)S + T / (2 * (kRows / group)) + 1; }
inline int part_count() { return sm_count() > 255 ? 255 : sm_count() > 0 ? sm_count() : 1; }

// ------------------------------------------------------------------ prepare

// The tokens of request s: cu is the caller's, so whatever it holds the range
// returned lies within [0, T); `sane` is cleared where it begins below 0 or
// decreases. Ranges of a cu that does neither are disjoint, which is what the
// number of items (most_items) rests on.
struct Request {
  int tok0, m, len;
  int seen;  // new tokens that are keys
  Fate fate;
};
__device__ __forceinline__ Request request_of(const AttnArgs& a, int s, bool& sane) {
  Request r;
  const int end = a.cu[s + 1];
  r.tok0 = a.cu[s];
  r.len = a.lens[s];
  sane = r.tok0 >= 0 && end >= r.tok0;
  r.tok0 = max(0, min(r.tok0, a.T));
  r.m = max(r.tok0, min(end, a.T)) - r.tok0;
  // the keys that the request's rows may see, within its pages? (lengths that
  // are keep all arithmetic on them in 32 bits)
  r.seen = a.tree ? min(r.m, 64) : r.m;
  r.fate = r.len >= 0 && r.len <= (a.width << a.page_shift) - r.seen ? kAttend : kFillNan;
  if (a.granted && a.granted[s] == 0) r.fate = kFillZero;
  if (r.fate != kAttend) r.len = 0;
  return r;
}

__device__ __forceinline__ Item make_item(const AttnArgs& a, int s, const Request& r, int x,
                                          int tile_tok) {
  Item it;
  it.s = s;
  it.i0 = x * 2 * tile_tok;
  it.tok0 = r.tok0 + it.i0;
  it.ntok = min(r.m - it.i0, 2 * tile_tok);
  it.len = r.len;
  it.ntile = it.ntok > tile_tok ? 2 : 1;
  it.kend = r.len + r.seen;
  const int end = a.tree ? it.kend : r.len + it.i0 + it.ntok;
  const int beg = a.window > 0 ? max(0, r.len + it.i0 + 1 - a.window) : 0;
  it.kb0 = beg / kKeys;
  it.nblk = r.fate == kAttend ? (end + kKeys - 1) / kKeys - it.kb0 : 0;
  it.kbeg = beg >> a.page_shift << a.page_shift;
  it.prefix = 0;
  it.fate = r.fate;
  return it;
}

// The items of all requests with the units before each, and where each CTA
// starts: CTA c of `parts` has the units [c U / parts, (c + 1) U / parts) of the
// sequence (K/V head, item).
__device__ void make_plan(const AttnArgs& a, const Scratch& sc, int most_parts, int* err) {
  constexpr int kKept = 1024;
  __shared__ int sh_n[kPrepThreads / 32];
  __shared__ long long sh_w[kPrepThreads / 32];
  __shared__ int sh_prefix[kKept];
  __shared__ int sh_bad, sh_fill;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int tile_tok = kRows / (a.heads / a.kv_heads);
  if (tid == 0) sh_bad = sh_fill = 0;
  cta_sync();
  int base_n = 0;
  long long base_w = 0;
  bool bad = false;
  for (int s0 = 0; s0 < a.S; s0 += kPrepThreads) {
    const int s = s0 + tid;
    Request req = {};
    int n = 0;
    long long w = 0;
    if (s < a.S) {
      bool sane;
      req = request_of(a, s, sane);
      if (!sane) sh_bad = 1;
      n = req.m > 0 ? (req.m - 1) / (2 * tile_tok) + 1 : 0;
      for (int x = 0; x < n; ++x) {
        const Item it = make_item(a, s, req, x, tile_tok);
        w += item_units(it.nblk, it.ntile);
      }
      if (n > 0 && req.fate != kAttend) {
        sh_fill = 1;
        if (req.fate == kFillNan) record_error(err, kDevErrBadId);
      }
    }
    int sn = n;
    long long sw = w;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int pn = __shfl_up_sync(0xFFFFFFFFu, sn, o);
      const long long pw = __shfl_up_sync(0xFFFFFFFFu, sw, o);
      if (lane >= o) {
        sn += pn;
        sw += pw;
      }
    }
    if (lane == 31) {
      sh_n[warp] = sn;
      sh_w[warp] = sw;
    }
    cta_sync();
    int bn = base_n;
    long long bw = base_w;
    for (int i = 0; i < kPrepThreads / 32; ++i) {
      if (i < warp) {
        bn += sh_n[i];
        bw += sh_w[i];
      }
      base_n += sh_n[i];
      base_w += sh_w[i];
    }
    // nothing of a cu that decreases is planned (its items might be more than the
    // scratch has places for), nor more units than their 32 bits can count
    bad = sh_bad || base_w > INT32_MAX;
    if (bad) break;
    int at = bn + sn - n, pre = (int)(bw + sw - w);
    for (int x = 0; x < n; ++x, ++at) {
      Item it = make_item(a, s, req, x, tile_tok);
      it.prefix = pre;
      pre += item_units(it.nblk, it.ntile);
      sc.items[at] = it;
      if (at < kKept) sh_prefix[at] = it.prefix;
    }
    cta_sync();
  }
  if (bad) base_n = 0, base_w = 0;
  const long long units = base_w * a.kv_heads;
  // a CTA has work for both warpgroups at least
  const int parts = (int)min((long long)most_parts, (units + 1) / 2);
  if (tid == 0) {
    sc.head->units = units;
    sc.head->items = base_n;
    sc.head->per_head = (int)base_w;
    sc.head->parts = parts;
    sc.head->fill = bad ? kFillAll : sh_fill ? kFillSome : kFillNone;
    if (bad) record_error(err, kDevErrBadId);
  }
  for (int c = tid; c < parts; c += kPrepThreads) {
    const long long u = units * c / parts;
    const int hk = (int)(u / base_w), rem = (int)(u - (long long)hk * base_w);
    int lo = 0, hi = base_n;  // the last item that starts at or before rem
    while (hi - lo > 1) {
      const int mid = (lo + hi) / 2;
      const int p = mid < kKept ? sh_prefix[mid] : sc.items[mid].prefix;
      if (p <= rem) lo = mid; else hi = mid;
    }
    const int p = lo < kKept ? sh_prefix[lo] : sc.items[lo].prefix;
    sc.start[c] = make_int4(lo, hk, rem - p, 0);
  }
}

// CTA 0 plans; the others clear the counts of finished blocks and copy K and V of
// the new tokens to their slots, 16 bytes a thread.
__global__ void __launch_bounds__(kPrepThreads)
prepare_kernel(AttnArgs a, Scratch sc, int most_parts, int64_t counts, int pieces, int* err) {
  pdl_wait();
  pdl_trigger();
  if (blockIdx.x == 0) {
    make_plan(a, sc, most_parts, err);
    return;
  }
  const int64_t first = (int64_t)(blockIdx.x - 1) * blockDim.x + threadIdx.x;
  const int64_t stride = (int64_t)(gridDim.x - 1) * blockDim.x;
  for (int64_t e = first * 4; e < counts; e += stride * 4)  // a multiple of 8 of them
    *reinterpret_cast<int4*>(sc.done + e) = make_int4(0, 0, 0, 0);
  if (!a.k) return;
  const int per = a.kv_heads * pieces;
  const int64_t all = (int64_t)a.T * per;
  const int64_t num_slots = a.pages << a.page_shift;
  for (int64_t e = first; e < all; e += stride) {
    const int t = (int)(e / per), x = (int)(e - (int64_t)t * per);
    const int hd = x / pieces, c = (x - hd * pieces) * 16;
    const int32_t slot = a.slots[t];
    if (slot < 0) continue;  // a token without a place
    if (slot >= num_slots) {
      record_error(err, kDevErrBadId);
      continue;
    }
    const int64_t pg = slot >> a.page_shift, off = slot & ((1 << a.page_shift) - 1);
    const char *k = static_cast<const char*>(a.k), *v = static_cast<const char*>(a.v);
    char *kc = static_cast<char*>(a.k_cache), *vc = static_cast<char*>(a.v_cache);
    const uint4 kv = *reinterpret_cast<const uint4*>(k + t * a.k_tok + hd * a.k_head + c);
    const uint4 vv = *reinterpret_cast<const uint4*>(v + t * a.v_tok + hd * a.v_head + c);
    *reinterpret_cast<uint4*>(kc + pg * a.ks.page + off * a.ks.token + hd * a.ks.head + c) = kv;
    *reinterpret_cast<uint4*>(vc + pg * a.vs.page + off * a.vs.token + hd * a.vs.head + c) = vv;
  }
}

// ------------------------------------------------------------------- attend

template <int D> struct Shape {
  static constexpr int kHalves = D / 64;             // 64-element (128-byte) columns of a row
  static constexpr int kBuf = kKeys * D * 2;         // one K or V block
  static constexpr int kStages = D == 128 ? 5 : 10;  // 160 KB
  static constexpr int kQ = 2 * kRows * D * 2;
  static constexpr int kSmem = kQ + kStages * kBuf + 1024;
};

constexpr int kBadSlots = 16;  // more pieces than the TMA warp can be ahead

template <int NS> struct Ctl {
  uint64_t full[NS], empty[NS];
  uint64_t q_full[2], s_full[2], p_half[2], h_done[2], p_full[2], o_full[2];
  uint64_t ex1, ex2, drain;
  uint32_t tmem;
  int abort;
  int bad[kBadSlots];
};

// The CTA's pieces, in order; every role walks over them by itself.
struct Cursor {
  const Item* items;
  long long units, left;
  int parts, per_head;
  int idx, hk, off, n_items;
  // the piece
  Item it;
  int b0, b1, p_hk, p_idx;

  // The units of CTA c begin at floor(units c / parts).
  __device__ long long start_of(int c) const {
    if (units < (1 << 24)) return (uint32_t)units * (uint32_t)c / (uint32_t)parts;  // parts < 256
    return units * c / parts;
  }
  // The CTA that has unit u.
  __device__ int cta_of(long long u) const {
    if (units < (1 << 24))
      return (int)(((uint32_t)(u + 1) * (uint32_t)parts + (uint32_t)units - 1) / (uint32_t)units) - 1;
    return (int)(((u + 1) * parts + units - 1) / units) - 1;
  }
  __device__ void init(const Scratch& sc, int cta) {
    // all under way before any is looked at (every CTA has a place in `start`)
    const Header head = *sc.head;
    const int4 st = sc.start[cta];
    items = sc.items;
    parts = head.parts;
    units = head.units;
    per_head = head.per_head;
    n_items = head.items;
    left = cta < parts ? start_of(cta + 1) - start_of(cta) : 0;
    idx = st.x;
    hk = st.y;
    off = st.z;
  }
  // On to the next piece; with FILLED also to an item that is only filled, which
  // is the CTA's that has its one unit.
  template <bool FILLED = false> __device__ bool next() {
    while (left > 0) {
      const int4* src = reinterpret_cast<const int4*>(items + idx);
      const int4 x = src[0], y = src[1], z = src[2];
      it.s = x.x; it.tok0 = x.y; it.ntok = x.z; it.len = x.w;
      it.i0 = y.x; it.kb0 = y.y; it.nblk = y.z; it.ntile = y.w;
      it.kend = z.x; it.kbeg = z.y; it.prefix = z.z; it.fate = z.w;
      const int w = item_units(it.nblk, it.ntile);
      const int end = (int)min((long long)w, off + left);
      b0 = block_at(off, it.nblk, it.ntile);
      b1 = block_at(end, it.nblk, it.ntile);
      left -= end - off;
      off = 0;
      p_hk = hk;
      p_idx = idx;
      if (++idx == n_items) {
        idx = 0;
        ++hk;
      }
      if (b1 > b0 || (FILLED && it.nblk == 0)) return true;
    }
    return false;
  }
};

// A warp's wait. The one that issues the MMAs is on the way of every block: it
// polls for a while before it lets itself be suspended, from which a warp takes a
// few hundred cycles to return (two prompts of 2048 tokens, one set of inputs
// replayed, 351 to 325 us; with the softmax's warps polling too, which takes issue
// slots from their neighbours, 332).
template <bool POLL>
__device__ __forceinline__ bool wait_all(uint64_t* bar, uint32_t parity, volatile int* abort,
                                         long long budget) {
  if (POLL && budget > 0) {
#pragma unroll 1
    for (int i = 0; i < 200; ++i)
      if (__all_sync(0xFFFFFFFFu, tc::mbar_test(bar, parity))) return true;
  }
  const bool now = budget > 0 && tc::mbar_try_wait(bar, parity);
  return __all_sync(0xFFFFFFFFu, now || tc::mbar_wait(bar, parity, abort, budget));
}

// Bits [lo, hi) of 32, either end anywhere.
__device__ __forceinline__ uint32_t span_bits(int lo, int hi) {
  const uint32_t below_hi = hi >= 32 ? ~0u : hi <= 0 ? 0u : (1u << hi) - 1u;
  const uint32_t below_lo = lo >= 32 ? ~0u : lo <= 0 ? 0u : (1u << lo) - 1u;
  return below_hi & ~below_lo;
}

template <bool BF16> __device__ __forceinline__ uint32_t pack2(float lo, float hi) {
  uint32_t r;
  if (BF16)
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  else
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

// 32 columns of an output row from column c on: 16-bit results, or fp32 parts.
template <bool BF16>
__device__ __forceinline__ void store_cols(const float (&v)[32], char* out16, float* out32, int c) {
  if (out16) {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      *reinterpret_cast<uint4*>(out16 + (c + 8 * i) * 2) =
          make_uint4(pack2<BF16>(v[8 * i], v[8 * i + 1]), pack2<BF16>(v[8 * i + 2], v[8 * i + 3]),
                     pack2<BF16>(v[8 * i + 4], v[8 * i + 5]), pack2<BF16>(v[8 * i + 6], v[8 * i + 7]));
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      *reinterpret_cast<float4*>(out32 + c + 4 * i) =
          make_float4(v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]);
  }
}

template <int N> struct Const {
  static constexpr int value = N;
};

// Joins the pieces of 32 rows (of row tile `tile`, quarter `quarter`) in COLS
// columns from col on, by one warp:
//   o = sum_p 2^(m_p - M) o_p / sum_p 2^(m_p - M) l_p.
// Lane r holds row r's references and sums; the lanes share the elements. What
// it costs is latency, so many loads are under way together.
template <bool BF16, int D, int COLS>
__device__ void join_rows(const AttnArgs& a, const Scratch& sc, const Cursor& cur, const Item& it,
                          int hk, int tile, int quarter, int col, int64_t out_row, bool valid) {
  constexpr int N4 = COLS / 4, EL = COLS / 4;  // float4 of a row; of a lane at 32 rows
  const int lane = threadIdx.x & 31;
  const int w = item_units(it.nblk, it.ntile);
  const long long ub = (long long)hk * cur.per_head + it.prefix;
  // its first CTA, and the piece of CTA c: its place, -1 if it has none, -2 past
  // the item's last
  const int c0 = cur.cta_of(ub);
  auto place_of = [&](int c) -> int {
    if (c >= cur.parts) return -2;
    const long long lo = cur.start_of(c), hi = cur.start_of(c + 1);
    if (lo >= ub + w) return -2;
    const int b0 = block_at((int)max(lo - ub, 0ll), it.nblk, it.ntile);
    const int b1 = block_at((int)min(hi - ub, (long long)w), it.nblk, it.ntile);
    return b1 > b0 ? 2 * c + (b0 == 0 ? 1 : 0) : -1;
  };
  const int row0 = tile * kRows + quarter * 32;
  const int rows = __popc(__ballot_sync(0xFFFFFFFFu, valid)), elems = rows * N4;
  float top = kNegInf;
  for (int c = c0;; c += 32) {
    const int place = place_of(c + lane);
    const uint32_t past = __ballot_sync(0xFFFFFFFFu, place == -2);
    const int count = past ? __ffs(past) - 1 : 32;
    for (int p0 = 0; p0 < count; p0 += 8) {
      float m[8];
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        const int p = __shfl_sync(0xFFFFFFFFu, place, (p0 + k) & 31);
        m[k] = p0 + k < count && p >= 0 && valid ? sc.ml[(int64_t)p * 256 + row0 + lane].x : kNegInf;
      }
#pragma unroll
      for (int k = 0; k < 8; ++k) top = fmaxf(top, m[k]);
    }
    if (past) break;
  }
  const float ref = top == kNegInf ? 0.f : top;
  float l = 0.f;
  float4 acc[EL];
#pragma unroll
  for (int i = 0; i < EL; ++i) acc[i] = make_float4(0.f, 0.f, 0.f, 0.f);
  // pieces p0.. (NP of them), NI elements of a lane at a time
  auto add_pieces = [&](auto np, auto ni, int place, int p0, int count) {
    constexpr int NP = decltype(np)::value, NI = decltype(ni)::value;
    float f[NP];
    const float* from[NP];
#pragma unroll
    for (int k = 0; k < NP; ++k) {
      const int p = __shfl_sync(0xFFFFFFFFu, place, (p0 + k) & 31);
      const bool some = p0 + k < count && p >= 0;
      const float2 ml = some && valid ? sc.ml[(int64_t)p * 256 + row0 + lane]
                                      : make_float2(kNegInf, 0.f);
      f[k] = tc::exp2_approx(ml.x - ref);
      l = fmaf(f[k], ml.y, l);
      from[k] = some ? sc.o + ((int64_t)p * 256 + row0) * D + col : nullptr;
    }
#pragma unroll
    for (int i0 = 0; i0 < EL; i0 += NI) {
      if (i0 * 32 >= elems) break;
      float4 v[NI][NP];
#pragma unroll
      for (int i = 0; i < NI; ++i)
#pragma unroll
        for (int k = 0; k < NP; ++k) {
          const int e = (i0 + i) * 32 + lane;
          v[i][k] = from[k] && e < elems
                        ? __ldcg(reinterpret_cast<const float4*>(from[k] + (e / N4) * D) + e % N4)
                        : make_float4(0.f, 0.f, 0.f, 0.f);
        }
#pragma unroll
      for (int i = 0; i < NI; ++i)
#pragma unroll
        for (int k = 0; k < NP; ++k) {
          const float fr = __shfl_sync(0xFFFFFFFFu, f[k], (((i0 + i) * 32 + lane) / N4) & 31);
          float4& s = acc[i0 + i];
          s.x = fmaf(fr, v[i][k].x, s.x);
          s.y = fmaf(fr, v[i][k].y, s.y);
          s.z = fmaf(fr, v[i][k].z, s.z);
          s.w = fmaf(fr, v[i][k].w, s.w);
        }
    }
  };
  for (int c = c0;; c += 32) {
    const int place = place_of(c + lane);
    const uint32_t past = __ballot_sync(0xFFFFFFFFu, place == -2);
    const int count = past ? __ffs(past) - 1 : 32;
    if (elems <= 64)
      for (int p0 = 0; p0 < count; p0 += 8)
        add_pieces(Const<8>{}, Const<2>{}, place, p0, count);
    else
      for (int p0 = 0; p0 < count; p0 += 4)
        add_pieces(Const<4>{}, Const<4>{}, place, p0, count);
    if (past) break;
  }
  const float inv = l == 0.f ? 0.f : 1.f / l;
  if (a.lse && valid && col == 0) a.lse[out_row] = l == 0.f ? kNegInf : ref * kLn2 + logf(l);
#pragma unroll
  for (int i = 0; i < EL; ++i) {
    if (i * 32 >= elems) break;
    const int e = i * 32 + lane, r = e / N4;
    const float s = __shfl_sync(0xFFFFFFFFu, inv, r & 31);
    const int64_t to = __shfl_sync(0xFFFFFFFFu, out_row, r & 31);
    if (e < elems)
      *reinterpret_cast<uint2*>(static_cast<char*>(a.out) + (to * D + col) * 2 + e % N4 * 8) =
          make_uint2(pack2<BF16>(acc[i].x * s, acc[i].y * s), pack2<BF16>(acc[i].z * s, acc[i].w * s));
  }
}

// One row of the output and its log-sum-exp that were not computed, by a warp.
template <bool BF16, int D>
__device__ __forceinline__ void fill_row(const AttnArgs& a, int64_t row, float v, float lse) {
  const int lane = threadIdx.x & 31;
  const uint32_t two = pack2<BF16>(v, v);
  if (lane < D / 8)
    *reinterpret_cast<uint4*>(static_cast<char*>(a.out) + (row * D + lane * 8) * 2) =
        make_uint4(two, two, two, two);
  if (lane == 0 && a.lse) a.lse[row] = lse;
}

// The CTA's share of the rows that are only filled, by eight warps.
template <bool BF16, int D>
__device__ __forceinline__ void fill_rows(const AttnArgs& a, const Scratch& sc, int warp) {
  const float nan = __int_as_float(0x7fc00000);
  if (sc.head->fill == kFillAll) {
    const int64_t rows = (int64_t)a.T * a.heads;
    for (int64_t r = (int64_t)blockIdx.x * 8 + warp; r < rows; r += (int64_t)gridDim.x * 8)
      fill_row<BF16, D>(a, r, nan, nan);
  }
  const int group = a.heads / a.kv_heads;
  Cursor cur;
  cur.init(sc, blockIdx.x);
  while (cur.next<true>()) {
    if (cur.it.nblk > 0) continue;
    const bool zero = cur.it.fate == kFillZero;
    for (int i = warp; i < cur.it.ntok * group; i += 8) {
      const int tk = i / group;
      fill_row<BF16, D>(a, (int64_t)(cur.it.tok0 + tk) * a.heads + cur.p_hk * group + i - tk * group,
                        zero ? 0.f : nan, zero ? kNegInf : nan);
    }
  }
}

template <bool BF16, int D>
__global__ void __launch_bounds__(kThreads, 1)
attend_kernel(const __grid_constant__ CUtensorMap kmap, const __grid_constant__ CUtensorMap vmap,
              const AttnArgs a, const Scratch sc, int k_head_first, int v_head_first,
              long long budget, int* err) {
  using Sh = Shape<D>;
  constexpr int NS = Sh::kStages;
  extern __shared__ uint8_t dsmem_raw[];
  __shared__ Ctl<NS> ctl;
  uint8_t* base = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(dsmem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  uint8_t* q_s = base;
  uint8_t* ring = base + Sh::kQ;
  const int warp = __shfl_sync(0xFFFFFFFFu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
  volatile int* abort_flag = &ctl.abort;

  if (threadIdx.x == 0) {
    for (int i = 0; i < NS; ++i) {
      tc::mbar_init(&ctl.full[i], 1);
      tc::mbar_init(&ctl.empty[i], 1);
    }
    for (int w = 0; w < 2; ++w) {
      tc::mbar_init(&ctl.q_full[w], kRows);
      tc::mbar_init(&ctl.s_full[w], 1);
      tc::mbar_init(&ctl.p_half[w], kRows);
      tc::mbar_init(&ctl.h_done[w], 1);
      tc::mbar_init(&ctl.p_full[w], kRows);
      tc::mbar_init(&ctl.o_full[w], 1);
    }
    tc::mbar_init(&ctl.ex1, 2 * kRows);
    tc::mbar_init(&ctl.ex2, 2 * kRows);
    tc::mbar_init(&ctl.drain, 1);
    ctl.abort = 0;
    tc::fence_mbar_init();
  }
  if (warp == 9) {
    tc::tmem_alloc(&ctl.tmem, 512);
    tc::tmem_relinquish();
  }
  if (warp == 8 && lane == 0) {
    tc::prefetch_tmap(&kmap);
    tc::prefetch_tmap(&vmap);
  }
  tc::fence_before_sync();
  cta_sync();
  tc::fence_after_sync();
  // all 512 columns: scores and weights at 0 and 128, outputs at 256 and 384
  constexpr uint32_t tmem = 0;
  pdl_wait();
  pdl_trigger();
  const int group = a.heads / a.kv_heads, tile_tok = kRows / group;
  Cursor cur;
  cur.init(sc, blockIdx.x);
  if (warp >= 8) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegsLess));
    if (warp == 8) {
      // ------------------------------------------------------------ pages by TMA
      // the cache was written by the launch before through the other proxy
      asm volatile("fence.proxy.async;" ::: "memory");
      const int unit_tok = min(kKeys, 1 << a.page_shift), units = kKeys / unit_tok;
      const int u = lane / Sh::kHalves, half = lane % Sh::kHalves;
      const bool mine = u < units;
      uint32_t n = 0;
      int piece = 0;
      bool ok = true;
      while (ok && cur.next()) {
        if (lane == 0) *(volatile int*)&ctl.bad[piece % kBadSlots] = 0;
        const int32_t* row = a.table + (size_t)cur.it.s * a.width;
        for (int b = cur.b0; b < cur.b1 && ok; ++b) {
          const int key = (cur.it.kb0 + b) * kKeys + u * unit_tok;
          const bool want = mine && key < cur.it.kend && key + unit_tok > cur.it.kbeg;
          int32_t id = 0;
          bool bad = false;
          if (want) {
            const int pg = key >> a.page_shift;
            id = pg < a.width ? row[pg] : -1;
            bad = id < 0 || id >= a.pages;
          }
          const uint32_t load = __ballot_sync(0xFFFFFFFFu, want && !bad);
          if (__any_sync(0xFFFFFFFFu, bad) && lane == 0) {
            *(volatile int*)&ctl.bad[piece % kBadSlots] = 1;
            record_error(err, kDevErrBadId);
          }
          const int off = key & ((1 << a.page_shift) - 1);
#pragma unroll
          for (int kv = 0; kv < 2; ++kv, ++n) {
            const int slot = (int)(n % NS);
            if (n >= (uint32_t)NS) {
              ok = wait_all<false>(&ctl.empty[slot], ((n / NS) & 1) ^ 1, abort_flag, budget);
              if (!ok) break;
            }
            if (lane == 0)
              tc::mbar_arrive_expect_tx(&ctl.full[slot], (uint32_t)(__popc(load) * unit_tok * 128));
            __syncwarp();
            if (want && !bad) {
              uint8_t* dst = ring + slot * Sh::kBuf + half * (kKeys * 128) + u * unit_tok * 128;
              const bool hf = kv ? v_head_first : k_head_first;
              tc::tma_load_4d(dst, kv ? &vmap : &kmap, &ctl.full[slot], half * 64,
                              hf ? cur.p_hk : off, hf ? off : cur.p_hk, id);
            }
          }
        }
        ++piece;
      }
      if (!ok && lane == 0) {
        *abort_flag = 1;
        record_error(err, kDevErrTimeout);
      }
      __syncwarp();
      if (lane == 0) {
        // no copy may be under way when the CTA ends, whichever role gave up
        // (bounded; in a run that did not, all of them are long done)
        const uint32_t first = n > (uint32_t)NS ? n - NS : 0;
        for (uint32_t j = first; j < n; ++j) {
          const long long t0 = clock64();
          while (!tc::mbar_try_wait(&ctl.full[j % NS], (j / NS) & 1) &&
                 clock64() - t0 < tc::kWaitCycles) {
          }
        }
      }
    } else if (warp == 9) {
      // ------------------------------------------------------------ MMAs
      // A step is one tile x one block; steps alternate between the warpgroups.
      // Scores of step k + 2 are issued behind the values of step k, which read
      // the weights that they overwrite (MMAs of one thread run in order).
      const uint32_t idesc_s = tc::idesc_f16_f32(BF16, kRows, kKeys, false);
      const uint32_t idesc_o = tc::idesc_f16_f32(BF16, kRows, D, true);
      const bool issuer = tc::elect_one();
      const uint64_t q_desc = tc::sw128_kmajor_desc(tc::smem_addr(q_s));
      const uint64_t k_desc = tc::sw128_kmajor_desc(tc::smem_addr(ring));
      const uint64_t v_desc = tc::sw128_mnmajor_desc(tc::smem_addr(ring), kKeys * 128);
      uint32_t blocks = 0, nq0 = 0, nq1 = 0, np0 = 0, np1 = 0;
      bool ok = true;
      while (ok) {
        // what branches and operands depend on comes by shuffle from lane 0, so
        // that the compiler knows it to be the warp's own
        const int found = cur.next() ? (cur.b1 - cur.b0) << 2 | (cur.it.ntile == 2) << 1 | 1 : 0;
        const int info = __shfl_sync(0xFFFFFFFFu, found, 0);
        if (info == 0) break;
        const bool pair = info & 2;
        const int nb = info >> 2, steps = pair ? 2 * nb : nb;
#pragma unroll 1
        for (int k = -2; k < steps && ok; ++k) {
          // values of step k, then scores of step k + 2; everything but the
          // weights is waited for first
          const bool has_v = k >= 0, has_s = k + 2 < steps;
          const int jv = pair ? k >> 1 : k, js = pair ? (k + 2) >> 1 : k + 2;
          const uint32_t nv = 2 * (blocks + jv) + 1, nk = 2 * (blocks + js);
          const int v_slot = (int)(nv % NS), k_slot = (int)(nk % NS), w = k & 1;
          const int tile = pair ? w : 0;
          // a pair's second step uses the block of its first
          const bool opens = !pair || w == 0, closes = !pair || w == 1;
          if (has_v && opens) {
            ok = wait_all<true>(&ctl.full[v_slot], (nv / NS) & 1, abort_flag, budget);
            if (!ok) break;
            // keys that are no token's, or whose page was not loaded, hold anything
            // at all, and weight 0 times NaN is NaN: they are zeroed
            const int first = (cur.it.kb0 + cur.b0 + jv) * kKeys;
            const int lo = max(0, min(kKeys, cur.it.kbeg - first));
            const int hi = min(kKeys, cur.it.kend - first);
            if (lo > 0 || hi < kKeys) {
              uint8_t* v = ring + v_slot * Sh::kBuf;
              for (int e = lane; e < kKeys * 8; e += 32) {
                const int r = e >> 3;
                if (r < lo || r >= hi)
#pragma unroll
                  for (int h = 0; h < Sh::kHalves; ++h)
                    *reinterpret_cast<uint4*>(v + h * (kKeys * 128) + e * 16) =
                        make_uint4(0, 0, 0, 0);
              }
              tc::fence_async_smem();
              __syncwarp();
            }
          }
          if (has_s) {
            if (k + 2 == 0 || (pair && k + 2 == 1)) {
              const uint32_t use = w ? nq1++ : nq0++;
              ok = wait_all<true>(&ctl.q_full[w], use & 1, abort_flag, budget);
            }
            if (!ok) break;
          }
          if (has_v) {  // the weights come in two halves
            const uint32_t use = w ? np1++ : np0++;
            const uint64_t vd = v_desc + v_slot * (Sh::kBuf / 16);
            ok = wait_all<true>(&ctl.p_half[w], use & 1, abort_flag, budget);
            if (!ok) break;
            tc::fence_after_sync();
#pragma unroll
            for (int c = 0; c < kKeys / 32; ++c)
              tc::mma_ts_one(issuer, tmem + 256 + w * 128, tmem + w * 128 + c * 8,
                             vd + c * (16 * 128 / 16), idesc_o, c > 0 ? 1u : (uint32_t)(k >= 2));
            tc::commit_one(issuer, &ctl.h_done[w]);
            ok = wait_all<true>(&ctl.p_full[w], use & 1, abort_flag, budget);
            if (!ok) break;
            tc::fence_after_sync();
#pragma unroll
            for (int c = kKeys / 32; c < kKeys / 16; ++c)
              tc::mma_ts_one(issuer, tmem + 256 + w * 128, tmem + w * 128 + c * 8,
                             vd + c * (16 * 128 / 16), idesc_o, 1u);
            if (closes) tc::commit_one(issuer, &ctl.empty[v_slot]);
            if (!has_s) tc::commit_one(issuer, &ctl.o_full[w]);
          }
          if (has_s) {
            if (opens) {
              ok = wait_all<true>(&ctl.full[k_slot], (nk / NS) & 1, abort_flag, budget);
              if (!ok) break;
            }
            tc::fence_after_sync();
            // addresses count 16 bytes and stay below 2^14 of them
            const uint64_t qd = q_desc + tile * (kRows * D * 2 / 16);
            const uint64_t kd = k_desc + k_slot * (Sh::kBuf / 16);
#pragma unroll
            for (int c = 0; c < D / 16; ++c) {
              constexpr int kHalf = kRows * 128 / 16;
              tc::mma_ss_one(issuer, tmem + w * 128, qd + (c / 4) * kHalf + (c % 4) * 2,
                             kd + (c / 4) * kHalf + (c % 4) * 2, idesc_s, c > 0);
            }
            tc::commit_one(issuer, &ctl.s_full[w]);
            if (closes) tc::commit_one(issuer, &ctl.empty[k_slot]);
          }
          __syncwarp();
        }
        blocks += nb;
      }
      if (!ok && lane == 0) {
        *abort_flag = 1;
        record_error(err, kDevErrTimeout);
      }
      if (issuer) tc::mma_drain(&ctl.drain);  // TMEM is freed below
      __syncwarp();
    }
  } else {
    // ------------------------------------------------------------ softmax
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRegsMore));
    const int w = warp >> 2;                // warpgroup
    const int r = threadIdx.x & 127;        // row of the tile = TMEM lane
    const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16;
    const uint32_t t_s = tmem + lanes + w * 128, t_o = tmem + lanes + 256 + w * 128;
    const float sl = a.scale * kLog2e;
    const int row_tok = min(r / group, tile_tok - 1);  // rows past the tile go along
    const int row_head = r - r / group * group;
    uint32_t ns = 0, no0 = 0, no1 = 0, nx = 0;
    int piece = 0;
    bool ok = true;
    // Rows of the piece at the cursor into the tile of this warpgroup, if it has
    // one there: 16 bytes a lane, row by row; rows that are none are zeroed.
    auto load_q = [&]() {
      if (cur.it.ntile == 1 && w == 1) return;
      const int t = cur.it.ntile == 2 ? w : 0, quarter = warp & 3;
      const uint32_t dst = tc::smem_addr(q_s) + t * (kRows * D * 2);
#pragma unroll 4
      for (int i = 0; i < D / 8; ++i) {
        const int e = i * 32 + lane, row = quarter * 32 + e / (D / 8), c = e % (D / 8);
        const int rt = row / group, tk = t * tile_tok + rt;
        const bool in = rt < tile_tok && tk < cur.it.ntok;
        const char* src = static_cast<const char*>(a.q) + c * 16;
        if (in)
          src += (int64_t)(cur.it.tok0 + tk) * a.q_tok +
                 (int64_t)(cur.p_hk * group + row - rt * group) * a.q_head;
        const int size = in ? 16 : 0;
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(
                         dst + (c / 8) * (kRows * 128) + row * 128 + (((c % 8) ^ (row & 7)) << 4)),
                     "l"(src), "r"(size)
                     : "memory");
      }
    };
    auto q_loaded = [&]() {
      asm volatile("cp.async.wait_all;" ::: "memory");
      if (cur.it.ntile == 1 && w == 1) return;
      tc::fence_async_smem();
      tc::mbar_arrive(&ctl.q_full[cur.it.ntile == 2 ? w : 0]);
    };
    bool have = cur.next();
    if (have) {
      load_q();
      q_loaded();
    }
    for (; ok && have; ++piece) {
      const Item it = cur.it;
      const int p_hk = cur.p_hk, p_idx = cur.p_idx, b_first = cur.b0;
      const bool pair = it.ntile == 2;
      const int nb = cur.b1 - cur.b0;
      const int tile = pair ? w : 0;
      const bool first = cur.b0 == 0, last = cur.b1 == it.nblk;
      const int tok = tile * tile_tok + row_tok;
      const bool valid = r < tile_tok * group && tok < it.ntok;
      const int tokc = min(tok, it.ntok - 1);
      const int head = p_hk * group + row_head;
      const int64_t out_row = (int64_t)(it.tok0 + tok) * a.heads + head;
      // the row's keys: [lo, hi), and the new tokens of its tree word
      const int hi = a.tree ? it.len : it.len + it.i0 + tokc + 1;
      const int lo = a.window > 0 ? max(0, hi - a.window) : 0;
      uint64_t bits = 0;
      if (a.tree) {
        bits = a.tree[it.tok0 + tokc];
        const int m = it.kend - it.len;
        if (m < 64) bits &= (1ull << m) - 1;
      }
      // keys [lo_most, hi_least) are seen by every row of the warp
      const int hi_least = __reduce_min_sync(0xFFFFFFFFu, hi);
      const int lo_most = __reduce_max_sync(0xFFFFFFFFu, lo);
      const bool idle = !__any_sync(0xFFFFFFFFu, valid);  // no row of this warp is one
      float ref = kNegInf;
      float2 sum = make_float2(0.f, 0.f);
      const int steps = pair ? nb : (nb + 1 - w) / 2;
      for (int j = 0; j < steps; ++j) {
        const int b = b_first + (pair ? j : 2 * j + w);
        const int key0 = (it.kb0 + b) * kKeys;
        ok = wait_all<false>(&ctl.s_full[w], ns++ & 1, abort_flag, budget);
        if (!ok) break;
        tc::fence_after_sync();
        if (!idle) {
          uint32_t s[kKeys] = {};
          auto val = [&](int c) { return __uint_as_float(s[c]); };
#pragma unroll
          for (int c = 0; c < 4; ++c)
            tc::tmem_ld32(t_s + c * 32, *reinterpret_cast<uint32_t(*)[32]>(&s[c * 32]));
          tc::tmem_ld_wait(s);
          if (key0 < lo_most || key0 + kKeys > hi_least) {
            // an edge of the mask in this warp's rows
#pragma unroll
            for (int c = 0; c < 4; ++c) {
              const int k0 = key0 + 32 * c;
              uint32_t see = span_bits(lo - k0, hi - k0);
              if (a.tree) {
                const int x = k0 - it.len;
                if (x > -32 && x < 64) see |= (uint32_t)(x < 0 ? bits << -x : bits >> x);
              }
#pragma unroll
              for (int i = 0; i < 32; ++i)
                s[c * 32 + i] = (see >> i) & 1 ? s[c * 32 + i] : __float_as_uint(kNegInf);
            }
          }
          const float2 sl2 = make_float2(sl, sl);
          uint32_t pk[32];
          // The weights of one half of the keys, into pk; returns their sum.
          auto half = [&](int h) {
            const float neg = ref == kNegInf ? 0.f : -ref;
            const float2 neg2 = make_float2(neg, neg);
            float2 part[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
#pragma unroll
            for (int i = 0; i < 32; ++i) {
              const int c = h * 64 + 2 * i;
              float2 x = tc::fma_x2(make_float2(val(c), val(c + 1)), sl2, neg2);
              x.x = tc::exp2_approx(x.x);
              x.y = tc::exp2_approx(x.y);
              part[i & 1] = tc::add_x2(part[i & 1], x);
              pk[i] = pack2<BF16>(x.x, x.y);
            }
            return tc::add_x2(part[0], part[1]);
          };
          // The block's maximum becomes the reference of the rows that it passes
          // by more than 2^8; what they have summed up is scaled to it.
          auto set_reference = [&](bool live) {
            float mx[4] = {val(0), val(1), val(2), val(3)};
#pragma unroll
            for (int c = 4; c < kKeys; ++c) mx[c & 3] = fmaxf(mx[c & 3], val(c));
            const float top = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])) * sl;
            const bool grow = top > ref + 8.f || (ref == kNegInf && top > kNegInf);
            if (!__any_sync(0xFFFFFFFFu, grow)) return;
            const float f = grow ? tc::exp2_approx(ref - top) : 1.f;
            if (grow) ref = top;
            sum.x *= f;
            sum.y *= f;
            if (live) {
#pragma unroll 1
              for (int c = 0; c < D / 16; ++c) {
                uint32_t v[16];
                tc::tmem_ld16(t_o + c * 16, v);
                tc::tmem_ld_wait(v);
#pragma unroll
                for (int i = 0; i < 16; ++i) v[i] = __float_as_uint(__uint_as_float(v[i]) * f);
                tc::tmem_st16(t_o + c * 16, v);
              }
            }
          };
          // A row's sum over half a block tells when weights have become large,
          // so that the maximum is looked for only then, and while a row has
          // no reference. Weights up to 2^15 are as exact as weights up to 1.
          auto large = [&](float2 p) {
            return __any_sync(0xFFFFFFFFu, !(p.x + p.y <= 32768.f));
          };
          bool sure = __any_sync(0xFFFFFFFFu, ref == kNegInf);
          if (sure) set_reference(j > 0);
          float2 p = half(0);
          if (!sure && large(p)) {
            sure = true;
            set_reference(j > 0);
            p = half(0);
          }
          tc::tmem_st32(t_s, pk);
          tc::tmem_st_wait();
          tc::fence_before_sync();
          tc::mbar_arrive(&ctl.p_half[w]);
          sum = tc::add_x2(sum, p);
          p = half(1);
          if (!sure && large(p)) {
            // the first half is with the MMAs: its values are summed up before
            // the accumulators are scaled
            ok = wait_all<false>(&ctl.h_done[w], (ns - 1) & 1, abort_flag, budget);
            if (!ok) break;
            tc::fence_after_sync();
            set_reference(true);
            p = half(1);
          }
          tc::tmem_st32(t_s + 32, pk);
          sum = tc::add_x2(sum, p);
          tc::tmem_st_wait();
        } else {
          tc::mbar_arrive(&ctl.p_half[w]);
        }
        tc::fence_before_sync();
        tc::mbar_arrive(&ctl.p_full[w]);
      }
      if (!ok) break;
      // with one tile and two blocks or more both warpgroups have values
      const bool join = !pair && nb > 1;
      const bool both = pair || nb > 1;  // warpgroup 1 has values
      if (w == 0 || join) ok = wait_all<false>(&ctl.o_full[0], no0 & 1, abort_flag, budget);
      if (ok && both && (w == 1 || join)) ok = wait_all<false>(&ctl.o_full[1], no1 & 1, abort_flag, budget);
      ++no0;
      no1 += both;
      if (!ok) break;
      tc::fence_after_sync();
      // every product of this piece with Q is done: the next piece's rows are on
      // their way while this one's are written
      have = cur.next();
      if (have) load_q();
      const float l_row = sum.x + sum.y;
      const bool bad = *(volatile int*)&ctl.bad[piece % kBadSlots] != 0;
      const float nan = __int_as_float(0x7fc00000);
      // where the row goes: the output, or the piece's place in the scratch
      const int64_t prow = ((int64_t)blockIdx.x * 2 + (first ? 1 : 0)) * 256 + tile * kRows + r;
      char* out16 = first && last ? static_cast<char*>(a.out) + out_row * (D * 2) : nullptr;
      float* out32 = sc.o + prow * D;
      auto finish = [&](float m, float l) -> float {  // what the sums are scaled by
        if (first && last) {
          if (valid && a.lse && (pair || w == 0))
            a.lse[out_row] = bad ? nan : l == 0.f ? kNegInf : m * kLn2 + logf(l);
          return bad ? nan : l == 0.f ? 0.f : 1.f / l;
        }
        if (valid && (pair || w == 0)) sc.ml[prow] = bad ? make_float2(0.f, nan) : make_float2(m, l);
        return 1.f;
      };
      if (!join) {
        if (pair || w == 0) {
          const float f = finish(ref, l_row);
          if (!idle) {
#pragma unroll
            for (int c = 0; c < D / 32; ++c) {
              uint32_t v[32];
              tc::tmem_ld32(t_o + c * 32, v);
              tc::tmem_ld_wait(v);
              float x[32];
#pragma unroll
              for (int i = 0; i < 32; ++i) x[i] = l_row == 0.f && !bad ? 0.f : __uint_as_float(v[i]) * f;
              if (valid) store_cols<BF16>(x, out16, out32, c * 32);
            }
          }
        }
      } else {
        // the warpgroups join: they exchange references and sums in the columns
        // of the scores, and each finishes one half of both outputs' columns
        if (!idle) {
          tc::tmem_st2(t_s, ref, l_row);
          tc::tmem_st_wait();
        }
        tc::fence_before_sync();
        tc::mbar_arrive(&ctl.ex1);
        ok = wait_all<false>(&ctl.ex1, nx & 1, abort_flag, budget);
        if (!ok) break;
        tc::fence_after_sync();
        if (!idle) {
          const float2 other = tc::tmem_ld2(tmem + lanes + (1 - w) * 128);
          const float m = fmaxf(ref, other.x), ms = m == kNegInf ? 0.f : m;
          const float f0 = tc::exp2_approx(ref - ms), f1 = tc::exp2_approx(other.x - ms);
          const float l = l_row * f0 + other.y * f1;
          const float f = finish(m, l);
          const bool none = l == 0.f && !bad;
#pragma unroll
          for (int c = 0; c < D / 64; ++c) {
            uint32_t v[32], u[32];
            const uint32_t at = w * (D / 2) + c * 32;
            tc::tmem_ld32(t_o + at, v);
            tc::tmem_ld32(tmem + lanes + 256 + (1 - w) * 128 + at, u);
            tc::tmem_ld_wait(v);
            tc::tmem_ld_wait(u);
            float x[32];
#pragma unroll
            for (int i = 0; i < 32; ++i)
              x[i] = none ? 0.f : (__uint_as_float(v[i]) * f0 + __uint_as_float(u[i]) * f1) * f;
            if (valid) store_cols<BF16>(x, out16, out32, at);
          }
        }
        tc::fence_before_sync();
        tc::mbar_arrive(&ctl.ex2);
        ok = wait_all<false>(&ctl.ex2, nx++ & 1, abort_flag, budget);
        if (!ok) break;
      }
      if (!(first && last) && !idle && (pair || join || w == 0)) {
        // a piece of an item: its blocks are counted for each warp's rows, of a
        // tile, or of a half of the columns where a single tile's are divided
        constexpr int kCols = D < 64 * 2 ? D / 2 : 64;
        const int only = pair || join ? w : -1;
        for (int h = only < 0 ? 0 : only; h < (only < 0 ? 2 : only + 1); ++h) {
          __threadfence();
          __syncwarp();
          int before = 0;
          if (lane == 0)
            before = atomicAdd(sc.done + ((int64_t)p_idx * a.kv_heads + p_hk) * 8 + h * 4 + (warp & 3), nb);
          before = __shfl_sync(0xFFFFFFFFu, before, 0);
          if (before + nb != it.nblk) continue;
          __threadfence();
          const int from = pair ? 0 : h * (D / 2), to = pair ? D : from + D / 2;
          for (int c = from; c < to; c += kCols)
            join_rows<BF16, D, kCols>(a, sc, cur, it, p_hk, tile, warp & 3, c, out_row, valid);
        }
      }
      if (have) q_loaded();
      // the next piece's first values overwrite what was read here
      tc::fence_before_sync();
    }
    if (!ok && lane == 0) {
      *abort_flag = 1;
      record_error(err, kDevErrTimeout);
    }
  }
  tc::fence_before_sync();
  cta_sync();
  if (warp == 9) {
    tc::fence_after_sync();
    tc::tmem_dealloc(tmem, 512);
  }
  // at the end, so that a call without such rows pays one look at the header (on the
  // softmax's way to its next piece it took 8 us of the 346 of two prompts)
  if (warp < 8 && sc.head->fill != kFillNone) fill_rows<BF16, D>(a, sc, warp);
}

template <bool BF16, int D>
cudaError_t launch_all(const AttnArgs& a, const Scratch& sc, int parts, int* err, cudaStream_t s) {
  const bool kf = a.ks.head <= a.ks.token, vf = a.vs.head <= a.vs.token;
  const int page = 1 << a.page_shift, box = page < kKeys ? page : kKeys;
  CUtensorMap kmap, vmap;
  if (!make_cache_map(&kmap, a.k_cache, BF16, D, page, a.kv_heads, a.pages, a.ks, box, kf) ||
      !make_cache_map(&vmap, a.v_cache, BF16, D, page, a.kv_heads, a.pages, a.vs, box, vf))
    return cudaErrorInvalidValue;
  const int64_t counts = most_items(a.S, a.T, a.heads / a.kv_heads) * a.kv_heads * 8;
  int64_t work = counts / 4;
  if (a.k && (int64_t)a.T * a.kv_heads * (D / 8) > work) work = (int64_t)a.T * a.kv_heads * (D / 8);
  int64_t ctas = (work + kPrepThreads - 1) / kPrepThreads;
  if (ctas > (int64_t)parts * 8) ctas = (int64_t)parts * 8;
  cudaError_t e = launch_kernel(true, prepare_kernel, dim3((unsigned)ctas + 1), dim3(kPrepThreads),
                                0, s, a, sc, parts, counts, D / 8, err);
  if (e != cudaSuccess) return e;
  static int smem_set[64] = {0};
  e = ensure_dynamic_smem(attend_kernel<BF16, D>, Shape<D>::kSmem, smem_set);
  if (e != cudaSuccess) return e;
  return launch_kernel(true, attend_kernel<BF16, D>, dim3(parts), dim3(kThreads),
                       Shape<D>::kSmem, s, kmap, vmap, a, sc, (int)kf, (int)vf, role_wait_cycles(),
                       err);
}

}  // namespace

size_t attention_scratch_bytes(int S, int T, int heads, int kv_heads, int dim) {
  return scratch_size(part_count(), most_items(S, T, heads / kv_heads), kv_heads, dim).total;
}

cudaError_t launch_attention(const AttnArgs& a, void* scratch, int* err, cudaStream_t s) {
  const int parts = part_count();
  const ScratchSize z = scratch_size(parts, most_items(a.S, a.T, a.heads / a.kv_heads), a.kv_heads,
                                     a.dim);
  char* p = static_cast<char*>(scratch);
  const Scratch sc = {reinterpret_cast<Header*>(p),           reinterpret_cast<int4*>(p + z.start),
                      reinterpret_cast<float2*>(p + z.ml),    reinterpret_cast<float*>(p + z.o),
                      reinterpret_cast<Item*>(p + z.items),   reinterpret_cast<int*>(p + z.done)};
  if (a.dtype == LMHEAD_BF16)
    return a.dim == 64 ? launch_all<true, 64>(a, sc, parts, err, s)
                       : launch_all<true, 128>(a, sc, parts, err, s);
  return a.dim == 64 ? launch_all<false, 64>(a, sc, parts, err, s)
                     : launch_all<false, 128>(a, sc, parts, err, s);
}

}  // namespace lmhead
