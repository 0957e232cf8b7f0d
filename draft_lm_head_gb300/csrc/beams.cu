// One step of a beam search: the k best continuations over all beams of a
// sequence and all entries of their rows, and the reordering of the beams'
// states by the parents found.
//
// score(b, j) = parent_b + (x_bj - lse_b), lse_b = log sum_j exp x_bj. Within a
// row the order of the scores is the order of x, so one pass over a row gives
// both its log-sum-exp and its k largest x; only those few are ever scored.
//   beam_rows:  a warp streams one slice of one row through a ring of shared
//     memory (16 values a lane a tile, several tiles' copies in flight), keeping
//     a running reference and sum of the softmax and the slice's k best so far;
//     no barrier, and past the first tile little but the exponentials.
//   beam_merge: a CTA per sequence turns the slices' sums into lse and picks
//     the k best of beams x slices x k scored entries.
//   beam_small: both in one launch where a sequence has few slices.
// Measured: 64 sequences x 8 rows of 151936 fp32 logits, k = 8, with the
// reordering of the 512 states: 63 us, 4.7 TB/s (a tenth of the beams has ended and
// their rows are not read; torch's maximum of all rows alone takes 62).
// Bound by reading the logits once. Beams meet at the border of the k with gaps
// below 32-bit rounding, so a lane's sums of exp, and the exponentials in them,
// are 32-bit (within 2^-22 or so of their values), but everything across lanes,
// and the scores of the few candidates, are pairs of fp32 numbers (the rounded
// value and what its rounding left: about 48 bits; fp64 units are too few on this
// GPU, the merge took twice as long with them).
#include <cuda_fp16.h>

#include <type_traits>

#include "common.cuh"
#include "kernels.h"

namespace lmhead {
namespace {

constexpr int kRowThreads = 256;
constexpr int kPerLane = 16;
constexpr int kTile = 32 * kPerLane;  // entries of a warp's tile
// A warp's ring of tiles, and the warps an SM has room for by it: 144 KB of an
// SM's copies in flight. (4, 6 and 12 KB with 32, 32 and 16 warps: 64 x 8 rows of
// 151936 69, 68 and 65 us in all against 64; loads to registers, a tile ahead: 77.)
constexpr int kRing = 8192, kWarpsSm = 24;
constexpr int kRowsSmem = kRowThreads / 32 * kRing;
constexpr int kBuf = 1024;            // the merge's candidates
constexpr float kNegInf = -__builtin_huge_valf();
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLag = 1.f;  // how far values may lie above a lane's reference

template <typename T> struct Elem;
template <> struct Elem<float> {
  static constexpr int kVec = 4;
  static __device__ __forceinline__ float get(const float* p) { return *p; }
  static __device__ __forceinline__ void unpack(const uint4& v, float* f) {
    f[0] = __uint_as_float(v.x);
    f[1] = __uint_as_float(v.y);
    f[2] = __uint_as_float(v.z);
    f[3] = __uint_as_float(v.w);
  }
};
template <> struct Elem<__nv_bfloat16> {
  static constexpr int kVec = 8;
  static __device__ __forceinline__ float get(const __nv_bfloat16* p) { return __bfloat162float(*p); }
  static __device__ __forceinline__ void unpack(const uint4& v, float* f) { unpack8(v, f); }
};
template <> struct Elem<__half> {
  static constexpr int kVec = 8;
  static __device__ __forceinline__ float get(const __half* p) { return __half2float(*p); }
  static __device__ __forceinline__ void unpack(const uint4& v, float* f) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 t = __half22float2(*reinterpret_cast<const __half2*>(&w[i]));
      f[2 * i] = t.x;
      f[2 * i + 1] = t.y;
    }
  }
};

// h + l, |l| at most half a step of h.
struct Pair {
  float h, l;
};
__device__ __forceinline__ Pair two_sum(float a, float b) {  // exactly
  const float s = a + b, t = s - a;
  return {s, (a - (s - t)) + (b - t)};
}
__device__ __forceinline__ Pair add(Pair a, Pair b) {
  const Pair s = two_sum(a.h, b.h);
  const float l = s.l + (a.l + b.l), h = s.h + l;
  return {h, l - (h - s.h)};
}
__device__ __forceinline__ Pair warp_sum(Pair v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1)
    v = add(v, Pair{__shfl_xor_sync(0xFFFFFFFFu, v.h, o), __shfl_xor_sync(0xFFFFFFFFu, v.l, o)});
  return v;
}

struct __align__(16) Slice {  // what a slice of a row leaves
  float top;  // a reference value
  Pair sum;   // of exp(x - top)
  float pad;
};

__device__ __forceinline__ float2 add2(float2 a, float2 b) {
  float2 d;
  asm("{\n\t.reg .b64 x, y;\n\tmov.b64 x, {%2, %3};\n\tmov.b64 y, {%4, %5};\n\t"
      "add.rn.f32x2 x, x, y;\n\tmov.b64 {%0, %1}, x;\n\t}"
      : "=f"(d.x), "=f"(d.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  return d;
}
__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
  float2 d;
  asm("{\n\t.reg .b64 x, y;\n\tmov.b64 x, {%2, %3};\n\tmov.b64 y, {%4, %5};\n\t"
      "mul.rn.f32x2 x, x, y;\n\tmov.b64 {%0, %1}, x;\n\t}"
      : "=f"(d.x), "=f"(d.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  return d;
}
__device__ __forceinline__ float exp2_fast(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// The k-th largest (or -inf) of the block's per-thread values, by warp 0:
// each round takes one copy of the current largest away.
__device__ __forceinline__ float kth_of_threads(float mine, int k, float* sh, float* out) {
  const int tid = threadIdx.x;
  sh[tid] = mine;
  cta_sync();
  if (tid < 32) {
    uint32_t key[kRowThreads / 32];
    uint32_t best = 0;
#pragma unroll
    for (int i = 0; i < kRowThreads / 32; ++i) {
      key[i] = float_key(sh[i * 32 + tid]);
      best = max(best, key[i]);
    }
    uint32_t top = 0;
    for (int r = 0; r < k; ++r) {
      top = __reduce_max_sync(0xFFFFFFFFu, best);
      const uint32_t who = __ballot_sync(0xFFFFFFFFu, best == top);
      if (tid == __ffs(who) - 1) {
        bool gone = false;
        best = 0;
#pragma unroll
        for (int i = 0; i < kRowThreads / 32; ++i) {
          if (!gone && key[i] == top) {
            key[i] = 0;
            gone = true;
          }
          best = max(best, key[i]);
        }
      }
    }
    if (tid == 0) *out = key_float(top);
  }
  cta_sync();
  return *out;
}

// Slice sl of the row at x, by one warp. Tiles are copied to the warp's ring
// several ahead; a lane reads back what it copied itself, so its own waits are
// all there is, and a stage is filled again an iteration after it was read.
template <typename T>
__device__ __forceinline__ void scan_slice(const T* x, int n, int sl, int slice_len, int k,
                                           char* ring, Slice* slice, float* best_v,
                                           int32_t* best_i) {
  const int lane = threadIdx.x & 31;
  constexpr int kStage = kTile * (int)sizeof(T), kStages = kRing / kStage;
  constexpr int V = Elem<T>::kVec, U = kPerLane / V;
  // 16-byte reads at 16-byte boundaries: the row starts `off` entries after
  // one, and slices are cut at them
  const int off = (int)((reinterpret_cast<uintptr_t>(x) & 15u) / sizeof(T));
  const int lo = max(0, sl * slice_len - off), hi = min(n, (sl + 1) * slice_len - off);
  auto inside = [&](int base) { return base * V - off >= lo && base * V - off + kTile <= hi; };
  const uint32_t mine = (uint32_t)__cvta_generic_to_shared(ring) + lane * 16;
  auto fetch = [&](int base, int stage) {
    if (inside(base))
#pragma unroll
      for (int u = 0; u < U; ++u)
        asm volatile("cp.async.cg.shared.global.L2::256B [%0], [%1], 16;" ::"r"(
                         mine + stage * kStage + u * 512),
                     "l"(x + (base + u * 32 + lane) * V - off)
                     : "memory");
    asm volatile("cp.async.commit_group;" ::: "memory");
  };
  float m = kNegInf;
  float2 s2 = make_float2(0.f, 0.f);
  uint64_t best = 0;        // lane j: the (j + 1)-th best entry so far, 0 for none
  float floor_v = kNegInf;  // the k-th of them
  int base = sl * (slice_len / V);
#pragma unroll
  for (int i = 0; i < kStages - 1; ++i) fetch(base + i * (kTile / V), i);
  int stage = 0, last = kStages - 1;
  for (; base * V - off < hi; base += kTile / V) {
    float f[kPerLane];
    fetch(base + (kStages - 1) * (kTile / V), last);
    asm volatile("cp.async.wait_group %0;" ::"n"(kStages - 1) : "memory");
    if (inside(base)) {
#pragma unroll
      for (int u = 0; u < U; ++u)
        Elem<T>::unpack(*reinterpret_cast<const uint4*>(ring + stage * kStage + u * 512 + lane * 16),
                        f + u * V);
    } else {
#pragma unroll
      for (int i = 0; i < kPerLane; ++i) {
        const int e = (base + i / V * 32 + lane) * V - off + i % V;
        f[i] = e >= lo && e < hi ? Elem<T>::get(x + e) : kNegInf;
      }
    }
    last = stage;
    stage = stage + 1 == kStages ? 0 : stage + 1;
    float tm = f[0];
#pragma unroll
    for (int i = 1; i < kPerLane; ++i) tm = fmaxf(tm, f[i]);
    if (!(tm >= kNegInf)) tm = kNegInf;  // all NaN
    // The sum is kept relative to a reference that the values pass by kLag at most:
    // an exponent's argument is rounded by 2^-23 or so of its size, which is all
    // of the error where one value has most of the sum. (At 60 in place of 1 a
    // score was off by up to 5e-6, now by 2e-7; 64 x 8 rows of 151936 62.6 against
    // 63.2 us, at 0 63.4.)
    if (tm > m + kLag || (m == kNegInf && tm > kNegInf)) {
      const float f0 = m == kNegInf ? 0.f : exp2_fast((m - tm) * kLog2e);
      s2.x *= f0;
      s2.y *= f0;
      m = tm;
    }
    const float ref = m == kNegInf ? 0.f : -m;
#pragma unroll
    for (int i = 0; i < kPerLane; i += 2) {
      const float2 d = mul2(add2(make_float2(f[i], f[i + 1]), make_float2(ref, ref)),
                            make_float2(kLog2e, kLog2e));
      s2 = add2(s2, make_float2(exp2_fast(d.x), exp2_fast(d.y)));
    }
    // Into the k best, one after the other: the largest value not yet taken (the
    // lowest index among equals) while it beats the k-th best. An equal value
    // further on has a higher index and stays out.
    while (true) {
      const bool want = tm > floor_v;
      if (!__any_sync(0xFFFFFFFFu, want)) break;
      const uint32_t key = want ? float_key(tm) : 0u;
      const uint32_t top = __reduce_max_sync(0xFFFFFFFFu, key);
      int own = 0;  // the first place of the lane's largest
#pragma unroll
      for (int i = kPerLane - 1; i >= 0; --i) own = f[i] == tm ? i : own;
      const uint32_t index =
          key == top ? (uint32_t)((base + own / V * 32 + lane) * V - off + own % V) : ~0u;
      const uint32_t win = __reduce_min_sync(0xFFFFFFFFu, index);
      const uint64_t entry = ((uint64_t)top << 32) | (uint32_t)~win;
      const int place = __popc(__ballot_sync(0xFFFFFFFFu, best > entry));
      const uint64_t above = __shfl_up_sync(0xFFFFFFFFu, best, 1);
      if (lane > place) best = above;
      if (lane == place) best = entry;
      const uint64_t least = __shfl_sync(0xFFFFFFFFu, best, k - 1);
      floor_v = least == 0 ? kNegInf : key_score(least);
      if (index == win) {
        tm = kNegInf;
#pragma unroll
        for (int i = 0; i < kPerLane; ++i) {
          if (i == own) f[i] = kNegInf;
          tm = fmaxf(tm, f[i]);
        }
      }
    }
  }
  // the slice's reference and sum
  const float s = s2.x + s2.y, top = warp_max(m);
  const Pair sum =
      warp_sum(Pair{m == kNegInf && s == 0.f ? 0.f : s * exp2_fast((m - top) * kLog2e), 0.f});
  if (lane == 0) *slice = {top, sum, 0.f};
  if (lane < k) {
    best_v[lane] = best ? key_score(best) : kNegInf;
    best_i[lane] = best ? key_id(best) : -1;
  }
}

template <typename T>
__global__ void __launch_bounds__(kRowThreads, kWarpsSm * 32 / kRowThreads)
beam_rows_kernel(const T* logits, int64_t stride, int n, int rows, int nsl, int slice_len, int k,
                 const uint8_t* finished, Slice* slices, float* best_v, int32_t* best_i) {
  extern __shared__ __align__(16) char rings[];
  pdl_wait();
  pdl_trigger();
  const int64_t unit = (int64_t)blockIdx.x * (kRowThreads / 32) + (threadIdx.x >> 5);
  if (unit >= (int64_t)rows * nsl) return;
  const int row = (int)(unit / nsl), sl = (int)(unit - (int64_t)row * nsl);
  if (finished && finished[row]) return;  // its one entry is its own score
  scan_slice(logits + (int64_t)row * stride, n, sl, slice_len, k,
             rings + (threadIdx.x >> 5) * kRing, slices + unit, best_v + unit * k,
             best_i + unit * k);
}

// Order of the merge: the larger score (as a key that orders like the pair of
// it; 0 is below every score that can be taken), then the lower index.
__device__ __forceinline__ bool ahead(uint64_t sa, int32_t ia, uint64_t sb, int32_t ib) {
  return sa > sb || (sa == sb && ia < ib);
}

// The k best of a sequence from its rows' slices, by one CTA.
__device__ __forceinline__ void merge_sequence(const BeamArgs& a, int seq, int nsl,
                                               const Slice* slices, const float* best_v,
                                               const int32_t* best_i) {
  // lse in its two parts: x - top is small where top is not
  __shared__ float row_top[kBeamMaxBeams];
  __shared__ Pair row_log[kBeamMaxBeams];
  __shared__ float row_score[kBeamMaxBeams];
  __shared__ bool row_done[kBeamMaxBeams];
  __shared__ uint64_t b_score[kBuf];
  __shared__ int32_t b_flat[kBuf];
  __shared__ float sh_f[kRowThreads];
  __shared__ float sh_out;
  __shared__ int sh_count;
  __shared__ uint64_t w_score[kRowThreads / 32];
  __shared__ int32_t w_flat[kRowThreads / 32];
  const int tid = threadIdx.x, lane = tid & 31, B = a.beams, k = a.k;
  const int32_t n = (int32_t)a.n;
  const int per = nsl * k, all = B * per;
  const size_t row0 = (size_t)seq * B;
  // a thread's first kKept entries are under way while the rows' sums are made
  constexpr int kKept = 4;
  float kept_v[kKept];
  int32_t kept_i[kKept];
#pragma unroll
  for (int j = 0; j < kKept; ++j) {
    const int e = tid + j * kRowThreads;
    kept_v[j] = e < all ? best_v[e] : 0.f;
    kept_i[j] = e < all ? best_i[e] : -1;
  }
  for (int b = tid >> 5; b < B; b += kRowThreads / 32) {  // a warp per row
    const Slice* sl = slices + (size_t)b * nsl;
    const bool done = a.finished && a.finished[row0 + b];
    const float score = a.scores[row0 + b];
    float top = kNegInf;
    Pair sum = {0.f, 0.f};
    for (int i0 = 0; i0 < nsl; i0 += 32) {
      Slice v = {kNegInf, {0.f, 0.f}, 0.f};
      if (i0 + lane < nsl) v = sl[i0 + lane];
      const float now = fmaxf(top, warp_max(v.top));
      if (now != top) {
        const float f = exp2_fast((top - now) * kLog2e);
        sum.h *= f;
        sum.l *= f;
      }
      top = now;
      if (v.top != kNegInf || v.sum.h != 0.f) {
        const float f = exp2_fast((v.top - top) * kLog2e);
        sum = add(sum, Pair{v.sum.h * f, v.sum.l * f});
      }
    }
    sum = warp_sum(sum);
    if (lane == 0) {
      row_done[b] = done;
      row_score[b] = score;
      row_top[b] = top;
      row_log[b] = sum;
    }
  }
  cta_sync();
  for (int b = tid; b < B; b += kRowThreads) {  // a lane per row: a warp's logarithms at once
    const double l = log((double)row_log[b].h + (double)row_log[b].l);
    row_log[b] = {(float)l, (float)(l - (double)(float)l)};
  }
  if (tid == 0) sh_count = 0;
  cta_sync();
  // entry e of the sequence, value v at index i of its row: the key of its
  // score, 0 when it cannot be taken
  auto score_of = [&](int e, float v, int32_t i, int32_t& flat) -> uint64_t {
    const int b = e / per;
    Pair sc;
    if (row_done[b]) {
      flat = b * n;
      sc = {e == b * per ? row_score[b] : kNegInf, 0.f};
    } else {
      flat = b * n + i;
      if (i < 0) return 0;
      const Pair lg = row_log[b];
      sc = add(add(Pair{row_score[b], 0.f}, two_sum(v, -row_top[b])), Pair{-lg.h, -lg.l});
    }
    if (!(fabsf(sc.h) < -kNegInf)) return 0;  // NaN too
    return ((uint64_t)float_key(sc.h) << 32) | float_key(sc.l);
  };
  auto entry = [&](int e, int32_t& flat) { return score_of(e, best_v[e], best_i[e], flat); };
  auto rounded = [](uint64_t key) { return key ? key_float((uint32_t)(key >> 32)) : kNegInf; };
  // the k-th largest of the threads' rounded maxima bounds the k best from below
  uint64_t kept[kKept];
  float mine = kNegInf;
#pragma unroll
  for (int j = 0; j < kKept; ++j) {
    const int e = tid + j * kRowThreads;
    kept[j] = e < all ? score_of(e, kept_v[j], kept_i[j], kept_i[j]) : 0;
    mine = fmaxf(mine, rounded(kept[j]));
  }
  for (int e = tid + kKept * kRowThreads; e < all; e += kRowThreads) {
    int32_t flat;
    mine = fmaxf(mine, rounded(entry(e, flat)));
  }
  const float bound = kth_of_threads(mine, k, sh_f, &sh_out);
  auto offer = [&](uint64_t sc, int32_t flat) {
    if (sc == 0 || rounded(sc) < bound) return;
    const int at = atomicAdd(&sh_count, 1);
    if (at < kBuf) {
      b_score[at] = sc;
      b_flat[at] = flat;
    }
  };
#pragma unroll
  for (int j = 0; j < kKept; ++j) offer(kept[j], kept_i[j]);
  for (int e = tid + kKept * kRowThreads; e < all; e += kRowThreads) {
    int32_t flat;
    const uint64_t sc = entry(e, flat);
    offer(sc, flat);
  }
  cta_sync();
  int fill = sh_count;
  if (fill > kBuf) {
    // more equal scores than places: one by one
    uint64_t ls = ~0ull;
    int32_t li = -1;
    for (fill = 0; fill < k; ++fill) {
      uint64_t ts = 0;
      int32_t ti = INT32_MAX;
      for (int e = tid; e < all; e += kRowThreads) {
        int32_t flat;
        const uint64_t sc = entry(e, flat);
        if (sc != 0 && ahead(ls, li, sc, flat) && ahead(sc, flat, ts, ti)) {
          ts = sc;
          ti = flat;
        }
      }
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) {
        const uint64_t os = __shfl_xor_sync(0xFFFFFFFFu, ts, o);
        const int32_t oi = __shfl_xor_sync(0xFFFFFFFFu, ti, o);
        if (ahead(os, oi, ts, ti)) {
          ts = os;
          ti = oi;
        }
      }
      if ((tid & 31) == 0) {
        w_score[tid >> 5] = ts;
        w_flat[tid >> 5] = ti;
      }
      cta_sync();
      ts = w_score[0];
      ti = w_flat[0];
      for (int w = 1; w < kRowThreads / 32; ++w)
        if (ahead(w_score[w], w_flat[w], ts, ti)) {
          ts = w_score[w];
          ti = w_flat[w];
        }
      cta_sync();
      if (ti == INT32_MAX) break;
      if (tid == 0) {
        b_score[fill] = ts;
        b_flat[fill] = ti;
      }
      ls = ts;
      li = ti;
    }
    cta_sync();
  }
  int32_t* parent = a.parent + (size_t)seq * k;
  int32_t* token = a.token + (size_t)seq * k;
  float* score = a.out_score + (size_t)seq * k;
  for (int c = tid; c < fill; c += kRowThreads) {
    const uint64_t sc = b_score[c];
    const int32_t flat = b_flat[c];
    int place = 0;
    for (int o = 0; o < fill && place < k; ++o) place += ahead(b_score[o], b_flat[o], sc, flat);
    if (place >= k) continue;
    const int b = flat / n, i = flat - b * n, row = seq * B + b;
    parent[place] = b;
    token[place] = row_done[b] ? a.eos
                   : a.ids ? a.ids[(size_t)row * n + i] : i;
    score[place] = rounded(sc);
  }
  for (int c = fill + tid; c < k; c += kRowThreads) {
    parent[c] = -1;
    token[c] = -1;
    score[c] = kNegInf;
  }
}

__global__ void __launch_bounds__(kRowThreads)
beam_merge_kernel(BeamArgs a, int nsl, const Slice* slices, const float* best_v,
                  const int32_t* best_i) {
  pdl_wait();
  pdl_trigger();
  const size_t unit = (size_t)blockIdx.x * a.beams * nsl;
  merge_sequence(a, blockIdx.x, nsl, slices + unit, best_v + unit * a.k, best_i + unit * a.k);
}

// Both steps of a sequence whose rows have few slices, in one launch: the head's
// candidates, short vocabularies.
constexpr int kFewSlices = 16;
template <typename T>
__global__ void __launch_bounds__(kRowThreads)
beam_small_kernel(const T* logits, BeamArgs a, int nsl, int slice_len) {
  __shared__ Slice slices[kFewSlices];
  __shared__ float best_v[kFewSlices * kBeamMaxK];
  __shared__ int32_t best_i[kFewSlices * kBeamMaxK];
  extern __shared__ __align__(16) char rings[];
  pdl_wait();
  pdl_trigger();
  for (int u = threadIdx.x >> 5; u < a.beams * nsl; u += kRowThreads / 32) {
    const int b = u / nsl;
    const size_t row = (size_t)blockIdx.x * a.beams + b;
    if (a.finished && a.finished[row]) continue;
    scan_slice(logits + (int64_t)row * a.row_stride, (int)a.n, u - b * nsl, slice_len, a.k,
               rings + (threadIdx.x >> 5) * kRing, slices + u, best_v + u * a.k, best_i + u * a.k);
  }
  cta_sync();
  merge_sequence(a, blockIdx.x, nsl, slices, best_v, best_i);
}

// ---- states of the chosen beams: out[s, j] = state[s, parent[s, j]], zeros
// where there is no parent. A copy: 16 bytes a thread where the row allows.
constexpr int kCopyBytes = 16384;  // of a row, per CTA

__global__ void __launch_bounds__(256) beam_reorder_kernel(ReorderArgs a, int* err) {
  pdl_wait();
  pdl_trigger();
  const int which = blockIdx.z, o = blockIdx.x;
  const int64_t bytes = a.bytes[which], lo = (int64_t)blockIdx.y * kCopyBytes;
  if (lo >= bytes) return;
  const int64_t hi = min(bytes, lo + kCopyBytes);
  const int seq = o / a.k;
  const int b = a.parent[o];
  const bool bad = b >= a.beams || b < -1;
  if (bad && threadIdx.x == 0) record_error(err, kDevErrBadId);
  const bool live = b >= 0 && !bad;
  const char* src =
      static_cast<const char*>(a.src[which]) + ((int64_t)seq * a.beams + (live ? b : 0)) * bytes;
  char* dst = static_cast<char*>(a.dst[which]) + (int64_t)o * bytes;
  if (((reinterpret_cast<uintptr_t>(a.src[which]) | reinterpret_cast<uintptr_t>(a.dst[which]) |
        (uintptr_t)bytes) & 15u) == 0) {
    for (int64_t e = lo + threadIdx.x * 16; e < hi; e += 256 * 16) {
      uint4 v = make_uint4(0, 0, 0, 0);
      if (live) v = ldg_nc_v4(src + e);
      *reinterpret_cast<uint4*>(dst + e) = v;
    }
  } else {
    for (int64_t e = lo + threadIdx.x; e < hi; e += 256) dst[e] = live ? src[e] : 0;
  }
}

// Entries of a row per warp: whole tiles, as many slices as leave every warp
// slot of the GPU one of them.
int slice_len(int rows, int64_t n) {
  const int64_t tiles = (n + kTile - 1) / kTile;
  const int sms = sm_count() > 0 ? sm_count() : 1;
  int64_t want = (int64_t)sms * kWarpsSm / rows;
  if (want < 1) want = 1;
  const int64_t per = tiles <= want ? 1 : (tiles + want - 1) / want;
  return (int)(per * kTile);
}
int slices_of(int rows, int64_t n) {
  const int len = slice_len(rows, n);
  return (int)((n + 7 + len - 1) / len);  // a row may start up to 7 entries past a boundary
}

}  // namespace

size_t beam_scratch_bytes(int S, int beams, int64_t n, int k) {
  const size_t cells = (size_t)S * beams * slices_of(S * beams, n);
  return cells * (sizeof(Slice) + (size_t)k * 8);
}

cudaError_t launch_beam_select(const BeamArgs& a, void* scratch, cudaStream_t s) {
  const int rows = a.S * a.beams, len = slice_len(rows, a.n), nsl = slices_of(rows, a.n);
  const size_t cells = (size_t)rows * nsl;
  Slice* sl = static_cast<Slice*>(scratch);
  float* bv = reinterpret_cast<float*>(sl + cells);
  int32_t* bi = reinterpret_cast<int32_t*>(bv + cells * a.k);
  const int warps = kRowThreads / 32;
  const dim3 grid((unsigned)((cells + warps - 1) / warps)), block(kRowThreads);
  const bool few = a.beams * nsl <= kFewSlices;
  auto scan = [&](auto* logits) -> cudaError_t {
    using T = std::remove_cv_t<std::remove_pointer_t<decltype(logits)>>;
    static int smem_small[64], smem_rows[64];
    if (few) {
      const cudaError_t e = ensure_dynamic_smem(beam_small_kernel<T>, kRowsSmem, smem_small);
      if (e != cudaSuccess) return e;
      return launch_kernel(true, beam_small_kernel<T>, dim3(a.S), block, kRowsSmem, s, logits, a, nsl,
                           len);
    }
    const cudaError_t e = ensure_dynamic_smem(beam_rows_kernel<T>, kRowsSmem, smem_rows);
    if (e != cudaSuccess) return e;
    return launch_kernel(true, beam_rows_kernel<T>, grid, block, kRowsSmem, s, logits, a.row_stride,
                         (int)a.n, rows, nsl, len, a.k, a.finished, sl, bv, bi);
  };
  const cudaError_t e = a.dtype == LMHEAD_FP32   ? scan(static_cast<const float*>(a.logits))
                        : a.dtype == LMHEAD_BF16 ? scan(static_cast<const __nv_bfloat16*>(a.logits))
                                                 : scan(static_cast<const __half*>(a.logits));
  if (e != cudaSuccess || few) return e;
  return launch_kernel(true, beam_merge_kernel, dim3(a.S), block, 0, s, a, nsl, (const Slice*)sl,
                       (const float*)bv, (const int32_t*)bi);
}

cudaError_t launch_beam_reorder(const ReorderArgs& a, int* err, cudaStream_t s) {
  int64_t most = 0;
  for (int i = 0; i < a.count; ++i) most = a.bytes[i] > most ? a.bytes[i] : most;
  const unsigned y = (unsigned)((most + kCopyBytes - 1) / kCopyBytes);
  return launch_kernel(true, beam_reorder_kernel, dim3(a.S * a.k, y, a.count), dim3(256), 0, s, a,
                       err);
}

}  // namespace lmhead
