// One step of a beam search: the k best continuations over all beams of a
// sequence and all entries of their rows, and the reordering of the beams'
// states by the parents found.
//
// score(b, j) = parent_b + (x_bj - lse_b), lse_b = log sum_j exp x_bj. Within a
// row the order of the scores is the order of x, so one pass over a row gives
// both its log-sum-exp and its k largest x; only those few are ever scored.
//   beam_rows:  a CTA streams one slice of one row through registers (32
//     values a thread a tile), keeping the running maximum and sum of the
//     softmax and the slice's k best so far.
//   beam_merge: a CTA per sequence turns the slices' sums into lse and picks
//     the k best of beams x slices x k scored entries.
// Bound by reading the logits once. The sums of exp are 32-bit within a
// thread (at most 32 x tiles terms) and 64-bit across threads, and the scores
// of the few candidates are formed and compared in 64 bits: beams meet at the
// border of the k with gaps below 32-bit rounding.
#include <cuda_fp16.h>

#include "common.cuh"
#include "kernels.h"

namespace lmhead {
namespace {

constexpr int kRowThreads = 256;
constexpr int kPerThread = 32;
constexpr int kTile = kRowThreads * kPerThread;  // 8192 entries
constexpr int kBuf = 1024;                       // candidates held between compactions
constexpr float kNegInf = -__builtin_huge_valf();

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

struct Slice {  // what a slice of a row leaves
  float top;    // its largest value
  float pad;
  double sum;   // of exp(x - top)
};

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

template <typename T>
__global__ void __launch_bounds__(kRowThreads)
beam_rows_kernel(const T* logits, int64_t stride, int n, int slice_len, int k,
                 const uint8_t* finished, Slice* slices, float* best_v, int32_t* best_i) {
  __shared__ uint64_t buf[kBuf + kBeamMaxK];
  __shared__ uint64_t best[kBeamMaxK];
  __shared__ float sh_f[kRowThreads];
  __shared__ double sh_d[kRowThreads / 32];
  __shared__ float sh_out;
  __shared__ int sh_count[3];  // in turn: one counts, the next one is cleared
  __shared__ uint64_t sh_key[kRowThreads / 32];
  pdl_wait();
  pdl_trigger();
  const int tid = threadIdx.x;
  const int row = blockIdx.y, sl = blockIdx.x;
  if (finished && finished[row]) return;  // its one entry is its own score
  constexpr int V = Elem<T>::kVec;
  const T* x = logits + (int64_t)row * stride;
  // 16-byte reads at 16-byte boundaries: the row starts `off` entries after
  // one, and slices are cut at them
  const int off = (int)((reinterpret_cast<uintptr_t>(x) & 15u) / sizeof(T));
  const int lo = max(0, sl * slice_len - off), hi = min(n, (sl + 1) * slice_len - off);
  float m = kNegInf, s = 0.f;
  int have = 0;              // entries in `best`, sorted, best first
  float floor_v = kNegInf;   // the k-th best so far once have == k
  if (tid < 3) sh_count[tid] = 0;
  cta_sync();
  int turn = 0;
  for (int base = sl * (slice_len / V); base * V - off < hi; base += kTile / V) {
    float f[kPerThread];
    float tm = kNegInf;
#pragma unroll
    for (int u = 0; u < kPerThread / V; ++u) {
      const int e = (base + u * kRowThreads + tid) * V - off;
      if (e >= lo && e + V <= hi) {
        Elem<T>::unpack(ldg_nc_v4(x + e), f + u * V);
      } else {
#pragma unroll
        for (int i = 0; i < V; ++i)
          f[u * V + i] = e + i >= lo && e + i < hi ? Elem<T>::get(x + e + i) : kNegInf;
      }
    }
#pragma unroll
    for (int i = 0; i < kPerThread; ++i) tm = fmaxf(tm, f[i]);
    // the softmax's running maximum and sum
    const float nm = fmaxf(m, tm), ref = nm == kNegInf ? 0.f : nm;
    if (m != nm) s *= expf(m - ref);
    m = nm;
    float ts = 0.f;
#pragma unroll
    for (int i = 0; i < kPerThread; ++i) ts += expf(f[i] - ref);
    s += ts;
    // candidates: everything that may be among the slice's k best. While fewer
    // than k are held, the k-th largest of the threads' maxima bounds them from
    // below; later entries must beat the k-th best (an equal one comes later).
    const bool first = have < k;
    const float bound = first ? kth_of_threads(tm, k, sh_f, &sh_out) : floor_v;
    int mine = 0;
#pragma unroll
    for (int i = 0; i < kPerThread; ++i)
      mine += (first ? f[i] >= bound : f[i] > bound) && f[i] > kNegInf;
    int at = 0;
    if (mine) at = atomicAdd(&sh_count[turn], mine);
    if (tid == 0) sh_count[turn == 2 ? 0 : turn + 1] = 0;
    cta_sync();
    const int total = sh_count[turn];
    turn = turn == 2 ? 0 : turn + 1;
    if (total == 0) continue;
    int fill = total;
    if (total <= kBuf) {
      if (mine) {
#pragma unroll
        for (int u = 0; u < kPerThread / V; ++u)
#pragma unroll
          for (int i = 0; i < V; ++i) {
            const float v = f[u * V + i];
            if ((first ? v >= bound : v > bound) && v > kNegInf)
              buf[at++] = select_key(v, (base + u * kRowThreads + tid) * V - off + i);
          }
      }
    } else {
      // many equal values: take the tile's k best one by one
      uint64_t last = ~0ull;
      for (fill = 0; fill < k; ++fill) {
        uint64_t top = 0;
#pragma unroll
        for (int u = 0; u < kPerThread / V; ++u)
#pragma unroll
          for (int i = 0; i < V; ++i) {
            const float v = f[u * V + i];
            const uint64_t key = select_key(v, (base + u * kRowThreads + tid) * V - off + i);
            if (v > kNegInf && key < last && key > top) top = key;
          }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) {
          const uint64_t other = __shfl_xor_sync(0xFFFFFFFFu, top, o);
          top = other > top ? other : top;
        }
        if ((tid & 31) == 0) sh_key[tid >> 5] = top;
        cta_sync();
        top = 0;
        for (int w = 0; w < kRowThreads / 32; ++w) top = sh_key[w] > top ? sh_key[w] : top;
        cta_sync();
        if (top == 0) break;
        if (tid == 0) buf[fill] = top;
        last = top;
      }
    }
    // join with the best so far; an entry's place is the count of larger keys
    if (tid < have) buf[fill + tid] = best[tid];
    cta_sync();
    const int all = fill + have;
    for (int c = tid; c < all; c += kRowThreads) {
      const uint64_t key = buf[c];
      int place = 0;
      for (int o = 0; o < all && place < k; ++o) place += buf[o] > key;
      if (place < k) best[place] = key;
    }
    have = min(all, k);
    cta_sync();
    if (have == k) floor_v = key_score(best[k - 1]);
  }
  // the slice's maximum and sum
  sh_f[tid] = m;
  cta_sync();
  float top = kNegInf;
  for (int i = 0; i < kRowThreads; i += 32) top = fmaxf(top, sh_f[i + (tid & 31)]);
  top = warp_max(top);
  double part = s == 0.f && m == kNegInf ? 0.0 : (double)s * exp((double)m - (double)top);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) part += __shfl_xor_sync(0xFFFFFFFFu, part, o);
  if ((tid & 31) == 0) sh_d[tid >> 5] = part;
  cta_sync();
  const size_t at = (size_t)row * gridDim.x + sl;
  if (tid == 0) {
    double sum = 0;
    for (int w = 0; w < kRowThreads / 32; ++w) sum += sh_d[w];
    slices[at].top = top;
    slices[at].sum = sum;
  }
  if (tid < k) {
    best_v[at * k + tid] = tid < have ? key_score(best[tid]) : kNegInf;
    best_i[at * k + tid] = tid < have ? key_id(best[tid]) : -1;
  }
}

__device__ __forceinline__ bool ahead(double sa, int32_t ia, double sb, int32_t ib) {
  return sa > sb || (sa == sb && ia < ib);
}

__global__ void __launch_bounds__(kRowThreads)
beam_merge_kernel(BeamArgs a, int nsl, const Slice* slices, const float* best_v,
                  const int32_t* best_i) {
  // lse in its two parts: x - top is small where top is not
  __shared__ float row_top[kBeamMaxBeams];
  __shared__ double row_log[kBeamMaxBeams];
  __shared__ double b_score[kBuf];
  __shared__ int32_t b_flat[kBuf];
  __shared__ float sh_f[kRowThreads];
  __shared__ float sh_out;
  __shared__ int sh_count;
  __shared__ double w_score[kRowThreads / 32];
  __shared__ int32_t w_flat[kRowThreads / 32];
  pdl_wait();
  pdl_trigger();
  const int tid = threadIdx.x, seq = blockIdx.x, B = a.beams, k = a.k;
  const int32_t n = (int32_t)a.n;
  for (int b = tid; b < B; b += kRowThreads) {
    const int row = seq * B + b;
    if (a.finished && a.finished[row]) continue;
    float top = kNegInf;
    for (int i = 0; i < nsl; ++i) top = fmaxf(top, slices[(size_t)row * nsl + i].top);
    double sum = 0;
    for (int i = 0; i < nsl; ++i) {
      const Slice sl = slices[(size_t)row * nsl + i];
      if (sl.top != kNegInf || sl.sum != 0.0) sum += sl.sum * exp((double)sl.top - (double)top);
    }
    row_top[b] = top;
    row_log[b] = log(sum);
  }
  if (tid == 0) sh_count = 0;
  cta_sync();
  const int per = nsl * k, all = B * per;
  // entry e of the sequence: its score, -inf when it cannot be taken
  auto entry = [&](int e, int32_t& flat) -> double {
    const int b = e / per, r = e - b * per, row = seq * B + b;
    double sc;
    if (a.finished && a.finished[row]) {
      flat = b * n;
      sc = r == 0 ? (double)a.scores[row] : (double)kNegInf;
    } else {
      const int32_t i = best_i[(size_t)row * per + r];
      flat = b * n + i;
      if (i < 0) return (double)kNegInf;
      sc = (double)a.scores[row] +
           (((double)best_v[(size_t)row * per + r] - (double)row_top[b]) - row_log[b]);
    }
    return sc == sc ? sc : (double)kNegInf;
  };
  // scores rounded to 32 bits keep their order, so the k-th largest of the
  // threads' rounded maxima bounds the k best from below
  float mine = kNegInf;
  for (int e = tid; e < all; e += kRowThreads) {
    int32_t flat;
    mine = fmaxf(mine, (float)entry(e, flat));
  }
  const float bound = kth_of_threads(mine, k, sh_f, &sh_out);
  for (int e = tid; e < all; e += kRowThreads) {
    int32_t flat;
    const double sc = entry(e, flat);
    if (sc > (double)kNegInf && (float)sc >= bound) {
      const int at = atomicAdd(&sh_count, 1);
      if (at < kBuf) {
        b_score[at] = sc;
        b_flat[at] = flat;
      }
    }
  }
  cta_sync();
  int fill = sh_count;
  if (fill > kBuf) {
    // more equal scores than places: one by one
    double ls = __longlong_as_double(0x7ff0000000000000ll);
    int32_t li = -1;
    for (fill = 0; fill < k; ++fill) {
      double ts = (double)kNegInf;
      int32_t ti = INT32_MAX;
      for (int e = tid; e < all; e += kRowThreads) {
        int32_t flat;
        const double sc = entry(e, flat);
        if (sc > (double)kNegInf && ahead(ls, li, sc, flat) && ahead(sc, flat, ts, ti)) {
          ts = sc;
          ti = flat;
        }
      }
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) {
        const double os = __shfl_xor_sync(0xFFFFFFFFu, ts, o);
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
    const double sc = b_score[c];
    const int32_t flat = b_flat[c];
    int place = 0;
    for (int o = 0; o < fill && place < k; ++o) place += ahead(b_score[o], b_flat[o], sc, flat);
    if (place >= k) continue;
    const int b = flat / n, i = flat - b * n, row = seq * B + b;
    parent[place] = b;
    token[place] = a.finished && a.finished[row] ? a.eos
                   : a.ids ? a.ids[(size_t)row * n + i] : i;
    score[place] = (float)sc;
  }
  for (int c = fill + tid; c < k; c += kRowThreads) {
    parent[c] = -1;
    token[c] = -1;
    score[c] = kNegInf;
  }
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

// Entries of a row per CTA: whole tiles, enough CTAs to fill the GPU, but
// slices as long as that allows (each slice costs k merged entries).
int slice_len(int rows, int64_t n) {
  const int64_t tiles = (n + kTile - 1) / kTile;
  const int sms = sm_count() > 0 ? sm_count() : 1;
  const int64_t want = ((int64_t)sms * 8 + rows - 1) / rows;  // slices a row
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
  const dim3 grid(nsl, rows), block(kRowThreads);
  cudaError_t e;
  if (a.dtype == LMHEAD_FP32)
    e = launch_kernel(true, beam_rows_kernel<float>, grid, block, 0, s, (const float*)a.logits,
                      a.row_stride, (int)a.n, len, a.k, a.finished, sl, bv, bi);
  else if (a.dtype == LMHEAD_BF16)
    e = launch_kernel(true, beam_rows_kernel<__nv_bfloat16>, grid, block, 0, s,
                      (const __nv_bfloat16*)a.logits, a.row_stride, (int)a.n, len, a.k, a.finished,
                      sl, bv, bi);
  else
    e = launch_kernel(true, beam_rows_kernel<__half>, grid, block, 0, s, (const __half*)a.logits,
                      a.row_stride, (int)a.n, len, a.k, a.finished, sl, bv, bi);
  if (e != cudaSuccess) return e;
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
