// Which tokens of a paged cache stay, their rows moved together, and the pages
// behind them given back.
#include <cuda_runtime.h>
#include <stdint.h>

#include "common.cuh"
#include "kernels.h"

namespace lmhead {
namespace {

// ------------------------------------------------------------------ select
// Of a request's L tokens and one K/V head the first `sinks`, the last `recent`
// and, of those between, the ones with the largest weights (ties: the lower
// position) up to `budget` in all, in ascending order.
// One CTA a request and head: the weights' order-preserving keys go to shared
// memory, four passes of eight bits find the key of the last one to stay and how
// many equal to it stay with it, and a last pass writes the positions that pass,
// each warp those of a run of its own behind the counts of the runs before.
constexpr int kSelThreads = 1024;
constexpr int kSelWarps = kSelThreads / 32;

__device__ __forceinline__ uint32_t weight_key(float w) {
  return w != w ? 0u : float_key(w);  // a NaN comes last
}

__global__ void __launch_bounds__(kSelThreads)
select_kernel(const SelectArgs a, int staged, int* err) {
  extern __shared__ uint32_t keys[];
  __shared__ int hist[256];
  __shared__ int more_w[kSelWarps], same_w[kSelWarps];
  __shared__ int sh_need, sh_digit;
  pdl_wait();
  pdl_trigger();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int head = blockIdx.x;
  for (int s = blockIdx.y; s < a.S; s += gridDim.y) {
    int32_t* out = a.kept + ((int64_t)s * a.kv_heads + head) * a.budget;
    const int64_t room = (int64_t)a.width * a.page;
    int L = a.lens[s];
    if (L < 0 || L > room) {
      if (tid == 0) record_error(err, kDevErrBadId);
      L = 0;
    }
    if (L <= a.budget) {  // all of them
      for (int i = tid; i < a.budget; i += kSelThreads) out[i] = i < L ? i : -1;
      continue;
    }
    const int lo = min(a.sinks, L), hi = max(lo, L - a.recent);  // positions that are chosen from
    int need = a.budget - lo - (L - hi);
    const int32_t* row = a.table + (int64_t)s * a.width;
    auto key_of = [&](int j) -> uint32_t {
      const int pg = j / a.page;
      const int32_t id = row[pg];
      if (id < 0 || id >= a.pages) {
        record_error(err, kDevErrBadId);
        return 0u;
      }
      return weight_key(*reinterpret_cast<const float*>(static_cast<const char*>(a.weights) +
                                                        id * a.ws.page + (j - pg * a.page) * a.ws.token +
                                                        head * a.ws.head));
    };
    for (int j = lo + tid; j < hi && j - lo < staged; j += kSelThreads) keys[j - lo] = key_of(j);
    auto key = [&](int j) { return j - lo < staged ? keys[j - lo] : key_of(j); };
    uint32_t prefix = 0, mask = 0;
    for (int shift = 24; shift >= 0; shift -= 8) {
      if (tid < 256) hist[tid] = 0;
      cta_sync();
      for (int j = lo + tid; j < hi; j += kSelThreads) {
        const uint32_t k = key(j);
        if ((k & mask) == prefix) atomicAdd(&hist[(k >> shift) & 255], 1);
      }
      cta_sync();
      if (warp == 0) {
        // the digit in which the need-th largest lies: counts from the top
        int c[8], sum = 0;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          c[i] = hist[255 - (lane * 8 + i)];
          sum += c[i];
        }
        int incl = sum;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const int p = __shfl_up_sync(0xFFFFFFFFu, incl, o);
          if (lane >= o) incl += p;
        }
        int at = incl - sum;
        if (at < need && need <= incl) {
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            if (at < need && need <= at + c[i]) {
              sh_digit = 255 - (lane * 8 + i);
              sh_need = need - at;
            }
            at += c[i];
          }
        }
        if (need == 0 && lane == 0) sh_digit = 255, sh_need = 0;
      }
      cta_sync();
      prefix |= (uint32_t)sh_digit << shift;
      mask |= 255u << shift;
      need = sh_need;
      cta_sync();
    }
    // `need` of the keys equal to prefix stay, the first ones; with nothing to
    // choose prefix is the largest key of all, and none of its equals stays
    const int run = ((hi - lo + kSelWarps - 1) / kSelWarps + 31) / 32 * 32;
    const int r0 = min(hi, lo + warp * run), r1 = min(hi, r0 + run);
    int more = 0, same = 0;
    for (int j = r0 + lane; j < r1; j += 32) {
      const uint32_t k = key(j);
      more += k > prefix;
      same += k == prefix;
    }
    more = __reduce_add_sync(0xFFFFFFFFu, more);
    same = __reduce_add_sync(0xFFFFFFFFu, same);
    if (lane == 0) more_w[warp] = more, same_w[warp] = same;
    cta_sync();
    int before = 0, equal = 0;
    for (int w = 0; w < warp; ++w) before += more_w[w], equal += same_w[w];
    for (int j0 = r0; j0 < r1; j0 += 32) {
      const int j = j0 + lane;
      const uint32_t k = j < r1 ? key(j) : 0u;
      const bool is_more = j < r1 && k > prefix, is_same = j < r1 && k == prefix;
      const uint32_t m = __ballot_sync(0xFFFFFFFFu, is_more), e = __ballot_sync(0xFFFFFFFFu, is_same);
      const uint32_t below = (1u << lane) - 1u;
      const int eq = equal + __popc(e & below);
      if (is_more || (is_same && eq < need))
        out[lo + before + __popc(m & below) + min(eq, need)] = j;
      before += __popc(m);
      equal += __popc(e);
    }
    for (int i = tid; i < lo; i += kSelThreads) out[i] = i;
    for (int i = tid; i < L - hi; i += kSelThreads) out[a.budget - (L - hi) + i] = hi + i;
    cta_sync();
  }
}

// -------------------------------------------------------------------- keep
// Row first + i of a request becomes what row first + kept[i] was, kept[i] >= i.
// A row is read from its own place or from one behind it, so rows moved in
// ascending order are read before they are overwritten. A CTA moves one slice of
// the rows' bytes of one tensor and head, for all of the request's list, tile
// after tile: it reads a tile's rows, waits for all its threads, and writes them;
// what it reads later lies behind all that it has written. CTAs share no bytes.
constexpr int kKeepThreads = 256;
constexpr int kKeepUnroll = 8;

template <typename V>
__device__ __forceinline__ void move_slice(const KeepArgs& a, const KeepTensor& t, int s, int head,
                                           int byte0, int bytes, int* err) {
  const int lanes = bytes / (int)sizeof(V);  // of a row; 256 at most
  const int per = kKeepThreads / lanes;      // rows a pass
  const int c = threadIdx.x % lanes, r = threadIdx.x / lanes;
  const bool in = r < per;
  const int32_t* row = a.table + (int64_t)s * a.width;
  const int32_t* kept = a.kept + ((int64_t)s * (a.per_head ? a.kv_heads : 1) + (a.per_head ? head : 0)) * a.n;
  const int64_t first = a.first ? a.first[s] : 0, room = (int64_t)a.width * a.page;
  char* base = static_cast<char*>(t.base) + head * t.st.head + byte0 + c * sizeof(V);
  auto place = [&](int64_t pos) -> char* {
    const int pg = (int)(pos / a.page);
    const int32_t id = row[pg];
    if (id < 0 || id >= a.pages) return nullptr;
    return base + id * t.st.page + (pos - (int64_t)pg * a.page) * t.st.token;
  };
  for (int i0 = 0; i0 < a.n; i0 += per * kKeepUnroll) {
    V v[kKeepUnroll];
    char* to[kKeepUnroll];
#pragma unroll
    for (int k = 0; k < kKeepUnroll; ++k) {
      const int i = i0 + k * per + r;
      to[k] = nullptr;
      const int32_t from = in && i < a.n ? kept[i] : -1;
      if (from < 0 || from == i) continue;
      char* src = nullptr;
      if (from > i && first + from < room) {
        src = place(first + from);
        to[k] = place(first + i);
      }
      if (!src || !to[k]) {
        to[k] = nullptr;
        record_error(err, kDevErrBadId);
        continue;
      }
      v[k] = *reinterpret_cast<const V*>(src);
    }
    cta_sync();
#pragma unroll
    for (int k = 0; k < kKeepUnroll; ++k)
      if (to[k]) *reinterpret_cast<V*>(to[k]) = v[k];
  }
}

__global__ void __launch_bounds__(kKeepThreads)
keep_kernel(const KeepArgs a, int* err) {
  pdl_wait();
  pdl_trigger();
  // the slice: of which tensor, head and bytes
  int x = blockIdx.x, ti = 0;
  while (x >= a.t[ti].slices * a.kv_heads) x -= a.t[ti++].slices * a.kv_heads;
  const KeepTensor& t = a.t[ti];
  const int head = x / t.slices, sl = x - head * t.slices;
  const int byte0 = sl * t.slice, bytes = min(t.slice, t.row - byte0);
  for (int s = blockIdx.y; s < a.S; s += gridDim.y) {
    const int32_t first = a.first ? a.first[s] : 0;
    if (blockIdx.x == 0) {
      // the rows that the list leaves: up to its last entry that is one
      const int32_t* kept = a.kept + (int64_t)s * (a.per_head ? a.kv_heads : 1) * a.n;
      __shared__ int sh_last;
      if (threadIdx.x == 0) sh_last = 0;
      cta_sync();
      int last = 0;
      for (int i = threadIdx.x; i < a.n; i += kKeepThreads)
        if (kept[i] >= 0) last = i + 1;
      last = __reduce_max_sync(0xFFFFFFFFu, last);
      if ((threadIdx.x & 31) == 0) atomicMax(&sh_last, last);
      cta_sync();
      if (threadIdx.x == 0) {
        a.new_lens[s] = first + (first >= 0 ? sh_last : 0);
        if (first < 0) record_error(err, kDevErrBadId);
      }
    }
    if (first < 0) continue;
    switch (t.vec) {
      case 16: move_slice<uint4>(a, t, s, head, byte0, bytes, err); break;
      case 4: move_slice<uint32_t>(a, t, s, head, byte0, bytes, err); break;
      case 2: move_slice<uint16_t>(a, t, s, head, byte0, bytes, err); break;
      default: move_slice<uint8_t>(a, t, s, head, byte0, bytes, err); break;
    }
    cta_sync();
  }
}

// ----------------------------------------------------------------- release
// Pages ceil(new / P) .. ceil(held / P) - 1 of each request go back behind the
// free ones, request after request. As in the page plan, each CTA takes
// kReleaseReqs requests and counts the pages of all earlier ones by itself.
constexpr int kReleaseThreads = 256;
constexpr int kReleaseReqs = 8;

struct Gone {
  int first, count;  // pages of the request's table that go
  bool sane;
};

__device__ __forceinline__ Gone gone_of(const ReleaseArgs& a, int s) {
  const int64_t len = a.lens[s], now = a.new_lens[s];
  int64_t fresh = 0;
  bool sane = true;
  if (a.cu && !(a.granted && a.granted[s] == 0)) {
    fresh = (int64_t)a.cu[s + 1] - a.cu[s];
    sane = fresh >= 0;
  }
  const int64_t held = len + fresh;
  sane = sane && len >= 0 && now >= 0 && now <= held && held <= (int64_t)a.width * a.page;
  Gone g = {0, 0, sane};
  if (sane) {
    g.first = (int)((now + a.page - 1) / a.page);
    g.count = (int)((held + a.page - 1) / a.page) - g.first;
  }
  return g;
}

__global__ void __launch_bounds__(kReleaseThreads)
release_kernel(const ReleaseArgs a, int* err) {
  __shared__ int sh_sum[kReleaseThreads / 32];
  __shared__ int r_at[kReleaseReqs], r_first[kReleaseReqs], r_count[kReleaseReqs];
  pdl_wait();
  pdl_trigger();
  const int tid = threadIdx.x, first = blockIdx.x * kReleaseReqs;
  const int count = min(kReleaseReqs, a.S - first);
  int sum = 0;  // S * width fits 32 bits
  for (int s = tid; s < first; s += kReleaseThreads) sum += gone_of(a, s).count;
  sum = __reduce_add_sync(0xFFFFFFFFu, sum);
  if ((tid & 31) == 0) sh_sum[tid >> 5] = sum;
  cta_sync();
  if (tid == 0) {
    const int F = max(0, min(*a.free_count, a.free_cap));
    int64_t at = F;
    for (int w = 0; w < kReleaseThreads / 32; ++w) at += sh_sum[w];
    for (int i = 0; i < count; ++i) {
      const Gone g = gone_of(a, first + i);
      if (!g.sane) record_error(err, kDevErrBadId);
      // what has no room in the list is not put there
      const int fit = (int)max((int64_t)0, min((int64_t)g.count, a.free_cap - at));
      if (fit < g.count) record_error(err, kDevErrBadId);
      r_at[i] = (int)min(at, (int64_t)a.free_cap);
      r_first[i] = g.first;
      r_count[i] = fit;
      at += g.count;
    }
    if (first + count == a.S) *a.free_left = (int32_t)min(at, (int64_t)a.free_cap);
  }
  cta_sync();
  for (int i = tid >> 5; i < count; i += kReleaseThreads / 32)
    for (int j = tid & 31; j < r_count[i]; j += 32)
      a.free_pages[r_at[i] + j] = a.table[(int64_t)(first + i) * a.width + r_first[i] + j];
}

}  // namespace

cudaError_t launch_cache_select(const SelectArgs& a, int* err, cudaStream_t s) {
  // keys that do not fit in shared memory are read again in each pass
  constexpr int kMost = 48 * 1024;
  const int64_t room = (int64_t)a.width * a.page;
  const int staged = (int)(room < kMost ? room : kMost);
  static int smem_set[64] = {0};
  const size_t smem = (size_t)staged * 4;
  cudaError_t e = ensure_dynamic_smem(select_kernel, smem, smem_set);
  if (e != cudaSuccess) return e;
  return launch_kernel(true, select_kernel, dim3(a.kv_heads, a.S < 65535 ? a.S : 65535),
                       dim3(kSelThreads), smem, s, a, staged, err);
}

cudaError_t launch_cache_keep(KeepArgs a, int* err, cudaStream_t s) {
  int64_t slices = 0;
  for (int i = 0; i < a.count; ++i) {
    KeepTensor& t = a.t[i];
    const uintptr_t bits = reinterpret_cast<uintptr_t>(t.base) | (uintptr_t)t.st.page |
                           (uintptr_t)t.st.token | (uintptr_t)t.st.head | (uintptr_t)t.row;
    t.vec = (bits & 15) == 0 ? 16 : (bits & 3) == 0 ? 4 : (bits & 1) == 0 ? 2 : 1;
    // long lists are moved in narrow slices, so that a request's rows are many CTAs'
    // work; short ones in whole rows, of no more vectors than a CTA has threads
    t.slice = a.n > 64 ? 64 : t.vec * kKeepThreads;
    t.slices = (t.row + t.slice - 1) / t.slice;
    slices += (int64_t)t.slices * a.kv_heads;
  }
  return launch_kernel(true, keep_kernel, dim3((unsigned)slices, a.S < 65535 ? a.S : 65535),
                       dim3(kKeepThreads), 0, s, a, err);
}

cudaError_t launch_page_release(const ReleaseArgs& a, int* err, cudaStream_t s) {
  return launch_kernel(true, release_kernel, dim3((a.S + kReleaseReqs - 1) / kReleaseReqs),
                       dim3(kReleaseThreads), 0, s, a, err);
}

}  // namespace lmhead
