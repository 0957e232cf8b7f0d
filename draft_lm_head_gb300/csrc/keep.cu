// Which tokens of a paged cache stay, their rows moved together, and the pages
// behind them given back.
#include <cuda_runtime.h>
#include <stdint.h>

#include "common.cuh"
#include "kernels.h"

namespace lmhead {
namespace {

// Page and place in it of a position: pages of a power of two by shift, others by
// division.
__device__ __forceinline__ void split_pos(uint32_t pos, int page, int shift, int& pg, int& off) {
  if (shift >= 0) {
    pg = (int)(pos >> shift);
    off = (int)(pos & ((1u << shift) - 1u));
  } else {
    pg = (int)(pos / (uint32_t)page);
    off = (int)(pos - (uint32_t)pg * (uint32_t)page);
  }
}

// ------------------------------------------------------------------ select
// Of a request's L tokens and one K/V head the first `sinks`, the last `recent`
// and, of those between, the ones with the largest weights (ties: the lower
// position) up to `budget` in all, in ascending order.
// One CTA a request and head: the weights' order-preserving keys go to shared
// memory and are counted by digits from the top (11, 11 and 10 bits, while the digit
// of the last one to stay holds others that do not) in four copies, as weights crowd
// in few exponents; a last pass writes the positions that pass, each warp those of
// a run of its own behind the counts of the runs before. Where a page's weights of a head
// lie side by side they are read four at a time, page and place looked up once for them. Bound by
// latency for one list (4096 tokens x 8 heads: 11 us alone, passes over shared memory and
// the waits between them), by instructions for long ones (16 lists of up to 32768 x 8 heads:
// 38 us one by one, 22 by fours; eight copies of the counts 4 us more; keys in registers
// and a search bit by bit 44).
constexpr int kSelThreads = 1024;
constexpr int kSelWarps = kSelThreads / 32;
constexpr int kSelLoads = 8, kSelQuads = 4;
constexpr int kBins = 2048, kCopies = 4, kCopy = kBins + 8;  // (copies begin in other banks)
constexpr int kMostStaged = 48 * 1024 - kCopy * kCopies;  // keys; those behind are read again

__device__ __forceinline__ uint32_t weight_key(float w) {
  return w != w ? 0u : float_key(w);  // a NaN comes last
}

__global__ void __launch_bounds__(kSelThreads)
select_kernel(const SelectArgs a, int shift, int staged, int quads, int* err) {
  extern __shared__ __align__(16) int hist[];  // kCopies counts of each bin, then the keys
  uint32_t* keys = reinterpret_cast<uint32_t*>(hist + kCopy * kCopies);
  int* mine = hist + (threadIdx.x & (kCopies - 1)) * kCopy;
  __shared__ int more_w[kSelWarps], same_w[kSelWarps];
  __shared__ int sh_need, sh_digit, sh_count;
  pdl_wait();
  pdl_trigger();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int head = blockIdx.x;
  for (int s = blockIdx.y; s < a.S; s += gridDim.y) {
    int32_t* out = a.kept + ((int64_t)s * a.kv_heads + head) * a.budget;
    int L = a.lens[s];
    if (L < 0 || L > min((int64_t)a.width * a.page, (int64_t)kMaxTokens)) {
      if (tid == 0) record_error(err, kDevErrBadId);
      L = 0;
    }
    if (L <= a.budget) {  // all of them
      for (int i = tid; i < a.budget; i += kSelThreads) out[i] = i < L ? i : -1;
      continue;
    }
    const int lo = min(a.sinks, L), hi = max(lo, L - a.recent);  // positions that are chosen from
    int need = a.budget - lo - (L - hi);
    for (int i = tid; i < lo; i += kSelThreads) out[i] = i;
    for (int i = tid; i < L - hi; i += kSelThreads) out[a.budget - (L - hi) + i] = hi + i;
    if (need == 0) continue;
    const int32_t* row = a.table + (int64_t)s * a.width;
    const char* weights = static_cast<const char*>(a.weights) + head * a.ws.head;
    bool bad = false;
    auto page_at = [&](int j, int& off) -> int32_t {  // or -1
      int pg;
      split_pos((uint32_t)j, a.page, shift, pg, off);
      const int32_t id = row[pg];
      return id < 0 || id >= a.pages ? -1 : id;
    };
    auto key_at = [&](int32_t id, int off) -> uint32_t {
      if (id < 0) return 0u;
      return weight_key(*reinterpret_cast<const float*>(weights + id * a.ws.page + off * a.ws.token));
    };
    auto key_of = [&](int j) -> uint32_t {
      int off;
      const int32_t id = page_at(j, off);
      return key_at(id, off);
    };
    // keys by their place behind `base`; those from `begin` to `end` are chosen from
    const int base = quads ? lo & ~3 : lo, begin = lo - base, end = hi - base;
    const int kept_keys = min(staged, end);
    auto key = [&](int i) { return i < kept_keys ? keys[i] : key_of(base + i); };
    auto each = [&](auto f) {
      if (end <= kept_keys) {
#pragma unroll 4
        for (int i = 4 * tid; i < end; i += 4 * kSelThreads) {
          const uint4 k = *reinterpret_cast<const uint4*>(keys + i);
          if (i >= begin) f(k.x);
          if (i + 1 >= begin && i + 1 < end) f(k.y);
          if (i + 2 >= begin && i + 2 < end) f(k.z);
          if (i + 3 >= begin && i + 3 < end) f(k.w);
        }
      } else {
        for (int i = begin + tid; i < end; i += kSelThreads) f(key(i));
      }
    };
    uint32_t prefix = 0, mask = 0;
    int top = 21, bits = 11;
    for (;;) {
      for (int i = tid; i < kCopy * kCopies / 4; i += kSelThreads)
        reinterpret_cast<int4*>(hist)[i] = make_int4(0, 0, 0, 0);
      cta_sync();
      if (mask == 0) {  // the first time the keys are read, several of a thread under way together
        if (quads) {
          for (int i0 = 4 * tid; i0 < end; i0 += 4 * kSelQuads * kSelThreads) {
            int32_t id[kSelQuads];
            int off[kSelQuads];
            float4 w[kSelQuads];
#pragma unroll
            for (int n = 0; n < kSelQuads; ++n) {
              const int i = i0 + 4 * n * kSelThreads;
              id[n] = i < end ? page_at(base + i, off[n]) : -1;
              bad |= i < end && id[n] < 0;
            }
#pragma unroll
            for (int n = 0; n < kSelQuads; ++n)
              if (id[n] >= 0) w[n] = *reinterpret_cast<const float4*>(weights + id[n] * a.ws.page + off[n] * 4ll);
#pragma unroll
            for (int n = 0; n < kSelQuads; ++n) {
              const int i = i0 + 4 * n * kSelThreads;
              if (i >= end) break;
              uint4 k = {0u, 0u, 0u, 0u};
              if (id[n] >= 0) k = {weight_key(w[n].x), weight_key(w[n].y), weight_key(w[n].z), weight_key(w[n].w)};
              if (i < kept_keys) *reinterpret_cast<uint4*>(keys + i) = k;
              if (i >= begin) atomicAdd(&mine[k.x >> top], 1);
              if (i + 1 >= begin && i + 1 < end) atomicAdd(&mine[k.y >> top], 1);
              if (i + 2 >= begin && i + 2 < end) atomicAdd(&mine[k.z >> top], 1);
              if (i + 3 >= begin && i + 3 < end) atomicAdd(&mine[k.w >> top], 1);
            }
          }
        } else {
          for (int i0 = tid; i0 < end; i0 += kSelLoads * kSelThreads) {
            int32_t id[kSelLoads];
            int off[kSelLoads];
            uint32_t k[kSelLoads];
#pragma unroll
            for (int n = 0; n < kSelLoads; ++n) {
              id[n] = -1;
              if (i0 + n * kSelThreads < end) {
                id[n] = page_at(lo + i0 + n * kSelThreads, off[n]);
                bad |= id[n] < 0;
              }
            }
#pragma unroll
            for (int n = 0; n < kSelLoads; ++n) k[n] = key_at(id[n], off[n]);
#pragma unroll
            for (int n = 0; n < kSelLoads; ++n) {
              const int i = i0 + n * kSelThreads;
              if (i >= end) break;
              if (i < kept_keys) keys[i] = k[n];
              atomicAdd(&mine[k[n] >> top], 1);
            }
          }
        }
        if (bad) record_error(err, kDevErrBadId);
      } else {
        each([&](uint32_t k) {
          if ((k & mask) == prefix) atomicAdd(&mine[(k >> top) & ((1u << bits) - 1u)], 1);
        });
      }
      cta_sync();
      // the digit in which the need-th largest lies: counts from the top, two bins a thread
      constexpr int kPer = kBins / kSelThreads;
      int c[kPer], sum = 0;
#pragma unroll
      for (int i = 0; i < kPer; ++i) {
        const int* h = hist + kBins - 1 - (tid * kPer + i);
        c[i] = (h[0] + h[kCopy]) + (h[2 * kCopy] + h[3 * kCopy]);
        sum += c[i];
      }
      int incl = sum;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int p = __shfl_up_sync(0xFFFFFFFFu, incl, o);
        if (lane >= o) incl += p;
      }
      if (lane == 31) more_w[warp] = incl;
      cta_sync();
      int at = incl - sum;
      {
        const int w = more_w[lane];
        int before = w;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const int p = __shfl_up_sync(0xFFFFFFFFu, before, o);
          if (lane >= o) before += p;
        }
        at += __shfl_sync(0xFFFFFFFFu, before - w, warp);
      }
#pragma unroll
      for (int i = 0; i < kPer; ++i) {
        if (at < need && need <= at + c[i]) {
          sh_digit = kBins - 1 - (tid * kPer + i);
          sh_need = need - at;
          sh_count = c[i];
        }
        at += c[i];
      }
      cta_sync();
      prefix |= (uint32_t)sh_digit << top;
      mask |= ((1u << bits) - 1u) << top;
      need = sh_need;
      if (sh_count == need || top == 0) break;  // all of the digit's stay, or they are equal
      bits = top >= 11 ? min(11, top) : top;
      top -= bits;
    }
    // keys above prefix (in the digits looked at) stay, and the first `need` equal to it
    const int run = ((end + kSelWarps - 1) / kSelWarps + 31) / 32 * 32;
    const int r1 = min(end, (warp + 1) * run), r0 = max(begin, min(r1, warp * run));
    int more = 0, same = 0;
    auto count = [&](auto key) {
#pragma unroll 8
      for (int i = r0 + lane; i < r1; i += 32) {
        const uint32_t k = key(i) & mask;
        more += k > prefix;
        same += k == prefix;
      }
    };
    if (r1 <= kept_keys)
      count([&](int i) { return keys[i]; });
    else
      count(key);
    more = __reduce_add_sync(0xFFFFFFFFu, more);
    same = __reduce_add_sync(0xFFFFFFFFu, same);
    cta_sync();
    if (lane == 0) more_w[warp] = more, same_w[warp] = same;
    cta_sync();
    int before = __reduce_add_sync(0xFFFFFFFFu, lane < warp ? more_w[lane] : 0);
    int equal = __reduce_add_sync(0xFFFFFFFFu, lane < warp ? same_w[lane] : 0);
    const uint32_t below = (1u << lane) - 1u;
    constexpr int kAhead = 4;  // chunks of 32 looked at together
    int32_t* to = out + lo + before + min(equal, need);
    // of a run whose equal keys all stay, or none, what passes is one comparison
    auto place = [&](auto key, uint32_t least) {
      for (int i0 = r0; i0 < r1; i0 += 32 * kAhead) {
        uint32_t m[kAhead];
        bool in[kAhead];
#pragma unroll
        for (int n = 0; n < kAhead; ++n) {
          const int i = i0 + 32 * n + lane;
          in[n] = i < r1 && (key(i) & mask) >= least;
          m[n] = __ballot_sync(0xFFFFFFFFu, in[n]);
        }
#pragma unroll
        for (int n = 0; n < kAhead; ++n) {
          if (in[n]) to[__popc(m[n] & below)] = base + i0 + 32 * n + lane;
          to += __popc(m[n]);
        }
      }
    };
    const bool all = equal + same <= need, none = equal >= need;
    if (all || (none && prefix + ~mask != 0xFFFFFFFFu)) {
      const uint32_t least = all ? prefix : (prefix | ~mask) + 1;
      if (r1 <= kept_keys)
        place([&](int i) { return keys[i]; }, least);
      else
        place(key, least);
    } else {
      for (int i0 = r0; i0 < r1; i0 += 32) {
        const int i = i0 + lane;
        const uint32_t k = i < r1 ? key(i) & mask : 0u;
        const bool is_more = i < r1 && k > prefix, is_same = i < r1 && k == prefix;
        const uint32_t m = __ballot_sync(0xFFFFFFFFu, is_more), e = __ballot_sync(0xFFFFFFFFu, is_same);
        const int eq = equal + __popc(e & below);
        if (is_more || (is_same && eq < need)) out[lo + before + __popc(m & below) + min(eq, need)] = base + i;
        before += __popc(m);
        equal += __popc(e);
      }
    }
    cta_sync();
  }
}

// -------------------------------------------------------------------- keep
// Row first + i of a request becomes what row first + kept[i] was, kept[i] >= i.
// A row is read from its own place or from one behind it, so rows moved in
// ascending order are read before they are overwritten. A CTA moves one slice of
// the rows' bytes of one tensor and head, for all of the request's list, chunk after
// chunk: where the rows lie is worked out once for each (a thread a row), then their
// vectors are read into registers, all threads waited for, and written; what is read
// later lies behind all that has been written. CTAs share no bytes.
// Bound by memory: 16 prompts' rows, 4097 of up to 32768 a head (540 MB read and written),
// 96 us, 5.6 TB/s, rows of 256 bytes in no order; by latency for short lists. More in flight
// does not help: an eviction of the 16 prompts took 128 us as it is (131 since the pages
// given back are looked over), 136 to 156 with rings of
// 12 to 48 KB in shared memory written while the next rows come, 131 and 140 with three
// and two rows a thread, 131 with loads that do not stay in caches; and, of 145 then, 149
// to 199 with slices of 64 and 128 bytes, 8 rows a thread, 3 or 6 CTAs an SM.
constexpr int kKeepThreads = 256;
constexpr int kKeepUnroll = 4;
constexpr int kKeepChunk = 1024;  // rows

struct KeepRows {
  int64_t from[kKeepChunk], to[kKeepChunk];  // byte offsets; from < 0: not moved
};

template <typename V>
__device__ __forceinline__ void move_rows(const KeepRows& rows, int count, char* base, int bytes) {
  const int lanes = bytes / (int)sizeof(V);  // of a row; no more than the CTA has threads
  const int per = kKeepThreads / lanes;      // rows a pass
  const int c = threadIdx.x % lanes, r = threadIdx.x / lanes;
  base += c * sizeof(V);
  for (int i0 = 0; i0 < count; i0 += per * kKeepUnroll) {
    V v[kKeepUnroll];
    uint32_t some = 0;
#pragma unroll
    for (int k = 0; k < kKeepUnroll; ++k) {
      const int i = i0 + k * per + r;
      if (r < per && i < count && rows.from[i] >= 0) {
        v[k] = *reinterpret_cast<const V*>(base + rows.from[i]);
        some |= 1u << k;
      }
    }
    cta_sync();
#pragma unroll
    for (int k = 0; k < kKeepUnroll; ++k)
      if (some >> k & 1) *reinterpret_cast<V*>(base + rows.to[i0 + k * per + r]) = v[k];
  }
}

__global__ void __launch_bounds__(kKeepThreads, 5)
keep_kernel(const KeepArgs a, int shift, int* err) {
  __shared__ KeepRows rows;
  __shared__ int sh_last, sh_first;
  pdl_wait();
  pdl_trigger();
  // the slice: of which tensor, head and bytes
  const int tid = threadIdx.x;
  int x = blockIdx.x, ti = 0;
  while (x >= a.t[ti].slices * a.kv_heads) x -= a.t[ti++].slices * a.kv_heads;
  const KeepTensor& t = a.t[ti];
  const int head = x / t.slices, sl = x - head * t.slices;
  const int byte0 = sl * t.slice, bytes = min(t.slice, t.row - byte0);
  char* base = static_cast<char*>(t.base) + head * t.st.head + byte0;
  const int64_t room = (int64_t)a.width * a.page;
  for (int s = blockIdx.y; s < a.S; s += gridDim.y) {
    const int32_t first = a.first ? a.first[s] : 0;
    const int32_t* table = a.table + (int64_t)s * a.width;
    const int32_t* kept = a.kept + ((int64_t)s * (a.per_head ? a.kv_heads : 1) + (a.per_head ? head : 0)) * a.n;
    auto place = [&](int64_t pos) -> int64_t {
      int pg, off;
      split_pos((uint32_t)pos, a.page, shift, pg, off);
      const int32_t id = table[pg];
      return id < 0 || id >= a.pages ? -1 : id * t.st.page + off * t.st.token;
    };
    // the first row that moves and the last one of the list
    if (tid == 0) sh_last = 0, sh_first = a.n;
    cta_sync();
    int last = 0, from0 = a.n;
#pragma unroll 8
    for (int i = tid; i < a.n; i += kKeepThreads) {
      const int32_t x = kept[i];
      if (x >= 0) {
        last = i + 1;
        if (x != i) from0 = min(from0, i);
      }
    }
    last = __reduce_max_sync(0xFFFFFFFFu, last);
    from0 = __reduce_min_sync(0xFFFFFFFFu, from0);
    if ((tid & 31) == 0) {
      atomicMax(&sh_last, last);
      atomicMin(&sh_first, from0);
    }
    cta_sync();
    last = sh_last;
    from0 = sh_first;
    if (tid == 0) {
      const int64_t now = first >= 0 ? (int64_t)first + last : first;
      if (blockIdx.x == 0) a.new_lens[s] = (int32_t)min(now, (int64_t)INT32_MAX);
      // (entries at their own place are not looked at below: the last is past the table here)
      if (first < 0 || (last > 0 && now > room)) record_error(err, kDevErrBadId);
    }
    for (int i0 = from0; i0 < last; i0 += kKeepChunk) {
      const int count = min(kKeepChunk, last - i0);
      cta_sync();  // the chunk before has been moved
#pragma unroll
      for (int k = 0; k < kKeepChunk / kKeepThreads; ++k) {
        const int i = i0 + k * kKeepThreads + tid;
        const int32_t from = i < last ? kept[i] : -1;
        int64_t src = -1, dst = -1;
        if (from >= 0 && from != i && first >= 0) {
          if (from > i && (int64_t)first + from < room) {
            src = place((int64_t)first + from);
            dst = place((int64_t)first + i);
          }
          if (src < 0 || dst < 0) {
            src = -1;
            record_error(err, kDevErrBadId);
          }
        }
        rows.from[i - i0] = src;
        rows.to[i - i0] = dst;
      }
      cta_sync();
      switch (t.vec) {
        case 16: move_rows<uint4>(rows, count, base, bytes); break;
        case 4: move_rows<uint32_t>(rows, count, base, bytes); break;
        case 2: move_rows<uint16_t>(rows, count, base, bytes); break;
        default: move_rows<uint8_t>(rows, count, base, bytes); break;
      }
    }
    cta_sync();
  }
}

// ----------------------------------------------------------------- release
// Pages ceil(new / P) .. ceil(held / P) - 1 of each request go back behind the
// free ones, request after request. As in the page plan, each CTA takes a few
// requests and counts the pages of all earlier ones by itself, which means to read
// them: a request counts only if all of its entries are pages. Bound by latency (device
// time, graphs replayed): one request 2.1 us (1.7 without the look), 64 of a page each 2.6,
// 1024 3.8, 16 of 1000 to 1800 pages 4.6 (3.6 without); 16384 of a page each 40.
constexpr int kReleaseThreads = 512;
constexpr int kReleaseReqs = 8, kReleaseMost = 32;  // of a CTA: few requests in all, many
constexpr int kReleaseUnroll = 4;  // pages of a thread under way together
constexpr int kReleaseFew = 16;    // pages of a request that a lane looks over by itself

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

// The same with the pages looked over: a request with an entry that is no page gives none
// back, so that what is in the free list can be handed out. Whole warps come here, a
// request each lane (s < 0: none); long lists are read by the warp, 16 bytes a lane.
__device__ __forceinline__ Gone gone_checked(const ReleaseArgs& a, int s, int lane) {
  Gone g = {0, 0, true};
  const int32_t* pages = a.table;
  if (s >= 0) {
    g = gone_of(a, s);
    pages += (int64_t)s * a.width + g.first;
  }
  int bits = 0;
  if (g.count <= kReleaseFew) {
#pragma unroll 4
    for (int j = 0; j < g.count; ++j) bits |= pages[j];
  }
  for (uint32_t many = __ballot_sync(0xFFFFFFFFu, g.count > kReleaseFew); many; many &= many - 1) {
    const int l = __ffs((int)many) - 1, n = __shfl_sync(0xFFFFFFFFu, g.count, l);
    const int32_t* p = reinterpret_cast<const int32_t*>(
        __shfl_sync(0xFFFFFFFFu, reinterpret_cast<unsigned long long>(pages), l));
    const int lead = min(n, (int)(-(reinterpret_cast<uintptr_t>(p) >> 2) & 3));
    const int quads = (n - lead) / 4, tail = lead + 4 * quads;
    const int4* q = reinterpret_cast<const int4*>(p + lead);
    int some = 0;
    if (lane < lead) some |= p[lane];
    if (tail + lane < n) some |= p[tail + lane];
#pragma unroll 4
    for (int i = lane; i < quads; i += 32) {
      const int4 v = q[i];
      some |= v.x | v.y | v.z | v.w;
    }
    some = __reduce_or_sync(0xFFFFFFFFu, (uint32_t)some);
    if (lane == l) bits = some;
  }
  if (bits < 0) {
    g.count = 0;
    g.sane = false;
  }
  return g;
}

__global__ void __launch_bounds__(kReleaseThreads)
release_kernel(const ReleaseArgs a, int reqs, int* err) {
  constexpr int kWarps = kReleaseThreads / 32;
  __shared__ int sh_sum[kWarps], r_count[kReleaseMost];
  __shared__ int r_end[kReleaseMost + 1], r_first[kReleaseMost];
  __shared__ int64_t sh_at;
  pdl_wait();
  pdl_trigger();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, first = blockIdx.x * reqs;
  const int count = min(reqs, a.S - first);
  // all requests up to the CTA's last; where each thread has one, neighbours are in
  // different warps, which share out long lists
  const bool spread = first + count <= kReleaseThreads;
  int sum = 0;  // S * width fits 32 bits
  for (int s0 = 0; s0 < first + count; s0 += kReleaseThreads) {
    const int s = spread ? lane * kWarps + warp : s0 + tid, i = s - first;
    const Gone g = gone_checked(a, i < count ? s : -1, lane);
    if (i < 0) {
      sum += g.count;
    } else if (i < count) {
      r_count[i] = g.count;
      r_first[i] = g.first;
      if (!g.sane && blockIdx.y == 0) record_error(err, kDevErrBadId);
    }
  }
  sum = __reduce_add_sync(0xFFFFFFFFu, sum);
  if (lane == 0) sh_sum[warp] = sum;
  cta_sync();
  if (warp == 0) {
    // where the pages of the CTA's requests, a lane each, lie among the CTA's
    int incl = lane < count ? r_count[lane] : 0;
#pragma unroll
    for (int o = 1; o < kReleaseMost; o <<= 1) {
      const int p = __shfl_up_sync(0xFFFFFFFFu, incl, o);
      if (lane >= o) incl += p;
    }
    r_end[lane + 1] = incl;
    if (lane == 0) r_end[0] = 0;
  }
  cta_sync();
  if (tid == 0) {
    int64_t at = max(0, min(*a.free_count, a.free_cap));
    for (int w = 0; w < kWarps; ++w) at += sh_sum[w];
    sh_at = at;
    const int64_t end = at + r_end[count];
    // what has no room in the list is not put there
    if (blockIdx.y == 0 && end > a.free_cap) record_error(err, kDevErrBadId);
    if (blockIdx.y == 0 && first + count == a.S) *a.free_left = (int32_t)min(end, (int64_t)a.free_cap);
  }
  cta_sync();
  const int64_t at = sh_at;
  const int total = (int)max((int64_t)0, min((int64_t)r_end[count], a.free_cap - at));
  const int stride = gridDim.y * kReleaseThreads;
  for (int64_t e0 = blockIdx.y * kReleaseThreads + tid; e0 < total; e0 += kReleaseUnroll * stride) {
    int32_t id[kReleaseUnroll];
#pragma unroll
    for (int k = 0; k < kReleaseUnroll; ++k) {
      const int64_t e = e0 + k * stride;
      if (e >= total) break;
      int i = 0;
      while (e >= r_end[i + 1]) ++i;
      id[k] = a.table[(int64_t)(first + i) * a.width + r_first[i] + (e - r_end[i])];
    }
#pragma unroll
    for (int k = 0; k < kReleaseUnroll; ++k) {
      const int64_t e = e0 + k * stride;
      if (e < total) a.free_pages[at + e] = id[k];
    }
  }
}

}  // namespace

namespace {

inline int shift_of(int page) {  // log2 of a power of two, else -1
  int s = 0;
  while ((1 << s) < page) ++s;
  return (1 << s) == page ? s : -1;
}

}  // namespace

cudaError_t launch_cache_select(const SelectArgs& a, int* err, cudaStream_t s) {
  const int64_t room = (int64_t)a.width * a.page;
  const int staged = (int)(room < kMostStaged ? (room + 3) / 4 * 4 : kMostStaged);
  const uintptr_t bits = reinterpret_cast<uintptr_t>(a.weights) | (uintptr_t)a.ws.page | (uintptr_t)a.ws.head;
  const int quads = a.ws.token == 4 && a.page % 4 == 0 && (bits & 15) == 0;
  static int smem_set[64] = {0};
  const size_t smem = (size_t)(kCopy * kCopies + staged) * 4;
  cudaError_t e = ensure_dynamic_smem(select_kernel, smem, smem_set);
  if (e != cudaSuccess) return e;
  return launch_kernel(true, select_kernel, dim3(a.kv_heads, a.S < 65535 ? a.S : 65535),
                       dim3(kSelThreads), smem, s, a, shift_of(a.page), staged, quads, err);
}

cudaError_t launch_cache_keep(KeepArgs a, int* err, cudaStream_t s) {
  // Short lists are moved in whole rows, long ones in slices of 256 bytes, or fewer
  // down to 64 where there are too few of them to fill the GPU, to 32 where they do not
  // reach every SM (2048 of 4096 rows of one request, 8 heads of 256 bytes: with them the
  // eviction takes 23 us in place of 25, with 16 bytes 26).
  int slice = a.n > 64 ? 256 : kKeepThreads * 16;
  const int64_t want = 4ll * (sm_count() > 0 ? sm_count() : 1);
  auto slices_of = [&](int width) {
    int64_t n = 0;
    for (int i = 0; i < a.count; ++i) n += (a.t[i].row + width - 1) / width;
    return n * a.kv_heads;
  };
  while (a.n > 64 && slice > 64 && slices_of(slice) * a.S < want) slice /= 2;
  while (a.n > 64 && slice > 32 && slices_of(slice) * a.S < want / 4) slice /= 2;
  int64_t slices = 0;
  for (int i = 0; i < a.count; ++i) {
    KeepTensor& t = a.t[i];
    const uintptr_t bits = reinterpret_cast<uintptr_t>(t.base) | (uintptr_t)t.st.page |
                           (uintptr_t)t.st.token | (uintptr_t)t.st.head | (uintptr_t)t.row;
    t.vec = (bits & 15) == 0 ? 16 : (bits & 3) == 0 ? 4 : (bits & 1) == 0 ? 2 : 1;
    // no more vectors than a CTA has threads
    t.slice = slice < t.vec * kKeepThreads ? slice : t.vec * kKeepThreads;
    t.slices = (t.row + t.slice - 1) / t.slice;
    slices += (int64_t)t.slices * a.kv_heads;
  }
  if (slices > INT32_MAX) return cudaErrorInvalidValue;
  return launch_kernel(true, keep_kernel, dim3((unsigned)slices, a.S < 65535 ? a.S : 65535),
                       dim3(kKeepThreads), 0, s, a, shift_of(a.page), err);
}

cudaError_t launch_page_release(const ReleaseArgs& a, int* err, cudaStream_t s) {
  const int reqs = a.S <= 1024 ? kReleaseReqs : kReleaseMost;
  // several CTAs for the pages of the same requests where tables are wide
  int64_t y = (int64_t)a.width * reqs / (kReleaseThreads * kReleaseUnroll);
  y = y < 1 ? 1 : y > 64 ? 64 : y;
  return launch_kernel(true, release_kernel, dim3((a.S + reqs - 1) / reqs, (unsigned)y),
                       dim3(kReleaseThreads), 0, s, a, reqs, err);
}

}  // namespace lmhead
