// Verification of a draft tree: which path of it the target accepts, and the
// token behind that path ("Speculative decoding and EAGLE", the exactness rule,
// with several proposals a place tried in turn).
//
// A request's nodes are walked in index order; a node is tried when its parent is
// the node that the walk stands on. What is left of the target's probabilities
// there are weights w of mass Z, at first p itself and 1.
//   Children that are given (the drafter's most likely ones): x is accepted if
//     r Z < w(x), else w(x) = 0 and Z falls by what it was.
//   Children drawn from q without replacement: with g = q / Q over what has not been
//     drawn yet, x is accepted if r Z g(x) < w(x), else w becomes (w - Z g)+, Z falls
//     by sum min(w, Z g), and g(x) = 0. q is nothing outside the candidates, so only
//     they change: the vocabulary is not read before the last token.
// Then one token is drawn from w by inverse CDF. Either way the tokens that come
// out are distributed as the target's.
// Weights are fp32 (w - fl(fl(Z / Q) g) is rounded once each); masses, running sums and
// what is compared are pairs of fp32 numbers, some 48 bits. (This GPU adds two fp64
// numbers a cycle and SM, one after the other in some hundred cycles: with fp64 in their
// place a draw took 12700 cycles in place of 3400, and sums made by every thread two
// thirds of the time.)
//
// One cluster of CTAs a request. Its first CTA takes the walk: the candidates of the
// node it stands on lie in shared memory, a rejection changes them all and sums up
// what was taken. Then each CTA takes its share of the last node's row of p, from
// memory to shared memory, where the changed weights replace what was read; the sums
// meet in distributed shared memory and the CTA that has the draw finds its place.
// Bound by latency: of dependent reads, one row of candidates a node, then the row of
// p. Measured (device time, graphs replayed; with the launches that keep the path's rows
// and give pages back): one tree of 10 given nodes over 128256 entries 19 us; 8 of 10
// drawn nodes, 1572 candidates a place, over 201088 38 us; 64 of 60 over 128256 86 us, where
// the longest walk of the batch bounds it (0.4 instructions a cycle, 8 % of the bandwidth).
#include "common.cuh"
#include "kernels.h"
#include "tc_util.cuh"

namespace lmhead {
namespace {

constexpr int kThreads = 512;
constexpr int kWarps = kThreads / 32;
constexpr int kMaxCluster = 8;
constexpr int kNodes = 64;      // of a request
constexpr int kLoads = 4;       // of a thread under way together
// Entries of p that a warp has in shared memory at a time: fewer where two CTAs are to
// share an SM.
constexpr int kMaxRun = 2048, kMaxRunShared = 1024;

// What is in shared memory: the candidates, then `chunk` entries of p (in their
// place, while the walk lasts, a table of 2^slot_bits keys and places).
struct Layout {
  int cluster;
  int run, chunk;  // a warp's entries (a multiple of 32), a CTA's
  int slot_bits, cands;
  size_t bytes;
};

inline Layout layout_of(int64_t n, int K, int S) {
  Layout l;
  // no more CTAs than the GPU holds at once, two an SM
  l.cluster = kMaxCluster;
  while (l.cluster > 2 && (int64_t)l.cluster * S > 2 * (sm_count() > 0 ? sm_count() : 1)) l.cluster /= 2;
  const int64_t per = ((n + l.cluster - 1) / l.cluster + 3) / 4 * 4;
  const int64_t run = ((per + kWarps - 1) / kWarps + 31) / 32 * 32;
  const int most = (int64_t)l.cluster * S > (sm_count() > 0 ? sm_count() : 1) ? kMaxRunShared : kMaxRun;
  l.run = (int)(run < most ? run : most);
  l.chunk = l.run * kWarps;
  l.cands = (K + 3) / 4 * 4;
  l.slot_bits = 6;
  while ((1 << l.slot_bits) < 2 * K) ++l.slot_bits;  // half empty at least
  const size_t row = (size_t)l.chunk * 4, table = K > 0 ? (size_t)8 << l.slot_bits : 0;
  l.bytes = (row > table ? row : table) + (size_t)l.cands * 12;
  return l;
}

__device__ __forceinline__ float weight_of(float p) { return p > 0.f ? p : 0.f; }  // NaN: nothing

__device__ __forceinline__ float2 ld_cluster_f32x2(uint32_t addr) {
  float2 v;
  asm volatile("ld.shared::cluster.v2.f32 {%0, %1}, [%2];" : "=f"(v.x), "=f"(v.y) : "r"(addr) : "memory");
  return v;
}
__device__ __forceinline__ int ld_cluster_s32(uint32_t addr) {
  int v;
  asm volatile("ld.shared::cluster.s32 %0, [%1];" : "=r"(v) : "r"(addr) : "memory");
  return v;
}
// What p points to in CTA 0 of the cluster.
__device__ __forceinline__ int of_first(const int* p) {
  return ld_cluster_s32(tc::map_to_rank(tc::smem_addr(p), 0));
}

// ---- a sum of two fp32 numbers, the second below half a step of the first
struct alignas(8) Pair {
  float hi, lo;
};
__device__ __forceinline__ Pair joined(float hi, float lo) {  // |hi| >= |lo|
  const float s = __fadd_rn(hi, lo);
  return {s, __fsub_rn(lo, __fsub_rn(s, hi))};
}
__device__ __forceinline__ Pair add(Pair a, Pair b) {
  const float s = __fadd_rn(a.hi, b.hi), t = __fsub_rn(s, a.hi);
  const float e = __fadd_rn(__fsub_rn(a.hi, __fsub_rn(s, t)), __fsub_rn(b.hi, t));
  return joined(s, __fadd_rn(e, __fadd_rn(a.lo, b.lo)));
}
__device__ __forceinline__ Pair minus(Pair a) { return {-a.hi, -a.lo}; }
__device__ __forceinline__ Pair times(Pair a, float b) {
  const float p = __fmul_rn(a.hi, b);
  return joined(p, __fmaf_rn(a.lo, b, __fmaf_rn(a.hi, b, -p)));
}
__device__ __forceinline__ bool less(Pair a, Pair b) { return a.hi < b.hi || (a.hi == b.hi && a.lo < b.lo); }
// a / b rounded to fp32, b > 0.
__device__ __forceinline__ float ratio(Pair a, Pair b) {
  const float q = __fdiv_rn(a.hi, b.hi);
  const Pair rest = add(a, minus(times(b, q)));
  return __fadd_rn(q, __fdiv_rn(rest.hi, b.hi));
}
// (hi, lo) += x, not joined: lo gathers what hi rounds off.
__device__ __forceinline__ void add_exact(Pair& a, float x) {
  const float s = __fadd_rn(a.hi, x), b = __fsub_rn(s, a.hi);
  a.lo = __fadd_rn(a.lo, __fadd_rn(__fsub_rn(a.hi, __fsub_rn(s, b)), __fsub_rn(x, b)));
  a.hi = s;
}
__device__ __forceinline__ Pair shuffled(Pair a, int lane) {
  return {__shfl_sync(0xFFFFFFFFu, a.hi, lane), __shfl_sync(0xFFFFFFFFu, a.lo, lane)};
}
// The sum of a warp's pairs, in every lane (of the first `lanes` of them, a power of two).
template <int LANES = 32> __device__ __forceinline__ Pair warp_sum_exact(Pair a) {
#pragma unroll
  for (int o = LANES / 2; o > 0; o >>= 1)
    a = add(a, {__shfl_xor_sync(0xFFFFFFFFu, a.hi, o), __shfl_xor_sync(0xFFFFFFFFu, a.lo, o)});
  return a;
}
// The sum up to and with each lane.
__device__ __forceinline__ Pair warp_scan_exact(Pair a, int lane) {
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const Pair t = {__shfl_up_sync(0xFFFFFFFFu, a.hi, o), __shfl_up_sync(0xFFFFFFFFu, a.lo, o)};
    if (lane >= o) a = add(t, a);
  }
  return a;
}

struct Cands {
  int32_t* ids;
  float *w, *g;
};

struct Walk {
  int parent[kNodes];
  int32_t token[kNodes];
  float r[kNodes], px[kNodes];
  int hit[kNodes];
  Pair part[kWarps];
  // where it ended, for all CTAs
  int cur, count, changed, state;
  unsigned long long path;
};
enum State { kWalked, kIdle, kBad };

// (What runs once or twice a launch takes its time mostly for its instructions, which
// come from memory the first time: such loops are not unrolled.)
__device__ void clear_table(int* key, int slot_bits) {  // keys -1, places INT32_MAX
#pragma unroll 1
  for (int i = threadIdx.x; i < 2 << slot_bits; i += kThreads) key[i] = i < 1 << slot_bits ? -1 : INT32_MAX;
}

// Of candidates listed twice the first counts: the others lose their id. The table is
// clear before and afterwards.
__device__ void drop_repeats(const Cands& c, int K, int* key, int slot_bits) {
  const int slots = 1 << slot_bits;
  int* at = key + slots;
  auto slot_of = [&](int32_t id) {  // where id is, or its place
    uint32_t h = ((uint32_t)id * 2654435761u) >> (32 - slot_bits);
    for (int probe = 0; probe < slots; ++probe) {
      const int was = atomicCAS(&key[h], -1, id);
      if (was == -1 || was == id) break;
      h = (h + 1) & (slots - 1);
    }
    return (int)h;
  };
#pragma unroll 1
  for (int j = threadIdx.x; j < K; j += kThreads)
    if (c.ids[j] >= 0) atomicMin(&at[slot_of(c.ids[j])], j);
  cta_sync();
#pragma unroll 1
  for (int j = threadIdx.x; j < K; j += kThreads)
    if (c.ids[j] >= 0 && at[slot_of(c.ids[j])] != j) {
      c.ids[j] = -1;
      c.w[j] = c.g[j] = 0.f;
    }
  cta_sync();
  clear_table(key, slot_bits);
}

// The nodes whose parent is c, c < kNodes.
__device__ __forceinline__ uint64_t children(const Walk& wk, int c, int lane) {
  const uint32_t lo = __ballot_sync(0xFFFFFFFFu, wk.parent[lane] == c);
  const uint32_t hi = __ballot_sync(0xFFFFFFFFu, wk.parent[lane + 32] == c);
  const uint64_t kids = (uint64_t)hi << 32 | lo;
  return c >= 63 ? 0 : kids >> (c + 1) << (c + 1);  // a parent comes before its children
}

// The walk over children that are given, by one warp.
__device__ void walk_given(const TreeArgs& a, Walk& wk, int lane) {
  int cur = 0, count = 0, state = kWalked;
  unsigned long long path = 1;
  bool changed = false;
  for (bool on = true; on;) {
    on = false;
    changed = false;
    Pair Z = {1.f, 0.f};
    for (uint64_t kids = children(wk, cur, lane); kids; kids &= kids - 1) {
      const int x = __ffsll((long long)kids) - 1;
      const int32_t tok = wk.token[x];
      if (tok < 0 || tok >= a.n) {
        state = kBad;
        break;
      }
      // nothing is left of a token that was tried before
      const bool twin = (lane < x && wk.parent[lane] == cur && wk.token[lane] == tok) ||
                        (lane + 32 < x && wk.parent[lane + 32] == cur && wk.token[lane + 32] == tok);
      const float w = __any_sync(0xFFFFFFFFu, twin) ? 0.f : wk.px[x];
      if (less(times(Z, wk.r[x]), {w, 0.f})) {
        if (count == a.depth) {  // deeper than there is room for
          state = kBad;
          break;
        }
        ++count;
        path |= 1ull << x;
        cur = x;
        on = true;
        break;
      }
      Z = less({w, 0.f}, Z) ? add(Z, {-w, 0.f}) : Pair{0.f, 0.f};
      changed = true;
    }
    if (state == kBad) break;
  }
  if (lane == 0) {
    wk.cur = cur;
    wk.count = count;
    wk.changed = changed;
    wk.state = state;
    wk.path = path;
  }
}

// The walk over children drawn from their parent's candidates, by a CTA.
__device__ void walk_drawn(const TreeArgs& a, Walk& wk, const Cands& c, int* table, int slot_bits,
                           int base) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int64_t n = a.n;
  clear_table(table, slot_bits);
  int cur = 0, count = 0, state = kWalked;
  unsigned long long path = 1;
  bool changed = false;
  for (;;) {
    changed = false;
    const uint64_t all = children(wk, cur, lane);
    if (!all) break;
    const int64_t row = (int64_t)(base + cur);
    for (int j0 = tid; j0 < a.K; j0 += kLoads * kThreads) {  // a few of a thread under way together
      int32_t id[kLoads];
      float g[kLoads], w[kLoads];
#pragma unroll
      for (int i = 0; i < kLoads; ++i) {
        const int j = j0 + i * kThreads;
        id[i] = j < a.K ? a.cand_ids[row * a.K + j] : -1;
        g[i] = j < a.K ? a.cand_q[row * a.K + j] : 0.f;
      }
#pragma unroll
      for (int i = 0; i < kLoads; ++i) {
        if (id[i] < 0 || id[i] >= n) id[i] = -1;
        w[i] = id[i] < 0 ? 0.f : a.p[row * n + id[i]];
      }
#pragma unroll
      for (int i = 0; i < kLoads; ++i) {
        const int j = j0 + i * kThreads;
        if (j >= a.K) break;
        c.ids[j] = id[i];
        c.g[j] = id[i] < 0 ? 0.f : weight_of(g[i]);
        c.w[j] = weight_of(w[i]);
        for (uint64_t kids = all; kids; kids &= kids - 1) {
          const int x = __ffsll((long long)kids) - 1;
          if (wk.token[x] == id[i] && id[i] >= 0) atomicMin(&wk.hit[x], j);
        }
      }
    }
    cta_sync();
    Pair Z = {1.f, 0.f}, Q = {1.f, 0.f};  // the same in every thread
    int next = -1;
    for (uint64_t kids = all; kids; kids &= kids - 1) {
      const int x = __ffsll((long long)kids) - 1;
      const int hit = wk.hit[x];
      if (hit == a.K) {  // no candidate of its parent's
        state = kBad;
        break;
      }
      const float gx = c.g[hit];
      if (less(times(times(Z, wk.r[x]), gx), times(Q, c.w[hit]))) {
        if (count == a.depth)  // deeper than there is room for
          state = kBad;
        else
          next = x;
        break;
      }
      const float f = Q.hi > 0.f ? ratio(Z, Q) : 0.f;
      cta_sync();  // seen by all before it changes
      if (!changed) drop_repeats(c, a.K, table, slot_bits);
      changed = true;
      Pair took = {0.f, 0.f};
      for (int j = tid; j < a.K; j += kThreads) {
        const float w = c.w[j], t = fminf(w, __fmul_rn(f, c.g[j]));
        c.w[j] = __fsub_rn(w, t);
        add_exact(took, t);
        if (j == hit) c.g[j] = 0.f;
      }
      took = warp_sum_exact(joined(took.hi, took.lo));
      if (lane == 0) wk.part[warp] = took;
      cta_sync();
      took = warp_sum_exact<kWarps>(wk.part[lane % kWarps]);
      Z = less(took, Z) ? add(Z, minus(took)) : Pair{0.f, 0.f};
      Q = add(Q, {-gx, 0.f});
    }
    if (next < 0) break;
    ++count;
    path |= 1ull << next;
    cur = next;
    cta_sync();  // the candidates have been read before the next node's come
  }
  if (tid == 0) {
    wk.cur = cur;
    wk.count = count;
    wk.changed = changed;
    wk.state = state;
    wk.path = path;
  }
}

__global__ void __launch_bounds__(kThreads, 2)
verify_tree_kernel(const TreeArgs a, const Layout lay, int* err) {
  extern __shared__ __align__(16) uint8_t dsmem[];
  float* row_s = reinterpret_cast<float*>(dsmem);
  Cands cand;
  cand.g = reinterpret_cast<float*>(dsmem + lay.bytes) - lay.cands;
  cand.w = cand.g - lay.cands;
  cand.ids = reinterpret_cast<int32_t*>(cand.w - lay.cands);
  __shared__ Walk wk;
  __shared__ Pair seg[kWarps], seg_at[kWarps + 1];  // each warp's sum, and the sum before it
  __shared__ Pair cta_total, sh_target, sh_off, sh_base;
  __shared__ int cta_last, sh_pick, sh_owner;
  __shared__ bool sh_past;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int rank = (int)tc::cluster_ctarank(), ranks = lay.cluster;
  const int64_t n = a.n;
  pdl_wait();
  pdl_trigger();
  for (int s = blockIdx.y; s < a.S; s += gridDim.y) {
    int32_t* out_tokens = a.out_tokens + (int64_t)s * (a.depth + 1);
    int32_t* out_path = a.out_path + (int64_t)s * (a.depth + 1);
    const int base = a.cu[s], m = a.cu[s + 1] - base;
    if (rank == 0) {
      const bool idle = (a.granted && a.granted[s] == 0) || a.cu[s + 1] == base;
      const bool sane = base >= 0 && m >= 0 && m <= kNodes && base <= a.T - m;
      cta_sync();
      if (idle || !sane) {
        if (tid == 0) wk.state = idle ? kIdle : kBad;
      } else {
        if (tid < kNodes) {
          const bool in = tid < m;
          const int parent = in && tid > 0 ? a.parent[base + tid] : -1;
          const int32_t token = in ? a.tokens[base + tid] : -1;
          wk.parent[tid] = parent;
          wk.token[tid] = token;
          wk.r[tid] = in ? a.r[base + tid] : 0.f;
          wk.hit[tid] = a.K;
          if (!a.cand_ids)
            wk.px[tid] = token >= 0 && token < n && parent >= 0 && parent < tid
                             ? weight_of(a.p[(int64_t)(base + parent) * n + token])
                             : 0.f;
        }
        cta_sync();
        if (a.cand_ids)
          walk_drawn(a, wk, cand, reinterpret_cast<int*>(row_s), lay.slot_bits, base);
        else if (warp == 0)
          walk_given(a, wk, lane);
      }
      cta_sync();
      if (wk.state != kWalked) {
        if (wk.state == kBad && tid == 0) record_error(err, kDevErrBadId);
        for (int i = tid; i <= a.depth; i += kThreads) out_tokens[i] = out_path[i] = -1;
        if (tid == 0) a.out_accepted[s] = -1;
      } else {
        // entry i: the i-th node of the path, the (i + 1)-th node's token
        for (int i = tid; i <= a.depth; i += kThreads) {
          unsigned long long rest = wk.path;
          for (int k = 0; k < i; ++k) rest &= rest - 1;
          const unsigned long long after = rest & (rest - 1);
          out_path[i] = i <= wk.count ? __ffsll((long long)rest) - 1 : -1;
          if (i != wk.count) out_tokens[i] = i < wk.count ? wk.token[__ffsll((long long)after) - 1] : -1;
        }
        if (tid == 0) a.out_accepted[s] = wk.count;
      }
    }
    tc::cluster_sync();
    const int state = of_first(&wk.state);
    if (state != kWalked) {
      tc::cluster_sync();  // read before the first CTA goes on or ends
      continue;
    }
    const int cur = of_first(&wk.cur), count = of_first(&wk.count);
    const bool changed = of_first(&wk.changed) != 0;
    // ---- the token behind the path
    const float* row = a.p + (int64_t)(base + cur) * n;
    const int64_t per = ((n + ranks - 1) / ranks + 3) / 4 * 4;
    const int64_t v0 = min(n, rank * per), v1 = min(n, v0 + per);
    const bool quads = (reinterpret_cast<uintptr_t>(row) & 15) == 0;
    const float u = a.u[s] < 0.f ? 0.f : a.u[s];  // (a NaN stays one, and passes nothing)
    for (int pass = 0; pass < 2; ++pass) {
      const bool patch = changed && pass == 0;  // what is left may be nothing: then p itself
      // a chunk of the row into shared memory, as it is left, and each warp's sum of
      // its run of it; returns the last place with a weight in this thread's part
      auto load = [&](int64_t at, int len) -> int {
        cta_sync();
        if (quads) {  // (what a chunk begins at is a multiple of four)
          const float4* src = reinterpret_cast<const float4*>(row + at);
          constexpr int kQuads = 8;
          for (int i0 = tid; i0 < len / 4; i0 += kQuads * kThreads) {
            float4 v[kQuads];
#pragma unroll
            for (int k = 0; k < kQuads; ++k)
              v[k] = i0 + k * kThreads < len / 4 ? src[i0 + k * kThreads] : make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
            for (int k = 0; k < kQuads; ++k)
              if (i0 + k * kThreads < len / 4)
                reinterpret_cast<float4*>(row_s)[i0 + k * kThreads] =
                    make_float4(weight_of(v[k].x), weight_of(v[k].y), weight_of(v[k].z), weight_of(v[k].w));
          }
          for (int i = (len & ~3) + tid; i < len; i += kThreads) row_s[i] = weight_of(row[at + i]);
        } else {
#pragma unroll 8
          for (int i = tid; i < len; i += kThreads) row_s[i] = weight_of(row[at + i]);
        }
        cta_sync();
        if (patch && a.cand_ids) {
          for (int j = tid; j < a.K; j += kThreads) {
            const int id = of_first(cand.ids + j);
            const int64_t i = id - at;
            if (id >= 0 && i >= 0 && i < len)
              row_s[i] = __int_as_float(of_first(reinterpret_cast<const int*>(cand.w) + j));
          }
        } else if (patch && tid < kNodes && tid > cur && of_first(&wk.parent[tid]) == cur) {
          const int64_t i = of_first(&wk.token[tid]) - at;
          if (i >= 0 && i < len) row_s[i] = 0.f;
        }
        cta_sync();
        Pair sum[2] = {};
        int last = -1;
        const int end = min(len, (warp + 1) * lay.run);
#pragma unroll 4
        for (int i = warp * lay.run + lane, odd = 0; i < end; i += 32, odd ^= 1) {
          const float w = row_s[i];
          add_exact(sum[odd], w);
          if (w > 0.f) last = i;
        }
        const Pair whole = warp_sum_exact(add(joined(sum[0].hi, sum[0].lo), joined(sum[1].hi, sum[1].lo)));
        if (lane == 0) seg[warp] = whole;
        cta_sync();
        if (warp == 0) {
          // where each warp's run begins in the running sum
          const Pair from = sh_base;
          Pair mine = lane < kWarps ? seg[lane] : Pair{0.f, 0.f};
          mine = warp_scan_exact(mine, lane);
          const Pair before = shuffled(mine, lane > 0 ? lane - 1 : 0);
          if (lane <= kWarps) seg_at[lane] = lane > 0 ? add(from, before) : from;
          __syncwarp();
          if (lane == kWarps - 1) sh_base = add(from, mine);
        }
        cta_sync();
        return last;
      };
      if (tid == 0) cta_last = -1, sh_pick = -1, sh_base = {0.f, 0.f};
      int last = -1;
      for (int64_t at = v0; at < v1; at += lay.chunk) {
        const int l = load(at, (int)min((int64_t)lay.chunk, v1 - at));
        if (l >= 0) last = (int)(at + l);
      }
      cta_sync();
      last = __reduce_max_sync(0xFFFFFFFFu, last);
      if (lane == 0) atomicMax(&cta_last, last);
      if (tid == 0) cta_total = sh_base;
      cta_sync();
      tc::cluster_sync();
      if (warp == 0) {  // the sums of the CTAs before this one and of all
        Pair t = {0.f, 0.f};
        int l = -1;
        if (lane < ranks) {
          const float2 v = ld_cluster_f32x2(tc::map_to_rank(tc::smem_addr(&cta_total), (uint32_t)lane));
          t = {v.x, v.y};
          l = ld_cluster_s32(tc::map_to_rank(tc::smem_addr(&cta_last), (uint32_t)lane));
        }
        const Pair to = warp_scan_exact(t, lane);
        const Pair before = shuffled(to, rank > 0 ? rank - 1 : 0);
        const Pair target = times(shuffled(to, 31), u);
        const uint32_t some = __ballot_sync(0xFFFFFFFFu, l >= 0);
        const uint32_t over = __ballot_sync(0xFFFFFFFFu, l >= 0 && less(target, to));
        if (lane == 31) {
          sh_off = rank > 0 ? before : Pair{0.f, 0.f};
          sh_target = target;
          sh_past = over == 0;
          sh_owner = over ? __ffs(over) - 1 : 31 - __clz(some);
        }
      }
      cta_sync();
      // The draw's place: the first with a weight whose running sum passes the target, or,
      // where none does (u is 1, or rounding), the last with a weight. It is looked for
      // by the same rule among the CTAs, a CTA's warps, their lanes and a lane's
      // entries. Running sums of one level are rounded in other places than those of
      // the next; an interval with ends of both could hold a target that no other holds
      // either, or two hold, where this names one place whatever the target.
      const int owner = sh_owner;
      const bool none = owner < 0;
      if (!none) {
        if (rank == owner) {
          if (!sh_past) {
            const Pair target = sh_target, off = sh_off;
            cta_sync();
            if (tid == 0) sh_base = {0.f, 0.f};
            for (int64_t at = v0; at < v1; at += lay.chunk) {
              const int len = (int)min((int64_t)lay.chunk, v1 - at);
              if (v1 - v0 > lay.chunk) load(at, len);  // a single chunk is still there
              const bool passes = lane < kWarps && seg[lane % kWarps].hi > 0.f &&
                                  less(target, add(off, seg_at[lane % kWarps + 1]));
              const uint32_t runs = __ballot_sync(0xFFFFFFFFu, passes);
              if (runs && warp == __ffs(runs) - 1) {
                // a lane sums neighbours (each lane beginning elsewhere, for the banks), and
                // those of the lane that passes the target are looked at 32 at a time
                const int many = lay.run / 32, first = warp * lay.run + lane * many, from0 = lane % many;
                const Pair mine = add(off, seg_at[warp]);
                Pair own = {0.f, 0.f};
#pragma unroll 4
                for (int i = 0; i < many; ++i) {
                  const int e = first + (from0 + i < many ? from0 + i : from0 + i - many);
                  if (e < len) add_exact(own, row_s[e]);
                }
                own = joined(own.hi, own.lo);
                const Pair run = add(mine, warp_scan_exact(own, lane));
                const uint32_t has = __ballot_sync(0xFFFFFFFFu, own.hi > 0.f);
                const uint32_t more = __ballot_sync(0xFFFFFFFFu, own.hi > 0.f && less(target, run));
                const int k = more ? __ffs(more) - 1 : max(0, 31 - __clz(has)), from = warp * lay.run + k * many;
                const Pair prior = shuffled(run, k > 0 ? k - 1 : 0);
                Pair under = k > 0 ? prior : mine;
                int pick = -1;
                for (int i = 0; i < many; i += 32) {
                  const int e = from + i + lane;
                  const float w = i + lane < many && e < len ? row_s[e] : 0.f;
                  const Pair sum = add(under, warp_scan_exact({w, 0.f}, lane));
                  const uint32_t some = __ballot_sync(0xFFFFFFFFu, w > 0.f);
                  const uint32_t hit = __ballot_sync(0xFFFFFFFFu, w > 0.f && less(target, sum));
                  if (some) pick = from + i + 31 - __clz(some);  // where none passes: the last
                  if (hit) {
                    pick = from + i + __ffs(hit) - 1;
                    break;
                  }
                  under = shuffled(sum, 31);
                }
                if (lane == 0 && pick >= 0) sh_pick = (int)(at + pick);
              }
              cta_sync();
              if (sh_pick >= 0) break;
            }
          }
          if (tid == 0) out_tokens[count] = sh_pick >= 0 ? sh_pick : cta_last;
        }
      } else if (pass == 1 && rank == ranks - 1 && tid == 0) {
        out_tokens[count] = (int32_t)(n - 1);
      }
      tc::cluster_sync();  // what the others read is kept until all are done
      if (!none) break;
    }
  }
}

}  // namespace

cudaError_t launch_verify_tree(const TreeArgs& a, int* err, cudaStream_t s) {
  const Layout lay = layout_of(a.n, a.cand_ids ? a.K : 0, a.S);
  static int smem_set[64] = {0};
  const cudaError_t e = ensure_dynamic_smem(verify_tree_kernel, lay.bytes, smem_set);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(lay.cluster, a.S < 65535 ? a.S : 65535);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = lay.bytes;
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = lay.cluster;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, verify_tree_kernel, a, lay, err);
}

}  // namespace lmhead
