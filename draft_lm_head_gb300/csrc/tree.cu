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
// Weights are fp32 (w - fl(fl(Z / Q) g) is rounded once each), masses and
// running sums 64 bits or pairs of fp32 numbers.
//
// One cluster of 8 CTAs a request: each takes the same walk, then an eighth of the
// last node's row of p, from memory to shared memory, where the changed weights
// replace what was read; the sums meet in distributed shared memory and the CTA that
// has the draw finds its place. Bound by latency: of dependent reads, one row of
// candidates a node, then the row of p.
#include "common.cuh"
#include "kernels.h"
#include "tc_util.cuh"

namespace lmhead {
namespace {

constexpr int kThreads = 512;
constexpr int kWarps = kThreads / 32;
constexpr int kCluster = 8;
constexpr int kNodes = 64;      // of a request
constexpr int kMaxRun = 2048;   // entries of p that a warp has in shared memory at a time

// What is in shared memory: `chunk` entries of p (in their place, while the walk
// lasts, a table of 2^slot_bits keys and places), then the candidates.
struct Layout {
  int run, chunk;  // a warp's entries (a multiple of 32), a CTA's
  int slot_bits, cands;
  size_t bytes;
};
struct Shared {
  float* row;
  int32_t* ids;
  float *w, *g;
};

inline Layout layout_of(int64_t n, int K) {
  Layout l;
  const int64_t per = (n + kCluster - 1) / kCluster;
  const int64_t run = ((per + kWarps - 1) / kWarps + 31) / 32 * 32;
  l.run = (int)(run < kMaxRun ? run : kMaxRun);
  l.chunk = l.run * kWarps;
  l.cands = (K + 3) / 4 * 4;
  l.slot_bits = 6;
  while ((1 << l.slot_bits) < 2 * K) ++l.slot_bits;  // half empty at least
  const size_t row = (size_t)l.chunk * 4, table = K > 0 ? (size_t)8 << l.slot_bits : 0;
  l.bytes = (row > table ? row : table) + (size_t)l.cands * 12;
  return l;
}

__device__ __forceinline__ float weight_of(float p) { return p > 0.f ? p : 0.f; }  // NaN: nothing

__device__ __forceinline__ double ld_cluster_f64(uint32_t addr) {
  double v;
  asm volatile("ld.shared::cluster.f64 %0, [%1];" : "=d"(v) : "r"(addr) : "memory");
  return v;
}
__device__ __forceinline__ int ld_cluster_s32(uint32_t addr) {
  int v;
  asm volatile("ld.shared::cluster.s32 %0, [%1];" : "=r"(v) : "r"(addr) : "memory");
  return v;
}

__device__ __forceinline__ double warp_sum_f64(double v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
  return v;
}

// (hi, lo) += x without a rounding of hi + lo but in lo.
__device__ __forceinline__ void add_exact(float& hi, float& lo, float x) {
  const float s = __fadd_rn(hi, x), b = __fsub_rn(s, hi);
  lo = __fadd_rn(lo, __fadd_rn(__fsub_rn(hi, __fsub_rn(s, b)), __fsub_rn(x, b)));
  hi = s;
}

// The sum over the CTA of v, the same in every thread.
__device__ __forceinline__ double cta_sum(double v, double* part) {
  v = warp_sum_f64(v);
  cta_sync();
  if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = v;
  cta_sync();
  double t = 0;
#pragma unroll
  for (int i = 0; i < kWarps; ++i) t += part[i];
  return t;
}

// Of candidates listed twice the first counts: the others lose their id.
__device__ void drop_repeats(const Shared& sh, int K, int slot_bits) {
  const int slots = 1 << slot_bits;
  int* key = reinterpret_cast<int*>(sh.row);
  int* at = key + slots;
  for (int i = threadIdx.x; i < slots; i += kThreads) key[i] = -1, at[i] = INT32_MAX;
  cta_sync();
  auto slot_of = [&](int32_t id) {  // where id is, or its place
    uint32_t h = ((uint32_t)id * 2654435761u) >> (32 - slot_bits);
    for (int probe = 0; probe < slots; ++probe) {
      const int was = atomicCAS(&key[h], -1, id);
      if (was == -1 || was == id) break;
      h = (h + 1) & (slots - 1);
    }
    return (int)h;
  };
  for (int j = threadIdx.x; j < K; j += kThreads)
    if (sh.ids[j] >= 0) atomicMin(&at[slot_of(sh.ids[j])], j);
  cta_sync();
  for (int j = threadIdx.x; j < K; j += kThreads)
    if (sh.ids[j] >= 0 && at[slot_of(sh.ids[j])] != j) {
      sh.ids[j] = -1;
      sh.w[j] = sh.g[j] = 0.f;
    }
  cta_sync();
}

__global__ void __cluster_dims__(kCluster, 1, 1) __launch_bounds__(kThreads, 1)
verify_tree_kernel(const TreeArgs a, const Layout lay, int* err) {
  extern __shared__ __align__(16) uint8_t dsmem[];
  Shared sh;
  sh.g = reinterpret_cast<float*>(dsmem);
  sh.w = sh.g + lay.cands;
  sh.ids = reinterpret_cast<int32_t*>(sh.w + lay.cands);
  sh.row = reinterpret_cast<float*>(sh.ids + lay.cands);
  __shared__ int parent[kNodes];
  __shared__ int32_t token[kNodes];
  __shared__ float r[kNodes], px[kNodes];
  __shared__ double part[kWarps], seg[kWarps];
  __shared__ double cta_total;
  __shared__ int cta_last, sh_hit, sh_pick;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int rank = (int)tc::cluster_ctarank();
  const int64_t n = a.n;
  pdl_wait();
  pdl_trigger();
  for (int s = blockIdx.y; s < a.S; s += gridDim.y) {
    cta_sync();  // what follows overwrites the last request's
    int32_t* out_tokens = a.out_tokens + (int64_t)s * (a.depth + 1);
    int32_t* out_path = a.out_path + (int64_t)s * (a.depth + 1);
    const int base = a.cu[s], m = a.cu[s + 1] - base;
    const bool idle = (a.granted && a.granted[s] == 0) || a.cu[s + 1] == base;
    const bool sane = base >= 0 && m >= 0 && m <= kNodes && base <= a.T - m;
    bool bad = !idle && !sane;
    int count = -1, cur = 0;
    uint64_t path = 1;  // nodes of the accepted path
    bool changed = false;
    if (!idle && !bad) {
      if (tid < kNodes) {
        parent[tid] = tid > 0 && tid < m ? a.parent[base + tid] : -1;
        token[tid] = tid < m ? a.tokens[base + tid] : -1;
        r[tid] = tid < m ? a.r[base + tid] : 0.f;
        const bool in = token[tid] >= 0 && token[tid] < n && parent[tid] >= 0 && parent[tid] < tid;
        px[tid] = in ? weight_of(a.p[(int64_t)(base + parent[tid]) * n + token[tid]]) : 0.f;
      }
      cta_sync();
      count = 0;
      double Z = 1, Q = 1;
      // the children of node c behind node `behind`
      auto next_child = [&](int c, int behind) -> int {
        const uint32_t lo = __ballot_sync(0xFFFFFFFFu, parent[lane] == c);
        const uint32_t hi = __ballot_sync(0xFFFFFFFFu, parent[lane + 32] == c);
        uint64_t kids = (uint64_t)hi << 32 | lo;
        kids = behind >= 63 ? 0 : kids >> (behind + 1) << (behind + 1);
        return kids ? __ffsll((long long)kids) - 1 : -1;
      };
      int x = next_child(0, 0);
      bool fresh = true;  // the candidates of `cur` are not loaded yet
      while (x >= 0) {
        const int32_t tok = token[x];
        if (tok < 0 || tok >= n) {
          bad = true;
          break;
        }
        bool yes;
        if (a.cand_ids) {
          const int64_t row = (int64_t)(base + cur);
          if (fresh) {
            for (int j = tid; j < a.K; j += kThreads) {
              int32_t id = a.cand_ids[row * a.K + j];
              if (id < 0 || id >= n) id = -1;
              sh.ids[j] = id;
              sh.g[j] = id < 0 ? 0.f : weight_of(a.cand_q[row * a.K + j]);
              sh.w[j] = id < 0 ? 0.f : weight_of(a.p[row * n + id]);
            }
            Z = Q = 1;
            changed = false;
          }
          if (tid == 0) sh_hit = a.K;
          cta_sync();
          for (int j = tid; j < a.K; j += kThreads)
            if (sh.ids[j] == tok) atomicMin(&sh_hit, j);
          cta_sync();
          const int hit = sh_hit;
          if (hit == a.K) {  // no candidate of its parent's
            bad = true;
            break;
          }
          const double gx = sh.g[hit];
          yes = (double)r[x] * Z * gx < (double)sh.w[hit] * Q;
          cta_sync();  // seen by all before it changes
          if (!yes) {
            if (!changed) drop_repeats(sh, a.K, lay.slot_bits);
            changed = true;
            const float f = Q > 0 ? (float)(Z / Q) : 0.f;
            float hi = 0.f, lo = 0.f;
            for (int j = tid; j < a.K; j += kThreads) {
              const float took = fminf(sh.w[j], __fmul_rn(f, sh.g[j]));
              sh.w[j] = __fsub_rn(sh.w[j], took);
              add_exact(hi, lo, took);
            }
            const double took = cta_sum((double)hi + (double)lo, part);  // (its barriers order the reads of g)
            Z = Z > took ? Z - took : 0;
            Q -= gx;
            if (tid == 0) sh.g[hit] = 0.f;
          }
        } else {
          if (fresh) Z = 1;
          // nothing is left of a token that was tried before
          const bool twin0 = lane < x && parent[lane] == cur && token[lane] == tok;
          const bool twin1 = lane + 32 < x && parent[lane + 32] == cur && token[lane + 32] == tok;
          const double w = __any_sync(0xFFFFFFFFu, twin0 || twin1) ? 0.0 : (double)px[x];
          yes = (double)r[x] * Z < w;
          if (!yes) Z = Z > w ? Z - w : 0;
          changed = true;
        }
        fresh = yes;
        if (yes) {
          if (count == a.depth) {  // deeper than there is room for
            bad = true;
            break;
          }
          ++count;
          path |= 1ull << x;
          cur = x;
          changed = false;
        }
        cta_sync();
        x = next_child(cur, x);
      }
    }
    if (bad || idle) {
      if (rank == 0) {
        if (bad && tid == 0) record_error(err, kDevErrBadId);
        for (int i = tid; i <= a.depth; i += kThreads) out_tokens[i] = out_path[i] = -1;
        if (tid == 0) a.out_accepted[s] = -1;
      }
      continue;  // every CTA of the cluster alike
    }
    if (rank == 0) {
      // entry i: the i-th node of the path, the (i + 1)-th node's token
      for (int i = tid; i <= a.depth; i += kThreads) {
        uint64_t rest = path;
        for (int k = 0; k < i; ++k) rest &= rest - 1;
        const uint64_t after = rest & (rest - 1);
        out_path[i] = i <= count ? __ffsll((long long)rest) - 1 : -1;
        if (i != count) out_tokens[i] = i < count ? token[__ffsll((long long)after) - 1] : -1;
      }
      if (tid == 0) a.out_accepted[s] = count;
    }
    // ---- the token behind the path
    const float* row = a.p + (int64_t)(base + cur) * n;
    const int64_t per = (n + kCluster - 1) / kCluster;
    const int64_t v0 = min(n, rank * per), v1 = min(n, v0 + per);
    const float u = a.u[s];
    for (int pass = 0; pass < 2; ++pass) {
      const bool patch = changed && pass == 0;  // what is left may be nothing: then p itself
      // a chunk of the row into shared memory, as it is left, and each warp's sum of
      // its run of it; returns the last place with a weight in this thread's part
      auto load = [&](int64_t at, int len) -> int {
        cta_sync();
#pragma unroll 8
        for (int i = tid; i < len; i += kThreads) sh.row[i] = weight_of(row[at + i]);
        cta_sync();
        if (patch && a.cand_ids) {
          for (int j = tid; j < a.K; j += kThreads) {
            const int64_t i = sh.ids[j] - at;
            if (sh.ids[j] >= 0 && i >= 0 && i < len) sh.row[i] = sh.w[j];
          }
        } else if (patch && tid < kNodes && parent[tid] == cur) {
          const int64_t i = token[tid] - at;
          if (i >= 0 && i < len) sh.row[i] = 0.f;
        }
        cta_sync();
        float hi = 0.f, lo = 0.f;
        int last = -1;
        for (int i = warp * lay.run + lane; i < min(len, (warp + 1) * lay.run); i += 32) {
          const float w = sh.row[i];
          add_exact(hi, lo, w);
          if (w > 0.f) last = i;
        }
        const double sum = warp_sum_f64((double)hi + (double)lo);
        if (lane == 0) seg[warp] = sum;
        cta_sync();
        return last;
      };
      double total = 0;
      int64_t last = -1;
      for (int64_t at = v0; at < v1; at += lay.chunk) {
        const int l = load(at, (int)min((int64_t)lay.chunk, v1 - at));
        if (l >= 0) last = at + l;
        for (int w = 0; w < kWarps; ++w) total += seg[w];
      }
      last = __reduce_max_sync(0xFFFFFFFFu, (int)last);
      if (tid == 0) cta_last = -1, cta_total = total, sh_pick = -1;
      cta_sync();
      if (lane == 0) atomicMax(&cta_last, (int)last);
      cta_sync();
      tc::cluster_sync();
      double all = 0, off = 0;
      int last_rank = -1;
      for (int q = 0; q < kCluster; ++q) {
        const double t = ld_cluster_f64(tc::map_to_rank(tc::smem_addr(&cta_total), (uint32_t)q));
        if (ld_cluster_s32(tc::map_to_rank(tc::smem_addr(&cta_last), (uint32_t)q)) >= 0) last_rank = q;
        if (q == rank) off = all;
        all += t;
      }
      tc::cluster_sync();  // read before any CTA goes on or ends
      if (!(all > 0)) {
        if (pass == 1 && rank == kCluster - 1 && tid == 0) out_tokens[count] = (int32_t)(n - 1);
        continue;
      }
      const double target = (double)u * all;
      const bool past = !(target < all);  // u * total rounded up to the total
      const double end = rank + 1 < kCluster ? off + total : all;
      if (past ? rank == last_rank : off <= target && target < end) {
        if (!past) {
          double before = off;
          for (int64_t at = v0; at < v1; at += lay.chunk) {
            const int len = (int)min((int64_t)lay.chunk, v1 - at);
            if (v1 - v0 > lay.chunk) load(at, len);  // a single chunk is still there
            double mine = before;
            for (int w = 0; w < kWarps; ++w) {
              if (w == warp) mine = before;
              before += seg[w];
            }
            if (mine <= target && target < mine + seg[warp]) {
              // a lane sums neighbours (each lane beginning elsewhere, for the banks), and
              // those of the lane that passes the target are looked at 32 at a time
              const int many = lay.run / 32, first = warp * lay.run + lane * many;
              float hi = 0.f, lo = 0.f;
              for (int i = 0, e = lane % many; i < many; ++i, e = e + 1 == many ? 0 : e + 1)
                if (first + e < len) add_exact(hi, lo, sh.row[first + e]);
              const double own = (double)hi + (double)lo;
              double run = own;
#pragma unroll
              for (int o = 1; o < 32; o <<= 1) {
                const double t = __shfl_up_sync(0xFFFFFFFFu, run, o);
                if (lane >= o) run += t;
              }
              const uint32_t over = __ballot_sync(0xFFFFFFFFu, own > 0 && mine + run > target);
              if (over) {
                const int k = __ffs(over) - 1, from = warp * lay.run + k * many;
                double under = mine + __shfl_sync(0xFFFFFFFFu, run - own, k);
                int pick = -1;
                for (int i = 0; i < many; i += 32) {
                  const int e = from + i + lane;
                  const float w = i + lane < many && e < len ? sh.row[e] : 0.f;
                  double sum = w;
#pragma unroll
                  for (int o = 1; o < 32; o <<= 1) {
                    const double t = __shfl_up_sync(0xFFFFFFFFu, sum, o);
                    if (lane >= o) sum += t;
                  }
                  const uint32_t some = __ballot_sync(0xFFFFFFFFu, w > 0.f);
                  const uint32_t hit = __ballot_sync(0xFFFFFFFFu, w > 0.f && under + sum > target);
                  if (some) pick = from + i + 31 - __clz(some);  // where none passes: the last
                  if (hit) {
                    pick = from + i + __ffs(hit) - 1;
                    break;
                  }
                  under += __shfl_sync(0xFFFFFFFFu, sum, 31);
                }
                if (lane == 0) atomicMax(&sh_pick, (int)(at + pick));
              }
            }
            cta_sync();
            if (sh_pick >= 0) break;
          }
        }
        // rounding kept the target from being passed: the last that has a weight
        if (tid == 0) out_tokens[count] = sh_pick >= 0 ? sh_pick : cta_last;
      }
      break;
    }
  }
}

}  // namespace

cudaError_t launch_verify_tree(const TreeArgs& a, int* err, cudaStream_t s) {
  const Layout lay = layout_of(a.n, a.cand_ids ? a.K : 0);
  static int smem_set[64] = {0};
  const cudaError_t e = ensure_dynamic_smem(verify_tree_kernel, lay.bytes, smem_set);
  if (e != cudaSuccess) return e;
  return launch_kernel(true, verify_tree_kernel, dim3(kCluster, a.S < 65535 ? a.S : 65535),
                       dim3(kThreads), lay.bytes, s, a, lay, err);
}

}  // namespace lmhead
