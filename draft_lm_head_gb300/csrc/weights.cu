// How much attention each cached token has drawn, summed up.
//
// For key j of request s and K/V head a, over the new tokens i and the heads h of
// a that see it:
//   w_j = decay w_j [j < len_s] + sum_i,h exp(scale q_ih . k_j - lse_ih),
// with lse as attention left it, so that a row's weights over all keys sum to 1.
//
// The products run on the tensor cores with the keys as their rows: 128 keys times
// a tile of up to 128 rows of queries (tokens x the G heads that share the K/V
// head), so a thread has a key and its sum runs along the tensor memory's columns,
// with no exchange between threads and no maximum to find. Four such tiles of keys
// make a unit: they are loaded once and stay in shared memory while the request's
// query tiles pass by; a decoding step has one query tile, and its keys stream.
// One CTA an SM, warp-specialised: a warp loads keys (TMA, page by page), one loads
// queries and their lse, one issues the MMAs, and four warpgroups (a key tile each,
// with 128 columns of tensor memory) exponentiate and sum; while one waits for its
// next product the others use the exponential units. The CTAs share out key tiles x
// query tiles evenly, in the order (K/V head, request, unit). Where requests bring
// many query tiles a unit may be cut between CTAs; each leaves its sums in the
// scratch and a second launch adds them up in order, so no result depends on which
// CTA came first.
// Bound: few rows, by reading the keys once; many rows, by the tensor cores and the
// exponential units (512 cycles each for a tile of keys x one of queries) and by what a
// warpgroup waits for its next product, in which time all four wait together for a
// part. Measured (device time, graphs replayed): 32 requests of 4000-8000 cached tokens
// and one new each, 32 heads over 8, dim 128: 76 us for 413 MB (5.4 TB/s); two chunks of
// 2048 tokens over 6144 cached: 174 us for 0.24 TFLOP (1.38 PFLOP/s), the tensor pipe busy
// for 59 % of it. On the way there: two tiles a unit 244; four 205; lse in a ring of
// its own 199; two warps that issue 184; units told by one warp in place of every role
// walking over them 174. Three tiles with 152 registers a thread, the columns loaded
// ahead: 228.
// Scores, exponentials and sums are fp32, each tile's sum joined to the row of sums
// before it by one addition: the error does not grow with the length of a chunk.

#include "common.cuh"
#include "kernels.h"
#include "lmhead.h"
#include "tc_util.cuh"

namespace lmhead {
namespace {

constexpr int kKeys = 128;         // keys of a tile
constexpr int kGroups = 4;         // tiles of a unit, a warpgroup each
constexpr int kUnit = kGroups * kKeys;
constexpr int kRows = 128;         // query rows of a tile
// Four warpgroups that sum, and four warps that load keys, load queries and issue the
// MMAs (two, of two tiles each); of the 96 registers a thread at launch the former get
// 104 and the latter 64.
constexpr int kThreads = kGroups * 128 + 128;
constexpr int kRegsMore = 104, kRegsLess = 64;
constexpr int kWarpK = kGroups * 4, kWarpQ = kWarpK + 1, kWarpMma = kWarpK + 2;  // and kWarpMma + 1
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kInf = __builtin_huge_valf();

template <int D> struct Shape {
  static constexpr int kHalves = D / 64;
  static constexpr int kTile = kKeys * D * 2;           // a key tile
  static constexpr int kSets = D == 128 ? 1 : 2;        // units whose keys are in shared memory
  static constexpr int kTiles = kSets * kGroups;
  static constexpr int kQ = kRows * D * 2;              // a query tile
  static constexpr int kQTiles = D == 128 ? 3 : 5;
  static constexpr int kLse = 4;                        // query tiles' lse
  static constexpr int kUnits = 2 * kSets;              // units ahead
  static constexpr int kSmem = kTiles * kTile + kQTiles * kQ;
};

// A unit as the other roles need it: they learn of it from the warp that loads the keys.
struct Unit {
  int s, p, hk, flags;
  int tok0, m, len, tiles;  // of the request; key tiles
  int first, steps;         // query tiles [first, first + steps); steps < 0: no unit, the end
  int unused[2];
  int32_t page[32];  // of its runs of keys, -1 where there is none
};
constexpr int kAgain = 1;  // its one query tile is the one of the unit before
constexpr int kKeep = 2;   // it has one query tile, which the next unit may use too
constexpr int kCutHead = 4, kCutTail = 8;  // of its steps the first, the last are not here

template <int NK, int NQ, int NL, int NU> struct Ctl {
  Unit unit[NU];
  uint64_t u_full[NU], u_empty[NU];
  uint64_t k_full[NK], k_empty[NK], q_full[NQ], q_empty[NQ], l_full[NL], l_empty[NL];
  uint64_t s_full[kGroups], s_empty[kGroups];
  uint64_t drain[2];
  uint32_t tmem;
  int abort;
  alignas(16) float neg_lse[NL][kRows];  // -lse in base 2; -inf where there is no row
  // the plan: the CTA's share of all cost, and the unit in which it begins
  long long lo, hi;
  int bad, s0, p0, off0, hk0;
};

// What a request has to do for one K/V head.
struct Req {
  int tok0, m, len;
  int np, qt;  // units, query tiles
};

// The query tiles [t0, t0 + n) that see any key of unit p.
struct Span {
  int t0, n;
};

__device__ __forceinline__ Req request_of(const WeightArgs& a, int s, int tile_tok, bool& sane) {
  Req r;
  r.tok0 = a.cu[s];
  r.m = a.cu[s + 1] - r.tok0;
  r.len = a.lens[s];
  sane = true;
  r.np = r.qt = 0;
  const bool refused = a.granted && a.granted[s] == 0;
  if (refused || r.len < 0 || r.len > min(a.width << a.page_shift, kMaxTokens) - r.m) {
    sane = refused;
    r.len = 0;  // (whatever it was, no arithmetic is done on it)
    return r;
  }
  if (r.m == 0 && a.decay == 1.f) return r;  // nothing changes
  r.np = (r.len + r.m + kUnit - 1) / kUnit;
  r.qt = (r.m + tile_tok - 1) / tile_tok;
  return r;
}

__device__ __forceinline__ Span span_of(const WeightArgs& a, const Req& r, int p, int tile_tok) {
  Span x = {0, r.qt};
  if (!a.tree) {
    const int first = p * kUnit - r.len;  // the first token that sees the unit's first key
    if (first > 0) x.t0 = min(r.qt, first / tile_tok);
    if (a.window > 0) {
      // the last key is out of sight from here on (64 bits: the window may be any)
      const long long past = (long long)first + kUnit - 1 + a.window;
      x.n = past <= 0 ? 0 : (int)min((long long)r.qt, (past + tile_tok - 1) / tile_tok);
    }
    x.n = max(0, x.n - x.t0);
  }
  return x;
}

// A unit's key tiles. They cost 1 each, and 1 for each query tile: the unit's step x
// (query tile) ends at cost tiles (x + 2), and what is cut at cost c falls to step
// step_at(c).
__device__ __forceinline__ int tiles_of(const Req& r, int p) {
  return min(kGroups, (r.len + r.m - p * kUnit + kKeys - 1) / kKeys);
}
__device__ __forceinline__ int step_at(int cost, int tiles) {
  return max(0, (cost + tiles - 1) / tiles - 1);
}
__device__ __forceinline__ int cost_of(const WeightArgs& a, const Req& r, int p, int tile_tok) {
  return tiles_of(r, p) * (1 + span_of(a, r, p, tile_tok).n);
}
// Units of four tiles that every query tile sees.
__device__ __forceinline__ int full_units(const WeightArgs& a, const Req& r) {
  if (a.window > 0) return 0;
  const int all = (r.len + r.m) / kUnit;  // of four tiles
  return min(r.np, a.tree ? all : min(all, r.len / kUnit + 1));
}
__device__ __forceinline__ long long cost_of(const WeightArgs& a, const Req& r, int tile_tok) {
  const int full = full_units(a, r);
  long long c = (long long)full * (kGroups * (1 + r.qt));
  for (int p = full; p < r.np; ++p) c += cost_of(a, r, p, tile_tok);
  return c;
}

// The CTA's share of all units, found by the CTA for itself.
template <typename C>
__device__ void make_plan(const WeightArgs& a, C& ctl, int tile_tok, int* err) {
  __shared__ long long warp_sum[kThreads / 32];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  if (tid == 0) ctl.bad = 0;
  cta_sync();
  long long target = 0;
  // The request in which the target lies, `before` it and of cost c, says where.
  auto locate = [&](int s, const Req& r, long long before, long long c) {
    if (target < before || target >= before + c) return;
    long long rem = target - before;
    const int each = kGroups * (1 + r.qt);
    int p = (int)min((long long)full_units(a, r), rem / each);
    rem -= (long long)p * each;
    for (; p < r.np; ++p) {
      const int w = cost_of(a, r, p, tile_tok);
      if (rem < w) break;
      rem -= w;
    }
    ctl.s0 = s;
    ctl.p0 = p;
    ctl.off0 = (int)rem;
  };
  // pass 0 sums up, and pass 1 finds the request in which the share begins (at once where
  // every thread has one request)
  for (int pass = 0; pass < 2; ++pass) {
    long long base = 0, c = 0, before = 0;
    Req r = {};
    for (int s0 = 0; s0 < a.S; s0 += kThreads) {
      const int s = s0 + tid;
      c = 0;
      if (s < a.S) {
        const int b = a.cu[s], e = a.cu[s + 1];
        if (b < 0 || e < b || e > a.T) {
          ctl.bad = 1;
        } else {
          bool sane;
          r = request_of(a, s, tile_tok, sane);
          c = cost_of(a, r, tile_tok);
          if (!sane && pass == 0 && blockIdx.x == 0) record_error(err, kDevErrBadId);
        }
      }
      long long incl = c;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const long long x = __shfl_up_sync(0xFFFFFFFFu, incl, o);
        if (lane >= o) incl += x;
      }
      if (lane == 31) warp_sum[warp] = incl;
      cta_sync();
      before = base + incl - c;
      for (int w = 0; w < kThreads / 32; ++w) {
        if (w < warp) before += warp_sum[w];
        base += warp_sum[w];
      }
      if (pass == 1) locate(s, r, before, c);
      cta_sync();
    }
    if (pass == 1) break;
    const long long all = ctl.bad ? 0 : base * a.kv_heads;
    // no CTA's share is empty before another's that is not
    const long long parts = min((long long)gridDim.x, all), x = blockIdx.x;
    long long lo = all, hi = all;
    if (x < parts) {
      lo = all / parts * x + all % parts * x / parts;
      hi = all / parts * (x + 1) + all % parts * (x + 1) / parts;
    }
    if (tid == 0) {
      ctl.lo = lo;
      ctl.hi = hi;
      ctl.hk0 = base > 0 ? (int)(lo / base) : 0;
      if (ctl.bad && blockIdx.x == 0) record_error(err, kDevErrBadId);
    }
    if (lo >= hi) break;  // the same in every thread
    target = lo - lo / base * base;
    if (a.S <= kThreads) {
      locate(tid, r, before, c);
      break;
    }
  }
  cta_sync();
}

// A CTA's units, in order.
struct Cursor {
  int s, p, hk, off, tile_tok;
  bool whole_only;
  long long left;
  Req r;
  // the unit: its place, its key tiles, its query tiles [a, b) of n from t0 on
  int u_s, u_p, u_hk, tiles, t0, n, a, b, kend;
  bool again;  // its one query tile is that of the unit's before it, whose step this CTA took too
  bool ran;    // it has a step here

  template <typename C> __device__ void init(const WeightArgs& w, const C& ctl, int tok, bool whole) {
    tile_tok = tok;
    whole_only = whole;
    left = ctl.hi - ctl.lo;
    u_s = -1;
    u_p = u_hk = tiles = t0 = n = a = b = kend = 0;
    r = {};
    again = ran = false;
    if (left <= 0) return;
    s = ctl.s0;
    p = ctl.p0;
    hk = ctl.hk0;
    off = ctl.off0;
    bool sane;
    r = request_of(w, s, tile_tok, sane);
  }
  __device__ bool next(const WeightArgs& w) {
    while (left > 0) {
      while (p >= r.np) {  // on to the next request with a unit: there is one while any cost is left
        if (++s == w.S) s = 0, ++hk;
        p = 0;
        bool sane;
        r = request_of(w, s, tile_tok, sane);
      }
      const Span x = span_of(w, r, p, tile_tok);
      tiles = tiles_of(r, p);
      const int cost = tiles * (1 + x.n);
      again = ran && n == 1 && x.n == 1 && x.t0 == t0 && u_s == s && u_hk == hk;
      u_s = s;
      u_p = p++;
      u_hk = hk;
      t0 = x.t0;
      n = x.n;
      kend = r.len + r.m;
      const int from = off, to = (int)min((long long)cost, off + left);
      off = 0;
      if (whole_only) {
        // a unit is the CTA's in whose share it begins
        left -= cost - from;
        a = 0;
        b = n;
        ran = from == 0 && n > 0;
        if (from == 0) return true;
        continue;
      }
      left -= to - from;
      a = step_at(from, tiles);
      b = step_at(to, tiles);
      ran = b > a;
      if (b > a || (n == 0 && from == 0)) return true;
    }
    return false;
  }
};

// Pieces of cut units: of CTA c one that began earlier (place 2 c) and one that
// begins there and goes on (2 c + 1), with the latter's unit.
struct Piece {
  int s, p, hk, flags;
};
constexpr int kBegins = 1;  // there is a piece in place 2 c + 1
constexpr int kHas = 2, kEnds = 4;  // there is one in place 2 c; the unit ends with it
struct Scratch {
  Piece* piece;
  float* sums;  // kUnit a place
};

__device__ __forceinline__ float* weight_at(const WeightArgs& a, int32_t id, int j, int hk) {
  return reinterpret_cast<float*>(static_cast<char*>(a.weights) + id * a.ws.page +
                                  (j & ((1 << a.page_shift) - 1)) * a.ws.token + hk * a.ws.head);
}

constexpr int kPlanBytes = kThreads / 32 * 8;  // make_plan's own
// (the tiles begin on a multiple of 1024 bytes)
static_assert(Shape<128>::kSmem + 3 * 1024 <= 227 * 1024 && sizeof(Ctl<4, 3, 4, 2>) + kPlanBytes <= 3 * 1024, "shared memory");
static_assert(Shape<64>::kSmem + 4096 <= 227 * 1024 && sizeof(Ctl<8, 5, 4, 4>) + kPlanBytes <= 4096, "shared memory");

template <bool BF16, int D>
__global__ void __launch_bounds__(kThreads, 1)
weights_kernel(const __grid_constant__ CUtensorMap kmap, const __grid_constant__ CUtensorMap qmap,
               const WeightArgs a, const Scratch sc, int k_head_first, int q_by_tma, int whole_only,
               long long budget, int* err) {
  using Sh = Shape<D>;
  constexpr int NK = Sh::kTiles, NQ = Sh::kQTiles, NL = Sh::kLse, NU = Sh::kUnits;
  extern __shared__ __align__(1024) uint8_t k_s[];
  __shared__ Ctl<NK, NQ, NL, NU> ctl;
  if (tc::smem_addr(k_s) & 1023) {  // (the same in every thread; swizzles count from there)
    if (threadIdx.x == 0) record_error(err, kDevErrTimeout);
    return;
  }
  uint8_t* q_s = k_s + NK * Sh::kTile;
  const int warp = __shfl_sync(0xFFFFFFFFu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
  volatile int* abort_flag = &ctl.abort;

  if (threadIdx.x == 0) {
    for (int i = 0; i < NK; ++i) {
      tc::mbar_init(&ctl.k_full[i], 1);
      tc::mbar_init(&ctl.k_empty[i], 1);
    }
    for (int i = 0; i < NQ; ++i) {
      tc::mbar_init(&ctl.q_full[i], 33);  // the warp's lanes, and one for a copy's bytes
      tc::mbar_init(&ctl.q_empty[i], 2);  // from both issuing warps
    }
    for (int i = 0; i < NL; ++i) {
      tc::mbar_init(&ctl.l_full[i], 32);
      tc::mbar_init(&ctl.l_empty[i], 4 * kGroups);  // a warp each of the readers
    }
    for (int i = 0; i < NU; ++i) {
      tc::mbar_init(&ctl.u_full[i], 32);
      tc::mbar_init(&ctl.u_empty[i], 3 + 4 * kGroups);  // a warp each of its readers
    }
    for (int w = 0; w < kGroups; ++w) {
      tc::mbar_init(&ctl.s_full[w], 1);
      tc::mbar_init(&ctl.s_empty[w], 4);
    }
    tc::mbar_init(&ctl.drain[0], 1);
    tc::mbar_init(&ctl.drain[1], 1);
    ctl.abort = 0;
    tc::fence_mbar_init();
  }
  if (warp == kWarpMma) {
    tc::tmem_alloc(&ctl.tmem, 512);
    tc::tmem_relinquish();
  }
  if (warp == kWarpK && lane == 0) {
    tc::prefetch_tmap(&kmap);
    tc::prefetch_tmap(&qmap);
  }
  const int group = a.heads / a.kv_heads, tile_tok = kRows / group;
  if (tile_tok * group < kRows) {
    // rows that no tile has: zeros throughout
    for (int e = threadIdx.x; e < NQ * Sh::kQ / 16; e += kThreads)
      reinterpret_cast<uint4*>(q_s)[e] = make_uint4(0, 0, 0, 0);
    tc::fence_async_smem();
  }
  tc::fence_before_sync();
  cta_sync();
  tc::fence_after_sync();
  constexpr uint32_t tmem = 0;  // all 512 columns: 128 a key tile
  pdl_wait();
  pdl_trigger();
  make_plan(a, ctl, tile_tok, err);
  const int run_tok = min(kKeys, 1 << a.page_shift), runs = kKeys / run_tok;  // keys of a page, of a tile
  // Unit number n of the CTA, for a reader: waited for, and given back.
  auto unit_wait = [&](uint32_t n) {
    return tc::wait_all<false>(&ctl.u_full[n % NU], (n / NU) & 1, abort_flag, budget);
  };
  auto unit_done = [&](uint32_t n) {
    __syncwarp();
    if (lane == 0) tc::mbar_arrive(&ctl.u_empty[n % NU]);
  };
  if (warp >= kWarpK) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegsLess));
    if (warp == kWarpK) {
      // ------------------------------------------------------------ keys by TMA
      // the cache was written by the launch before through the other proxy
      asm volatile("fence.proxy.async;" ::: "memory");
      const int run = lane / Sh::kHalves, half = lane % Sh::kHalves;
      uint32_t n = 0, units = 0;  // units, and those with a step
      uint32_t used = 0;  // a bit a slot: whether it was used, and above them, an odd number of times
      Cursor cur;
      cur.init(a, ctl, tile_tok, whole_only != 0);
      bool ok = true, more = true;
      while (ok && more) {
        more = cur.next(a);
        // a lane looks up the page of one run of the unit's keys (32 of them at most)
        int32_t id = -1;
        if (more) {
          const int key = cur.u_p * kUnit + lane * run_tok;
          if (lane < kGroups * runs && key < cur.kend) {
            id = a.table[(int64_t)cur.u_s * a.width + (key >> a.page_shift)];
            if (id < 0 || id >= a.pages) {
              id = -1;
              record_error(err, kDevErrBadId);
            }
          }
        }
        // the other roles are told
        if (n >= (uint32_t)NU) {
          ok = tc::wait_all<false>(&ctl.u_empty[n % NU], ((n / NU) & 1) ^ 1, abort_flag, budget);
          if (!ok) break;
        }
        Unit& u = ctl.unit[n % NU];
        u.page[lane] = id;
        if (lane == 0) {
          u.s = cur.u_s;
          u.p = cur.u_p;
          u.hk = cur.u_hk;
          u.flags = (cur.again ? kAgain : 0) | (cur.n == 1 ? kKeep : 0) | (cur.a > 0 ? kCutHead : 0) |
                    (cur.b < cur.n ? kCutTail : 0);
          u.tok0 = cur.r.tok0;
          u.m = cur.r.m;
          u.len = cur.r.len;
          u.tiles = cur.tiles;
          u.first = cur.t0 + cur.a;
          u.steps = more ? cur.b - cur.a : -1;
        }
        tc::mbar_arrive(&ctl.u_full[n % NU]);
        ++n;
        if (!more || cur.b == cur.a) continue;  // (no row sees the unit)
        const int set = (int)(units++ % Sh::kSets) * kGroups;
#pragma unroll 1
        for (int t = 0; t < cur.tiles; ++t) {
          const int slot = set + t;
          if (used >> slot & 1) {
            ok = tc::wait_all<false>(&ctl.k_empty[slot], (used >> (slot + 16) & 1) ^ 1, abort_flag, budget);
            if (!ok) break;
          }
          used = (used | 1u << slot) ^ 1u << (slot + 16);
          // and loads one of the tile, or half its dimensions
          const int32_t page = __shfl_sync(0xFFFFFFFFu, id, (t * runs + run) & 31);
          const bool want = run < runs && page >= 0;
          const uint32_t load = __ballot_sync(0xFFFFFFFFu, want);
          if (lane == 0)
            tc::mbar_arrive_expect_tx(&ctl.k_full[slot], (uint32_t)(__popc(load) * run_tok * 128));
          __syncwarp();
          if (want) {
            const int off = (cur.u_p * kUnit + t * kKeys + run * run_tok) & ((1 << a.page_shift) - 1);
            tc::tma_load_4d(k_s + slot * Sh::kTile + half * (kKeys * 128) + run * run_tok * 128, &kmap,
                            &ctl.k_full[slot], half * 64, k_head_first ? cur.u_hk : off,
                            k_head_first ? off : cur.u_hk, page);
          }
        }
      }
      if (!ok && lane == 0) {
        *abort_flag = 1;
        record_error(err, kDevErrTimeout);
      }
      __syncwarp();
      if (lane == 0) {
        // no copy may be under way when the CTA ends, whichever role gave up
#pragma unroll 1
        for (int i = 0; i < NK; ++i) {
          if (!(used >> i & 1)) continue;
          const long long t = clock64();
          while (!tc::mbar_try_wait(&ctl.k_full[i], (used >> (i + 16) & 1) ^ 1) &&
                 clock64() - t < tc::kWaitCycles) {
          }
        }
      }
    } else if (warp == kWarpQ) {
      // ------------------------------------------------------------ queries and lse
      asm volatile("fence.proxy.async;" ::: "memory");
      uint32_t n = 0;  // query tiles
      bool ok = true;
      for (uint32_t un = 0;; ++un) {
        ok = unit_wait(un);
        if (!ok) break;
        const Unit& u = ctl.unit[un % NU];
        const int steps = u.steps, first = u.first, tok0 = u.tok0, m = u.m, head0 = u.hk * group;
        const bool again = u.flags & kAgain;
        unit_done(un);
        if (steps < 0) break;
        if (again) continue;
#pragma unroll 1
        for (int t = first; t < first + steps; ++t, ++n) {
          const int slot = (int)(n % NQ), l_slot = (int)(n % NL);
          if (n >= (uint32_t)NQ) {
            ok = tc::wait_all<false>(&ctl.q_empty[slot], ((n / NQ) & 1) ^ 1, abort_flag, budget);
            if (!ok) break;
          }
          if (n >= (uint32_t)NL) {
            ok = tc::wait_all<false>(&ctl.l_empty[l_slot], ((n / NL) & 1) ^ 1, abort_flag, budget);
            if (!ok) break;
          }
          uint8_t* dst = q_s + slot * Sh::kQ;
          const int tok = tok0 + t * tile_tok, toks = min(tile_tok, m - t * tile_tok);
          const bool tma = q_by_tma && toks == tile_tok;
          if (lane == 0)
            tc::mbar_arrive_expect_tx(&ctl.q_full[slot],
                                      tma ? (uint32_t)(tile_tok * group * 128 * Sh::kHalves) : 0u);
          __syncwarp();
          if (tma) {
            if (lane < Sh::kHalves)
              tc::tma_load_3d(dst + lane * (kRows * 128), &qmap, &ctl.q_full[slot], lane * 64,
                              head0, tok);
          } else {
            // a tile that is not full: row by row, zeros up to the product's columns
            const int rows = toks * group, cols = (rows + 15) & ~15;
            const uint32_t to = tc::smem_addr(dst);
#pragma unroll 1
            for (int e = lane; e < cols * (D / 8); e += 32) {
              const int row = e / (D / 8), c = e % (D / 8), tk = row / group;
              const bool in = row < rows;
              const char* src = static_cast<const char*>(a.q) + c * 16;
              if (in)
                src += (int64_t)(tok + tk) * a.q_tok + (int64_t)(head0 + row - tk * group) * a.q_head;
              const int size = in ? 16 : 0;
              asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(
                               to + (c / 8) * (kRows * 128) + row * 128 + (((c % 8) ^ (row & 7)) << 4)),
                           "l"(src), "r"(size)
                           : "memory");
            }
          }
          float l[kRows / 32];
#pragma unroll
          for (int i = 0; i < kRows / 32; ++i) {
            const int row = i * 32 + lane, tk = row / group;
            l[i] = -kInf;
            if (tk < toks) l[i] = a.lse[(int64_t)(tok + tk) * a.heads + head0 + row - tk * group];
          }
#pragma unroll
          for (int i = 0; i < kRows / 32; ++i)  // a row that sees nothing draws nothing
            ctl.neg_lse[l_slot][i * 32 + lane] = l[i] == -kInf ? -kInf : l[i] * -kLog2e;
          tc::mbar_arrive(&ctl.l_full[l_slot]);
          if (!tma) {
            asm volatile("cp.async.wait_all;" ::: "memory");
            tc::fence_async_smem();
          }
          tc::mbar_arrive(&ctl.q_full[slot]);
        }
        if (!ok) break;
      }
      if (!ok && lane == 0) {
        *abort_flag = 1;
        record_error(err, kDevErrTimeout);
      }
      __syncwarp();
      if (lane == 0) {
        const uint32_t first = n > (uint32_t)NQ ? n - NQ : 0;
        for (uint32_t j = first; j < n; ++j) {
          const long long t = clock64();
          while (!tc::mbar_try_wait(&ctl.q_full[j % NQ], (j / NQ) & 1) &&
                 clock64() - t < tc::kWaitCycles) {
          }
        }
      }
    } else {
      // ------------------------------------------------------------ MMAs
      // of tiles w0 and w0 + 1. One warp for all four spends about half of the tensor
      // cores' time between tiles, waiting and forming descriptors (two chunks of 2048
      // tokens 207 us, with two warps 184).
      const int w0 = (warp - kWarpMma) * 2;
      const bool issuer = tc::elect_one();
      // (addresses count 16 bytes in the low 14 bits: sums stay in the low word)
      const uint64_t k_desc = tc::sw128_kmajor_desc(tc::smem_addr(k_s) + w0 * Sh::kTile);
      const uint64_t q_desc = tc::sw128_kmajor_desc(tc::smem_addr(q_s));
      const uint32_t hi = (uint32_t)(k_desc >> 32);
      auto desc = [&](uint32_t lo) { return (uint64_t)hi << 32 | lo; };
      uint32_t units = 0, count = 0;  // units with a step, query tiles
      uint32_t uses = 0;  // a bit a tile: whether it was used, and above them, an odd number of times
      bool held = false;  // the last query tile is not given back yet
      uint32_t seen = 0;  // a bit a slot of keys: whether it was used an odd number of times
      bool ok = true;
      for (uint32_t un = 0; ok; ++un) {
        ok = unit_wait(un);
        if (!ok) break;
        // what branches and operands depend on comes by shuffle from lane 0, so that
        // the compiler knows it to be the warp's own
        const Unit& u = ctl.unit[un % NU];
        const int steps = __shfl_sync(0xFFFFFFFFu, u.steps, 0), flags = __shfl_sync(0xFFFFFFFFu, u.flags, 0);
        const int tiles = __shfl_sync(0xFFFFFFFFu, u.tiles, 0) - w0;
        const int first = __shfl_sync(0xFFFFFFFFu, u.m - u.first * tile_tok, 0);
        unit_done(un);
        if (steps < 0) break;
        if (steps == 0) continue;
        const uint32_t set = __shfl_sync(0xFFFFFFFFu, units, 0) % Sh::kSets;
        const uint32_t kd = (uint32_t)k_desc + set * (kGroups * Sh::kTile / 16);
        ++units;
        const bool again = flags & kAgain, keep = flags & kKeep;
        const uint32_t base = __shfl_sync(0xFFFFFFFFu, count, 0) - (again ? 1u : 0u);
#pragma unroll 1
        for (int t = 0; t < steps && ok; ++t) {
          const int rows = min(tile_tok, first - t * tile_tok) * group;
          const uint32_t idesc = tc::idesc_f16_f32(BF16, kKeys, (uint32_t)((rows + 15) & ~15), false);
          const uint32_t q_slot = (base + t) % NQ;
          if (!again) {
            if (held && t == 0) tc::commit_one(issuer, &ctl.q_empty[(base - 1) % NQ]);
            ok = tc::wait_all<true>(&ctl.q_full[q_slot], ((base + t) / NQ) & 1, abort_flag, budget);
            if (!ok) break;
          }
          const uint32_t qd = (uint32_t)q_desc + q_slot * (Sh::kQ / 16);
#pragma unroll
          for (int w = 0; w < 2; ++w) {
            if (w >= tiles) break;
            uint64_t* k_empty = &ctl.k_empty[set * kGroups + w0 + w];
            if (t == 0) {
              ok = tc::wait_all<true>(&ctl.k_full[set * kGroups + w0 + w], seen >> (set * kGroups + w) & 1, abort_flag,
                                      budget);
              if (!ok) break;
              seen ^= 1u << (set * kGroups + w);
            }
            if (uses >> w & 1) {
              ok = tc::wait_all<true>(&ctl.s_empty[w0 + w], (uses >> (w + 4) & 1) ^ 1, abort_flag, budget);
              if (!ok) break;
            }
            uses = (uses | 1u << w) ^ 1u << (w + 4);
            tc::fence_after_sync();
#pragma unroll
            for (int c = 0; c < D / 16; ++c) {
              constexpr int kHalf = kKeys * 128 / 16;
              tc::mma_ss_one(issuer, tmem + (w0 + w) * 128,
                             desc(kd + w * (Sh::kTile / 16) + (c / 4) * kHalf + (c % 4) * 2),
                             desc(qd + (c / 4) * kHalf + (c % 4) * 2), idesc, c > 0);
            }
            tc::commit_one(issuer, &ctl.s_full[w0 + w]);
            if (t + 1 == steps) tc::commit_one(issuer, k_empty);
          }
          if (!ok) break;
          if (!keep) tc::commit_one(issuer, &ctl.q_empty[q_slot]);
          __syncwarp();
        }
        count = base + steps;
        held = keep;
      }
      if (!ok && lane == 0) {
        *abort_flag = 1;
        record_error(err, kDevErrTimeout);
      }
      if (issuer) tc::mma_drain(&ctl.drain[warp - kWarpMma]);  // TMEM is freed below
      __syncwarp();
    }
  } else {
    // ------------------------------------------------------------ exponentials and sums
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRegsMore));
    const int w = warp >> 2, r = threadIdx.x & 127;  // key tile, key of it = TMEM lane
    const uint32_t t_s = tmem + ((uint32_t)((warp & 3) * 32) << 16) + w * 128;
    const float sl = a.scale * kLog2e;
    const float2 sl2 = make_float2(sl, sl);
    uint32_t slot = NL - 1, phase = 1, used = 0;  // the query tile's lse; products that this warpgroup had
    bool held = false;            // the last tile's lse is not given back yet
    bool ok = true;
    Piece piece = {0, 0, 0, 0};
    // sum += 2^(s sl - lse), two columns at once
    auto add_weights = [&](float2& to, uint32_t s0, uint32_t s1, float l0, float l1) {
      float2 x = tc::fma_x2(make_float2(__uint_as_float(s0), __uint_as_float(s1)), sl2, make_float2(l0, l1));
      x.x = tc::exp2_approx(x.x);
      x.y = tc::exp2_approx(x.y);
      to = tc::add_x2(to, x);
    };
    for (uint32_t un = 0;; ++un) {
      ok = unit_wait(un);
      if (!ok) break;
      const Unit& u = ctl.unit[un % NU];  // (kept until its sums are written)
      const int steps = u.steps;
      if (steps < 0) break;
      const int flags = u.flags, len = u.len;
      const int j = u.p * kUnit + w * kKeys + r;
      const bool idle = w >= u.tiles;  // no key of this tile is one
      const int32_t id = j < len + u.m ? u.page[(w * kKeys + r) >> min(7, a.page_shift)] : -1;
      const bool add = id >= 0 && j < len && a.decay != 0.f, cut = flags & (kCutHead | kCutTail);
      if (cut) {
        if (!(flags & kCutHead)) piece = {u.s, u.p, u.hk, piece.flags | kBegins};
        else piece.flags |= kHas | (flags & kCutTail ? 0 : kEnds);
      }
      // what the weight was, under way while the products are waited for
      float* at = id >= 0 ? weight_at(a, id, j, u.hk) : nullptr;
      float old = 0.f;
      if (add && !cut) old = *at;
      float sum = 0.f;
      // the query tiles of which every row is one and sees every key of this warp
      int fast0 = 0, fast1 = 0;
      if (tile_tok * group > kRows - 16 && steps > 1) {
        const int j1 = (j | 31) - len;  // the warp's last key, counted from the first new token
        fast1 = u.m / tile_tok;
        if (a.tree)
          fast1 = j1 < 0 ? fast1 : 0;
        else if (j1 > 0)
          fast0 = (j1 + tile_tok - 1) / tile_tok;
        if (a.window > 0) {
          // its first key is in sight of a tile's last token
          const long long past = (long long)(j & ~31) - len + a.window;
          fast1 = past <= 0 ? 0 : (int)min((long long)fast1, past / tile_tok);
        }
      }
      const int t0 = u.first;
      for (int t = t0; t < t0 + steps; ++t) {
        if (!(flags & kAgain)) {
          if (held) {
            __syncwarp();
            if (lane == 0) tc::mbar_arrive(&ctl.l_empty[slot]);
          }
          if (++slot == NL) slot = 0, phase ^= 1;
          ok = tc::wait_all<false>(&ctl.l_full[slot], phase, abort_flag, budget);
          if (!ok) break;
        }
        held = flags & kKeep;
        if (!idle) {
          ok = tc::wait_all<false>(&ctl.s_full[w], used & 1, abort_flag, budget);
          if (!ok) break;
          ++used;
          tc::fence_after_sync();
          const float4* l4 = reinterpret_cast<const float4*>(ctl.neg_lse[slot]);
          if (t >= fast0 && t < fast1) {
            // every row of a whole product (what is behind the last has -lse -inf and
            // zeros for q): 32 columns are summed while the next are loaded
            uint32_t s[2][32];
            tc::tmem_ld32(t_s, s[0]);
            float2 part[4] = {};
#pragma unroll
            for (int q = 0; q < kRows / 32; ++q) {
              uint32_t(&v)[32] = s[q & 1];
              tc::tmem_ld_wait(v);
              if (q + 1 < kRows / 32) {
                tc::tmem_ld32(t_s + (q + 1) * 32, s[(q + 1) & 1]);
              } else {
                tc::fence_before_sync();
                __syncwarp();
                if (lane == 0) tc::mbar_arrive(&ctl.s_empty[w]);
              }
#pragma unroll
              for (int c = 0; c < 8; ++c) {
                const float4 l = l4[q * 8 + c];
                add_weights(part[c % 2 * 2], v[4 * c], v[4 * c + 1], l.x, l.y);
                add_weights(part[c % 2 * 2 + 1], v[4 * c + 2], v[4 * c + 3], l.z, l.w);
              }
            }
            const float2 x = tc::add_x2(tc::add_x2(part[0], part[1]), tc::add_x2(part[2], part[3]));
            sum += x.x + x.y;
          } else {
            const int i0 = t * tile_tok, toks = min(tile_tok, u.m - i0), cols = toks * group;
            // columns [lo, hi) see the key
            int lo = 0, hi = cols;
            if (!a.tree) {
              const int late = j - len - i0;  // tokens of the tile that come before the key
              lo = late <= 0 ? 0 : late >= toks ? cols : late * group;
              if (a.window > 0) {
                const long long past = (long long)late + a.window;
                hi = past <= 0 ? 0 : past >= toks ? cols : (int)past * group;
              }
            } else if (j >= len) {
              lo = cols;  // by their words, below
            }
            float some = 0.f;
#pragma unroll 1
            for (int c = 0; c < cols; c += 32) {
              uint32_t see = tc::span_bits(lo - c, hi - c);
              if (a.tree && j >= len && j - len < 64) {
                for (int i = c / group; i <= (c + 31) / group && i < toks; ++i)
                  if (a.tree[u.tok0 + i0 + i] >> (j - len) & 1)
                    see |= tc::span_bits(i * group - c, (i + 1) * group - c);
              }
              if (!__any_sync(0xFFFFFFFFu, see != 0)) continue;
              uint32_t v[32];
              tc::tmem_ld32(t_s + c, v);
              tc::tmem_ld_wait(v);
              if (__all_sync(0xFFFFFFFFu, see == ~0u)) {
                float2 part[2] = {};
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                  const float4 l = l4[c / 4 + i];
                  add_weights(part[0], v[4 * i], v[4 * i + 1], l.x, l.y);
                  add_weights(part[1], v[4 * i + 2], v[4 * i + 3], l.z, l.w);
                }
                const float2 x = tc::add_x2(part[0], part[1]);
                some += x.x + x.y;
              } else {
#pragma unroll
                for (int i = 0; i < 32; ++i) {
                  const float x = tc::exp2_approx(fmaf(__uint_as_float(v[i]), sl, ctl.neg_lse[slot][c + i]));
                  some += (see >> i) & 1 ? x : 0.f;
                }
              }
            }
            sum += some;
            tc::fence_before_sync();
            __syncwarp();
            if (lane == 0) tc::mbar_arrive(&ctl.s_empty[w]);
          }
        }
        if (!held) {
          __syncwarp();
          if (lane == 0) tc::mbar_arrive(&ctl.l_empty[slot]);
        }
      }
      if (!ok) break;
      if (cut)
        sc.sums[((int64_t)blockIdx.x * 2 + (flags & kCutHead ? 0 : 1)) * kUnit + w * kKeys + r] = sum;
      else if (id >= 0)
        *at = add ? fmaf(a.decay, old, sum) : sum;
      unit_done(un);
    }
    if (!ok && lane == 0) {
      *abort_flag = 1;
      record_error(err, kDevErrTimeout);
    }
    if (threadIdx.x == 0 && !whole_only) sc.piece[blockIdx.x] = piece;
  }
  tc::fence_before_sync();
  cta_sync();
  if (warp == kWarpMma) {
    tc::fence_after_sync();
    tc::tmem_dealloc(tmem, 512);
  }
}

// The sums of the unit that begins in CTA c and goes on behind it, in order.
__global__ void __launch_bounds__(kUnit) join_kernel(const WeightArgs a, const Scratch sc, int parts) {
  pdl_wait();
  pdl_trigger();
  const int k = threadIdx.x;
  int c = blockIdx.x;
  const Piece u = sc.piece[c];
  if (!(u.flags & kBegins)) return;
  float sum = sc.sums[((int64_t)c * 2 + 1) * kUnit + k];
  for (++c; c < parts; ++c) {
    const int flags = sc.piece[c].flags;
    if (flags & kHas) sum += sc.sums[(int64_t)c * 2 * kUnit + k];
    if (flags & kEnds) break;
  }
  const int j = u.p * kUnit + k, len = a.lens[u.s];
  if (j >= len + a.cu[u.s + 1] - a.cu[u.s]) return;
  const int32_t id = a.table[(int64_t)u.s * a.width + (j >> a.page_shift)];
  if (id < 0 || id >= a.pages) return;
  float* w = weight_at(a, id, j, u.hk);
  *w = j < len && a.decay != 0.f ? fmaf(a.decay, *w, sum) : sum;
}

inline int part_count() { return sm_count() > 0 ? sm_count() : 1; }

template <bool BF16, int D>
cudaError_t launch_all(const WeightArgs& a, const Scratch& sc, int parts, int* err, cudaStream_t s) {
  const int page = 1 << a.page_shift, group = a.heads / a.kv_heads, tile_tok = kRows / group;
  const bool head_first = a.ks.head <= a.ks.token;
  CUtensorMap kmap, qmap;
  if (!make_cache_map(&kmap, a.k_cache, BF16, D, page, a.kv_heads, a.pages, a.ks,
                      page < kKeys ? page : kKeys, head_first))
    return cudaErrorInvalidValue;
  // a full tile of queries comes by one copy where a token's heads lie within its stride
  const int64_t row = (int64_t)D * 2;
  const int64_t q_head = a.heads > 1 ? a.q_head : row;
  const int64_t q_tok = a.T > 1 ? a.q_tok : q_head * a.heads;
  const bool by_tma = q_tok >= (a.heads - 1) * q_head + row && a.T >= tile_tok;
  qmap = kmap;
  if (by_tma && !make_rows_map(&qmap, a.q, BF16, D, a.heads, a.T, q_head, q_tok, group, tile_tok))
    return cudaErrorInvalidValue;
  // Cutting units between CTAs costs the second launch; it pays where a request has
  // several query tiles a unit. (Told by the average: the host does not know the requests. A
  // prompt among many single tokens stays whole, and its units are the longest shares.)
  const bool whole = a.T <= (int64_t)2 * tile_tok * a.S;
  static int smem_set[64] = {0};
  cudaError_t e = ensure_dynamic_smem(weights_kernel<BF16, D>, Shape<D>::kSmem, smem_set);
  if (e != cudaSuccess) return e;
  e = launch_kernel(true, weights_kernel<BF16, D>, dim3(parts), dim3(kThreads), Shape<D>::kSmem, s, kmap,
                    qmap, a, sc, (int)head_first, (int)by_tma, (int)whole, role_wait_cycles(), err);
  if (e != cudaSuccess || whole) return e;
  return launch_kernel(true, join_kernel, dim3(parts), dim3(kUnit), 0, s, a, sc, parts);
}

inline size_t sums_at(int parts) { return ((size_t)parts * sizeof(Piece) + 255) / 256 * 256; }

}  // namespace

size_t weights_scratch_bytes() {
  const int parts = part_count();
  return sums_at(parts) + (size_t)parts * 2 * kUnit * sizeof(float);
}

cudaError_t launch_cache_weights(const WeightArgs& a, void* scratch, int* err, cudaStream_t s) {
  const int parts = part_count();
  char* p = static_cast<char*>(scratch);
  const Scratch sc = {reinterpret_cast<Piece*>(p), reinterpret_cast<float*>(p + sums_at(parts))};
  if (a.dtype == LMHEAD_BF16)
    return a.dim == 64 ? launch_all<true, 64>(a, sc, parts, err, s)
                       : launch_all<true, 128>(a, sc, parts, err, s);
  return a.dim == 64 ? launch_all<false, 64>(a, sc, parts, err, s)
                     : launch_all<false, 128>(a, sc, parts, err, s);
}

}  // namespace lmhead
