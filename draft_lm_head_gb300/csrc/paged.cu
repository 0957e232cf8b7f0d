// The pages of a paged K/V cache: which pages and slots a step's new tokens
// get (block tables and slot maps, from request lengths alone).
#include <cuda_runtime.h>
#include <stdint.h>

#include "common.cuh"
#include "kernels.h"

namespace lmhead {
namespace {

// ---- page plan
// With held = ceil(len/P) and need = ceil((len+new)/P) - held, request s gets
// the pages free[F-1-e_s-j], j < need_s, e_s the sum of the needs before it.
// A CTA takes kPlanReqs consecutive requests and sums the needs and the new
// tokens of every request before its first one by itself (8 bytes a request
// from L2), so the whole plan is one launch with no state between CTAs; the
// tokens of a CTA's requests are spread over gridDim.y CTAs when there are
// many. Bound by latency: 8 us for 64 requests of a token each, 11-12 us for 1500
// requests and 525000 new tokens (4 + 4 bytes written a token). The sums of all
// CTAs together grow with the square of the requests: 50 us for 16384, 2 ms
// for 131072, 120 ms for 2^20.
constexpr int kPlanThreads = 256;
constexpr int kPlanReqs = 8;

struct Plan {
  int64_t need, fresh;  // pages to take, tokens to place
  bool fits;
};

__device__ __forceinline__ Plan plan_of(int32_t len, int32_t fresh, int page, int width) {
  Plan p;
  const bool sane = len >= 0 && fresh >= 0;
  const int64_t l = sane ? len : 0, m = sane ? fresh : 0;
  p.fits = sane && l + m <= min((int64_t)width * page, (int64_t)INT32_MAX - page);
  p.fresh = fresh > 0 ? fresh : 0;
  // a page less one added, lengths that fit stay within 32 bits
  const uint32_t up = (uint32_t)page - 1u;
  p.need = p.fits ? ((uint32_t)(l + m) + up) / (uint32_t)page - ((uint32_t)l + up) / (uint32_t)page : 0;
  return p;
}

__device__ __forceinline__ int64_t warp_sum64(int64_t v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
  return v;
}

__global__ void __launch_bounds__(kPlanThreads)
page_plan_kernel(const int32_t* lens, const int32_t* fresh, int S, int32_t* table, int width,
                 const int32_t* free_pages, int free_cap, const int32_t* free_count, int page,
                 int T, int32_t* slots, int32_t* positions, int32_t* cu, int32_t* granted,
                 int32_t* free_left, int* err) {
  __shared__ int64_t sh_need[kPlanThreads / 32], sh_new[kPlanThreads / 32];
  __shared__ int64_t r_excl[kPlanReqs], r_cu[kPlanReqs + 1];
  __shared__ int r_held[kPlanReqs], r_need[kPlanReqs], r_len[kPlanReqs], r_ok[kPlanReqs];
  pdl_wait();
  pdl_trigger();
  const int tid = threadIdx.x, first = blockIdx.x * kPlanReqs;
  const int count = min(kPlanReqs, S - first);
  int64_t a = 0, b = 0;
  for (int s = tid; s < first; s += kPlanThreads) {
    const Plan p = plan_of(lens[s], fresh[s], page, width);
    a += p.need;
    b += p.fresh;
  }
  a = warp_sum64(a);
  b = warp_sum64(b);
  if ((tid & 31) == 0) {
    sh_need[tid >> 5] = a;
    sh_new[tid >> 5] = b;
  }
  cta_sync();
  const int64_t F = max(0, min(*free_count, free_cap));
  if (tid == 0) {
    int64_t excl = 0, c = 0;
    for (int w = 0; w < kPlanThreads / 32; ++w) {
      excl += sh_need[w];
      c += sh_new[w];
    }
    const int64_t before = excl;
    int64_t taken = excl;  // the largest running sum that still fits in F
    for (int i = 0; i < count; ++i) {
      const Plan p = plan_of(lens[first + i], fresh[first + i], page, width);
      const bool ok = p.fits && (p.need == 0 || excl + p.need <= F);
      r_excl[i] = excl;
      r_cu[i] = c;
      r_len[i] = lens[first + i];
      r_held[i] = ok ? (int)(((int64_t)r_len[i] + page - 1) / page) : 0;
      r_need[i] = ok ? (int)p.need : 0;
      r_ok[i] = ok;
      excl += p.need;
      if (excl <= F) taken = excl;
      c += p.fresh;
    }
    r_cu[count] = c;
    if (blockIdx.y == 0) {
      // the free count after the plan: written by the CTA in whose requests the
      // running sum passes F, or by the last one
      if (before <= F && (excl > F || first + count == S)) *free_left = (int32_t)(F - taken);
      if (first == 0) cu[0] = 0;
      if (first + count == S && c > T) record_error(err, kDevErrBadId);
    }
  }
  cta_sync();
  if (blockIdx.y == 0) {
    if (tid < count) {
      const int64_t c = r_cu[tid + 1];
      cu[first + tid + 1] = (int32_t)(c < INT32_MAX ? c : INT32_MAX);
      granted[first + tid] = r_ok[tid];
    }
    for (int i = tid >> 5; i < count; i += kPlanThreads / 32)
      for (int j = tid & 31; j < r_need[i]; j += 32)
        table[(size_t)(first + i) * width + r_held[i] + j] = free_pages[F - 1 - r_excl[i] - j];
  }
  // slots and positions of the CTA's tokens; the last CTA also clears what is
  // left of the buffers. Held pages are read from the table and new ones from
  // the free list, so nothing read here is written above.
  const int64_t t0 = r_cu[0], t1 = min(r_cu[count], (int64_t)T);
  const int64_t end = first + count == S ? (int64_t)T : t1;
  int i = 0;
  for (int64_t t = t0 + blockIdx.y * kPlanThreads + tid; t < end;
       t += (int64_t)gridDim.y * kPlanThreads) {
    int32_t slot = -1, pos = -1;
    if (t < t1) {
      while (t >= r_cu[i + 1]) ++i;
      if (r_ok[i]) {
        pos = (int32_t)(r_len[i] + (t - r_cu[i]));
        const int pg = pos / page, at = pg - r_held[i];
        const int32_t id = at < 0 ? table[(size_t)(first + i) * width + pg]
                                  : free_pages[F - 1 - r_excl[i] - at];
        slot = id * page + (pos - pg * page);
      }
    }
    slots[t] = slot;
    positions[t] = pos;
  }
}

}  // namespace

cudaError_t launch_page_plan(const int32_t* lens, const int32_t* fresh, int S, int32_t* table,
                             int width, const int32_t* free_pages, int free_cap,
                             const int32_t* free_count, int page, int T, int32_t* slots,
                             int32_t* positions, int32_t* cu, int32_t* granted,
                             int32_t* free_left, int* err, cudaStream_t s) {
  const int groups = (S + kPlanReqs - 1) / kPlanReqs;
  int64_t y = (T / groups + 4 * kPlanThreads - 1) / (4 * kPlanThreads);
  y = y < 1 ? 1 : (y > 1024 ? 1024 : y);
  return launch_kernel(true, page_plan_kernel, dim3(groups, (unsigned)y), dim3(kPlanThreads), 0, s,
                       lens, fresh, S, table, width, free_pages, free_cap, free_count, page, T,
                       slots, positions, cu, granted, free_left, err);
}

}  // namespace lmhead
