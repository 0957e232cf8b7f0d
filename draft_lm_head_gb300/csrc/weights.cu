// How much attention each cached token has drawn, summed up.
//
// For key j of request s and K/V head a, over the new tokens i and the heads h of
// a that see it:
//   w_j = decay w_j [j < len_s] + sum_i,h exp(scale q_ih . k_j - lse_ih),
// with lse as attention left it, so that a token's weights over all keys sum to 1.
//
// A CTA takes 64 keys of one request and head: they are read once, to shared
// memory, and the queries in turn; a thread has a key and every fourth row.
#include <cuda_fp16.h>

#include "common.cuh"
#include "kernels.h"
#include "lmhead.h"

namespace lmhead {
namespace {

constexpr int kKeys = 64, kGroups = 4, kThreads = kKeys * kGroups, kRows = 16;

template <bool BF16> __device__ __forceinline__ float load16(const char* p) {
  const uint16_t x = *reinterpret_cast<const uint16_t*>(p);
  return BF16 ? __uint_as_float((uint32_t)x << 16) : __half2float(__ushort_as_half(x));
}

template <bool BF16, int D>
__global__ void __launch_bounds__(kThreads)
weights_kernel(const WeightArgs a, int* err) {
  __shared__ float ks[kKeys][D + 1];
  __shared__ float qs[kRows][D];
  __shared__ float lse[kRows];
  __shared__ float part[kGroups][kKeys];
  pdl_wait();
  pdl_trigger();
  const int tid = threadIdx.x, x = tid % kKeys, grp = tid / kKeys;
  const int hk = blockIdx.y, group = a.heads / a.kv_heads;
  const int j = blockIdx.x * kKeys + x;
  __shared__ int bad;
  if (tid == 0) bad = 0;
  cta_sync();
  for (int s = tid; s < a.S; s += kThreads)
    if (a.cu[s] < 0 || a.cu[s + 1] < a.cu[s] || a.cu[s + 1] > a.T) bad = 1;
  cta_sync();
  if (bad) {
    if (tid == 0) record_error(err, kDevErrBadId);
    return;
  }
  for (int s = blockIdx.z; s < a.S; s += gridDim.z) {
    if (a.granted && a.granted[s] == 0) continue;
    const int tok0 = a.cu[s], end = a.cu[s + 1], len = a.lens[s];
    const int m = end - tok0;
    if (len < 0 || len > (a.width << a.page_shift) - m) {
      if (tid == 0) record_error(err, kDevErrBadId);
      continue;
    }
    const int kend = len + m;
    if ((int)blockIdx.x * kKeys >= kend) continue;
    // the key's place
    const int off = j & ((1 << a.page_shift) - 1);
    int32_t id = -1;
    if (j < kend) {
      id = a.table[(int64_t)s * a.width + (j >> a.page_shift)];
      if (id < 0 || id >= a.pages) {
        record_error(err, kDevErrBadId);
        id = -1;
      }
    }
    cta_sync();
    if (id >= 0) {
      const char* k = static_cast<const char*>(a.k_cache) + id * a.ks.page + off * a.ks.token + hk * a.ks.head;
      for (int d = grp; d < D; d += kGroups) ks[x][d] = load16<BF16>(k + d * 2);
    }
    float sum = 0.f;
    const int rows = m * group;
    for (int r0 = 0; r0 < rows; r0 += kRows) {
      cta_sync();
      for (int e = tid; e < kRows * D; e += kThreads) {
        const int r = r0 + e / D, d = e % D;
        if (r >= rows) break;
        const char* q = static_cast<const char*>(a.q) + (int64_t)(tok0 + r / group) * a.q_tok +
                        (int64_t)(hk * group + r % group) * a.q_head;
        qs[e / D][d] = load16<BF16>(q + d * 2);
      }
      if (tid < kRows && r0 + tid < rows) {
        const int r = r0 + tid;
        lse[tid] = a.lse[(int64_t)(tok0 + r / group) * a.heads + hk * group + r % group];
      }
      cta_sync();
      for (int y = grp; y < kRows && r0 + y < rows; y += kGroups) {
        const int i = (r0 + y) / group;
        bool see;
        if (a.tree) {
          see = j < len || (j - len < 64 && (a.tree[tok0 + i] >> (j - len) & 1));
        } else {
          see = j <= len + i && (a.window == 0 || j > len + i - a.window);
        }
        if (!see || lse[y] == -INFINITY) continue;
        float dot = 0.f;
        for (int d = 0; d < D; ++d) dot = fmaf(qs[y][d], ks[x][d], dot);
        sum += expf(fmaf(dot, a.scale, -lse[y]));
      }
    }
    part[grp][x] = sum;
    cta_sync();
    if (grp == 0 && id >= 0) {
      float* w = reinterpret_cast<float*>(static_cast<char*>(a.weights) + id * a.ws.page +
                                          off * a.ws.token + hk * a.ws.head);
      const float fresh = (part[0][x] + part[1][x]) + (part[2][x] + part[3][x]);
      *w = j < len && a.decay != 0.f ? fmaf(a.decay, *w, fresh) : fresh;
    }
    cta_sync();
  }
}

}  // namespace

size_t weights_scratch_bytes(int) { return 256; }

cudaError_t launch_cache_weights(const WeightArgs& a, void*, int* err, cudaStream_t s) {
  const dim3 grid((((unsigned)a.width << a.page_shift) + kKeys - 1) / kKeys, a.kv_heads,
                  a.S < 65535 ? a.S : 65535);
  if (a.dtype == LMHEAD_BF16)
    return a.dim == 64 ? launch_kernel(true, weights_kernel<true, 64>, grid, dim3(kThreads), 0, s, a, err)
                       : launch_kernel(true, weights_kernel<true, 128>, grid, dim3(kThreads), 0, s, a, err);
  return a.dim == 64 ? launch_kernel(true, weights_kernel<false, 64>, grid, dim3(kThreads), 0, s, a, err)
                     : launch_kernel(true, weights_kernel<false, 128>, grid, dim3(kThreads), 0, s, a, err);
}

}  // namespace lmhead
