// Attention of a chunk of new tokens over a paged K/V cache.
//
// For token i of request s (len_s tokens cached before the chunk) and head a:
//   o = sum_j p_j v_j,  p = softmax_j(scale * q . k_j),  lse = log sum exp,
// over the keys the mask leaves: j <= len + i (and j > len + i - window), or
// the cached ones and those whose bit is set in the token's tree word. A row
// left with no key gives o = 0 and lse = -inf.
//
// A warp per (token, head): 32 keys at a time, a key per lane for the scores,
// running maximum and sum of the softmax in 32 bits, then D/32 dimensions per
// lane for the sum over values.
#include <cuda_fp16.h>

#include "common.cuh"
#include "kernels.h"

namespace lmhead {
namespace {

template <bool BF16> __device__ __forceinline__ float2 pair_to_float(uint32_t w) {
  if (BF16) return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xFFFF0000u));
  return __half22float2(*reinterpret_cast<const __half2*>(&w));
}

template <bool BF16, int D>
__global__ void __launch_bounds__(128) attention_rows_kernel(AttnArgs a, int* err) {
  __shared__ float qs[4][D];
  pdl_wait();
  pdl_trigger();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int64_t unit = (int64_t)blockIdx.x * 4 + warp;
  if (unit >= (int64_t)a.T * a.heads) return;
  const int t = (int)(unit / a.heads), head = (int)(unit - (int64_t)t * a.heads);
  const int kvh = head / (a.heads / a.kv_heads);
  uint16_t* o = static_cast<uint16_t*>(a.out) + unit * D;
  // the request: the last one that starts at or before t
  int lo = 0, hi = a.S;
  while (hi - lo > 1) {
    const int mid = (lo + hi) / 2;
    if (a.cu[mid] <= t) lo = mid; else hi = mid;
  }
  const int s = lo, i = t - a.cu[s], fresh = a.cu[s + 1] - a.cu[s];
  if (i < 0 || i >= fresh) return;
  constexpr int E = D / 32;
  float acc[E];
#pragma unroll
  for (int e = 0; e < E; ++e) acc[e] = 0.f;
  float m = -__builtin_huge_valf(), l = 0.f;
  bool bad = false;
  const int len = max(a.lens[s], 0);
  const char* q = static_cast<const char*>(a.q) + t * a.q_tok + head * a.q_head;
  for (int e = lane; e < D / 2; e += 32) {
    const float2 f = pair_to_float<BF16>(*reinterpret_cast<const uint32_t*>(q + e * 4));
    qs[warp][2 * e] = f.x;
    qs[warp][2 * e + 1] = f.y;
  }
  __syncwarp();
  const uint64_t bits = a.tree ? a.tree[t] : 0;
  const int end = a.tree ? len + min(fresh, 64) : len + i + 1;
  const int begin = a.window > 0 ? max(0, len + i + 1 - a.window) : 0;
  for (int j0 = begin; j0 < end; j0 += 32) {
    const int j = j0 + lane;
    bool see = j < end;
    if (a.tree && j >= len) see = see && ((bits >> (j - len)) & 1);
    const int pg = j >> a.page_shift;
    int32_t id = -1;
    if (j < end) {
      if (pg < a.width) id = a.table[(size_t)s * a.width + pg];
      if (id < 0 || id >= a.pages) {
        bad = true;
        id = -1;
      }
    }
    const int64_t off = j & ((1 << a.page_shift) - 1);
    float x = -__builtin_huge_valf();
    if (see && id >= 0) {
      const char* k = static_cast<const char*>(a.k_cache) + id * a.ks.page + off * a.ks.token +
                      kvh * a.ks.head;
      x = 0.f;
      for (int c = 0; c < D / 8; ++c) {
        const uint4 v = *reinterpret_cast<const uint4*>(k + c * 16);
        const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const float2 f = pair_to_float<BF16>(w[e]);
          x = fmaf(f.x, qs[warp][c * 8 + 2 * e], x);
          x = fmaf(f.y, qs[warp][c * 8 + 2 * e + 1], x);
        }
      }
      x *= a.scale;
    }
    const float nm = fmaxf(m, warp_max(x)), ref = nm == -__builtin_huge_valf() ? 0.f : nm;
    const float p = expf(x - ref), f = expf(m - ref);
    l = l * f + warp_sum(p);
    m = nm;
#pragma unroll
    for (int e = 0; e < E; ++e) acc[e] *= f;
    const int64_t vo = id >= 0 ? id * a.vs.page + off * a.vs.token + kvh * a.vs.head : -1;
    for (int y = 0; y < 32; ++y) {
      const float py = __shfl_sync(0xFFFFFFFFu, p, y);
      const int64_t at = __shfl_sync(0xFFFFFFFFu, vo, y);
      const bool sy = __shfl_sync(0xFFFFFFFFu, (int)see, y);
      if (!sy || at < 0) continue;
      const char* v = static_cast<const char*>(a.v_cache) + at + lane * E * 2;
#pragma unroll
      for (int e = 0; e < E; e += 2) {
        const float2 z = pair_to_float<BF16>(*reinterpret_cast<const uint32_t*>(v + e * 2));
        acc[e] = fmaf(py, z.x, acc[e]);
        acc[e + 1] = fmaf(py, z.y, acc[e + 1]);
      }
    }
  }
  bad = __any_sync(0xFFFFFFFFu, bad);
  if (bad && lane == 0) record_error(err, kDevErrBadId);
  const float inv = l == 0.f ? 0.f : 1.f / l;
#pragma unroll
  for (int e = 0; e < E; ++e) {
    const float v = bad ? __int_as_float(0x7fc00000) : acc[e] * inv;
    if (BF16)
      reinterpret_cast<__nv_bfloat16*>(o)[lane * E + e] = __float2bfloat16(v);
    else
      reinterpret_cast<__half*>(o)[lane * E + e] = __float2half(v);
  }
  if (a.lse && lane == 0)
    a.lse[unit] = bad ? __int_as_float(0x7fc00000)
                      : (l == 0.f ? -__builtin_huge_valf() : m + logf(l));
}

}  // namespace

size_t attention_scratch_bytes(int S, int T, int heads, int kv_heads, int dim) {
  (void)S, (void)T, (void)heads, (void)kv_heads, (void)dim;
  return 256;
}

cudaError_t launch_attention(const AttnArgs& a, void* scratch, int* err, cudaStream_t s) {
  (void)scratch;
  const unsigned grid = (unsigned)(((int64_t)a.T * a.heads + 3) / 4);
#define RUN(B, D) return launch_kernel(true, attention_rows_kernel<B, D>, dim3(grid), dim3(128), 0, s, a, err)
  if (a.dtype == LMHEAD_BF16) {
    if (a.dim == 64) RUN(true, 64);
    RUN(true, 128);
  }
  if (a.dim == 64) RUN(false, 64);
  RUN(false, 128);
#undef RUN
}

}  // namespace lmhead
