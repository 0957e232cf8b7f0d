// Rotary positions of a step's queries and keys.
//
// A pair (a, b) of a head at position p turns by the angle t = 2 pi frac(p f):
//   (a, b) -> m (a cos t - b sin t, b cos t + a sin t),
// or by -t for the gradient (the rotation's transpose). A frequency f is given
// in units of 2^-64 turns, so the product with the position, taken modulo 2^64,
// is the fraction of a turn exactly, however far the position; its leading 32
// bits become a float in [-1, 1) half turns, which sincospi takes without any
// reduction of its own. The angle is off by 2 pi (2^-33 + 2^-26) at most.
//
// Bound by memory: every element is read and written once. A thread takes 16
// bytes of either half of a pair's places and keeps their sines and cosines for
// several heads of its token (their cost is that of about four heads), four of them
// under way together. Measured: 16384 tokens x 40 heads of 128 bf16 elements 52 us for
// 335 MB (6.4 TB/s; 90 with the elements unpacked one by one and two CTAs an SM, 58 to
// 72 with more CTAs and fewer loads of each thread); 5001 x 72 of 64 fp32 31 us for
// 184 MB (5.9 TB/s); a decoding step of 8 tokens 4 us, a launch's latency.
#include <cuda_fp16.h>

#include "common.cuh"
#include "kernels.h"
#include "lmhead.h"

namespace lmhead {
namespace {

constexpr int kThreads = 256;
constexpr int kResident = 3;  // CTAs an SM, of 80 registers a thread

// V elements as one load or store: 16 bytes, or (V = 1) the element itself.
template <int DT, int V> struct Pack;
template <int DT> struct Pack<DT, 8> {  // of 16 bits each
  uint4 v;
  __device__ __forceinline__ void get(float* f) const {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if (DT == LMHEAD_BF16) {
        f[2 * i] = __uint_as_float(w[i] << 16);
        f[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
      } else {
        const float2 x = __half22float2(*reinterpret_cast<const __half2*>(&w[i]));
        f[2 * i] = x.x;
        f[2 * i + 1] = x.y;
      }
    }
  }
  __device__ __forceinline__ void set(const float* f) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if (DT == LMHEAD_BF16)
        asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(w[i]) : "f"(f[2 * i + 1]), "f"(f[2 * i]));
      else
        asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(w[i]) : "f"(f[2 * i + 1]), "f"(f[2 * i]));
    }
    v = make_uint4(w[0], w[1], w[2], w[3]);
  }
};
template <> struct Pack<LMHEAD_FP32, 4> {
  float4 v;
  __device__ __forceinline__ void get(float* f) const { f[0] = v.x; f[1] = v.y; f[2] = v.z; f[3] = v.w; }
  __device__ __forceinline__ void set(const float* f) { v = make_float4(f[0], f[1], f[2], f[3]); }
};
template <> struct Pack<LMHEAD_FP32, 1> {
  float v;
  __device__ __forceinline__ void get(float* f) const { f[0] = v; }
  __device__ __forceinline__ void set(const float* f) { v = f[0]; }
};
template <int DT> struct Pack<DT, 1> {
  uint16_t v;
  __device__ __forceinline__ void get(float* f) const {
    f[0] = DT == LMHEAD_BF16 ? __uint_as_float((uint32_t)v << 16) : __half2float(__ushort_as_half(v));
  }
  __device__ __forceinline__ void set(const float* f) {
    v = DT == LMHEAD_BF16 ? __bfloat16_as_ushort(__float2bfloat16_rn(f[0]))
                          : __half_as_ushort(__float2half_rn(f[0]));
  }
};

// Thread x of a token: place u of a row (of `units`, the last of them copies
// what does not turn) and the heads h0, h0 + groups, ...
template <int DT, int V, bool PAIRS>
__global__ void __launch_bounds__(kThreads, V == 1 ? 4 : kResident)
rotary_kernel(const RotaryArgs a, int units, int groups) {
  using P = Pack<DT, V>;
  constexpr int E = DT == LMHEAD_FP32 ? 4 : 2;  // bytes of an element
  pdl_wait();
  pdl_trigger();
  const int64_t x = (int64_t)blockIdx.x * kThreads + threadIdx.x;
  const int per = units * groups;
  const int64_t t = x / per;
  if (t >= a.T) return;
  const int rest = (int)(x - t * per);
  const int h0 = rest / units, u = rest - h0 * units;
  const int32_t pos = a.pos[t];
  if (pos < 0) return;
  const int half = a.rot / 2, turning = half / V;
  const int heads = a.heads + a.kv_heads;
  const bool copy = u >= turning;
  // the two packs of the place: V pairs, or 2 V neighbouring elements behind the part that turns
  int c0, c1;
  if (copy) {
    c0 = a.rot + (u - turning) * 2 * V;
    c1 = c0 + V < a.dim ? c0 + V : -1;
  } else if (PAIRS) {
    c0 = u * 2 * V;
    c1 = c0 + V;
  } else {
    c0 = u * V;
    c1 = c0 + half;
  }
  float co[V], si[V];
  if (!copy) {
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const uint64_t turn = (uint64_t)(uint32_t)pos * (uint64_t)a.turns[u * V + i];
      // rounded to 32 bits; past the last it wraps to the first, as turns do
      const int32_t part = (int32_t)(uint32_t)((turn + 0x80000000ull) >> 32);
      sincospif((float)part * 0x1p-31f, &si[i], &co[i]);
      co[i] *= a.magnitude;
      si[i] *= a.backward ? -a.magnitude : a.magnitude;
    }
  }
  // (byte offsets of a token's first heads)
  const char *q = static_cast<const char*>(a.q) + t * a.q_tok * E, *k = static_cast<const char*>(a.k) + t * a.k_tok * E;
  char *qo = static_cast<char*>(a.qo) + t * a.qo_tok * E, *ko = static_cast<char*>(a.ko) + t * a.ko_tok * E;
  constexpr int N = 4;  // heads under way together
#pragma unroll 1
  for (int h = h0; h < heads; h += N * groups) {
    P v0[N], v1[N];
#pragma unroll
    for (int n = 0; n < N; ++n) {
      const int hn = h + n * groups;
      if (hn >= heads) break;
      const char* src = hn < a.heads ? q + hn * a.q_head * E : k + (hn - a.heads) * a.k_head * E;
      v0[n] = *reinterpret_cast<const P*>(src + c0 * E);
      if (c1 >= 0) v1[n] = *reinterpret_cast<const P*>(src + c1 * E);
    }
#pragma unroll
    for (int n = 0; n < N; ++n) {
      const int hn = h + n * groups;
      if (hn >= heads) break;
      if (!copy) {
        float f[2 * V];  // v0's, then v1's
        v0[n].get(f);
        v1[n].get(f + V);
#pragma unroll
        for (int i = 0; i < V; ++i) {
          float &fa = PAIRS ? f[2 * i] : f[i], &fb = PAIRS ? f[2 * i + 1] : f[V + i];
          const float x = fa, y = fb;
          fa = fmaf(x, co[i], -(y * si[i]));
          fb = fmaf(y, co[i], x * si[i]);
        }
        v0[n].set(f);
        v1[n].set(f + V);
      }
      char* dst = hn < a.heads ? qo + hn * a.qo_head * E : ko + (hn - a.heads) * a.ko_head * E;
      *reinterpret_cast<P*>(dst + c0 * E) = v0[n];
      if (c1 >= 0) *reinterpret_cast<P*>(dst + c1 * E) = v1[n];
    }
  }
}

template <int DT, int V>
cudaError_t launch_packs(const RotaryArgs& a, cudaStream_t s) {
  const bool in_place = a.q == a.qo && (!a.k || a.k == a.ko);
  const int rest = in_place ? 0 : a.dim - a.rot;
  const int units = a.rot / 2 / V + (rest + 2 * V - 1) / (2 * V);
  const int heads = a.heads + a.kv_heads;
  // enough threads to fill the GPU, heads shared out no further than that and no
  // coarser than eight a thread
  const int64_t want = (int64_t)(sm_count() > 0 ? sm_count() : 1) * 1024;
  int64_t groups = want / ((int64_t)a.T * units);
  groups = groups < (heads + 7) / 8 ? (heads + 7) / 8 : groups > heads ? heads : groups;
  const int64_t blocks = ((int64_t)a.T * units * groups + kThreads - 1) / kThreads;
  if (blocks > INT32_MAX) return cudaErrorInvalidValue;
  return launch_kernel(true, a.interleaved ? rotary_kernel<DT, V, true> : rotary_kernel<DT, V, false>,
                       dim3((unsigned)blocks), dim3(kThreads), 0, s, a, units, (int)groups);
}

template <int DT>
cudaError_t launch_typed(const RotaryArgs& a, cudaStream_t s) {
  constexpr int V = DT == LMHEAD_FP32 ? 4 : 8;  // 16 bytes
  const uintptr_t at = reinterpret_cast<uintptr_t>(a.q) | reinterpret_cast<uintptr_t>(a.qo) |
                       reinterpret_cast<uintptr_t>(a.k) | reinterpret_cast<uintptr_t>(a.ko);
  const int64_t st = a.q_tok | a.q_head | a.k_tok | a.k_head | a.qo_tok | a.qo_head | a.ko_tok | a.ko_head;
  // whole packs of 16 bytes where addresses, strides and the parts of a row allow them
  const bool packs = (at & 15) == 0 && st % V == 0 && a.rot % (2 * V) == 0 && a.dim % V == 0;
  return packs ? launch_packs<DT, V>(a, s) : launch_packs<DT, 1>(a, s);
}

}  // namespace

cudaError_t launch_rotary(const RotaryArgs& a, cudaStream_t s) {
  switch (a.dtype) {
    case LMHEAD_BF16: return launch_typed<LMHEAD_BF16>(a, s);
    case LMHEAD_FP16: return launch_typed<LMHEAD_FP16>(a, s);
    default: return launch_typed<LMHEAD_FP32>(a, s);
  }
}

}  // namespace lmhead
