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
// several heads of its token (their cost is that of about four heads).
#include <cuda_fp16.h>

#include "common.cuh"
#include "kernels.h"
#include "lmhead.h"

namespace lmhead {
namespace {

constexpr int kThreads = 256;

template <int DT> struct Elem;
template <> struct Elem<LMHEAD_BF16> {
  using type = uint16_t;
  static __device__ float load(uint16_t x) { return __uint_as_float((uint32_t)x << 16); }
  static __device__ uint16_t store(float f) { return __bfloat16_as_ushort(__float2bfloat16_rn(f)); }
};
template <> struct Elem<LMHEAD_FP16> {
  using type = uint16_t;
  static __device__ float load(uint16_t x) { return __half2float(__ushort_as_half(x)); }
  static __device__ uint16_t store(float f) { return __half_as_ushort(__float2half_rn(f)); }
};
template <> struct Elem<LMHEAD_FP32> {
  using type = float;
  static __device__ float load(float x) { return x; }
  static __device__ float store(float f) { return f; }
};

// V elements as one load or store (V = 1: the element itself).
template <typename T, int V> struct alignas(sizeof(T) * V) Pack {
  T x[V];
};

// Thread x of a token: place u of a row (of `units`, the last of them copies
// what does not turn) and the heads h0, h0 + groups, ...
template <int DT, int V, bool PAIRS>
__global__ void __launch_bounds__(kThreads)
rotary_kernel(const RotaryArgs a, int units, int groups) {
  using E = Elem<DT>;
  using T = typename E::type;
  using P = Pack<T, V>;
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
  auto in_row = [&](int h) {
    return h < a.heads ? static_cast<const T*>(a.q) + t * a.q_tok + h * a.q_head
                       : static_cast<const T*>(a.k) + t * a.k_tok + (h - a.heads) * a.k_head;
  };
  auto out_row = [&](int h) {
    return h < a.heads ? static_cast<T*>(a.qo) + t * a.qo_tok + h * a.qo_head
                       : static_cast<T*>(a.ko) + t * a.ko_tok + (h - a.heads) * a.ko_head;
  };
  constexpr int N = 4;  // heads under way together
  for (int h = h0; h < heads; h += N * groups) {
    P v0[N], v1[N];
#pragma unroll
    for (int n = 0; n < N; ++n) {
      const int hn = h + n * groups;
      if (hn >= heads) break;
      const T* src = in_row(hn);
      v0[n] = *reinterpret_cast<const P*>(src + c0);
      if (c1 >= 0) v1[n] = *reinterpret_cast<const P*>(src + c1);
    }
#pragma unroll
    for (int n = 0; n < N; ++n) {
      const int hn = h + n * groups;
      if (hn >= heads) break;
      if (!copy) {
#pragma unroll
        for (int i = 0; i < V; ++i) {
          T& ra = PAIRS ? (2 * i < V ? v0[n].x[(2 * i) % V] : v1[n].x[(2 * i) % V]) : v0[n].x[i];
          T& rb = PAIRS ? (2 * i + 1 < V ? v0[n].x[(2 * i + 1) % V] : v1[n].x[(2 * i + 1) % V]) : v1[n].x[i];
          const float fa = E::load(ra), fb = E::load(rb);
          ra = E::store(fmaf(fa, co[i], -(fb * si[i])));
          rb = E::store(fmaf(fb, co[i], fa * si[i]));
        }
      }
      T* dst = out_row(hn);
      *reinterpret_cast<P*>(dst + c0) = v0[n];
      if (c1 >= 0) *reinterpret_cast<P*>(dst + c1) = v1[n];
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
  constexpr int V = 16 / (int)sizeof(typename Elem<DT>::type);
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
