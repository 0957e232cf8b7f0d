// Products of hidden vectors with rows of 4-bit codes and group scales:
//   y[m, i] = sum_G ( s[i,G] sum_{k in G} (c[i,k] - 8) h[m,k] + o[i,G] H[m,G] ),
// H[m,G] = sum_{k in G} h[m,k]; o = 0 for symmetric codes, and min + 8 s for
// codes with an offset (w = c s + min).
//
// Bound by reading the codes: d/2 + 2 d/group bytes a row. Every code costs an
// unpack, so the products have to be cheap: a code minus 8 is exact in 16
// bits, and a warp multiplies 16 rows x 16 codes with up to 8 hidden vectors
// in one matrix instruction from registers (products exact, sums in 32 bits).
// The codes go from global memory to the operand registers with no shuffle
// and no shared memory: the sum over k may take k in any order, so the order
// in which a lane's own codes unpack is the order of k, and h is laid out to
// match once per CTA. Group sums are scaled in 32 bits after the matrix
// products; no weight is ever rounded. (Operands of the tcgen05 instructions
// would have to be written to shared or tensor memory first, at a store per
// two codes; here they never leave registers.)
//   Unpacking a 32-bit word of 8 codes: (w >> 4j) & 0x000f000f joined with the
// bit pattern of 128 (bf16) or 1024 (fp16), where one unit is the lowest
// mantissa bit, gives 128 + c (1024 + c) for codes j and j + 4; one packed
// subtraction leaves c - 8.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "common.cuh"
#include "kernels.h"

namespace lmhead {
namespace {

constexpr int kBlockK = 128;  // codes of a row that four lanes take together
constexpr int kRowsWarp = 32;

template <bool BF16> struct Half2 {
  // codes j and j + 4 of word w, minus 8
  static __device__ __forceinline__ uint32_t codes(uint32_t w, int j) {
    uint32_t v = ((w >> (4 * j)) & 0x000f000fu) | (BF16 ? 0x43004300u : 0x64006400u);
    if (BF16) {
      const __nv_bfloat162 r = __hsub2(*reinterpret_cast<__nv_bfloat162*>(&v),
                                       __floats2bfloat162_rn(136.f, 136.f));
      return *reinterpret_cast<const uint32_t*>(&r);
    }
    const __half2 r = __hsub2(*reinterpret_cast<__half2*>(&v), __floats2half2_rn(1032.f, 1032.f));
    return *reinterpret_cast<const uint32_t*>(&r);
  }
  static __device__ __forceinline__ float to_float(uint16_t b) {
    if (BF16) return __uint_as_float((uint32_t)b << 16);
    return __half2float(__ushort_as_half(b));
  }
  static __device__ __forceinline__ void mma(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                             uint32_t a3, uint32_t b0, uint32_t b1) {
    if (BF16)
      asm volatile(
          "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
          "{%8,%9}, {%0,%1,%2,%3};"
          : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
          : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
    else
      asm volatile(
          "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
          "{%8,%9}, {%0,%1,%2,%3};"
          : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
          : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
  }
};

// Word i (of 4) of lane chunk t in a 128-code block, so that each matrix
// instruction stays within one group: bytes t*16 + i*4 for groups of 128,
// 8 bytes from each of two groups of 64, 4 from each of four groups of 32.
template <int G> __host__ __device__ __forceinline__ constexpr int word_of(int t, int i) {
  return G == 128 ? 4 * t + i : G == 64 ? (i >> 1) * 8 + 2 * t + (i & 1) : 4 * i + t;
}

template <int G> __device__ __forceinline__ uint4 load_codes(const uint8_t* row, int t, int left) {
  // row: at the block; left: codes of the row from here on (>= G)
  uint4 v = make_uint4(0, 0, 0, 0);
  if (G == 128) {
    v = ldg_nc_v4(row + t * 16);
  } else if (G == 64) {
    const uint2 a = __ldg(reinterpret_cast<const uint2*>(row + t * 8));
    v.x = a.x;
    v.y = a.y;
    if (left > 64) {
      const uint2 b = __ldg(reinterpret_cast<const uint2*>(row + 32 + t * 8));
      v.z = b.x;
      v.w = b.y;
    }
  } else {
    v.x = __ldg(reinterpret_cast<const uint32_t*>(row + t * 4));
    if (left > 32) v.y = __ldg(reinterpret_cast<const uint32_t*>(row + 16 + t * 4));
    if (left > 64) v.z = __ldg(reinterpret_cast<const uint32_t*>(row + 32 + t * 4));
    if (left > 96) v.w = __ldg(reinterpret_cast<const uint32_t*>(row + 48 + t * 4));
  }
  return v;
}

struct Q4Launch {
  const uint8_t* codes;
  const uint16_t *scales, *mins, *h;
  const int32_t* ids;
  int64_t n;
  int d, M, K;     // M hidden vectors from h; K candidates a vector (gather)
  int k_lo, k_hi;  // codes [k_lo, k_hi) of each row are summed
  int add;         // add to out instead of writing it
  int64_t ldo;
  float* out;
  int tiles;       // row tiles (of each vector in the gather)
  int split;       // warps that share a tile's codes
};

// Shared memory: h of the call's vectors, [vector][block][i][t] 16-byte words
// (8 codes' worth, codes 0,4,1,5,2,6,3,7), rows 64 bytes off a multiple of
// 128 so that the 8 lanes of a 16-byte read phase (2 vectors x 4 chunks) hit
// all banks once; then H per group and vector; then the warps' partial sums.
__host__ __device__ inline int h_stride(int blocks) { return blocks * 256 + 64; }

template <bool BF16, int G, int NT, int WARPS, bool MINS, bool GATHER>
__global__ void __launch_bounds__(WARPS * 32, GATHER || NT == 1 ? 2 : 1)
q4_kernel(Q4Launch a, int* err) {
  extern __shared__ __align__(128) unsigned char smem[];
  using P = Half2<BF16>;
  constexpr int GB = kBlockK / G;             // groups a block
  constexpr int HC = GATHER ? 1 : NT * 8;     // vectors of H
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, t = lane & 3;
  const int kd = a.k_hi - a.k_lo;
  const int blocks = (kd + kBlockK - 1) / kBlockK, groups = kd / G;
  const int stride = h_stride(blocks);
  const int nv = GATHER ? 1 : min(a.M, NT * 8);
  unsigned char* hs = smem;
  float* Hs = reinterpret_cast<float*>(smem + (size_t)nv * stride);  // [group][HC]
  float* part = Hs + (MINS ? (size_t)(blocks * GB) * HC : 0);
  pdl_wait();
  pdl_trigger();
  const int vec0 = GATHER ? blockIdx.y : 0;
  // ---- h, laid out as the codes unpack
  const int words = blocks * 16;
  for (int e = tid; e < nv * words; e += WARPS * 32) {
    const int v = e / words, w = e - v * words, b = w >> 4, p = w & 15;
    const int src = b * 16 + word_of<G>(p & 3, p >> 2);
    uint4 x = make_uint4(0, 0, 0, 0);
    if (src * 8 < kd)
      x = *reinterpret_cast<const uint4*>(a.h + (size_t)(vec0 + v) * a.d + a.k_lo + src * 8);
    uint4 y;
    y.x = __byte_perm(x.x, x.z, 0x5410);  // 0, 4
    y.y = __byte_perm(x.x, x.z, 0x7632);  // 1, 5
    y.z = __byte_perm(x.y, x.w, 0x5410);  // 2, 6
    y.w = __byte_perm(x.y, x.w, 0x7632);  // 3, 7
    *reinterpret_cast<uint4*>(hs + (size_t)v * stride + w * 16) = y;
  }
  if (MINS) {
    for (int e = tid; e < blocks * GB * HC; e += WARPS * 32) {
      const int v = e % HC, gi = e / HC;
      float s = 0.f;
      if (v < nv && gi < groups) {
        const uint16_t* src = a.h + (size_t)(vec0 + v) * a.d + a.k_lo + gi * G;
        for (int i = 0; i < G; ++i) s += P::to_float(src[i]);
      }
      Hs[e] = s;
    }
  }
  cta_sync();

  const int tiles_cta = WARPS / a.split;
  const int k_warp = warp % a.split, slot = warp / a.split;
  const int b_lo = blocks * k_warp / a.split, b_hi = blocks * (k_warp + 1) / a.split;
  const int64_t row_bytes = a.d / 2;
  const int row_groups = a.d / G;
  const int64_t count = GATHER ? a.K : a.n;
  for (int tile0 = blockIdx.x * tiles_cta; tile0 < a.tiles; tile0 += gridDim.x * tiles_cta) {
    const int tile = tile0 + slot;
    const bool on = tile < a.tiles;
    const int64_t first = (int64_t)tile * kRowsWarp;
    // the four rows of this lane: g, g + 8, g + 16, g + 24
    int64_t row[4];
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      const int64_t i = first + g + 8 * r;
      row[r] = 0;
      if (on && i < count) {
        if (GATHER) {
          const int32_t id = a.ids[(size_t)vec0 * a.K + i];
          row[r] = id >= 0 && id < a.n ? id : 0;
        } else {
          row[r] = i;
        }
      }
    }
    float acc[2][NT][4];
#pragma unroll
    for (int x = 0; x < 2; ++x)
#pragma unroll
      for (int y = 0; y < NT; ++y)
#pragma unroll
        for (int z = 0; z < 4; ++z) acc[x][y][z] = 0.f;
    if (on) {
      const uint8_t* cp[4];
      const uint16_t* sp[4];
      const uint16_t* op[4];
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        cp[r] = a.codes + row[r] * row_bytes + a.k_lo / 2;
        sp[r] = a.scales + row[r] * row_groups + a.k_lo / G;
        op[r] = MINS ? a.mins + row[r] * row_groups + a.k_lo / G : nullptr;
      }
#pragma unroll 2
      for (int b = b_lo; b < b_hi; ++b) {
        const int left = kd - b * kBlockK;
        uint4 c[4];
        float sc[4][GB], of[4][GB];
#pragma unroll
        for (int r = 0; r < 4; ++r) c[r] = load_codes<G>(cp[r] + b * (kBlockK / 2), t, left);
#pragma unroll
        for (int r = 0; r < 4; ++r)
#pragma unroll
          for (int q = 0; q < GB; ++q) {
            const bool in = q * G < left;
            sc[r][q] = in ? P::to_float(__ldg(sp[r] + b * GB + q)) : 0.f;
            if (MINS) of[r][q] = in ? P::to_float(__ldg(op[r] + b * GB + q)) + 8.f * sc[r][q] : 0.f;
          }
#pragma unroll
        for (int q = 0; q < GB; ++q) {
          float p[2][NT][4];
#pragma unroll
          for (int x = 0; x < 2; ++x)
#pragma unroll
            for (int y = 0; y < NT; ++y)
#pragma unroll
              for (int z = 0; z < 4; ++z) p[x][y][z] = 0.f;
#pragma unroll
          for (int i = q * (4 / GB); i < (q + 1) * (4 / GB); ++i) {
            uint4 hb[NT];
#pragma unroll
            for (int y = 0; y < NT; ++y) {
              hb[y] = make_uint4(0, 0, 0, 0);
              if (y * 8 + g < nv)
                hb[y] = *reinterpret_cast<const uint4*>(hs + (size_t)(y * 8 + g) * stride +
                                                        b * 256 + i * 64 + t * 16);
            }
#pragma unroll
            for (int x = 0; x < 2; ++x) {
              const uint32_t w0 = reinterpret_cast<const uint32_t*>(&c[2 * x])[i];
              const uint32_t w1 = reinterpret_cast<const uint32_t*>(&c[2 * x + 1])[i];
              uint32_t u0[4], u1[4];
#pragma unroll
              for (int j = 0; j < 4; ++j) {
                u0[j] = P::codes(w0, j);
                u1[j] = P::codes(w1, j);
              }
#pragma unroll
              for (int y = 0; y < NT; ++y) {
                P::mma(p[x][y], u0[0], u1[0], u0[1], u1[1], hb[y].x, hb[y].y);
                P::mma(p[x][y], u0[2], u1[2], u0[3], u1[3], hb[y].z, hb[y].w);
              }
            }
          }
#pragma unroll
          for (int x = 0; x < 2; ++x)
#pragma unroll
            for (int y = 0; y < NT; ++y)
#pragma unroll
              for (int z = 0; z < 4; ++z) {
                acc[x][y][z] = fmaf(sc[2 * x + (z >> 1)][q], p[x][y][z], acc[x][y][z]);
                if (MINS) {
                  const int col = GATHER ? 0 : y * 8 + 2 * t + (z & 1);
                  acc[x][y][z] = fmaf(of[2 * x + (z >> 1)][q], Hs[(b * GB + q) * HC + col],
                                      acc[x][y][z]);
                }
              }
        }
      }
    }
    if (a.split > 1) {
      // the tile's other warps hand their sums over in shared memory, and its
      // first one adds them in their order
      constexpr int PER = 2 * NT * 4;
      float* mine = part + (size_t)warp * PER * 32;
      if (k_warp > 0) {
#pragma unroll
        for (int x = 0; x < 2; ++x)
#pragma unroll
          for (int y = 0; y < NT; ++y)
#pragma unroll
            for (int z = 0; z < 4; ++z) mine[((x * NT + y) * 4 + z) * 32 + lane] = acc[x][y][z];
      }
      cta_sync();
      if (k_warp == 0) {
        for (int o = 1; o < a.split; ++o) {
          const float* from = part + (size_t)(warp + o) * PER * 32;
#pragma unroll
          for (int x = 0; x < 2; ++x)
#pragma unroll
            for (int y = 0; y < NT; ++y)
#pragma unroll
              for (int z = 0; z < 4; ++z) acc[x][y][z] += from[((x * NT + y) * 4 + z) * 32 + lane];
        }
      }
      cta_sync();
    }
    if (!on || k_warp != 0) continue;
#pragma unroll
    for (int x = 0; x < 2; ++x)
#pragma unroll
      for (int y = 0; y < NT; ++y)
#pragma unroll
        for (int z = 0; z < 4; ++z) {
          const int64_t i = first + 16 * x + g + 8 * (z >> 1);
          const int col = y * 8 + 2 * t + (z & 1);
          if (i >= count || col >= nv) continue;
          float* o = a.out + (size_t)(vec0 + col) * a.ldo + i;
          float v = acc[x][y][z];
          if (a.add) v += *o;
          if (GATHER) {
            const int32_t id = a.ids[(size_t)vec0 * a.K + i];
            if (id < 0 || id >= a.n) {
              record_error(err, kDevErrBadId);
              v = __int_as_float(0x7fc00000);
            }
          }
          *o = v;
        }
  }
}

constexpr size_t kSmemMost = 220 * 1024;

size_t smem_bytes(int kd, int group, int vecs, int cols, bool mins, int warps, int nt) {
  const int blocks = (kd + kBlockK - 1) / kBlockK;
  return (size_t)vecs * h_stride(blocks) +
         (mins ? (size_t)blocks * (kBlockK / group) * cols * sizeof(float) : 0) +
         (size_t)warps * nt * 8 * 32 * sizeof(float);
}

template <bool BF16, int G, int NT, int WARPS, bool MINS, bool GATHER>
cudaError_t launch_one(const Q4Launch& in, int* err, cudaStream_t s) {
  Q4Launch a = in;
  const int vecs = GATHER ? 1 : (a.M < NT * 8 ? a.M : NT * 8), cols = GATHER ? 1 : NT * 8;
  const int64_t rows = GATHER ? a.K : a.n;
  a.tiles = (int)((rows + kRowsWarp - 1) / kRowsWarp);
  // few tiles: more warps share one, until the GPU has about 16 warps an SM
  const int64_t all = (int64_t)a.tiles * (GATHER ? a.M : 1);
  const int blocks = (a.k_hi - a.k_lo + kBlockK - 1) / kBlockK;
  a.split = 1;
  while (a.split < WARPS && a.split * 2 <= blocks && all * a.split < (int64_t)sm_count() * 16)
    a.split *= 2;
  const size_t smem = smem_bytes(a.k_hi - a.k_lo, G, vecs, cols, MINS, WARPS, NT);
  static int smem_set[64] = {0};
  cudaError_t e = ensure_dynamic_smem(q4_kernel<BF16, G, NT, WARPS, MINS, GATHER>, smem, smem_set);
  if (e != cudaSuccess) return e;
  const int per = WARPS / a.split, ctas = (a.tiles + per - 1) / per;
  const int resident = sm_count() * ((smem <= 110 * 1024 && (GATHER || NT == 1)) ? 2 : 1);
  const unsigned gx = GATHER ? ctas : (ctas < resident ? ctas : resident);
  return launch_kernel(true, q4_kernel<BF16, G, NT, WARPS, MINS, GATHER>,
                       dim3(gx, GATHER ? a.M : 1), dim3(WARPS * 32), smem, s, a, err);
}

template <bool BF16, int G, bool MINS>
cudaError_t launch_cols(const Q4Launch& a, int* err, cudaStream_t s) {
  if (a.ids) return launch_one<BF16, G, 1, 8, MINS, true>(a, err, s);
  if (a.M <= 8) return launch_one<BF16, G, 1, 8, MINS, false>(a, err, s);
  return launch_one<BF16, G, 2, 16, MINS, false>(a, err, s);
}

template <bool BF16, int G>
cudaError_t launch_mins(const Q4Launch& a, int* err, cudaStream_t s) {
  return a.mins ? launch_cols<BF16, G, true>(a, err, s) : launch_cols<BF16, G, false>(a, err, s);
}

template <bool BF16>
cudaError_t launch_group(const Q4Launch& a, int group, int* err, cudaStream_t s) {
  if (group == 128) return launch_mins<BF16, 128>(a, err, s);
  if (group == 64) return launch_mins<BF16, 64>(a, err, s);
  return launch_mins<BF16, 32>(a, err, s);
}

}  // namespace

cudaError_t launch_q4(const Q4Args& q, int* err, cudaStream_t s) {
  Q4Launch a = {};
  a.codes = q.codes;
  a.scales = static_cast<const uint16_t*>(q.scales);
  a.mins = static_cast<const uint16_t*>(q.mins);
  a.ids = q.ids;
  a.n = q.n;
  a.d = q.d;
  a.K = q.K;
  a.ldo = q.ids ? q.K : q.n;
  // hidden vectors of one pass over the rows, then pieces of d, as far as h
  // fits in shared memory; a later piece adds to the former's sums
  const int most = q.ids ? q.M : 16;
  for (int m = 0; m < q.M; m += most) {
    a.M = q.M - m < most ? q.M - m : most;
    a.h = static_cast<const uint16_t*>(q.h) + (size_t)m * q.d;
    a.out = q.out + (size_t)m * a.ldo;
    const int nt = !q.ids && a.M > 8 ? 2 : 1, warps = nt == 2 ? 16 : 8;
    const int vecs = q.ids ? 1 : a.M, cols = q.ids ? 1 : nt * 8;
    int piece = q.d;
    while (smem_bytes(piece, q.group, vecs, cols, q.mins != nullptr, warps, nt) > kSmemMost)
      piece = ((piece + 1) / 2 + kBlockK - 1) / kBlockK * kBlockK;
    for (int k = 0; k < q.d; k += piece) {
      a.k_lo = k;
      a.k_hi = k + piece < q.d ? k + piece : q.d;
      a.add = k > 0;
      const cudaError_t e = q.dtype == LMHEAD_BF16 ? launch_group<true>(a, q.group, err, s)
                                                   : launch_group<false>(a, q.group, err, s);
      if (e != cudaSuccess) return e;
    }
  }
  return cudaSuccess;
}

}  // namespace lmhead
