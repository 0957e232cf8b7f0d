// Products of hidden vectors with rows of 4-bit codes and group scales:
//   y[m, i] = sum_G ( s[i,G] sum_{k in G} c[i,k] h[m,k] + o[i,G] H[m,G] ),
// H[m,G] = sum_{k in G} h[m,k]; o = -8 s for symmetric codes, the group's min
// for codes with an offset.
//
// Bound by reading the codes (d/2 + 2 d/group bytes a row) and by the
// instructions that unpack them. A warp multiplies 16 rows x 16 codes with up
// to 8 hidden vectors in one matrix instruction from registers (products
// exact, sums in 32 bits), and the codes need next to no work to become its
// operands: four bits among the ten of an fp16 mantissa are a subnormal number,
// exactly c times its place, so a 32-bit word of 8 codes takes two shifts and
// four masks. (Adding the bits of
// 1024 and subtracting 1032 instead, to have c - 8, took nine instructions; the
// term with H costs one multiply-add a group.) h is kept in fp16, scaled, with
// the sixteenth for the pairs that need it. The sum over k may take k in any
// order, so the order in which a lane's own codes unpack is the order of k, and
// h is laid out to match once per CTA: no shuffle is needed. Each warp streams
// its own 32 rows through a ring of shared memory with asynchronous copies (128
// bytes of a row at a time; loads straight to the operand registers touch 64
// bytes of 8 rows at once and were bound by the L1's tags). Group sums are
// scaled in 32 bits after the matrix products; no weight is ever rounded.
// (Operands of the tcgen05 instructions would have to be written to shared or
// tensor memory first, at a store per two codes; here they never leave
// registers.)
// Measured: 128256 rows of 4096 codes, groups of 128: 49-53 us for one hidden vector
// (5.1-5.5 TB/s of codes and scales, at 1.8 instructions a cycle and SM), 56 for
// eight, 31 for 1002 candidate rows of each of 64; 151936 rows of 5120, groups of
// 64 with mins: 124 us for 16 vectors.
//   The matrix instructions cut the products of a sum at a place set by the
// largest. With codes up to 15 in place of -8..7 a symmetric row's sums lose
// about two bits more; over long rows that stays near 2^-21 of the result, in
// short ones (kCentreD) 8 is subtracted from the codes, which costs four packed
// additions a word and makes H unnecessary.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "common.cuh"
#include "kernels.h"

namespace lmhead {
namespace {

constexpr int kBlockK = 128;  // codes of a row that four lanes take together
constexpr int kRowsWarp = 32;
constexpr int kCentreD = 256;

// What becomes of a code: c with a min per group, c with -8 s, or c - 8.
enum Mode { kMins, kPlain, kCentred };

// The 8 codes of word w as fp16 pairs (0,4), (1,5), (2,6), (3,7): subnormal
// numbers, 2^-22 c for the first and third pair and 2^-18 c for the others (the
// mantissa's top; the matrix instructions do not normalise their operands, so
// the higher the code sits the more bits its products keep).
template <bool CENTRE> __device__ __forceinline__ void unpack_codes(uint32_t w, uint32_t (&u)[4]) {
  const uint32_t v = w << 2, x = w >> 6;
  u[0] = v & 0x003c003cu;
  u[1] = v & 0x03c003c0u;
  u[2] = x & 0x003c003cu;
  u[3] = x & 0x03c003c0u;
  if (CENTRE) {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      uint32_t eight = j & 1 ? 0x82008200u : 0x80208020u;  // -8 times the unit
      const __half2 r = __hadd2(*reinterpret_cast<__half2*>(&u[j]),
                                *reinterpret_cast<__half2*>(&eight));
      u[j] = *reinterpret_cast<const uint32_t*>(&r);
    }
  }
}

__device__ __forceinline__ void mma_f16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                        uint32_t a3, uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
      "{%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
// The same with nothing to add to.
__device__ __forceinline__ void mma_f16_first(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                              uint32_t a3, uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
      "{%8,%9}, {%10,%10,%10,%10};"
      : "=f"(c[0]), "=f"(c[1]), "=f"(c[2]), "=f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.f));
}

template <bool BF16> __device__ __forceinline__ float2 pair_to_float(uint32_t w) {
  if (BF16) return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xFFFF0000u));
  return __half22float2(*reinterpret_cast<const __half2*>(&w));
}

// Two fp32 multiply-adds in one instruction.
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
  float2 d;
  asm("{\n\t.reg .b64 x, y, z;\n\t"
      "mov.b64 x, {%2, %3};\n\tmov.b64 y, {%4, %5};\n\tmov.b64 z, {%6, %7};\n\t"
      "fma.rn.f32x2 z, x, y, z;\n\tmov.b64 {%0, %1}, z;\n\t}"
      : "=f"(d.x), "=f"(d.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
  return d;
}

// N consecutive 16-bit values of a row, in shared memory or not.
template <int N> struct Packed {
  uint32_t w[(N + 1) / 2];
};
template <int N, bool SHARED> __device__ __forceinline__ Packed<N> load_whole(const uint16_t* p) {
  auto get = [](auto* q) { return SHARED ? *q : __ldg(q); };
  Packed<N> v;
  if (N == 4) {
    const uint2 x = get(reinterpret_cast<const uint2*>(p));
    v.w[0] = x.x;
    v.w[(N + 1) / 2 - 1] = x.y;
  } else if (N == 2) {
    v.w[0] = get(reinterpret_cast<const uint32_t*>(p));
  } else {
    v.w[0] = get(p);
  }
  return v;
}
// Those below `left` one by one, zeros behind them.
template <int N> __device__ __forceinline__ Packed<N> load_single(const uint16_t* p, int left) {
  Packed<N> v;
#pragma unroll
  for (int i = 0; i < (N + 1) / 2; ++i) {
    v.w[i] = 2 * i < left ? __ldg(p + 2 * i) : 0u;
    if (2 * i + 1 < N && 2 * i + 1 < left) v.w[i] |= (uint32_t)__ldg(p + 2 * i + 1) << 16;
  }
  return v;
}
// Values [N pos, N pos + N) of 8.
template <int N> __device__ __forceinline__ Packed<N> packed_of(const uint4& v, int pos) {
  Packed<N> r;
  if (N == 4) {
    r.w[0] = pos & 1 ? v.z : v.x;
    r.w[(N + 1) / 2 - 1] = pos & 1 ? v.w : v.y;
  } else {
    const int word = N == 2 ? pos : pos >> 1;
    const uint32_t x = word & 2 ? (word & 1 ? v.w : v.z) : (word & 1 ? v.y : v.x);
    r.w[0] = N == 1 && (pos & 1) ? x >> 16 : x;
  }
  return r;
}
template <bool BF16, int N> __device__ __forceinline__ float packed_at(const Packed<N>& v, int i) {
  const float2 f = pair_to_float<BF16>(v.w[i >> 1]);
  return i & 1 ? f.y : f.x;
}

// Word i (of 4) of lane chunk t in a 128-code block, so that each matrix
// instruction stays within one group: bytes t*16 + i*4 for groups of 128,
// 8 bytes from each of two groups of 64, 4 from each of four groups of 32.
template <int G> __host__ __device__ __forceinline__ constexpr int word_of(int t, int i) {
  return G == 128 ? 4 * t + i : G == 64 ? (i >> 1) * 8 + 2 * t + (i & 1) : 4 * i + t;
}

struct Q4Launch {
  const uint8_t* codes;
  const uint16_t *scales, *mins, *h;
  const int32_t* ids;
  int64_t n;
  int d, M, K;         // M hidden vectors from h; K candidates a vector (gather)
  int k_lo, k_hi;      // codes [k_lo, k_hi) of each row are summed
  int add;             // add to out instead of writing it
  int64_t ldo;
  float* out;
  int tiles;           // row tiles (of each vector in the gather)
  int scales_aligned;  // scales and mins at 16 bytes
  int share;           // a tile's codes may be divided between warps
};

// Shared memory: h of the call's vectors, [vector][block][i][t] 16-byte words
// (8 codes' worth, codes 0,4,1,5,2,6,3,7), rows 64 bytes off a multiple of
// 128 so that the 8 lanes of a 16-byte read phase (2 vectors x 4 chunks) hit
// all banks once; then H per group and vector; each warp's ring of codes; and
// a tile's sums per warp where warps share tiles.
__host__ __device__ inline int h_stride(int blocks) { return blocks * 256 + 64; }
// Bytes of h and H together: the rings behind them start at a multiple of 128.
__host__ __device__ inline int h_bytes(int blocks, int vecs, int sums) {
  return (vecs * h_stride(blocks) + sums * (int)sizeof(float) + 127) / 128 * 128;
}

// A stage of a warp's ring: SB blocks of 32 rows x 64 bytes. The 16-byte
// chunks of a row are permuted by it so that the reads of all three group
// sizes (16 bytes of 2 rows, 8 of 4 rows or 4 of 8 rows at a time) and the
// copies that write them meet every bank once.
__device__ __forceinline__ uint32_t ring_at(int blk, int row, int chunk) {
  const int x = (row & 2) | ((row >> 2) & 1);
  return (uint32_t)(blk * 2048 + (row ^ blk) * 64 + ((chunk ^ x) * 16));
}

__device__ __forceinline__ void copy16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global.L2::128B [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void copy16_or_zero(uint32_t dst, const void* src, bool in) {
  const int n = in ? 16 : 0;
  asm volatile("cp.async.cg.shared.global.L2::128B [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(n)
               : "memory");
}

// A warp's slot for the scales of 8 groups of 32 rows, and for the mins.
__host__ __device__ constexpr int slot_bytes(bool mins) { return mins ? 1024 : 512; }

// Hidden vectors that a CTA of the gather holds at a time.
constexpr int kGatherVecs = 2;

template <bool BF16, int G, int NT, int WARPS, int SB, int NS, int MODE, bool GATHER, bool COPIED>
__global__ void __launch_bounds__(WARPS * 32, WARPS == 8 ? 2 : 1)
q4_kernel(Q4Launch a, int* err) {
  extern __shared__ __align__(128) unsigned char smem[];
  __shared__ uint32_t sh_top[WARPS];
  __shared__ float sh_back[GATHER ? kGatherVecs : NT * 8];  // what a vector's sums are scaled back by
  constexpr bool MINS = MODE == kMins, SUMS = MODE != kCentred;
  constexpr int GB = kBlockK / G;          // groups a block
  constexpr int HC = GATHER ? kGatherVecs : NT * 8;  // vectors of H
  constexpr int CPY = SB * 4;              // copies a lane and stage
  constexpr int CR = 32 / CPY;             // rows a copy of the warp covers
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, t = lane & 3;
  const int kd = a.k_hi - a.k_lo;
  const int blocks = (kd + kBlockK - 1) / kBlockK;
  const int stride = h_stride(blocks);
  const int nv = GATHER ? kGatherVecs : min(a.M, NT * 8);
  unsigned char* hs = smem;
  float* Hs = reinterpret_cast<float*>(smem + (size_t)nv * stride);  // [group][HC]
  unsigned char* rings = smem + h_bytes(blocks, nv, SUMS ? blocks * GB * HC : 0);
  unsigned char* ring = rings + (size_t)warp * (NS * SB * 2048);
  constexpr int SLOT = COPIED ? slot_bytes(MINS) : 0;
  unsigned char* slots = rings + WARPS * NS * SB * 2048 + warp * (NS * SLOT);
  float* part = reinterpret_cast<float*>(rings + (size_t)WARPS * NS * (SB * 2048 + SLOT));
  pdl_wait();
  pdl_trigger();
  const int64_t count = GATHER ? a.K : a.n;
  const int row_bytes = a.d / 2, row_groups = a.d / G;

  // The CTA takes a run of tiles (of vector after vector in the gather) and
  // divides their stages evenly among its warps, wherever a tile's end falls, so
  // that no warp waits for another before the end: a warp whose stages begin
  // inside a tile and reach its end adds the sums that earlier warps left for it.
  // It goes through its tiles from the last to the first, so that what it
  // leaves itself is done first and what it waits for comes last. In the gather
  // this is repeated for each kGatherVecs vectors of the run.
  const int all_stages = (blocks + SB - 1) / SB;
  const int64_t tiles = (int64_t)a.tiles * (GATHER ? a.M : 1);
  const int64_t run_lo = tiles * blockIdx.x / gridDim.x, run_hi = tiles * (blockIdx.x + 1) / gridDim.x;
  int64_t part_lo = run_lo;  // of the run
  int mine_lo = 0, mine_hi = 0;  // this warp's stages of the part
  auto share_of = [&](int w, int64_t count_tiles) -> int {  // where warp w's stages begin
    return a.share ? (int)(count_tiles * all_stages * w / WARPS)
                   : (int)(count_tiles * w / WARPS) * all_stages;
  };
  auto row_id = [&](int vec, int64_t i) -> int32_t {  // the row behind entry i, 0 for none
    if (!GATHER) return i < count ? (int32_t)i : 0;
    if (i >= count) return 0;
    const int32_t id = a.ids[(size_t)vec * a.K + i];
    return id >= 0 && id < a.n ? id : 0;
  };

  // ---- the copies of this warp's codes run NS - 1 stages ahead, over the ends
  // of its tiles
  const int c_row = lane / CPY, c_chunk = lane % CPY;  // of the warp's first copy
  int c_end = 0, c_stage = 0, c_last = 0, c_slot = 0;  // c_end: stages not yet begun end here
  // where this lane's chunks go in a stage, and where the next ones come from
  const uint32_t ring_s = (uint32_t)__cvta_generic_to_shared(ring);
  uint32_t c_dst[CPY];
#pragma unroll
  for (int j = 0; j < CPY; ++j)
    c_dst[j] = ring_s + ring_at(c_chunk >> 2, j * CR + c_row, c_chunk & 3);
  const uint8_t* c_src[CPY];
  int c_rows = 0;  // of the tile
  // Where rows of scales allow 16-byte copies a lane copies those of 8 groups of
  // one row along with the first stage that needs them. (Loaded to registers
  // stage by stage, as other rows' are, they want the L1, which the rings leave
  // little of: one vector, groups of 64 with mins 68 us, so 60.)
  constexpr int SC = SB * GB;  // scales of a row and stage
  constexpr int PER = 8 / SC;  // stages they last
  int64_t c_scale = 0;  // the lane's row's first scale
  int c_scale_slot = 0, c_first = 0;
  auto copy_scales = [&]() {
    const uint32_t to =
        (uint32_t)__cvta_generic_to_shared(slots) + c_scale_slot * SLOT + lane * 16;
    c_scale_slot = c_scale_slot + 1 == NS ? 0 : c_scale_slot + 1;
    const int64_t at = c_scale + c_stage / PER * 8;
    copy16(to, a.scales + at);
    if (MINS) copy16(to + 512, a.mins + at);
  };
  auto copy_tile = [&]() {  // on to the tile before, if this warp has stages there
    c_stage = c_last = 0;
    if (c_end <= mine_lo) return;
    const int tl = (c_end - 1) / all_stages;
    c_stage = max(0, mine_lo - tl * all_stages);
    c_last = c_end - tl * all_stages;
    c_end = tl * all_stages;
    const int64_t flat = part_lo + tl;
    const int vec = GATHER ? (int)(flat / a.tiles) : 0;
    const int64_t first = (flat - (int64_t)vec * a.tiles) * kRowsWarp;
    c_rows = (int)min((int64_t)kRowsWarp, count - first);
    if (COPIED) c_scale = (int64_t)row_id(vec, first + lane) * row_groups + a.k_lo / G;
    c_first = c_stage;
    const uint8_t* src = a.codes + a.k_lo / 2 + (c_stage * SB * 4 + c_chunk) * 16;
#pragma unroll
    for (int j = 0; j < CPY; ++j) {
      const int64_t i = first + j * CR + c_row;
      c_src[j] = src + (GATHER ? (int64_t)row_id(vec, i) : i) * row_bytes;
    }
  };
  auto copy_stage = [&]() {
    if (c_stage < c_last) {
      const uint32_t slot_at = c_slot * (SB * 2048);
      if (c_rows == kRowsWarp && (c_stage + 1) * SB * kBlockK <= kd) {
#pragma unroll
        for (int j = 0; j < CPY; ++j) copy16(c_dst[j] + slot_at, c_src[j]);
      } else {
        const bool in = (c_stage * SB * 4 + c_chunk) * 32 < kd;  // of the piece
#pragma unroll
        for (int j = 0; j < CPY; ++j) {
          const bool there = in && j * CR + c_row < c_rows;
          copy16_or_zero(c_dst[j] + slot_at, there ? c_src[j] : a.codes, there);
        }
      }
      if (COPIED && (c_stage == c_first || c_stage % PER == 0)) copy_scales();
#pragma unroll
      for (int j = 0; j < CPY; ++j) c_src[j] += SB * (kBlockK / 2);
      if (++c_stage == c_last) copy_tile();
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
    c_slot = c_slot + 1 == NS ? 0 : c_slot + 1;
  };
  // ---- h, laid out as the codes unpack, in fp16: values are first scaled by
  // the power of two that takes the vector's largest to 2^14..2^15, which keeps
  // all bits of those down to 2^-25 of the largest, and 2^-36 of it throughout;
  // the pairs that meet 2^-18 c are divided by 16. A warp takes a vector, in the
  // gather all of them one after the other.
  auto lay_out = [&](int vec0, int vecs) {
    const int words = blocks * 16;
    const int lanes = GATHER ? WARPS * 32 : 32, me = GATHER ? tid : lane;
    for (int v = GATHER ? 0 : warp; v < vecs; v += GATHER ? 1 : WARPS) {
      const uint16_t* src = a.h + (size_t)(vec0 + v) * a.d + a.k_lo;
      unsigned char* dst = hs + (size_t)v * stride;
      uint32_t top = 0;  // the order of magnitudes is that of their bits
      for (int w = me; w * 8 < kd; w += lanes) {
        const uint4 x = *reinterpret_cast<const uint4*>(src + w * 8);
        const uint32_t u[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float2 f = pair_to_float<BF16>(u[i]);
          top = max(top, max(__float_as_uint(fabsf(f.x)), __float_as_uint(fabsf(f.y))));
        }
      }
      top = __reduce_max_sync(0xFFFFFFFFu, top);
      if (GATHER) {
        if (lane == 0) sh_top[warp] = top;
        cta_sync();
#pragma unroll
        for (int i = 0; i < WARPS; ++i) top = max(top, sh_top[i]);
        cta_sync();
      }
      const int e = (int)(top >> 23) - 127;  // floor of its logarithm
      const int k = top == 0 ? 0 : max(-126, min(126, 14 - e));
      const float scale = __uint_as_float((uint32_t)(127 + k) << 23), sixteenth = scale * 0.0625f;
      if (me == 0) sh_back[v] = __uint_as_float((uint32_t)(127 - k) << 23);
      for (int w = me; w < words; w += lanes) {
        const int b = w >> 4, p = w & 15, at = b * 16 + word_of<G>(p & 3, p >> 2);
        uint4 x = make_uint4(0, 0, 0, 0);
        if (at * 8 < kd) x = *reinterpret_cast<const uint4*>(src + at * 8);
        const uint32_t u[4] = {x.x, x.y, x.z, x.w};  // 0 1, 2 3, 4 5, 6 7
        uint32_t r[4];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const float2 lo = pair_to_float<BF16>(u[i]), hi = pair_to_float<BF16>(u[i + 2]);
          const __half2 even = __floats2half2_rn(lo.x * scale, hi.x * scale);
          const __half2 odd = __floats2half2_rn(lo.y * sixteenth, hi.y * sixteenth);
          r[2 * i] = *reinterpret_cast<const uint32_t*>(&even);
          r[2 * i + 1] = *reinterpret_cast<const uint32_t*>(&odd);
        }
        *reinterpret_cast<uint4*>(dst + w * 16) = make_uint4(r[0], r[1], r[2], r[3]);
      }
    }
    cta_sync();
    if (SUMS) {
      // H, times 2^-22 like the products; a group's words lie at i in
      // [q * 4 / GB, (q + 1) * 4 / GB), every t
      for (int e = tid; e < blocks * GB * HC; e += WARPS * 32) {
        const int v = e % HC, gi = e / HC, b = gi / GB, q = gi - b * GB;
        float even = 0.f, odd = 0.f;
        if (v < vecs) {
          const unsigned char* src = hs + (size_t)v * stride + b * 256 + q * (256 / GB);
#pragma unroll
          for (int w = 0; w < 16 / GB; ++w) {
            const uint4 x = *reinterpret_cast<const uint4*>(src + w * 16);
            const float2 f0 = pair_to_float<false>(x.x), f1 = pair_to_float<false>(x.y);
            const float2 f2 = pair_to_float<false>(x.z), f3 = pair_to_float<false>(x.w);
            even += (f0.x + f0.y) + (f2.x + f2.y);
            odd += (f1.x + f1.y) + (f3.x + f3.y);
          }
        }
        Hs[e] = fmaf(16.f, odd, even) * 2.384185791015625e-7f;
      }
      cta_sync();
    }
  };
  // This lane's vector columns (columns past the last repeat it and are not
  // stored) and its places in a stage: row g, with rows g + 8 r 512 bytes apart.
  const unsigned char* hp[NT];
  if (!GATHER)
#pragma unroll
    for (int y = 0; y < NT; ++y) hp[y] = hs + (size_t)min(y * 8 + g, nv - 1) * stride + t * 16;
  // From nine vectors on, where h leaves no room for slots, a lane loads the
  // scales of 8 groups of one row (g + 8 t) for PER stages and hands them round:
  // loaded stage by stage they took as much of the L2 as the codes, a sector a
  // row (194 against 136 us for 16 vectors over the wide head). Rows that allow
  // neither load theirs a stage ahead.
  constexpr bool CHUNKS = NT == 2;
  constexpr int ALIGN = CHUNKS ? 8 : SC;
  const bool whole = row_groups % ALIGN == 0 && a.scales_aligned && (a.k_lo / G) % ALIGN == 0;
  const int groups = kd / G;
  // the sums of tile `flat` to where they belong
  auto put = [&](int64_t flat, const float2 (&acc)[2][NT][2]) {
    const int vec = GATHER ? (int)(flat / a.tiles) : 0;
    const int64_t first = (flat - (int64_t)vec * a.tiles) * kRowsWarp;
    const int vec0 = GATHER ? (int)(part_lo / a.tiles) : 0;
#pragma unroll
    for (int x = 0; x < 2; ++x)
#pragma unroll
      for (int y = 0; y < NT; ++y)
#pragma unroll
        for (int z = 0; z < 4; ++z) {
          const int64_t i = first + 16 * x + g + 8 * (z >> 1);
          const int col = y * 8 + 2 * t + (z & 1);
          if (i >= count || col >= (GATHER ? 1 : nv)) continue;
          float* o = a.out + (size_t)(GATHER ? vec : col) * a.ldo + i;
          float v = (z & 1 ? acc[x][y][z >> 1].y : acc[x][y][z >> 1].x) * 4194304.f *
                    sh_back[GATHER ? vec - vec0 : col];
          if (a.add) v += *o;
          if (GATHER) {
            const int32_t id = a.ids[(size_t)vec * a.K + i];
            if (id < 0 || id >= a.n) {
              record_error(err, kDevErrBadId);
              v = __int_as_float(0x7fc00000);
            }
          }
          *o = v;
        }
  };
  constexpr int PER_LANE = 2 * NT * 2;  // pairs of sums
  float2* left = reinterpret_cast<float2*>(part) + lane;  // [warp][pair][lane]
  while (part_lo < run_hi) {
    int64_t part_hi = run_hi;
    const int vec0 = GATHER ? (int)(part_lo / a.tiles) : 0;
    if (GATHER) part_hi = min(run_hi, (int64_t)(vec0 + kGatherVecs) * a.tiles);
    mine_lo = share_of(warp, part_hi - part_lo);
    mine_hi = share_of(warp + 1, part_hi - part_lo);
    if (part_lo > run_lo) cta_sync();  // what the part before had laid out is read no more
    c_end = mine_hi;
    c_slot = c_scale_slot = 0;
    copy_tile();
#pragma unroll
    for (int i = 0; i < NS - 1; ++i) copy_stage();
    lay_out(vec0, GATHER ? (int)((part_hi - 1) / a.tiles) - vec0 + 1 : nv);
    int use = 0, scale_use = -1;  // ring slots
    int64_t waits = -1;  // the tile whose earlier stages other warps have
    float2 acc[2][NT][2];  // columns 2 t and 2 t + 1 of rows g + 16 x + 8 z
    for (int end = mine_hi; end > mine_lo;) {
      const int tl = (end - 1) / all_stages;
      const int s_lo = max(0, mine_lo - tl * all_stages), s_hi = end - tl * all_stages;
      end = tl * all_stages;
      const int64_t flat = part_lo + tl;
      const int vec = GATHER ? (int)(flat / a.tiles) : 0;
      const int64_t first = (flat - (int64_t)vec * a.tiles) * kRowsWarp;
      if (GATHER) hp[0] = hs + (size_t)(vec - vec0) * stride + t * 16;
#pragma unroll
      for (int x = 0; x < 2; ++x)
#pragma unroll
        for (int y = 0; y < NT; ++y)
#pragma unroll
          for (int z = 0; z < 2; ++z) acc[x][y][z] = make_float2(0.f, 0.f);
      // scales of this lane's rows g, g + 8, g + 16, g + 24 where they are not
      // copied: one stage ahead, or in chunks one chunk ahead
      const uint16_t *sp[4] = {}, *op[4] = {};
      uint4 s_now, s_next, o_now, o_next;
      Packed<SC> sc_n[4], of_n[4];
      auto load_chunk = [&](int ch) {
        if (ch * 8 >= groups) return;
        s_next = __ldg(reinterpret_cast<const uint4*>(sp[0]) + ch);
        if (MINS) o_next = __ldg(reinterpret_cast<const uint4*>(op[0]) + ch);
      };
      auto load_scales = [&](int st) {
        if (!CHUNKS && whole) {
#pragma unroll
          for (int r = 0; r < 4; ++r) {
            sc_n[r] = load_whole<SC, false>(sp[r] + st * SC);
            if (MINS) of_n[r] = load_whole<SC, false>(op[r] + st * SC);
          }
        } else {
#pragma unroll
          for (int r = 0; r < 4; ++r) {
            sc_n[r] = load_single<SC>(sp[r] + st * SC, groups - st * SC);
            if (MINS) of_n[r] = load_single<SC>(op[r] + st * SC, groups - st * SC);
          }
        }
      };
      if (!COPIED) {
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          if (CHUNKS && whole && r > 0) break;
          const int64_t at =
              (int64_t)row_id(vec, first + g + 8 * (CHUNKS && whole ? t : r)) * row_groups + a.k_lo / G;
          sp[r] = a.scales + at;
          op[r] = MINS ? a.mins + at : nullptr;
        }
        if (CHUNKS && whole) {
          load_chunk(s_lo / PER);
          s_now = s_next;
          if (MINS) o_now = o_next;
          load_chunk(s_lo / PER + 1);
        } else {
          load_scales(s_lo);
        }
      }
#pragma unroll 1
      for (int st = s_lo; st < s_hi; ++st) {
        copy_stage();
        asm volatile("cp.async.wait_group %0;" ::"n"(NS - 1) : "memory");
        __syncwarp();
        Packed<SC> sc[4], of[4];
        if (COPIED) {
          if (st == s_lo || st % PER == 0) scale_use = scale_use + 1 == NS ? 0 : scale_use + 1;
          const uint16_t* from = reinterpret_cast<const uint16_t*>(slots + scale_use * SLOT) + g * 8 +
                                 st % PER * SC;
#pragma unroll
          for (int r = 0; r < 4; ++r) {
            sc[r] = load_whole<SC, true>(from + r * 64);
            if (MINS) of[r] = load_whole<SC, true>(from + r * 64 + 256);
          }
        } else if (CHUNKS && whole) {
          if (st % PER == 0 && st != s_lo) {
            s_now = s_next;
            if (MINS) o_now = o_next;
            load_chunk(st / PER + 1);
          }
          const Packed<SC> ms = packed_of<SC>(s_now, st % PER);
          const Packed<SC> mo = MINS ? packed_of<SC>(o_now, st % PER) : ms;
#pragma unroll
          for (int r = 0; r < 4; ++r)
#pragma unroll
            for (int i = 0; i < (SC + 1) / 2; ++i) {
              sc[r].w[i] = __shfl_sync(0xFFFFFFFFu, ms.w[i], (lane & ~3) | r);
              if (MINS) of[r].w[i] = __shfl_sync(0xFFFFFFFFu, mo.w[i], (lane & ~3) | r);
            }
        } else {
#pragma unroll
          for (int r = 0; r < 4; ++r) {
            sc[r] = sc_n[r];
            if (MINS) of[r] = of_n[r];
          }
          if (st + 1 < s_hi) load_scales(st + 1);
        }
        const unsigned char* codes = ring + use * (SB * 2048);
        use = use + 1 == NS ? 0 : use + 1;
#pragma unroll
        for (int u = 0; u < SB; ++u) {
          const int b = st * SB + u;
          if (SB > 1 && u > 0 && b >= blocks) break;
          uint32_t c[4][4];
#pragma unroll
          for (int r = 0; r < 4; ++r) {
            if (G == 128) {
              const uint4 v = *reinterpret_cast<const uint4*>(codes + ring_at(u, g, t) + r * 512);
              c[r][0] = v.x, c[r][1] = v.y, c[r][2] = v.z, c[r][3] = v.w;
            } else if (G == 64) {
#pragma unroll
              for (int q = 0; q < 2; ++q) {
                const uint2 v = *reinterpret_cast<const uint2*>(
                    codes + ring_at(u, g, q * 2 + (t >> 1)) + (t & 1) * 8 + r * 512);
                c[r][2 * q] = v.x, c[r][2 * q + 1] = v.y;
              }
            } else {
#pragma unroll
              for (int q = 0; q < 4; ++q)
                c[r][q] =
                    *reinterpret_cast<const uint32_t*>(codes + ring_at(u, g, q) + t * 4 + r * 512);
            }
          }
#pragma unroll
          for (int q = 0; q < GB; ++q) {
            float p[2][NT][4];
#pragma unroll
            for (int i = q * (4 / GB); i < (q + 1) * (4 / GB); ++i) {
              uint4 hb[NT];
#pragma unroll
              for (int y = 0; y < NT; ++y)
                hb[y] = *reinterpret_cast<const uint4*>(hp[y] + b * 256 + i * 64);
#pragma unroll
              for (int x = 0; x < 2; ++x) {
                uint32_t u0[4], u1[4];
                unpack_codes<MODE == kCentred>(c[2 * x][i], u0);
                unpack_codes<MODE == kCentred>(c[2 * x + 1][i], u1);
#pragma unroll
                for (int y = 0; y < NT; ++y) {
                  if (i == q * (4 / GB))
                    mma_f16_first(p[x][y], u0[0], u1[0], u0[1], u1[1], hb[y].x, hb[y].y);
                  else
                    mma_f16(p[x][y], u0[0], u1[0], u0[1], u1[1], hb[y].x, hb[y].y);
                  mma_f16(p[x][y], u0[2], u1[2], u0[3], u1[3], hb[y].z, hb[y].w);
                }
              }
            }
            float s4[4], o4[4];
#pragma unroll
            for (int r = 0; r < 4; ++r) {
              s4[r] = packed_at<BF16, SC>(sc[r], u * GB + q);
              o4[r] = MINS ? packed_at<BF16, SC>(of[r], u * GB + q) : -8.f * s4[r];
            }
#pragma unroll
            for (int y = 0; y < NT; ++y) {
              float2 H = make_float2(0.f, 0.f);
              if (SUMS) {
                const float* hq = Hs + (b * GB + q) * HC + (GATHER ? vec - vec0 : y * 8 + 2 * t);
                H = GATHER ? make_float2(hq[0], 0.f) : *reinterpret_cast<const float2*>(hq);
              }
#pragma unroll
              for (int x = 0; x < 2; ++x)
#pragma unroll
                for (int z = 0; z < 2; ++z) {
                  const int r = 2 * x + z;
                  float2& d = acc[x][y][z];
                  d = fma2(make_float2(s4[r], s4[r]),
                           make_float2(p[x][y][2 * z], p[x][y][2 * z + 1]), d);
                  if (SUMS) d = fma2(make_float2(o4[r], o4[r]), H, d);
                }
            }
          }
        }
        __syncwarp();  // the next copy may overwrite what was read here
      }
      if (s_hi < all_stages) {
#pragma unroll
        for (int e = 0; e < PER_LANE; ++e)
          left[(warp * PER_LANE + e) * 32] = acc[e / (NT * 2)][e / 2 % NT][e % 2];
      } else if (s_lo > 0) {
        waits = flat;
      } else {
        put(flat, acc);
      }
    }
    if (a.share) {
      cta_sync();
      if (waits >= 0) {
        // the earlier warps' sums in their order, then this one's
        const int begin = (int)(waits - part_lo) * all_stages;
        float2 sum[2][NT][2] = {};
        for (int o = 0; o < warp; ++o) {
          const int lo = share_of(o, part_hi - part_lo), hi = share_of(o + 1, part_hi - part_lo);
          if (lo == hi || hi <= begin) continue;
#pragma unroll
          for (int e = 0; e < PER_LANE; ++e) {
            const float2 v = left[(o * PER_LANE + e) * 32];
            float2& d = sum[e / (NT * 2)][e / 2 % NT][e % 2];
            d.x += v.x;
            d.y += v.y;
          }
        }
#pragma unroll
        for (int e = 0; e < PER_LANE; ++e) {
          float2& d = acc[e / (NT * 2)][e / 2 % NT][e % 2];
          const float2 v = sum[e / (NT * 2)][e / 2 % NT][e % 2];
          d.x = v.x + d.x;
          d.y = v.y + d.y;
        }
        put(waits, acc);
      }
    }
    part_lo = part_hi;
  }
  asm volatile("cp.async.wait_all;" ::: "memory");
}

constexpr size_t kSmemMost = 226 * 1024;

// The kernel's shapes: stages of 256 codes (128 for groups of 32, which carry
// four scales a row and block), 16 warps an SM, in two CTAs for the gather. From
// 9 vectors on stages of 128 codes and 12 warps (h alone takes 160 KB at d = 5120).
struct Form {
  int nt, warps, sb, ns;
};
constexpr Form form_of(int nt, int group, bool gather) {
  return nt == 2 ? Form{2, 12, 1, 2}
                 : Form{1, gather ? 8 : 16, group == 32 ? 1 : 2, group == 32 ? 4 : 2};
}

size_t smem_bytes(const Form& f, int kd, int group, int vecs, int cols, int slot, bool share) {
  const int blocks = (kd + kBlockK - 1) / kBlockK;
  return (size_t)h_bytes(blocks, vecs, blocks * (kBlockK / group) * cols) +
         (size_t)f.warps * f.ns * (f.sb * 2048 + slot) +
         (share ? (size_t)f.warps * f.nt * 8 * 32 * sizeof(float) : 0);
}

template <bool BF16, int G, int NT, int MODE, bool GATHER, bool COPIED>
cudaError_t launch_one(const Q4Launch& in, int* err, cudaStream_t s) {
  constexpr Form f = form_of(NT, G, GATHER);
  auto kernel = q4_kernel<BF16, G, NT, f.warps, f.sb, f.ns, MODE, GATHER, COPIED>;
  Q4Launch a = in;
  const int kd = a.k_hi - a.k_lo;
  const int vecs = GATHER ? kGatherVecs : a.M < NT * 8 ? a.M : NT * 8;
  const int cols = GATHER ? kGatherVecs : NT * 8;
  const int64_t rows = GATHER ? a.K : a.n;
  const int slot = COPIED ? slot_bytes(MODE == kMins) : 0;
  a.tiles = (int)((rows + kRowsWarp - 1) / kRowsWarp);
  const int64_t tiles = (int64_t)a.tiles * (GATHER ? a.M : 1);
  // tiles are shared where the sums that this hands round fit beside the rest
  // (all but the widest rows with many vectors); a run of tiles counts its
  // stages in 32 bits
  size_t smem = smem_bytes(f, kd, G, vecs, cols, slot, true);
  a.share = smem <= kSmemMost;
  if (!a.share) smem = smem_bytes(f, kd, G, vecs, cols, slot, false);
  static int smem_set[64] = {0};
  cudaError_t e = ensure_dynamic_smem(kernel, smem, smem_set);
  if (e != cudaSuccess) return e;
  const int resident = sm_count() * (f.warps == 8 && 2 * (smem + 1024) <= 228 * 1024 ? 2 : 1);
  const int64_t want = a.share ? tiles : (tiles + f.warps - 1) / f.warps;
  return launch_kernel(true, kernel, dim3((unsigned)(want < resident ? want : resident)),
                       dim3(f.warps * 32), smem, s, a, err);
}

template <bool BF16, int G, int MODE, bool COPIED>
cudaError_t launch_cols(const Q4Launch& a, int* err, cudaStream_t s) {
  if (a.ids) return launch_one<BF16, G, 1, MODE, true, COPIED>(a, err, s);
  if (a.M <= 8 || MODE == kCentred) return launch_one<BF16, G, 1, MODE, false, COPIED>(a, err, s);
  return launch_one<BF16, G, MODE == kCentred ? 1 : 2, MODE, false, false>(a, err, s);
}

template <bool BF16, int G>
cudaError_t launch_mode(const Q4Launch& a, bool copied, int* err, cudaStream_t s) {
  if (a.mins)
    return copied ? launch_cols<BF16, G, kMins, true>(a, err, s)
                  : launch_cols<BF16, G, kMins, false>(a, err, s);
  if (a.d < kCentreD) return launch_cols<BF16, G, kCentred, false>(a, err, s);
  return copied ? launch_cols<BF16, G, kPlain, true>(a, err, s)
                : launch_cols<BF16, G, kPlain, false>(a, err, s);
}

template <bool BF16>
cudaError_t launch_group(const Q4Launch& a, int group, bool copied, int* err, cudaStream_t s) {
  if (group == 128) return launch_mode<BF16, 128>(a, copied, err, s);
  if (group == 64) return launch_mode<BF16, 64>(a, copied, err, s);
  return launch_mode<BF16, 32>(a, copied, err, s);
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
  const uintptr_t at = reinterpret_cast<uintptr_t>(q.scales) | reinterpret_cast<uintptr_t>(q.mins);
  a.scales_aligned = at % 16 == 0;
  const bool centred = !q.mins && q.d < kCentreD;
  // Scales are copied (kernel, COPIED) where rows of them allow it and the slots
  // leave room for h of whole rows and for shared tiles; groups of 32 over the
  // whole head gain nothing by it (one vector 62 us, with loads 60).
  const bool copies = !centred && a.scales_aligned && q.d / q.group % 8 == 0 &&
                      (q.group > 32 || q.ids);
  // hidden vectors of one pass over the rows, then pieces of d, as far as h
  // fits in shared memory; a later piece adds to the former's sums
  const int most = q.ids ? q.M : centred ? 8 : 16;
  for (int m = 0; m < q.M; m += most) {
    a.M = q.M - m < most ? q.M - m : most;
    a.h = static_cast<const uint16_t*>(q.h) + (size_t)m * q.d;
    a.out = q.out + (size_t)m * a.ldo;
    const Form f = form_of(!q.ids && a.M > 8 ? 2 : 1, q.group, q.ids != nullptr);
    const int vecs = q.ids ? kGatherVecs : a.M, cols = q.ids ? kGatherVecs : f.nt * 8;
    const bool copied = copies && f.nt == 1 &&
                        smem_bytes(f, q.d, q.group, vecs, cols, slot_bytes(q.mins), true) <= kSmemMost;
    int piece = q.d;
    // pieces begin at whole 16 bytes of scales
    const int unit = 8 * q.group > kBlockK ? 8 * q.group : kBlockK;
    while (!copied && piece > unit &&
           smem_bytes(f, piece, q.group, vecs, cols, 0, false) > kSmemMost)
      piece = ((piece + 1) / 2 + unit - 1) / unit * unit;
    for (int k = 0; k < q.d; k += piece) {
      a.k_lo = k;
      a.k_hi = k + piece < q.d ? k + piece : q.d;
      a.add = k > 0;
      const cudaError_t e = q.dtype == LMHEAD_BF16 ? launch_group<true>(a, q.group, copied, err, s)
                                                   : launch_group<false>(a, q.group, copied, err, s);
      if (e != cudaSuccess) return e;
    }
  }
  return cudaSuccess;
}

}  // namespace lmhead
