// qmv_kv_attn.cuh -- attention of one new token per sequence over the paged
// cache: the kernel behind kv_attention.  Each of qmv_kv_attn4.cu, 8 and 16
// instantiates it for one width.
//
// The mathematics.  Codes are multiplied as the integers they are, and scales
// and biases applied outside the products: with groups g of a row,
//   s_j   = f * sum_g (sk_jg * sum_{d in g} x_d q_jd + bk_jg * sum_{d in g} x_d)
//   out_d = (sum_j (p_j sv_jg) q_jd + sum_j p_j bv_jg) / sum_j p_j
// so a score costs two fp32 multiply-adds per group beyond its matrix product,
// and the values one multiplication of the probability per group.  Scores are
// kept in units of log2, p_j = 2^(s_j - m), with a running maximum m that is
// raised (and the sums rescaled) only when a score exceeds it by 3, so p <= 8.
//
// Matrix products.  A step takes 16 slots.  Scores: A = 16 slots x 16 elements
// of codes, B = 16 elements x 8 query heads, C = slots x heads.  Values: A = 16
// elements x 16 slots, B = slots x heads (the probabilities, transposed 8x8 in
// registers by movmatrix), C = elements x heads.  mma.sync m16n8k16 holds 8
// heads without padding its 16-row side; one tcgen05 instruction wants 64 or
// 128 rows of A and both products' operands staged through shared or tensor
// memory, which a few query heads over codes that have to be converted in
// registers do not pay for.
//   4- and 8-bit codes are fp16 numbers already: the bits q alone are the
//     subnormal q * 2^-24 (q * 2^-20 where a nibble stays in bits 4 .. 7, which
//     its query element or output makes up for), exactly.  Queries are scaled
//     per head by a power of two that brings the largest to [2^14, 2^15), exact
//     in fp16 for every bf16 within 2^24 of it.  p * scale is rounded once to
//     fp16, after a power of two, common to a warp's slots, that brings the largest
//     scale so far to [2^9, 2^10): by 2^-11 of itself, or below fp16's normal range
//     (2^-23 of that scale) by 2^-34 of the scale.  An output is then 2 to 6 % further
//     from the 64-bit value than its own rounding leaves it; the rest as a second
//     product took that away and 10 % longer at 4 bits (four sequences of 131072
//     slots: 123 -> 135 us), at 8 bits nothing where memory binds and up to 13 %
//     elsewhere (32 x 8192, 8 x 16 heads of 64: 79 -> 90 us).
//   bf16 rows are multiplied as they are, by p as the sum of two bf16 numbers, its
//     rounding and that of the rest (2^-16): with the first alone p's rounding was
//     as large as the output's.  The second product of a tile costs 0.5 % of a call
//     (64 x 255 .. 2047 slots, 4 x 4 heads of 256: 66.4 -> 67.1 us), 3 % with 16
//     heads to a kv head (16 x 512 .. 4096, 4 x 16 of 128: 20.1 -> 20.7).
//   Sums are fp32 throughout.
// The k index of a product may be any permutation of its 16 elements or slots
// as long as both operands agree: it is chosen so that a 32-bit word of codes
// yields whole operand registers (elements (0,4), (1,5), (2,6), (3,7) of a word
// of 4-bit codes) and shared-memory reads meet all 32 banks.
//
// Work.  All (sequence, kv head, 8 or 16 query heads) segments are cut into
// tiles of 16 or 32 slots, numbered through, and shared out evenly over all
// warps of the grid, whatever the lengths: a warp walks a contiguous range with
// a ring of tiles of its own in shared memory, filled by 16-byte cp.async a few
// tiles ahead, and needs no barrier but its own until its range is done.  A
// segment inside a warp's range is written out by it; pieces of a segment are
// joined within the CTA, and those of CTAs by a second kernel, in order.
//
// Bound, and measured (B200): 4-bit rows by the latency of instructions that wait
// for one another, at three warps a scheduler (some 590 for a 32-slot tile of heads of
// 128; 0.60 issued a cycle, and in 0.40 of the cycles no warp ready; full issue would
// take 0.56 of the time, the bytes 0.69: four sequences of 131072 slots, 604 MB, in
// 123 to 139 us); 8-bit rows by memory (8 of 32768, 571 MB, in 97 us, 0.90 of the
// measured copy rate); calls of a few hundred slots by the look-ups, one tile and
// the joins of two dependent kernels (10 us).  With weights the scores go out and
// come back to a second kernel, 7 of 28 us (8 x 1023 .. 8190 slots, 16 heads of 64).
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <cmath>
#include <cstdint>

#include "qmv_kv.h"

namespace qmvc {

struct AttnParams {
  CacheView c;
  const __nv_bfloat16 *q;
  long long q_stride;
  const int *lens;
  __nv_bfloat16 *out;
  int batch, Hq, R;
  int chunks;          // segments of a kv head: ceil(R / heads of a segment)
  int page_blocks;     // 16-slot blocks of a page
  unsigned page_rows;  // rows of a page: kv heads * slots
  float scale_log2;    // |scale| * log2(e)
  uint32_t q_sign;     // flips the queries where scale is negative
  float *weights;      // or null
  int state_width;
  long long room;
  // workspace
  int *cum;            // [batch + 1] tiles before a sequence
  float *scores;       // [batch][Hq][room], with weights
  float2 *stats;       // [batch][Hq] maximum and sum of segments not joined by the second kernel
  int2 *cuts;          // [ctas] segments whose later / first piece a CTA holds, or -1
  float2 *part_ml;     // [ctas][2][heads]
  float4 *part_o;      // [ctas][2] pieces of `quads` float4 (write_piece)
  float4 *warp_o;      // [ctas][warps] pieces
  int ctas;
};

constexpr float kNegInf = -__builtin_huge_valf();
constexpr float kLazy = 3.0f;  // p <= 2^kLazy

// A score in units of log2.  It is rounded before the maximum is subtracted, here as
// in the maximum itself and in the stored scores: their differences are then exact
// multiples of its last step.  (A fused multiply-add would subtract the maximum's
// rounding from a score without it, which at scores of 2^30 is 2^6 of an exponent,
// and at 2^9 3e-5 of a weight.)
__device__ __forceinline__ float scaled(float s, float f) { return __fmul_rn(s, f); }

template <int BITS_, int D_, int GS_, int NB_>
struct AttnCfg {
  static constexpr int BITS = BITS_, D = D_, GS = BITS_ == 16 ? D_ : GS_, NB = NB_;
  static constexpr int HEADS = 8 * NB;                 // query heads of a segment
  static constexpr int G = BITS == 16 ? 0 : D / GS;    // groups of a row
  static constexpr int RB = D * BITS / 8;              // bytes of a row
  static constexpr int CH = RB / 16;                   // 16-byte chunks of a row
  // Warps of an SM, by the registers of the accumulators: 16 in two CTAs where
  // they are 16 (128 registers a thread: heads of 64 took 28.4 us for 52 MB, 29.1
  // with 12 warps), 12 where they are up to 32 (168: heads of 128 took 126 us for
  // 604 MB and 47.7 us for 168 MB in groups of 32, with 16 warps 132 and 56.9 us),
  // else 8.  bf16 rows need few instructions and deep rings: 8, and 4 for heads
  // of 256, whose tiles are 16 KB.
  static constexpr bool LIGHT = BITS != 16 && D * NB <= 64, SMALL = BITS != 16 && D * NB <= 128;
  static constexpr int WARPS = LIGHT ? 8 : SMALL ? 12 : BITS == 16 && D == 256 ? 4 : 8;
  static constexpr int CTAS_PER_SM = LIGHT ? 2 : 1;
  static constexpr int ROOM = (LIGHT ? 110592 : SMALL ? 196608 : 204800) / WARPS;  // bytes of a warp's ring
  // 4-bit tiles are 32 slots where three of them fit: half as many softmax
  // steps for the same bytes
  static constexpr int SLOT = 2 * RB + 8 * G;          // bytes of a slot
  static constexpr int TB = BITS == 4 && SMALL && 3 * 32 * SLOT <= ROOM ? 2 : 1;  // 16-slot blocks
  static constexpr int TILE = 16 * TB;
  static constexpr int STAGE = TILE * SLOT;
  static constexpr int RING = ROOM / STAGE;
  // two tiles in flight, or 4 KB of them: 64 KB to an SM, where the latency of
  // a copy times its share of the bandwidth is about 45 KB (more only made
  // the start longer)
  static constexpr int WANT = 2 + (4096 + STAGE - 1) / STAGE;
  static constexpr int STAGES = RING < WANT ? RING : WANT;
  static_assert(STAGES >= 2, "a tile is fetched while another is computed");
  static constexpr int TAIL = HEADS * D * 4;           // a warp's last piece
  static constexpr int SMEM = WARPS * (STAGES * STAGE > TAIL ? STAGES * STAGE : TAIL);
  // attn_kernel's arrays of fixed size, and up to 128 bytes to align the rings
  static constexpr int FIXED = 40 * WARPS * HEADS + 8 * WARPS + 128 + 128;
  static_assert(SMEM + 4 * 4097 + FIXED <= 232448, "rings, the tiles' sums of 4096 sequences, and the rest");
  static constexpr int MT = D / 16;                    // 16-element accumulator tiles
  static constexpr int QUADS = HEADS * D / 4;          // float4 of a piece
  // elements that one set of value words covers
  static constexpr int VCH = BITS == 4 && GS >= 64 ? 64 : 32;
};

// Chunk swizzle of row r and the slot that product row r stands for, chosen
// per row size so that the score reads (8 rows, one chunk) and the value reads
// (4 rows, two chunks) each meet all banks.
template <int CH>
__device__ __forceinline__ int swizzle(int r) {
  if constexpr (CH == 2 || CH == 6) return (r >> 2) & 1;
  else if constexpr (CH == 4 || CH == 12) return (r >> 1) & 3;
  else if constexpr (CH == 3) return 0;
  else return r & 7;
}
template <int CH>
__device__ __forceinline__ int slot_of(int r) {  // r < 8
  if constexpr (CH == 2) return ((r & 1) << 2) | (r >> 1);
  else if constexpr (CH == 4) return (r & 4) | ((r & 1) << 1) | ((r >> 1) & 1);
  else return r;
}

// Address of 16-byte chunk `chunk` (a constant) of a row, from that of its chunk
// 0 (swizzled): the swizzle's bits are exchanged, the others added.
template <int CH>
__device__ __forceinline__ uint32_t chunk_at(uint32_t row0, int chunk) {
  constexpr int kBits = CH == 3 ? 0 : CH == 2 || CH == 6 ? 1 : CH == 4 || CH == 12 ? 3 : 7;
  return (row0 ^ ((chunk & kBits) << 4)) + ((chunk & ~kBits) << 4);
}

__device__ __forceinline__ uint32_t smem_addr(const void *p) {
  return static_cast<uint32_t>(__cvta_generic_to_shared(p));
}
__device__ __forceinline__ void cp_async16(uint32_t dst, const void *src, int bytes) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;\n" ::"r"(dst), "l"(src), "r"(bytes)
               : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;\n" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_wait() {
  asm volatile("cp.async.wait_group %0;\n" ::"n"(N) : "memory");
}
__device__ __forceinline__ uint32_t ld_s32(uint32_t a) {
  uint32_t v;
  asm volatile("ld.shared.u32 %0, [%1];\n" : "=r"(v) : "r"(a));
  return v;
}
template <bool TRANS>
__device__ __forceinline__ void ldmatrix4(uint32_t (&r)[4], uint32_t a) {
  if constexpr (TRANS)
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];\n"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(a));
  else
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];\n"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(a));
}
__device__ __forceinline__ uint32_t movmatrix(uint32_t v) {
  uint32_t r;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;\n" : "=r"(r) : "r"(v));
  return r;
}
template <bool BF16>
__device__ __forceinline__ void mma(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                    uint32_t a3, uint32_t b0, uint32_t b1) {
  if constexpr (BF16)
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
        "{%8,%9}, {%0,%1,%2,%3};\n"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
  else
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
        "{%8,%9}, {%0,%1,%2,%3};\n"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ float ex2(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;\n" : "=f"(r) : "f"(x));
  return r;
}
__device__ __forceinline__ float pow2(int e) {  // e in [-126, 127]
  return __uint_as_float(static_cast<uint32_t>(e + 127) << 23);
}
__device__ __forceinline__ __half2 as_half2(uint32_t v) {
  return *reinterpret_cast<const __half2 *>(&v);
}
__device__ __forceinline__ __nv_bfloat162 as_bf162(uint32_t v) {
  return *reinterpret_cast<const __nv_bfloat162 *>(&v);
}
__device__ __forceinline__ uint32_t as_u32(__half2 v) { return *reinterpret_cast<uint32_t *>(&v); }
template <bool BF16>
__device__ __forceinline__ uint32_t pack16(float lo, float hi) {
  if constexpr (BF16) {
    __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<uint32_t *>(&v);
  } else {
    return as_u32(__floats2half2_rn(lo, hi));
  }
}

// Codes as fp16 numbers without any conversion: the bits q alone are the fp16
// subnormal q * 2^-24, exactly, and products take subnormals as they are.
// Nibbles (j, j + 4) of x's 16-bit halves, j = 0 .. 3: q * 2^-24 for even j,
// q * 2^-20 for odd j (bits 4 .. 7 of the fraction).
__device__ __forceinline__ void nibbles(uint32_t x, uint32_t (&o)[4]) {
  const uint32_t y = x >> 8;
  o[0] = x & 0x000f000fu;
  o[1] = x & 0x00f000f0u;
  o[2] = y & 0x000f000fu;
  o[3] = y & 0x00f000f0u;
}
// Bytes (0, 1) or (2, 3) of x: q * 2^-24.
template <int PAIR>
__device__ __forceinline__ uint32_t bytes16(uint32_t x) {
  return __byte_perm(x, 0u, PAIR ? 0x4342 : 0x4140);
}
// Both nibbles' products of a byte come from the byte and its low nibble:
// sum p (16 hi + lo) and sum p lo give sum p hi, which spares a mask.  Bytes 0
// and 1 of x's 16-bit halves: o[0], o[2] the low nibbles, o[1], o[3] the bytes.
__device__ __forceinline__ void nibble_bytes(uint32_t x, uint32_t (&o)[4]) {
  o[1] = x & 0x00ff00ffu;
  o[3] = __byte_perm(x, 0u, 0x4341);
  o[0] = x & 0x000f000fu;
  o[2] = o[3] & 0x000f000fu;
}
constexpr float kUnit = 5.9604644775390625e-8f;  // 2^-24

// G bf16 values at shared address a, as pairs of bits.
template <int G>
__device__ __forceinline__ void ld_groups(uint32_t a, uint32_t (&v)[(G + 1) / 2]) {
  if constexpr (G == 1) {
    uint16_t x;
    asm volatile("ld.shared.u16 %0, [%1];\n" : "=h"(x) : "r"(a));
    v[0] = x;
  } else if constexpr (G == 2) {
    v[0] = ld_s32(a);
  } else if constexpr (G == 3) {  // heads of 96: 6 bytes, 2-byte aligned
    uint16_t x[3];
#pragma unroll
    for (int i = 0; i < 3; ++i)
      asm volatile("ld.shared.u16 %0, [%1];\n" : "=h"(x[i]) : "r"(a + 2 * i));
    v[0] = x[0] | (static_cast<uint32_t>(x[1]) << 16);
    v[1] = x[2];
  } else if constexpr (G == 4) {
    asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];\n" : "=r"(v[0]), "=r"(v[1]) : "r"(a));
  } else {
    asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];\n"
                 : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]) : "r"(a));
  }
}
__device__ __forceinline__ float group_value(const uint32_t *v, int g) {
  return (g & 1) ? __uint_as_float(v[g / 2] & 0xffff0000u) : __uint_as_float(v[g / 2] << 16);
}

// Element of accumulator tile mt, product row lane/4 + 8*half.
template <class C>
__device__ __forceinline__ int element_of(int mt, int half, int g) {
  if constexpr (C::BITS == 16) return 16 * mt + g + 8 * half;
  else if constexpr (C::BITS == 8) return 32 * (mt / 2) + 4 * g + 2 * half + mt % 2;
  else if constexpr (C::VCH == 64) return 64 * (mt / 4) + 8 * g + 4 * half + mt % 4;
  else return 32 * (mt / 2) + 8 * (g & 3) + 4 * (g >> 2) + 2 * half + mt % 2;
}

__device__ __forceinline__ int clipped_length(const AttnParams &p, int b) {
  const int len = __ldg(p.lens + b);
  return len < 0 ? 0 : len < p.room ? len : static_cast<int>(p.room);
}

// Fewest tiles of a CTA: with 8 a 2000-slot sequence of 8 kv heads took 11.5 us,
// with 4, 2 and 1 (more CTAs to join) 12.5, 14.2 and 19.6 us; calls of a few
// hundred slots did not differ.
constexpr int kFew = 8;

// How `total` tiles are shared out: over every CTA, or as many as have kFew
// each.  CTA i has `base` tiles, and one more where i < extra; within it its
// warps share them the same way.
struct Share {
  int ctas, base, extra;
  __device__ __forceinline__ Share(int total, int most) {
    const int need = (total + kFew - 1) / kFew;
    ctas = need < most ? need : most;
    base = ctas ? total / ctas : 0;
    extra = total - base * ctas;
  }
  __device__ __forceinline__ int first(int cta) const {
    return cta * base + (cta < extra ? cta : extra);
  }
  __device__ __forceinline__ int cta_of(int tile) const {
    const int bound = extra * (base + 1);
    return tile < bound ? tile / (base + 1) : extra + (tile - bound) / base;
  }
};

// Position in the numbered tiles.
struct Cursor {
  int b, hc, tile, tiles, n;  // sequence, segment within it, tile, tiles of a segment, slots
};

template <class C>
__device__ __forceinline__ void cursor_sequence(const AttnParams &p, Cursor &k) {
  k.n = clipped_length(p, k.b);
  k.tiles = (k.n + C::TILE - 1) / C::TILE;
}

// With at most 32 sequences, lane i knows sequence i: its slots, and the tiles
// up to its end.
struct Known {
  int n, upto;
};
template <class C>
__device__ __forceinline__ Cursor cursor_at(const AttnParams &p, const int *cum, Known known, int u) {
  int lo = 0;
  if (p.batch <= 32) {
    lo = __popc(__ballot_sync(0xffffffffu, known.upto <= u));
  } else {
    int hi = p.batch;  // cum[lo] <= u < cum[hi]
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (cum[mid] <= u) lo = mid;
      else hi = mid;
    }
  }
  Cursor k;
  k.b = lo;
  if (p.batch <= 32) {
    k.n = __shfl_sync(0xffffffffu, known.n, lo);
    k.tiles = (k.n + C::TILE - 1) / C::TILE;
  } else {
    cursor_sequence<C>(p, k);
  }
  const int rest = u - cum[lo];
  k.hc = rest / k.tiles;
  k.tile = rest - k.hc * k.tiles;
  return k;
}

// True when the next tile is another segment's.
template <class C>
__device__ __forceinline__ bool cursor_next(const AttnParams &p, const int *cum, Cursor &k) {
  if (++k.tile < k.tiles) return false;
  k.tile = 0;
  if (++k.hc == p.c.H * p.chunks) {
    k.hc = 0;
    do ++k.b;
    while (k.b < p.batch && cum[k.b + 1] == cum[k.b]);
    if (k.b < p.batch) cursor_sequence<C>(p, k);
  }
  return true;
}

// What a warp carries through a segment.  Lane (g, t) = (lane / 4, lane % 4)
// has heads 2t and 2t + 1 of each block of 8.
template <class C>
struct Segment {
  uint32_t q[C::NB][C::D / 8];                       // B operands of the scores
  float x[C::G ? C::G : 1][C::NB][2];                // sums of a group's queries
  float f[C::NB][2];                                 // score units of a head
  float o[C::MT][C::NB][4];
  float m[C::NB][2], l[C::NB][2];
  float pb[C::G ? C::G : 1][C::NB][2];               // sums of p * bias
  float allow[C::NB][2];                             // scores up to here leave m as it is
  uint32_t limit;                                    // largest scale for vexp, a pair of bf16
  int vexp;                                          // values are scaled by 2^vexp

  __device__ __forceinline__ void allow_scales(int e) {
    vexp = e;
    limit = (__float_as_uint(4096.0f * pow2(-e)) >> 16) * 0x10001u;  // a power of two
  }

  // elements of a lane's word, and words of a row that it has
  static constexpr int PER = C::BITS == 16 ? 2 : 32 / C::BITS, STEPS = C::D / (4 * PER);

  // The queries' bits, as they are (begin() makes operands of them): elements
  // of word t + 4 i, or for bf16 rows the operands themselves.
  __device__ __forceinline__ void load(const AttnParams &p, const Cursor &k, int lane) {
    const int g = lane >> 2, t = lane & 3;
    const int hk = p.chunks == 1 ? k.hc : k.hc / p.chunks, ch = k.hc - hk * p.chunks;
#pragma unroll
    for (int nb = 0; nb < C::NB; ++nb) {
      const int r = ch * C::HEADS + nb * 8 + g;
      const bool live = r < p.R;
      const __nv_bfloat16 *row = p.q + k.b * p.q_stride + (hk * p.R + (live ? r : 0)) * C::D;
#pragma unroll
      for (int i = 0; i < STEPS; ++i) {
        const __nv_bfloat16 *w = row + PER * (t + 4 * i);
        if constexpr (C::BITS == 4) {
          const uint4 v = live ? __ldg(reinterpret_cast<const uint4 *>(w)) : make_uint4(0, 0, 0, 0);
          q[nb][4 * i] = v.x; q[nb][4 * i + 1] = v.y; q[nb][4 * i + 2] = v.z; q[nb][4 * i + 3] = v.w;
        } else if constexpr (C::BITS == 8) {
          const uint2 v = live ? __ldg(reinterpret_cast<const uint2 *>(w)) : make_uint2(0, 0);
          q[nb][2 * i] = v.x; q[nb][2 * i + 1] = v.y;
        } else {
          q[nb][i] = live ? __ldg(reinterpret_cast<const uint32_t *>(w)) : 0u;
        }
      }
    }
  }

  __device__ __forceinline__ void begin(const AttnParams &p, int lane) {
    const int t = lane & 3;
#pragma unroll
    for (int nb = 0; nb < C::NB; ++nb) {
#pragma unroll
      for (int i = 0; i < C::D / 8; ++i) q[nb][i] ^= p.q_sign;
      if constexpr (C::BITS == 16) {
        f[nb][0] = f[nb][1] = p.scale_log2;
      } else {
        uint32_t top = 0u;
#pragma unroll
        for (int i = 0; i < C::D / 8; ++i)
          top = max(top, max(q[nb][i] & 0x7fffu, (q[nb][i] >> 16) & 0x7fffu));
        top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
        top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
        // 2^e brings the largest to [2^14, 2^15); -114 <= e <= 126 keeps 2^e normal
        int e = top >= 0x80u ? 14 - (static_cast<int>(top >> 7) - 127) : 126;
        e = e > 126 ? 126 : e;
        const float up = pow2(e);
        float sums[C::G];
#pragma unroll
        for (int i = 0; i < C::G; ++i) sums[i] = 0.0f;
#pragma unroll
        for (int i = 0; i < STEPS; ++i) {
          float v[PER];
#pragma unroll
          for (int j = 0; j < PER / 2; ++j) {
            const uint32_t raw = q[nb][PER / 2 * i + j];
            v[2 * j] = __uint_as_float(raw << 16) * up;
            v[2 * j + 1] = __uint_as_float(raw & 0xffff0000u) * up;
          }
          if constexpr (PER == 8) {
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              const float odd = j & 1 ? 0.0625f : 1.0f;  // those nibbles count 16 times
              q[nb][4 * i + j] = pack16<false>(v[j] * odd, v[j + 4] * odd);
            }
          } else {
            q[nb][2 * i] = pack16<false>(v[0], v[1]);
            q[nb][2 * i + 1] = pack16<false>(v[2], v[3]);
          }
#pragma unroll
          for (int j = 0; j < PER; ++j) sums[i * 4 * PER / C::GS] += v[j];
        }
        // never 0, so that a masked score times it is -inf
        const float unit = fmaxf(p.scale_log2 * pow2(-e) * (1.0f / kUnit), 1.17549435e-38f);
#pragma unroll
        for (int i = 0; i < C::G; ++i) {
          sums[i] += __shfl_xor_sync(0xffffffffu, sums[i], 1);
          sums[i] += __shfl_xor_sync(0xffffffffu, sums[i], 2);
          // head h's sums are in lanes 4 h .. 4 h + 3
          x[i][nb][0] = __shfl_sync(0xffffffffu, sums[i] * kUnit, 8 * t);
          x[i][nb][1] = __shfl_sync(0xffffffffu, sums[i] * kUnit, 8 * t + 4);
        }
        f[nb][0] = __shfl_sync(0xffffffffu, unit, 8 * t);
        f[nb][1] = __shfl_sync(0xffffffffu, unit, 8 * t + 4);
      }
      m[nb][0] = m[nb][1] = allow[nb][0] = allow[nb][1] = kNegInf;
      l[nb][0] = l[nb][1] = 0.0f;
#pragma unroll
      for (int i = 0; i < C::MT; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) o[i][nb][j] = 0.0f;
#pragma unroll
      for (int i = 0; i < C::G; ++i) pb[i][nb][0] = pb[i][nb][1] = 0.0f;
    }
    allow_scales(126);
  }

  // The sums over all lanes of the warp: l, and the values in true units.
  __device__ __forceinline__ void finish() {
    const float back = C::BITS == 16 ? 1.0f : pow2(-vexp);
#pragma unroll
    for (int nb = 0; nb < C::NB; ++nb)
#pragma unroll
      for (int i = 0; i < 2; ++i) {
#pragma unroll
        for (int s = 4; s < 32; s <<= 1) l[nb][i] += __shfl_xor_sync(0xffffffffu, l[nb][i], s);
        if constexpr (C::BITS != 16) {
#pragma unroll
          for (int g = 0; g < C::G; ++g)
#pragma unroll
            for (int s = 4; s < 32; s <<= 1)
              pb[g][nb][i] += __shfl_xor_sync(0xffffffffu, pb[g][nb][i], s);
#pragma unroll
          for (int mt = 0; mt < C::MT; ++mt) {
            const int g = mt * 16 / C::GS;
            if (C::BITS == 4 && mt % 2 == 0) {  // the odd tile held 16 hi + lo
              o[mt + 1][nb][i] = (o[mt + 1][nb][i] - o[mt][nb][i]) * 0.0625f;
              o[mt + 1][nb][i + 2] = (o[mt + 1][nb][i + 2] - o[mt][nb][i + 2]) * 0.0625f;
            }
            o[mt][nb][i] = fmaf(o[mt][nb][i] * (1.0f / kUnit), back, pb[g][nb][i]);
            o[mt][nb][i + 2] = fmaf(o[mt][nb][i + 2] * (1.0f / kUnit), back, pb[g][nb][i]);
          }
        }
      }
  }
};

// Whether a table entry names a page outside the cache.
static __device__ __noinline__ bool outside(const int *entry, int num_pages) {
  return static_cast<unsigned>(__ldg(entry)) >= static_cast<unsigned>(num_pages);
}

// One tile's scores, softmax step and value products.
template <class C>
__device__ __forceinline__ void attend_tile(Segment<C> &sg, const AttnParams &p, const Cursor &k,
                                            uint32_t stage, bool bad, int lane) {
  constexpr bool BF = C::BITS == 16;
  constexpr int GW = C::G ? (C::G + 1) / 2 : 1;
  const int g = lane >> 2, t = lane & 3;
  const int row = slot_of<C::CH>(g), sw = swizzle<C::CH>(row);
  const uint32_t kbase = stage, vbase = stage + C::TILE * C::RB;
  const uint32_t sbase = stage + 2 * C::TILE * C::RB;
  constexpr uint32_t kArr = C::TILE * C::G * 2;
  float s[C::TB][C::NB][4];

#pragma unroll
  for (int blk = 0; blk < C::TB; ++blk) {
    const uint32_t kb = kbase + blk * 16 * C::RB;
    if constexpr (BF) {
      float c[C::NB][4] = {};
      const uint32_t a0 = kb + (lane & 15) * C::RB + (((lane >> 4) ^ swizzle<C::CH>(lane & 7)) << 4);
#pragma unroll
      for (int i = 0; i < C::D / 16; ++i) {
        uint32_t a[4];
        ldmatrix4<false>(a, chunk_at<C::CH>(a0, 2 * i));
#pragma unroll
        for (int nb = 0; nb < C::NB; ++nb)
          mma<true>(c[nb], a[0], a[1], a[2], a[3], sg.q[nb][2 * i], sg.q[nb][2 * i + 1]);
      }
#pragma unroll
      for (int nb = 0; nb < C::NB; ++nb)
#pragma unroll
        for (int j = 0; j < 4; ++j) s[blk][nb][j] = c[nb][j];
    } else {
      uint32_t ska[GW], skb[GW], bka[GW], bkb[GW];
      const uint32_t sa = sbase + (blk * 16 + row) * C::G * 2;
      ld_groups<C::G>(sa, ska);
      ld_groups<C::G>(sa + 16 * C::G, skb);
      ld_groups<C::G>(sa + kArr, bka);
      ld_groups<C::G>(sa + kArr + 16 * C::G, bkb);
#pragma unroll
      for (int nb = 0; nb < C::NB; ++nb)
#pragma unroll
        for (int j = 0; j < 4; ++j) s[blk][nb][j] = 0.0f;
      constexpr int SPAN = C::BITS == 4 ? 32 : 16;  // elements of four lanes' words
      constexpr int PER_GROUP = C::GS / SPAN;
      const uint32_t ka = kb + row * C::RB + (sw << 4) + 4 * t;
#pragma unroll
      for (int gr = 0; gr < C::G; ++gr) {
        float c[C::NB][4] = {};
#pragma unroll
        for (int ii = 0; ii < PER_GROUP; ++ii) {
          const int i = gr * PER_GROUP + ii;
          const uint32_t at = chunk_at<C::CH>(ka, i);
          const uint32_t w0 = ld_s32(at), w1 = ld_s32(at + 8 * C::RB);
          if constexpr (C::BITS == 4) {
            uint32_t u[4], v[4];
            nibbles(w0, u);
            nibbles(w1, v);
#pragma unroll
            for (int nb = 0; nb < C::NB; ++nb) {
              mma<false>(c[nb], u[0], v[0], u[1], v[1], sg.q[nb][4 * i], sg.q[nb][4 * i + 1]);
              mma<false>(c[nb], u[2], v[2], u[3], v[3], sg.q[nb][4 * i + 2], sg.q[nb][4 * i + 3]);
            }
          } else {
            const uint32_t u0 = bytes16<0>(w0), u1 = bytes16<1>(w0);
            const uint32_t v0 = bytes16<0>(w1), v1 = bytes16<1>(w1);
#pragma unroll
            for (int nb = 0; nb < C::NB; ++nb)
              mma<false>(c[nb], u0, v0, u1, v1, sg.q[nb][2 * i], sg.q[nb][2 * i + 1]);
          }
        }
        const float s0 = group_value(ska, gr), s1 = group_value(skb, gr);
        const float b0 = group_value(bka, gr), b1 = group_value(bkb, gr);
#pragma unroll
        for (int nb = 0; nb < C::NB; ++nb)
#pragma unroll
          for (int j = 0; j < 4; ++j)
            s[blk][nb][j] = fmaf(j < 2 ? s0 : s1, c[nb][j],
                                 fmaf(j < 2 ? b0 : b1, sg.x[gr][nb][j & 1], s[blk][nb][j]));
      }
    }
  }

  // slots past the sequence's, or of a page outside the cache, take no part
  const int t0 = k.tile * C::TILE;
  if (bad || t0 + C::TILE > k.n) {
#pragma unroll
    for (int blk = 0; blk < C::TB; ++blk) {
      const int first = t0 + 16 * blk;
      const bool off = bad && first < k.n &&
                       outside(p.c.table + static_cast<long long>(k.b) * p.c.width + first / p.c.S,
                               p.c.num_pages);
#pragma unroll
      for (int j = 0; j < 4; ++j)
        if (off || t0 + 16 * blk + row + 8 * (j >> 1) >= k.n)
#pragma unroll
          for (int nb = 0; nb < C::NB; ++nb) s[blk][nb][j] = kNegInf;
    }
  }
  if (p.scores) {
    const int hk = p.chunks == 1 ? k.hc : k.hc / p.chunks, r0 = (k.hc - hk * p.chunks) * C::HEADS + 2 * t;
    float *to = p.scores + (static_cast<long long>(k.b) * p.Hq + hk * p.R + r0) * p.room + t0 + row;
    const int have = k.n - t0 - row;  // slots behind this lane's first that count
#pragma unroll
    for (int nb = 0; nb < C::NB; ++nb)
#pragma unroll
      for (int i = 0; i < 2; ++i)
        if (r0 + nb * 8 + i < p.R) {
          float *at = to + (nb * 8 + i) * p.room;
#pragma unroll
          for (int blk = 0; blk < C::TB; ++blk)
#pragma unroll
            for (int half = 0; half < 2; ++half)
              if (16 * blk + 8 * half < have) at[16 * blk + 8 * half] = scaled(s[blk][nb][i + 2 * half], sg.f[nb][i]);
        }
  }

  // The running maximum is looked at lane by lane: only when some lane's slots
  // exceed what it allows are the lanes' maxima brought together.
  float top[C::NB][2];
  bool raise = false;
#pragma unroll
  for (int nb = 0; nb < C::NB; ++nb)
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      float x = fmaxf(s[0][nb][i], s[0][nb][i + 2]);
#pragma unroll
      for (int blk = 1; blk < C::TB; ++blk) x = fmaxf(x, fmaxf(s[blk][nb][i], s[blk][nb][i + 2]));
      top[nb][i] = x;
      raise |= x > sg.allow[nb][i];
    }
  uint32_t sva[C::TB][GW], svb[C::TB][GW];
  __nv_bfloat162 wide[GW];  // the largest scales, in pairs
  if constexpr (!BF) {
#pragma unroll
    for (int blk = 0; blk < C::TB; ++blk) {
      const uint32_t a = sbase + 2 * kArr + (blk * 16 + row) * C::G * 2;
      ld_groups<C::G>(a, sva[blk]);
      ld_groups<C::G>(a + 16 * C::G, svb[blk]);
#pragma unroll
      for (int i = 0; i < GW; ++i) {
        const __nv_bfloat162 m = __hmax2(__habs2(as_bf162(sva[blk][i])), __habs2(as_bf162(svb[blk][i])));
        wide[i] = blk ? __hmax2(wide[i], m) : m;
      }
    }
#pragma unroll
    for (int i = 1; i < GW; ++i) wide[0] = __hmax2(wide[0], wide[i]);
    raise |= !__hble2(wide[0], as_bf162(sg.limit));  // NaN scales do not count as small
  }
  if (__any_sync(0xffffffffu, raise)) {
    float ratio = 1.0f;
    if constexpr (!BF) {
      float large = fmaxf(__low2float(wide[0]), __high2float(wide[0]));
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) large = fmaxf(large, __shfl_xor_sync(0xffffffffu, large, o));
      if (large > group_value(&sg.limit, 0)) {
        int e = 9 - (static_cast<int>(__float_as_uint(large) >> 23) - 127);
        e = e > 126 ? 126 : e < -118 ? -118 : e;
        const int step = e - sg.vexp;  // below 0
        ratio = step < -126 ? 0.0f : pow2(step);
        sg.allow_scales(e);
      }
    }
#pragma unroll
    for (int nb = 0; nb < C::NB; ++nb)
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        float x = top[nb][i];
#pragma unroll
        for (int o = 4; o < 32; o <<= 1) x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, o));
        const float m = fmaxf(sg.m[nb][i], scaled(x, sg.f[nb][i]));
        const float a = m == kNegInf ? 1.0f : ex2(sg.m[nb][i] - m);
        sg.m[nb][i] = m;
        // below the quotient by more than its roundings and the product's: a score
        // that is allowed is m + kLazy at most, whatever the steps at m are
        const float up = (m + kLazy) / sg.f[nb][i];
        sg.allow[nb][i] = m == kNegInf ? kNegInf : fmaf(fabsf(up), -0x1p-21f, up);
        sg.l[nb][i] *= a;
#pragma unroll
        for (int gr = 0; gr < C::G; ++gr) sg.pb[gr][nb][i] *= a;
        const float ar = a * ratio;
#pragma unroll
        for (int mt = 0; mt < C::MT; ++mt) {
          sg.o[mt][nb][i] *= ar;
          sg.o[mt][nb][i + 2] *= ar;
        }
      }
  }
  const float power = BF ? 1.0f : pow2(sg.vexp);
#pragma unroll
  for (int nb = 0; nb < C::NB; ++nb)
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const float m = sg.m[nb][i] == kNegInf ? 0.0f : sg.m[nb][i];
#pragma unroll
      for (int blk = 0; blk < C::TB; ++blk)
#pragma unroll
        for (int j = i; j < 4; j += 2) {
          s[blk][nb][j] = ex2(__fsub_rn(scaled(s[blk][nb][j], sg.f[nb][i]), m));
          sg.l[nb][i] += s[blk][nb][j];
        }
    }

  // values
#pragma unroll
  for (int blk = 0; blk < C::TB; ++blk) {
    const uint32_t vb = vbase + blk * 16 * C::RB;
    if constexpr (BF) {
      uint32_t b[C::NB][2], rest[C::NB][2];
#pragma unroll
      for (int nb = 0; nb < C::NB; ++nb)
#pragma unroll
        for (int half = 0; half < 2; ++half) {
          const float x0 = s[blk][nb][2 * half], x1 = s[blk][nb][2 * half + 1];
          const uint32_t hi = pack16<true>(x0, x1);
          b[nb][half] = movmatrix(hi);
          rest[nb][half] = movmatrix(pack16<true>(x0 - __uint_as_float(hi << 16),
                                                  x1 - __uint_as_float(hi & 0xffff0000u)));
        }
      const int r = (lane & 7) + ((lane >> 4) << 3);
      const uint32_t a0 = vb + r * C::RB + ((((lane >> 3) & 1) ^ swizzle<C::CH>(lane & 7)) << 4);
#pragma unroll
      for (int mt = 0; mt < C::MT; ++mt) {
        uint32_t a[4];
        ldmatrix4<true>(a, chunk_at<C::CH>(a0, 2 * mt));
#pragma unroll
        for (int nb = 0; nb < C::NB; ++nb) {
          mma<true>(sg.o[mt][nb], a[0], a[1], a[2], a[3], b[nb][0], b[nb][1]);
          mma<true>(sg.o[mt][nb], a[0], a[1], a[2], a[3], rest[nb][0], rest[nb][1]);
        }
      }
    } else {
      uint32_t bva[GW], bvb[GW];
      const uint32_t ba = sbase + 3 * kArr + (blk * 16 + row) * C::G * 2;
      ld_groups<C::G>(ba, bva);
      ld_groups<C::G>(ba + 16 * C::G, bvb);
      // the four slots of this lane's operand columns, and their rows
      const int ra = slot_of<C::CH>(2 * t), rb = slot_of<C::CH>(2 * t + 1);
      const int xa = swizzle<C::CH>(ra), xb = swizzle<C::CH>(rb);
      const int w0 = C::VCH == 32 && C::BITS == 4 ? g & 3 : g;  // word of the first set
      const uint32_t va = vb + ra * C::RB + (((w0 >> 2) ^ xa) << 4) + ((w0 & 3) << 2);
      const uint32_t vc = vb + rb * C::RB + (((w0 >> 2) ^ xb) << 4) + ((w0 & 3) << 2);
#pragma unroll
      for (int gr = 0; gr < C::G; ++gr) {
        uint32_t b[C::NB][2];
        const float s0 = group_value(sva[blk], gr) * power, s1 = group_value(svb[blk], gr) * power;
        const float b0 = group_value(bva, gr), b1 = group_value(bvb, gr);
#pragma unroll
        for (int nb = 0; nb < C::NB; ++nb) {
          const float(&x)[4] = s[blk][nb];
          b[nb][0] = movmatrix(pack16<false>(x[0] * s0, x[1] * s0));
          b[nb][1] = movmatrix(pack16<false>(x[2] * s1, x[3] * s1));
          sg.pb[gr][nb][0] += x[0] * b0 + x[2] * b1;
          sg.pb[gr][nb][1] += x[1] * b0 + x[3] * b1;
        }
#pragma unroll
        for (int cc = 0; cc < C::GS / C::VCH; ++cc) {
          const int c = gr * (C::GS / C::VCH) + cc;
          const int chunk = c * (C::VCH == 32 && C::BITS == 4 ? 1 : 2);
          const uint32_t aa = chunk_at<C::CH>(va, chunk), ab = chunk_at<C::CH>(vc, chunk);
          const uint32_t w0 = ld_s32(aa), w1 = ld_s32(ab);
          const uint32_t w2 = ld_s32(aa + 8 * C::RB), w3 = ld_s32(ab + 8 * C::RB);
          if constexpr (C::BITS == 8) {
            const uint32_t e0 = __byte_perm(w0, w1, 0x5140), e1 = __byte_perm(w0, w1, 0x7362);
            const uint32_t e2 = __byte_perm(w2, w3, 0x5140), e3 = __byte_perm(w2, w3, 0x7362);
            const uint32_t u0 = bytes16<0>(e0), u1 = bytes16<1>(e0), u2 = bytes16<0>(e1), u3 = bytes16<1>(e1);
            const uint32_t z0 = bytes16<0>(e2), z1 = bytes16<1>(e2), z2 = bytes16<0>(e3), z3 = bytes16<1>(e3);
#pragma unroll
            for (int nb = 0; nb < C::NB; ++nb) {
              mma<false>(sg.o[2 * c][nb], u0, u2, z0, z2, b[nb][0], b[nb][1]);
              mma<false>(sg.o[2 * c + 1][nb], u1, u3, z1, z3, b[nb][0], b[nb][1]);
            }
          } else if constexpr (C::VCH == 64) {
            uint32_t u[4], v[4], y[4], z[4];
            nibble_bytes(__byte_perm(w0, w1, 0x5410), u);
            nibble_bytes(__byte_perm(w0, w1, 0x7632), v);
            nibble_bytes(__byte_perm(w2, w3, 0x5410), y);
            nibble_bytes(__byte_perm(w2, w3, 0x7632), z);
#pragma unroll
            for (int j = 0; j < 4; ++j)
#pragma unroll
              for (int nb = 0; nb < C::NB; ++nb)
                mma<false>(sg.o[4 * c + j][nb], u[j], v[j], y[j], z[j], b[nb][0], b[nb][1]);
          } else {
            const uint32_t sel = g < 4 ? 0x5410u : 0x7632u;
            uint32_t u[4], y[4];
            nibble_bytes(__byte_perm(w0, w1, sel), u);
            nibble_bytes(__byte_perm(w2, w3, sel), y);
#pragma unroll
            for (int j = 0; j < 2; ++j)
#pragma unroll
              for (int nb = 0; nb < C::NB; ++nb)
                mma<false>(sg.o[2 * c + j][nb], u[j], u[j + 2], y[j], y[j + 2], b[nb][0], b[nb][1]);
          }
        }
      }
    }
  }
}

// Fetches tiles ahead of the computation.  A 16-slot block lies in one page, so
// its rows (and its scales of one kind) are contiguous: lane i copies their
// 16-byte chunks i, i + 32, ...
template <class C>
struct Fetcher {
  static constexpr int kCopies = (C::CH + 1) / 2;          // of a lane, for a block's keys
  static constexpr int kScaleCopies = (8 * C::G + 31) / 32;
  Cursor k;
  const int *entry;            // table entry of the next block's page
  int in_page;                 // its place in the page, in blocks
  int head_row;                // first row of the segment's head in a page
  int pages[C::TB];            // the pages of the next tile's blocks, looked up ahead
  int left;                    // tiles still to fetch
  int full;                    // of which these, of the segment, have every slot
  bool bad;                    // a page outside the cache was met
  uint32_t to, scale_to;       // this lane's first chunks in a stage
  const uint8_t *keys, *values;
  const uint16_t *scales[kScaleCopies ? kScaleCopies : 1];

  __device__ __forceinline__ void start(const AttnParams &p, const Cursor &at, int count, int lane) {
    k = at;
    left = count;
    bad = false;
    to = (lane / C::CH) * C::RB + (((lane % C::CH) ^ swizzle<C::CH>((lane / C::CH) & 7)) << 4);
    keys = p.c.k + lane * 16;
    values = p.c.v + lane * 16;
    if constexpr (C::BITS != 16) {
      const int a0 = lane / (2 * C::G), j0 = lane - a0 * 2 * C::G;
      scale_to = 2 * C::TILE * C::RB + a0 * C::TILE * C::G * 2 + j0 * 16;
#pragma unroll
      for (int i = 0; i < kScaleCopies; ++i) {
        const int a = (lane + 32 * i) / (2 * C::G), j = (lane + 32 * i) % (2 * C::G);
        scales[i] = (a == 0 ? p.c.k_scales : a == 1 ? p.c.k_biases : a == 2 ? p.c.v_scales
                                                                            : p.c.v_biases) + j * 8;
      }
    }
    if (left > 0) segment(p, lane);
  }
  __device__ __forceinline__ void segment(const AttnParams &p, int lane) {
    call_queries(p, lane);
    head_row = (p.chunks == 1 ? k.hc : k.hc / p.chunks) * p.c.S;
    entry = p.c.table + static_cast<long long>(k.b) * p.c.width;
    in_page = 0;
    if (k.tile > 0) {
      const int blk = k.tile * C::TB;
      entry += blk / p.page_blocks;
      in_page = blk % p.page_blocks;
    }
    look_up(p);
    full = k.n / C::TILE - k.tile;
  }
  // A block past the sequence's slots has no page.
  __device__ __forceinline__ void look_up(const AttnParams &p) {
    pages[0] = __ldg(entry);
    int in = in_page;
    const int *e = entry;
#pragma unroll
    for (int i = 1; i < C::TB; ++i) {
      pages[i] = pages[i - 1];
      if (++in == p.page_blocks) {
        in = 0;
        ++e;
        pages[i] = k.tile * C::TILE + 16 * i < k.n ? __ldg(e) : -1;
      }
    }
  }
  // Brings the queries of the segment closer: they are wanted a few tiles later.
  __device__ __forceinline__ void call_queries(const AttnParams &p, int lane) {
    constexpr int kLines = C::HEADS * C::D / 64;  // of 128 bytes
    const int hk = p.chunks == 1 ? k.hc : k.hc / p.chunks;
    const int r0 = hk * p.R + (k.hc - hk * p.chunks) * C::HEADS;
    const __nv_bfloat16 *q = p.q + k.b * p.q_stride + r0 * C::D;
#pragma unroll
    for (int i = 0; i < kLines; i += 32)
      if (lane + i < kLines && r0 + (lane + i) * 64 / C::D < p.Hq)
        asm volatile("prefetch.global.L1 [%0];\n" ::"l"(q + (lane + i) * 64));
  }
  // Copies BLOCKS blocks that follow one another in a page, from block `i` of
  // the stage on; `rows` of their slots are the sequence's, the others 0.
  template <bool ALL, int BLOCKS>
  __device__ __forceinline__ void copy(const AttnParams &p, int i, int from, int at, int rows,
                                       uint32_t stage, int lane) {
    const uint32_t first = static_cast<uint32_t>(from) * p.page_rows + (head_row + at);
    const uint8_t *ks = keys + static_cast<unsigned long long>(first) * C::RB;
    const uint8_t *vs = values + static_cast<unsigned long long>(first) * C::RB;
    const uint32_t base = stage + to;
#pragma unroll
    for (int blk = 0; blk < BLOCKS; ++blk)
#pragma unroll
      for (int c = 0; c < kCopies; ++c) {
        constexpr bool kEven = 32 % C::CH == 0;  // a copy is whole rows
        constexpr int kRows = kEven ? 32 / C::CH : 1;
        uint32_t dst;
        int r;
        if constexpr (kEven) {
          r = lane / C::CH + c * kRows;
          dst = (base ^ (swizzle<C::CH>((c * kRows) & 7) << 4)) + (16 * (i + blk) + c * kRows) * C::RB;
        } else {
          r = (c * 32 + lane) / C::CH;
          dst = stage + (16 * (i + blk) + r) * C::RB +
                (((c * 32 + lane) % C::CH ^ swizzle<C::CH>(r & 7)) << 4);
        }
        if (C::CH % 2 == 0 || c * 32 + lane < 16 * C::CH) {
          const int bytes = ALL || 16 * blk + r < rows ? 16 : 0;
          cp_async16(dst, ks + blk * 16 * C::RB + c * 512, bytes);
          cp_async16(dst + C::TILE * C::RB, vs + blk * 16 * C::RB + c * 512, bytes);
        }
      }
    if constexpr (C::BITS != 16) {
#pragma unroll
      for (int c = 0; c < kScaleCopies; ++c) {
        const uint16_t *ss = scales[c] + static_cast<unsigned long long>(first) * C::G;
        if (8 * C::G % 32 == 0 || c * 32 + lane < 8 * C::G) {
#pragma unroll
          for (int blk = 0; blk < BLOCKS; ++blk) {
            const int j = (c * 32 + lane) % (2 * C::G);
            int bytes = 16;
            if (!ALL) {
              bytes = (rows - 16 * blk) * C::G * 2 - j * 16;
              bytes = bytes < 0 ? 0 : bytes < 16 ? bytes : 16;
            }
            // the second copy's kinds (values) follow the first's (keys)
            cp_async16(stage + scale_to + c * 2 * C::TILE * C::G * 2 + (i + blk) * 32 * C::G,
                       ss + blk * 16 * C::G, bytes);
          }
        }
      }
    }
  }
  __device__ __forceinline__ bool inside(const AttnParams &p, int page) {
    return static_cast<unsigned>(page) < static_cast<unsigned>(p.c.num_pages);
  }
  // A tile of fewer slots, or of several pages, or with a page outside the cache.
  __device__ __forceinline__ void copy_apart(const AttnParams &p, uint32_t stage, int lane) {
    int in = in_page;
#pragma unroll
    for (int i = 0; i < C::TB; ++i) {
      int rows = k.n - k.tile * C::TILE - 16 * i, from = pages[i];
      rows = rows < 0 ? 0 : rows < 16 ? rows : 16;
      if (!inside(p, from)) {
        if (rows > 0) {
          bad = true;
          if (p.c.status && lane == 0) atomicOr(p.c.status, 1);
        }
        from = rows = 0;
      }
      copy<false, 1>(p, i, from, 16 * in, rows, stage, lane);
      if (++in == p.page_blocks) in = 0;
    }
  }
  // Starts the copies of the next tile.
  __device__ __forceinline__ void fetch(const AttnParams &p, const int *cum, uint32_t stage,
                                        int lane) {
    if (left > 0) {
      --left;
      if (full > 0 && in_page + C::TB <= p.page_blocks && inside(p, pages[0]))
        copy<true, C::TB>(p, 0, pages[0], 16 * in_page, 16 * C::TB, stage, lane);
      else
        copy_apart(p, stage, lane);
      --full;
      if (++k.tile < k.tiles) {
        const int *old = entry;
        in_page += C::TB;
        while (in_page >= p.page_blocks) {
          in_page -= p.page_blocks;
          ++entry;
        }
        if (left > 0 && (entry != old || in_page + C::TB > p.page_blocks)) look_up(p);
      } else if (left > 0) {
        --k.tile;
        cursor_next<C>(p, cum, k);
        segment(p, lane);
      }
    }
    cp_commit();
  }
};

// The output of a segment that was whole here.
template <class C>
__device__ __forceinline__ void write_out(const Segment<C> &sg, const AttnParams &p, const Cursor &k,
                                          int lane) {
  const int g = lane >> 2, t = lane & 3;
  const int hk = p.chunks == 1 ? k.hc : k.hc / p.chunks, r0 = (k.hc - hk * p.chunks) * C::HEADS;
#pragma unroll
  for (int nb = 0; nb < C::NB; ++nb)
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int r = r0 + nb * 8 + 2 * t + i;
      if (r >= p.R) continue;
      const long long head = static_cast<long long>(k.b) * p.Hq + hk * p.R + r;
      const float inv = sg.l[nb][i] > 0.0f ? 1.0f / sg.l[nb][i] : 0.0f;
      __nv_bfloat16 *to = p.out + head * C::D;
      auto val = [&](int mt, int half) { return sg.o[mt][nb][i + 2 * half] * inv; };
      if constexpr (C::BITS == 16) {
#pragma unroll
        for (int mt = 0; mt < C::MT; ++mt) {
          to[element_of<C>(mt, 0, g)] = __float2bfloat16_rn(val(mt, 0));
          to[element_of<C>(mt, 1, g)] = __float2bfloat16_rn(val(mt, 1));
        }
      } else if constexpr (C::VCH == 64) {  // 8 neighbours
#pragma unroll
        for (int mt = 0; mt < C::MT; mt += 4)
          *reinterpret_cast<uint4 *>(to + element_of<C>(mt, 0, g)) =
              make_uint4(pack16<true>(val(mt, 0), val(mt + 1, 0)), pack16<true>(val(mt + 2, 0), val(mt + 3, 0)),
                         pack16<true>(val(mt, 1), val(mt + 1, 1)), pack16<true>(val(mt + 2, 1), val(mt + 3, 1)));
      } else {  // 4
#pragma unroll
        for (int mt = 0; mt < C::MT; mt += 2)
          *reinterpret_cast<uint2 *>(to + element_of<C>(mt, 0, g)) =
              make_uint2(pack16<true>(val(mt, 0), val(mt + 1, 0)), pack16<true>(val(mt, 1), val(mt + 1, 1)));
      }
      if (p.scores && g == 0) p.stats[head] = make_float2(sg.m[nb][i], sg.l[nb][i]);
    }
}

// A piece of a segment: its accumulators as the lanes hold them (quad q of the
// piece is accumulator tile q / 32, all lanes side by side), and its heads'
// maxima and sums.
template <class C>
__device__ __forceinline__ void write_piece(const Segment<C> &sg, float4 *o, float2 *ml, int lane) {
  const int g = lane >> 2, t = lane & 3;
#pragma unroll
  for (int nb = 0; nb < C::NB; ++nb) {
#pragma unroll
    for (int mt = 0; mt < C::MT; ++mt)
      o[(mt * C::NB + nb) * 32 + lane] = make_float4(sg.o[mt][nb][0], sg.o[mt][nb][1], sg.o[mt][nb][2],
                                                     sg.o[mt][nb][3]);
    if (g == 0) {
      ml[nb * 8 + 2 * t] = make_float2(sg.m[nb][0], sg.l[nb][0]);
      ml[nb * 8 + 2 * t + 1] = make_float2(sg.m[nb][1], sg.l[nb][1]);
    }
  }
}

// Quad q of a segment's output: two elements of two neighbouring heads, from
// sums and the heads' l; `head0` is the segment's first head, `heads` how many
// it has.
template <class C>
__device__ __forceinline__ void store_quad(__nv_bfloat16 *head0, int heads, int q, float4 o, float l0,
                                           float l1) {
  const int lane = q & 31, g = lane >> 2, tile = q >> 5, mt = tile / C::NB;
  const int h = (tile % C::NB) * 8 + 2 * (lane & 3);
  const float i0 = l0 > 0.0f ? 1.0f / l0 : 0.0f, i1 = l1 > 0.0f ? 1.0f / l1 : 0.0f;
  __nv_bfloat16 *to = head0 + h * C::D;
  const int a = element_of<C>(mt, 0, g), b = element_of<C>(mt, 1, g);
  if (h < heads) {
    to[a] = __float2bfloat16_rn(o.x * i0);
    to[b] = __float2bfloat16_rn(o.z * i0);
  }
  if (h + 1 < heads) {
    to[C::D + a] = __float2bfloat16_rn(o.y * i1);
    to[C::D + b] = __float2bfloat16_rn(o.w * i1);
  }
}
template <class C>
__device__ __forceinline__ int quad_head(int q) {  // the first of its two heads
  return (q >> 5) % C::NB * 8 + 2 * (q & 3);
}
__device__ __forceinline__ void add_quad(float4 &o, float2 a, const float4 &x) {
  o.x = fmaf(a.x, x.x, o.x);
  o.y = fmaf(a.y, x.y, o.y);
  o.z = fmaf(a.x, x.z, o.z);
  o.w = fmaf(a.y, x.w, o.w);
}

// Tiles before every sequence, into shared memory (and the workspace, for the
// second kernel).
template <class C>
__device__ __forceinline__ Known sum_tiles(const AttnParams &p, int *cum, int threads) {
  __shared__ int part[32];
  static_assert(sizeof(part) == 128, "counted by AttnCfg::FIXED");
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int per = (p.batch + threads - 1) / threads;
  const int b0 = tid * per < p.batch ? tid * per : p.batch;
  const int b1 = b0 + per < p.batch ? b0 + per : p.batch;
  const int unit = p.c.H * p.chunks;
  if (p.batch <= 32) {  // every warp for itself (all write the same), without a barrier
    int n = 0;
    if (lane < p.batch) {
      n = __ldg(p.lens + lane);
      if (n > p.room) {
        n = static_cast<int>(p.room);
        if (p.c.status && blockIdx.x == 0) atomicOr(p.c.status, 1);
      }
      n = n < 0 ? 0 : n;
    }
    int upto = (n + C::TILE - 1) / C::TILE * unit;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int x = __shfl_up_sync(0xffffffffu, upto, o);
      if (lane >= o) upto += x;
    }
    if (lane < p.batch) {
      cum[lane + 1] = upto;
      if (blockIdx.x == 0) p.cum[lane + 1] = upto;
    }
    if (lane == 0) {
      cum[0] = 0;
      if (blockIdx.x == 0) p.cum[0] = 0;
    }
    __syncwarp();
    return {n, lane < p.batch ? upto : 0x7fffffff};
  }
  int sum = 0;
  for (int b = b0; b < b1; ++b) {
    if (p.c.status && blockIdx.x == 0 && __ldg(p.lens + b) > p.room) atomicOr(p.c.status, 1);
    sum += (clipped_length(p, b) + C::TILE - 1) / C::TILE * unit;
  }
  int before = sum;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int x = __shfl_up_sync(0xffffffffu, before, o);
    if (lane >= o) before += x;
  }
  if (lane == 31) part[warp] = before;
  __syncthreads();
  before -= sum;
  for (int w = 0; w < warp; ++w) before += part[w];
  for (int b = b0; b < b1; ++b) {
    cum[b] = before;
    if (blockIdx.x == 0) p.cum[b] = before;
    before += (clipped_length(p, b) + C::TILE - 1) / C::TILE * unit;
  }
  if (b1 == p.batch && (b0 < b1 || tid == 0)) {
    cum[p.batch] = before;
    if (blockIdx.x == 0) p.cum[p.batch] = before;
  }
  __syncthreads();
  return {0, 0};
}

template <class C>
__global__ void __launch_bounds__(C::WARPS * 32, C::CTAS_PER_SM)
attn_kernel(const AttnParams p) {
  extern __shared__ __align__(128) uint8_t attn_smem[];
  __shared__ float2 piece_ml[2][C::WARPS][C::HEADS];  // first and last pieces
  __shared__ int piece_seg[2][C::WARPS];              // segment, or -1
  __shared__ __align__(8) float factor[2 * C::WARPS][C::HEADS];
  __shared__ float2 joined[2 * C::WARPS][C::HEADS];   // maximum and sum of a piece's segment here
  static_assert(sizeof(piece_ml) + sizeof(piece_seg) + sizeof(factor) + sizeof(joined) + 128 + 128 == C::FIXED,
                "what the shared memory's limit is checked with");
  int *cum = reinterpret_cast<int *>(attn_smem + C::SMEM);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  wait_for_previous_grid();
  const Known known = sum_tiles<C>(p, cum, C::WARPS * 32);
  const int total = cum[p.batch], unit = p.c.H * p.chunks;

  // rows of sequences without slots
  for (int b = blockIdx.x; b < p.batch; b += gridDim.x) {
    if (cum[b + 1] == cum[b]) {
      uint4 *to = reinterpret_cast<uint4 *>(p.out + static_cast<long long>(b) * p.Hq * C::D);
      for (int i = tid; i < p.Hq * C::D / 8; i += C::WARPS * 32) to[i] = make_uint4(0u, 0u, 0u, 0u);
    }
  }
  const Share share(total, p.ctas);
  if (static_cast<int>(blockIdx.x) >= share.ctas) {
    if (tid == 0) p.cuts[blockIdx.x] = make_int2(-1, -1);
    return;
  }

  const int cta_warp = blockIdx.x * C::WARPS, me = cta_warp + warp;
  const int c0 = share.first(blockIdx.x), c1 = share.first(blockIdx.x + 1);
  const int each = (c1 - c0) / C::WARPS, more = (c1 - c0) % C::WARPS;
  const int u0 = c0 + warp * each + (warp < more ? warp : more), u1 = u0 + each + (warp < more ? 1 : 0);
  const uint32_t ring = smem_addr(attn_smem) + warp * C::STAGES * C::STAGE;
  if (lane == 0) piece_seg[0][warp] = piece_seg[1][warp] = -1;

  // (The code of what follows runs once or twice in a warp, from a cold
  // instruction cache: one copy of each part, in loops that are not unrolled.)
  bool tail = false;
  Segment<C> sg;
  if (u0 < u1) {
    Cursor k = cursor_at<C>(p, cum, known, u0);
    sg.load(p, k, lane);
    Fetcher<C> fetch;
    fetch.start(p, k, u1 - u0, lane);
    const uint32_t ring_end = ring + C::STAGES * C::STAGE;
    uint32_t stage = ring, ahead = ring;
    bool fresh = true;
#pragma unroll 1
    for (int u = u0 - (C::STAGES - 1); u < u1; ++u) {
      if (u >= u0) {
        cp_wait<C::STAGES - 2>();
        __syncwarp();
      }
      fetch.fetch(p, cum, ahead, lane);
      ahead = ahead + C::STAGE == ring_end ? ring : ahead + C::STAGE;
      if (u < u0) continue;
      if (fresh) {
        if (u > u0) sg.load(p, k, lane);
        sg.begin(p, lane);
        fresh = false;
      }
      attend_tile<C>(sg, p, k, stage, fetch.bad, lane);
      __syncwarp();
      stage = stage + C::STAGE == ring_end ? ring : stage + C::STAGE;
      const bool last = k.tile + 1 == k.tiles;
      if (last || u + 1 == u1) {
        sg.finish();
        if (!last) {  // the segment goes on in the next warp
          tail = true;
          if (lane == 0) piece_seg[1][warp] = k.b * unit + k.hc;
          break;
        }
        if (u + 1 - k.tiles >= u0) {  // the whole segment was here
          write_out<C>(sg, p, k, lane);
        } else {
          write_piece<C>(sg, p.warp_o + static_cast<long long>(me) * C::QUADS, piece_ml[0][warp], lane);
          if (lane == 0) piece_seg[0][warp] = k.b * unit + k.hc;
        }
        fresh = true;
        if (u + 1 < u1) cursor_next<C>(p, cum, k);
      } else {
        ++k.tile;
      }
    }
    cp_wait<0>();
  }
  __syncthreads();  // the rings are free
  float4 *tails = reinterpret_cast<float4 *>(attn_smem);
  if (tail) write_piece<C>(sg, tails + warp * C::QUADS, piece_ml[1][warp], lane);
  __syncthreads();

  // Join the pieces of a segment, in the order of its slots: piece 2 w (+ 1) is
  // warp w's first (last).  First each piece's factor for each head ...
  // A segment's pieces are the last ones of neighbouring warps and then, where
  // it ends, the first one of the next.
  const int mine = lane < 2 * C::WARPS ? piece_seg[lane & 1][lane >> 1] : -1;
  const unsigned all = __ballot_sync(0xffffffffu, mine >= 0);
  const unsigned alike = __match_any_sync(0xffffffffu, mine);
#pragma unroll 1
  for (int i = tid; i < 2 * C::WARPS * C::HEADS; i += C::WARPS * 32) {
    const int j = i / C::HEADS, h = i % C::HEADS;  // a whole warp takes this step or none
    const unsigned run = __shfl_sync(0xffffffffu, alike, j);
    if (!((all >> j) & 1u)) continue;
    const int j0 = __ffs(run) - 1, j1 = 31 - __clz(run);
    // (pieces between that are not there count nothing)
    float m = kNegInf, l = 0.0f;
#pragma unroll 4
    for (int r = j0; r <= j1; ++r)
      if ((run >> r) & 1u) m = fmaxf(m, piece_ml[r & 1][r >> 1][h].x);
    const float ms = m == kNegInf ? 0.0f : m;
#pragma unroll 4
    for (int r = j0; r <= j1; ++r)
      if ((run >> r) & 1u) {
        const float2 ml = piece_ml[r & 1][r >> 1][h];
        l += ex2(ml.x - ms) * ml.y;
      }
    factor[j][h] = ex2(piece_ml[j & 1][j >> 1][h].x - ms);
    joined[j][h] = make_float2(m, l);
  }
  __syncthreads();
  // ... then four sums a thread.
  int cut0 = -1, cut1 = -1;
#pragma unroll 1
  for (unsigned left = all; left;) {
    const int j0 = __ffs(left) - 1;
    const int seg = __shfl_sync(0xffffffffu, mine, j0);
    const unsigned run = __shfl_sync(0xffffffffu, alike, j0);
    left &= ~run;
    const unsigned lasts = run & 0xaaaaaaaau, ends = run & 0x55555555u;
    const int w0 = lasts ? (__ffs(lasts) - 1) >> 1 : 0, some = __popc(lasts);
    const int b = seg / unit, hc = seg - b * unit;
    const int tiles = (cum[b + 1] - cum[b]) / unit;
    const int first = cum[b] + hc * tiles;
    const int hk = hc / p.chunks, r0 = (hc - hk * p.chunks) * C::HEADS;
    const long long part = static_cast<long long>(blockIdx.x) * 2 + (first < c0 ? 0 : 1);
    const bool whole = first >= c0 && first + tiles <= c1;
    const long long head = static_cast<long long>(b) * p.Hq + hk * p.R + r0;
    if (tid == 0 && !whole) {
      if (first < c0) cut0 = seg;
      else cut1 = seg;
    }
    for (int q = tid; q < C::QUADS; q += C::WARPS * 32) {
      const int h = quad_head<C>(q);
      float4 o = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll 4
      for (int w = w0; w < w0 + some; ++w)
        add_quad(o, *reinterpret_cast<const float2 *>(&factor[2 * w + 1][h]), tails[w * C::QUADS + q]);
      if (ends) {
        const int w = (__ffs(ends) - 1) >> 1;
        add_quad(o, *reinterpret_cast<const float2 *>(&factor[2 * w][h]),
                 p.warp_o[static_cast<long long>(cta_warp + w) * C::QUADS + q]);
      }
      if (whole)
        store_quad<C>(p.out + head * C::D, p.R - r0, q, o, joined[j0][h].y, joined[j0][h + 1].y);
      else
        p.part_o[part * C::QUADS + q] = o;
    }
    if (tid < C::HEADS) {
      if (!whole) p.part_ml[part * C::HEADS + tid] = joined[j0][tid];
      else if (p.scores && r0 + tid < p.R) p.stats[head + tid] = joined[j0][tid];
    }
  }
  // the segments that this CTA holds a later and a first piece of
  if (tid == 0) p.cuts[blockIdx.x] = make_int2(cut0, cut1);
}

// CTAs that hold pieces of segment hc of sequence b: first and last, the same
// where no second step is needed.
template <class C>
__device__ __forceinline__ int2 segment_ctas(const AttnParams &p, int b, int hc) {
  const int total = __ldg(p.cum + p.batch), c0 = __ldg(p.cum + b), c1 = __ldg(p.cum + b + 1);
  const int tiles = (c1 - c0) / (p.c.H * p.chunks);
  const int first = c0 + hc * tiles;
  const Share share(total, p.ctas);
  return make_int2(share.cta_of(first), share.cta_of(first + tiles - 1));
}

// Maximum and sum of one head over the CTAs that hold its segment.
template <class C>
__device__ __forceinline__ float2 joined_stats(const AttnParams &p, int2 at, int h) {
  float m = kNegInf, l = 0.0f;
  for (int c = at.x; c <= at.y; ++c) {
    const float2 ml = p.part_ml[(static_cast<long long>(c) * 2 + (c == at.x)) * C::HEADS + h];
    const float up = fmaxf(m, ml.x), us = up == kNegInf ? 0.0f : up;
    l = l * ex2(m - us) + ex2(ml.x - us) * ml.y;  // (NaN stays)
    m = up;
  }
  return make_float2(m, l);
}

constexpr int kWeightSlots = 1024;  // slots of a block that adds weights
constexpr int kJoinThreads = 256;
constexpr int kJoinCtas = 32;       // pieces whose factors are kept at once

// Second kernel: block i joins the segment that begins in CTA i and goes on in
// the next ones, if there is one; further blocks add a kv head's probabilities
// into the weights.
template <class C>
__global__ void __launch_bounds__(kJoinThreads) attn_join_kernel(const AttnParams p, int weight_blocks) {
  const int tid = threadIdx.x, lane = tid & 31;
  wait_for_previous_grid();
  if (static_cast<int>(blockIdx.x) < p.ctas) {
    const int cta = blockIdx.x, unit = p.c.H * p.chunks;
    const int seg = p.cuts[cta].y;
    // the CTAs behind that hold more of it (a warp looks at 32 of them)
    int pieces = 1;
    for (bool more = true; more;) {
      const int c = cta + pieces + lane;
      const unsigned same = __ballot_sync(0xffffffffu, c < p.ctas && p.cuts[c].x == seg);
      pieces += same == 0xffffffffu ? 32 : __ffs(~same) - 1;
      more = same == 0xffffffffu;
    }
    if (seg < 0) return;
    const int b = seg / unit, hc = seg - b * unit;
    const int hk = p.chunks == 1 ? hc : hc / p.chunks, r0 = (hc - hk * p.chunks) * C::HEADS;
    constexpr int kOwn = (C::QUADS + kJoinThreads - 1) / kJoinThreads, kAhead = 4;
    __shared__ float2 ml[kJoinCtas][C::HEADS];
    __shared__ __align__(8) float factor[kJoinCtas][C::HEADS];
    __shared__ __align__(8) float scale_by[C::HEADS], l[C::HEADS];
    float4 o[kOwn] = {};
    float m = kNegInf, sum = 0.0f;  // of head `tid`
    for (int c0 = 0; c0 < pieces; c0 += kJoinCtas) {
      const int n = pieces - c0 < kJoinCtas ? pieces - c0 : kJoinCtas;
      // the first piece is its CTA's second
      auto piece = [&](int c) { return static_cast<long long>(cta + c0 + c) * 2 + (c0 + c == 0); };
      float4 x[kOwn][kAhead];  // the first pieces' sums, on their way meanwhile
#pragma unroll
      for (int i = 0; i < kOwn; ++i)
#pragma unroll
        for (int c = 0; c < kAhead; ++c)
          if (c < n && tid + i * kJoinThreads < C::QUADS)
            x[i][c] = p.part_o[piece(c) * C::QUADS + tid + i * kJoinThreads];
      for (int i = tid; i < n * C::HEADS; i += kJoinThreads)
        ml[i / C::HEADS][i % C::HEADS] = p.part_ml[piece(i / C::HEADS) * C::HEADS + i % C::HEADS];
      __syncthreads();
      if (tid < C::HEADS) {
        float up = m;
        for (int c = 0; c < n; ++c) up = fmaxf(up, ml[c][tid].x);
        const float us = up == kNegInf ? 0.0f : up;
        const float a = ex2(m - us);
        sum *= a;
        for (int c = 0; c < n; ++c) {
          const float f = ex2(ml[c][tid].x - us);
          factor[c][tid] = f;
          sum += f * ml[c][tid].y;
        }
        scale_by[tid] = a;
        l[tid] = sum;
        m = up;
      }
      __syncthreads();
#pragma unroll
      for (int i = 0; i < kOwn; ++i) {
        const int q = tid + i * kJoinThreads;
        if (q >= C::QUADS) break;
        const int h = quad_head<C>(q);
        const float2 a = *reinterpret_cast<const float2 *>(&scale_by[h]);
        o[i].x *= a.x; o[i].y *= a.y; o[i].z *= a.x; o[i].w *= a.y;
#pragma unroll
        for (int c = 0; c < kAhead; ++c)
          if (c < n) add_quad(o[i], *reinterpret_cast<const float2 *>(&factor[c][h]), x[i][c]);
#pragma unroll 8
        for (int c = kAhead; c < n; ++c)
          add_quad(o[i], *reinterpret_cast<const float2 *>(&factor[c][h]), p.part_o[piece(c) * C::QUADS + q]);
      }
    }
#pragma unroll
    for (int i = 0; i < kOwn; ++i) {
      const int q = tid + i * kJoinThreads;
      if (q < C::QUADS)
        store_quad<C>(p.out + (static_cast<long long>(b) * p.Hq + hk * p.R + r0) * C::D, p.R - r0, q, o[i],
                      l[quad_head<C>(q)], l[quad_head<C>(q) + 1]);
    }
    return;
  }
  const int ix = blockIdx.x - p.ctas, row = ix / weight_blocks, z = ix - row * weight_blocks;
  const int b = row / p.c.H, hk = row - b * p.c.H;
  const int n = clipped_length(p, b);
  const int j0 = z * kWeightSlots;
  if (j0 >= n) return;
  const int j1 = j0 + kWeightSlots < n ? j0 + kWeightSlots : n;
  __shared__ float2 all[64];
  float sum[kWeightSlots / kJoinThreads] = {};
  for (int r0 = 0; r0 < p.R; r0 += 64) {
    const int count = p.R - r0 < 64 ? p.R - r0 : 64;
    __syncthreads();
    if (tid < count) {
      const int r = r0 + tid, ch = r / C::HEADS;
      const int2 at = segment_ctas<C>(p, b, hk * p.chunks + ch);
      all[tid] = at.x == at.y ? p.stats[static_cast<long long>(b) * p.Hq + hk * p.R + r]
                              : joined_stats<C>(p, at, r - ch * C::HEADS);
    }
    __syncthreads();
    for (int r = 0; r < count; ++r) {
      const float m = all[r].x, inv = 1.0f / all[r].y;
      if (all[r].y == 0.0f) continue;  // no slot of the row takes part
      const float *s = p.scores + (static_cast<long long>(b) * p.Hq + hk * p.R + r0 + r) * p.room;
#pragma unroll
      for (int i = 0; i < kWeightSlots / kJoinThreads; ++i) {
        const int j = j0 + i * kJoinThreads + tid;
        if (j < j1) sum[i] += ex2(s[j] - m) * inv;
      }
    }
  }
  float *w = p.weights + static_cast<long long>(row) * p.state_width;
#pragma unroll
  for (int i = 0; i < kWeightSlots / kJoinThreads; ++i) {
    const int j = j0 + i * kJoinThreads + tid;
    if (j < j1) w[j] += sum[i];
  }
}

// ---------------------------------------------------------------------------
// Host side
// ---------------------------------------------------------------------------

template <class C>
int attn_ctas(int sms) { return sms * C::CTAS_PER_SM; }

// Lays the workspace out from `base` (null: only its size is wanted).
template <class C>
size_t lay_out(AttnParams &p, const CacheView &c, int batch, int num_q_heads, bool weights, int sms,
               uint8_t *base) {
  size_t at = 0;
  auto take = [&](size_t bytes) {
    uint8_t *r = base ? base + at : nullptr;
    at += (bytes + 127) / 128 * 128;
    return r;
  };
  const size_t ctas = attn_ctas<C>(sms), heads = static_cast<size_t>(batch) * num_q_heads;
  p.cum = reinterpret_cast<int *>(take(4 * (static_cast<size_t>(batch) + 1)));
  p.cuts = reinterpret_cast<int2 *>(take(ctas * 8));
  p.part_ml = reinterpret_cast<float2 *>(take(ctas * 2 * C::HEADS * 8));
  p.part_o = reinterpret_cast<float4 *>(take(ctas * 2 * C::HEADS * C::D * 4));
  p.warp_o = reinterpret_cast<float4 *>(take(ctas * C::WARPS * C::HEADS * C::D * 4));
  if (weights) {
    p.stats = reinterpret_cast<float2 *>(take(heads * 8));
    p.scores = reinterpret_cast<float *>(take(heads * c.width * c.S * 4));
  }
  return at;
}

template <class C>
cudaError_t attn_run(const AttnArgs &a, const Device &dev) {
  AttnParams p = {};
  p.c = a.cache;
  p.q = static_cast<const __nv_bfloat16 *>(a.q);
  p.q_stride = a.q_stride;
  p.lens = a.lens;
  p.out = static_cast<__nv_bfloat16 *>(a.out);
  p.batch = a.batch;
  p.Hq = a.num_q_heads;
  p.R = a.num_q_heads / a.cache.H;
  p.chunks = (p.R + C::HEADS - 1) / C::HEADS;
  p.page_blocks = a.cache.S / 16;
  p.page_rows = static_cast<unsigned>(a.cache.H) * a.cache.S;
  p.scale_log2 = fmaxf(fabsf(a.scale) * 1.4426950408889634f, 1.17549435e-38f);
  p.q_sign = a.scale < 0.0f ? 0x80008000u : 0u;
  p.weights = a.weights;
  p.state_width = a.state_width;
  p.room = static_cast<long long>(a.cache.width) * a.cache.S;
  p.ctas = attn_ctas<C>(dev.sms);
  lay_out<C>(p, a.cache, a.batch, a.num_q_heads, a.weights != nullptr, dev.sms,
             static_cast<uint8_t *>(a.workspace));
  const size_t smem = C::SMEM + 4 * (static_cast<size_t>(a.batch) + 1);
  static Granted granted;
  cudaError_t e = allow_smem(attn_kernel<C>, granted, dev, static_cast<int>(smem));
  if (e != cudaSuccess) return e;
  e = launch_overlapped(attn_kernel<C>, dim3(p.ctas), C::WARPS * 32, smem, 1, a.stream, p);
  if (e != cudaSuccess) return e;
  const int weight_blocks =
      a.weights ? static_cast<int>((p.room + kWeightSlots - 1) / kWeightSlots) : 0;
  const long long blocks = p.ctas + static_cast<long long>(a.batch) * p.c.H * weight_blocks;
  return launch_overlapped(attn_join_kernel<C>, dim3(static_cast<unsigned>(blocks)), kJoinThreads, 0, 1,
                           a.stream, p, weight_blocks);
}

// The kernel for a head size, group size and number of query heads to a kv
// head: 16 heads at a time where there are more than 8 (but 8 for heads of
// 256, whose accumulators fill the registers).
template <int BITS, class F>
auto attn_select(const CacheView &c, int R, F f) {
  const int gs = BITS == 16 ? 32 : c.D / c.G;
  const bool wide = R > 8;
  if constexpr (BITS == 16) {
    switch (c.D) {
      case 64: return wide ? f(AttnCfg<16, 64, 64, 2>{}) : f(AttnCfg<16, 64, 64, 1>{});
      case 96: return wide ? f(AttnCfg<16, 96, 96, 2>{}) : f(AttnCfg<16, 96, 96, 1>{});
      case 128: return wide ? f(AttnCfg<16, 128, 128, 2>{}) : f(AttnCfg<16, 128, 128, 1>{});
      default: return f(AttnCfg<16, 256, 256, 1>{});
    }
  } else {
    switch (c.D) {
      case 64:
        if (gs == 32) return wide ? f(AttnCfg<BITS, 64, 32, 2>{}) : f(AttnCfg<BITS, 64, 32, 1>{});
        return wide ? f(AttnCfg<BITS, 64, 64, 2>{}) : f(AttnCfg<BITS, 64, 64, 1>{});
      case 96:
        return wide ? f(AttnCfg<BITS, 96, 32, 2>{}) : f(AttnCfg<BITS, 96, 32, 1>{});
      case 128:
        if (gs == 32) return wide ? f(AttnCfg<BITS, 128, 32, 2>{}) : f(AttnCfg<BITS, 128, 32, 1>{});
        if (gs == 64) return wide ? f(AttnCfg<BITS, 128, 64, 2>{}) : f(AttnCfg<BITS, 128, 64, 1>{});
        return wide ? f(AttnCfg<BITS, 128, 128, 2>{}) : f(AttnCfg<BITS, 128, 128, 1>{});
      default:
        if (gs == 32) return f(AttnCfg<BITS, 256, 32, 1>{});
        if (gs == 64) return f(AttnCfg<BITS, 256, 64, 1>{});
        return f(AttnCfg<BITS, 256, 128, 1>{});
    }
  }
}

template <int BITS>
size_t attn_workspace_bits(const CacheView &c, int batch, int num_q_heads, bool weights, int sms) {
  return attn_select<BITS>(c, num_q_heads / c.H, [&](auto cfg) {
    AttnParams p = {};
    return lay_out<decltype(cfg)>(p, c, batch, num_q_heads, weights, sms, nullptr);
  });
}
template <int BITS>
cudaError_t attn_launch_bits(const AttnArgs &a, const Device &dev) {
  return attn_select<BITS>(a.cache, a.num_q_heads / a.cache.H,
                           [&](auto cfg) { return attn_run<decltype(cfg)>(a, dev); });
}

}  // namespace qmvc
