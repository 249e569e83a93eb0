// qmv_kv.cu -- the paged key-value cache in the packed affine format:
// kv_append (bf16 rows in, quantized or as they are), kv_read (dense bf16
// rows out), kv_evict (the slots with the least accumulated attention weight
// make room), and the C entry points, kv_attention's among them (its kernels
// are in qmv_kv_attn.cuh).  Contracts are in include/qmv.h.
//
// Append and read are streaming and element-wise: bf16 rows on one side, code
// rows, scales and biases on the other, in chunks of 16 elements (32 bytes of
// bf16).  A block takes a contiguous range of tokens, looks up where all of
// them lie first (a thread each), and then goes through them with every thread
// at a chunk of its own: its head and place in the head stay the same, so a
// token costs it one row number.  A group of 32, 64 or 128 elements is 2, 4 or
// 8 neighbouring lanes.  Measured (B200, 8 heads of 128): 73.7 thousand 4-bit
// tokens read in 71 us (5.4 TB/s, memory); 6656 tokens quantized to 8 bits, with
// state, in 16.8 us (6.4 us of bytes), by the barriers behind the tokens' look-ups
// and state (2.4 warps wait there for each instruction issued) and by the
// quantizer's arithmetic, whose 10.6 M instructions would issue in 9.3 us.
#include <cooperative_groups.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <atomic>
#include <cmath>
#include <cstdarg>
#include <cstdint>
#include <cstdio>

#include "qmv.h"
#include "qmv_affine.cuh"
#include "qmv_kv.h"

namespace qmvc {

using namespace qmva;

namespace cg = cooperative_groups;

constexpr int kRowThreads = 256;
constexpr int kRowBatch = 256;    // tokens looked up at once
constexpr int kRowAhead = 2;      // chunks of a thread in flight
constexpr int kStartsMax = 1024;  // token_starts kept in shared memory up to here

struct RowParams {
  CacheView c;
  uint16_t *k, *v;            // dense rows: read by append, written by read
  long long k_stride, v_stride;
  const int *lens, *starts;   // starts may be null: one token per sequence
  const int *seen;            // slot state (append), or null
  int *positions;
  float *weights;
  int batch, tokens, state_width;
  int block_tokens;           // tokens of a block
  bool wide;                  // dense and bf16 rows lie at multiples of 32 bytes
};

constexpr uint32_t kNowhere = 0xffffffffu;

// The row of token t's slot for head 0, or kNowhere where it has none (padding,
// an unused row of the batch, or a bad index).  `starts` may lie in shared
// memory.  Writes the slot's state where there is one.
__device__ __forceinline__ uint32_t place_of(const RowParams &p, const int *starts, int t) {
  int seq = t, first = t;
  if (p.starts) {
    // the last sequence that starts at or before t
    int lo = 0, hi = p.batch;
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (starts[mid] <= t) lo = mid;
      else hi = mid;
    }
    first = starts[lo];
    if (t < first || t >= starts[lo + 1]) return kNowhere;
    seq = lo;
  }
  const int len = __ldg(p.lens + seq);
  if (len < 0) return kNowhere;
  const int nth = t - first;
  const long long at = static_cast<long long>(len) + nth;
  if (at >= static_cast<long long>(p.c.width) * p.c.S) {
    if (p.c.status) atomicOr(p.c.status, 1);
    return kNowhere;
  }
  const int slot = static_cast<int>(at), of = slot / p.c.S;
  const int page = checked_page(p.c, __ldg(p.c.table + static_cast<long long>(seq) * p.c.width + of));
  if (page < 0) return kNowhere;
  if (p.positions) {
    const int pos = __ldg(p.seen + seq) + nth;
    for (int h = 0; h < p.c.H; ++h) {
      const long long j = (static_cast<long long>(seq) * p.c.H + h) * p.state_width + slot;
      p.positions[j] = pos;
      p.weights[j] = 0.0f;
    }
  }
  return cache_row(p.c, page, 0, slot - of * p.c.S);
}

// A chunk: 16 bf16 elements, or the words of 16 codes.
struct Chunk {
  uint32_t w[8];
};

// 32 bytes at once where they are aligned.  (Cache rows may be written in the
// same kernel by no one else, but other kernels do: no read-only path.)
__device__ __forceinline__ void load32(Chunk &x, const void *from, bool wide) {
  if (wide) {
    asm volatile("ld.global.v8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];\n"
                 : "=r"(x.w[0]), "=r"(x.w[1]), "=r"(x.w[2]), "=r"(x.w[3]), "=r"(x.w[4]), "=r"(x.w[5]),
                   "=r"(x.w[6]), "=r"(x.w[7])
                 : "l"(from));
  } else {
    const uint4 a = static_cast<const uint4 *>(from)[0], b = static_cast<const uint4 *>(from)[1];
    x.w[0] = a.x; x.w[1] = a.y; x.w[2] = a.z; x.w[3] = a.w;
    x.w[4] = b.x; x.w[5] = b.y; x.w[6] = b.z; x.w[7] = b.w;
  }
}
__device__ __forceinline__ void store32(void *to, const Chunk &x, bool wide) {
  if (wide) {
    asm volatile("st.global.v8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};\n" ::"l"(to), "r"(x.w[0]),
                 "r"(x.w[1]), "r"(x.w[2]), "r"(x.w[3]), "r"(x.w[4]), "r"(x.w[5]), "r"(x.w[6]), "r"(x.w[7])
                 : "memory");
  } else {
    static_cast<uint4 *>(to)[0] = make_uint4(x.w[0], x.w[1], x.w[2], x.w[3]);
    static_cast<uint4 *>(to)[1] = make_uint4(x.w[4], x.w[5], x.w[6], x.w[7]);
  }
}

// The range of a group, its chunks in GS / 16 neighbouring lanes: (largest, from 0
// up; smallest, from kRangeStart down).  In pairs of bf16, whose comparisons are
// exact and take the number beside a NaN.
template <int GS>
__device__ __forceinline__ float2 group_range(const Chunk &x) {
  auto pair = [](uint32_t v) { return *reinterpret_cast<const __nv_bfloat162 *>(&v); };
  __nv_bfloat162 lo = pair(x.w[0]), hi = lo;
#pragma unroll
  for (int i = 1; i < 8; ++i) {
    lo = __hmin2(lo, pair(x.w[i]));
    hi = __hmax2(hi, pair(x.w[i]));
  }
#pragma unroll
  for (int o = 1; o < GS / 16; o <<= 1) {
    lo = __hmin2(lo, __shfl_xor_sync(0xffffffffu, lo, o));
    hi = __hmax2(hi, __shfl_xor_sync(0xffffffffu, hi, o));
  }
  return make_float2(fmaxf(fmaxf(__low2float(hi), __high2float(hi)), 0.0f),
                     fminf(fminf(__low2float(lo), __high2float(lo)), kRangeStart));
}

// 16 bf16 elements to 16 codes (2 * BITS bytes), with the group's scale and bias.
template <int BITS>
__device__ __forceinline__ void quantize_chunk(Chunk &x, float scale, float bias, float rcp) {
#pragma unroll
  for (int part = 0; part < 2; ++part) {
    float v[8];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[2 * i] = __uint_as_float(x.w[4 * part + i] << 16);
      v[2 * i + 1] = __uint_as_float(x.w[4 * part + i] & 0xffff0000u);
    }
    codes_of<BITS>(v, bias, scale, rcp);
    // 16 bits of codes are an exact binary32 number: packed by multiply-adds,
    // taken out of the fraction under the exponent of 2^23
    uint32_t half[BITS / 2];
#pragma unroll
    for (int i = 0; i < BITS / 2; ++i) {
      float y;
      if constexpr (BITS == 4)
        y = fmaf(v[4 * i + 3], 4096.0f, fmaf(v[4 * i + 2], 256.0f, fmaf(v[4 * i + 1], 16.0f, v[4 * i])));
      else
        y = fmaf(v[2 * i + 1], 256.0f, v[2 * i]);
      half[i] = __float_as_uint(__fadd_rn(y, 8388608.0f));
    }
#pragma unroll
    for (int i = 0; i < BITS / 4; ++i)
      x.w[BITS / 4 * part + i] = __byte_perm(half[2 * i], half[2 * i + 1], 0x5410);
  }
}

// bf16(s * q + b) of 16 codes: the bf16 multiply-add rounds the exact value
// once; codes enter as exact bf16 numbers (those of 8 bits through binary32).
template <int BITS>
__device__ __forceinline__ void dequantize_chunk(Chunk &x, uint16_t s, uint16_t b) {
  const __nv_bfloat16 sb = __ushort_as_bfloat16(s), bb = __ushort_as_bfloat16(b);
  const __nv_bfloat162 s2 = __halves2bfloat162(sb, sb), b2 = __halves2bfloat162(bb, bb);
  auto pair = [](uint32_t v) { return *reinterpret_cast<const __nv_bfloat162 *>(&v); };
  uint32_t in[BITS / 2];
#pragma unroll
  for (int i = 0; i < BITS / 2; ++i) in[i] = x.w[i];
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    __nv_bfloat162 q;
    if constexpr (BITS == 4) {
      // both nibbles of a byte under the exponent of 128: 128 + q
      const uint32_t w = in[j / 4], m = __byte_perm(w, w >> 4, j % 4 * 0x0101 + 0x0400);
      q = __hsub2(pair((m & 0x000f000fu) | 0x43004300u), pair(0x43004300u));
    } else {
      const uint32_t c0 = __byte_perm(in[j / 2], 0x4b000000u, j & 1 ? 0x7652 : 0x7650);
      const uint32_t c1 = __byte_perm(in[j / 2], 0x4b000000u, j & 1 ? 0x7653 : 0x7651);
      q = __floats2bfloat162_rn(__fsub_rn(__uint_as_float(c0), 8388608.0f),
                                __fsub_rn(__uint_as_float(c1), 8388608.0f));
    }
    const __nv_bfloat162 r = __hfma2(q, s2, b2);
    x.w[j] = *reinterpret_cast<const uint32_t *>(&r);
  }
}

// ---------------------------------------------------------------------------
// Append and read
// ---------------------------------------------------------------------------

// Blocks of an SM: as many as leave the registers that the two directions need
// (one fewer or more took 5 to 20 % longer).
template <bool APPEND>
constexpr int row_blocks() { return APPEND ? 4 : 5; }

template <bool APPEND, int BITS, int GS, int D>
__global__ void __launch_bounds__(kRowThreads, row_blocks<APPEND>()) kv_rows_kernel(const RowParams p) {
  constexpr int kChunks = D / 16, kRow = D * BITS / 8;  // chunks and bytes of a row
  constexpr int kGroups = D / GS, kLanes = GS / 16;     // groups of a row, lanes of a group
  __shared__ uint32_t rows[kRowBatch];
  __shared__ int starts[kStartsMax + 1];
  const int tid = threadIdx.x;
  const int side = p.c.H * kChunks, per_token = 2 * side;  // chunks of a token
  // several tokens at once where a token has fewer chunks than the block threads
  const int at_once = per_token < kRowThreads ? kRowThreads / per_token : 1;
  const int sub = per_token < kRowThreads ? tid / per_token : 0;
  const int mine = tid - sub * per_token;              // this thread's first chunk
  const int t0 = blockIdx.x * p.block_tokens;
  const int t1 = t0 + p.block_tokens < p.tokens ? t0 + p.block_tokens : p.tokens;
  wait_for_previous_grid();
  const int *from = p.starts;
  if (p.starts && p.batch <= kStartsMax) {
    for (int i = tid; i <= p.batch; i += kRowThreads) starts[i] = __ldg(p.starts + i);
    from = starts;
    __syncthreads();
  }
  for (int base = t0; base < t1; base += kRowBatch) {
    const int count = t1 - base < kRowBatch ? t1 - base : kRowBatch;
    if (tid < count) rows[tid] = place_of(p, from, base + tid);
    __syncthreads();
    // the warp's lanes stay together (groups are reduced across lanes)
    for (int cc0 = 0; cc0 < per_token; cc0 += kRowThreads) {
      const int cc = cc0 + mine;
      const bool have = sub < at_once && cc < per_token;
      const bool value = cc >= side;
      const int rest = value ? cc - side : cc;
      const int h = rest / kChunks, i = rest - h * kChunks;
      uint8_t *codes = value ? p.c.v : p.c.k;
      uint16_t *scales = value ? p.c.v_scales : p.c.k_scales;
      uint16_t *biases = value ? p.c.v_biases : p.c.k_biases;
      const uint32_t head_row = static_cast<uint32_t>(h) * p.c.S;
      const long long stride = value ? p.v_stride : p.k_stride;
      uint16_t *dense = (value ? p.v : p.k) + static_cast<long long>(base) * stride + rest * 16;
      for (int n0 = 0; n0 < count; n0 += at_once * kRowAhead) {
        uint32_t row[kRowAhead];
        Chunk x[kRowAhead];
        uint16_t s[kRowAhead], b[kRowAhead];
#pragma unroll
        for (int a = 0; a < kRowAhead; ++a) {
          const int n = n0 + a * at_once + sub;
          row[a] = have && n < count ? rows[n] : kNowhere;
          if constexpr (APPEND) x[a] = Chunk{};
          if (row[a] == kNowhere) continue;
          row[a] += head_row;
          if constexpr (APPEND) {
            load32(x[a], dense + n * stride, p.wide);
          } else {
            const uint8_t *src = codes + static_cast<unsigned long long>(row[a]) * kRow + i * 2 * BITS;
            if constexpr (BITS == 16) {
              load32(x[a], src, p.wide);
            } else {
              if constexpr (BITS == 4) {
                const uint2 w = *reinterpret_cast<const uint2 *>(src);
                x[a].w[0] = w.x; x[a].w[1] = w.y;
              } else {
                const uint4 w = *reinterpret_cast<const uint4 *>(src);
                x[a].w[0] = w.x; x[a].w[1] = w.y; x[a].w[2] = w.z; x[a].w[3] = w.w;
              }
              const unsigned long long g = static_cast<unsigned long long>(row[a]) * kGroups + i / kLanes;
              s[a] = scales[g];
              b[a] = biases[g];
            }
          }
        }
        // The groups' scales take three divisions and a reciprocal each: of the
        // chunks in flight, lane a (mod 2) works out chunk a's, for all.
        float scale = 0.0f, bias = 0.0f, rcp = 0.0f;
        if constexpr (APPEND && BITS != 16) {
          static_assert(kRowAhead == 2, "a lane for each chunk of a group's lanes");
          const float2 r0 = group_range<GS>(x[0]), r1 = group_range<GS>(x[1]);
          const float2 sb = group_step_offset(tid & 1 ? r1.y : r0.y, tid & 1 ? r1.x : r0.x,
                                       static_cast<float>((1 << BITS) - 1));
          scale = sb.x;
          bias = sb.y;
          rcp = __frcp_rn(sb.x);
        }
#pragma unroll
        for (int a = 0; a < kRowAhead; ++a) {
          const int n = n0 + a * at_once + sub;
          if constexpr (APPEND) {
            uint8_t *dst = codes + static_cast<unsigned long long>(row[a]) * kRow + i * 2 * BITS;
            if constexpr (BITS == 16) {
              if (row[a] != kNowhere) store32(dst, x[a], p.wide);
            } else {
              const int from = (tid & 30) | a;
              const float sa = __shfl_sync(0xffffffffu, scale, from);
              const float ba = __shfl_sync(0xffffffffu, bias, from);
              const float ra = __shfl_sync(0xffffffffu, rcp, from);
              if (row[a] == kNowhere) continue;
              quantize_chunk<BITS>(x[a], sa, ba, ra);
              if constexpr (BITS == 4)
                *reinterpret_cast<uint2 *>(dst) = make_uint2(x[a].w[0], x[a].w[1]);
              else
                *reinterpret_cast<uint4 *>(dst) = make_uint4(x[a].w[0], x[a].w[1], x[a].w[2], x[a].w[3]);
              if (tid % kLanes == 0) {
                const unsigned long long g = static_cast<unsigned long long>(row[a]) * kGroups + i / kLanes;
                scales[g] = __bfloat16_as_ushort(__float2bfloat16_rn(sa));
                biases[g] = __bfloat16_as_ushort(__float2bfloat16_rn(ba));
              }
            }
          } else if (row[a] != kNowhere) {
            if constexpr (BITS != 16) dequantize_chunk<BITS>(x[a], s[a], b[a]);
            store32(dense + n * stride, x[a], p.wide);
          }
        }
      }
    }
    __syncthreads();
  }
}

// ---------------------------------------------------------------------------
// Evict
// ---------------------------------------------------------------------------

// A (sequence, kv head)'s slots are shared out over the CTAs of a cluster.
// The weights become keys in shared memory whose unsigned order is the order
// of the choice, are read from memory once, and the key of the last kept slot
// is found 8 bits at a time from histograms added up over the cluster, the last few
// candidates ranked at once.  Then
// each CTA lists its evicted slots below the new length (holes) and its kept
// ones at or above it (movers), in order, and the cluster's warps move the
// i-th mover's rows into the i-th hole.  Bound by that chain of steps, each of
// which waits for the one before: one of 1025 slots in 128 rows takes 9.5 us,
// 2048 of up to 16384 in 32 rows 27 us, 8 of them moving the rows at HBM rate.
constexpr int kEvictThreads = 512;
constexpr int kEvictWarps = kEvictThreads / 32;
constexpr int kEvictMaxCluster = 8;
constexpr int kEvictCopies = 8;  // of a histogram: weights share few leading bytes
constexpr int kEvictMaxSlots = 196608;
constexpr int kEvictPool = 256;

struct EvictParams {
  CacheView c;
  const int *lens, *seen;
  const float *weights;
  const int *positions;
  int *new_lens;
  float *new_weights;
  int *new_positions;
  int batch, state_width, budget, recent, sinks;
  int seg_max;  // keys that fit a CTA
};

// Unsigned order: NaN, then the numbers (both zeros alike), then protected.
__device__ __forceinline__ uint32_t evict_key(float w, int pos, int sinks, int from) {
  if (pos < sinks || pos >= from) return 0xffffffffu;
  if (w != w) return 0u;
  const uint32_t u = __float_as_uint(w + 0.0f);  // -0 + 0 = 0
  return (u >> 31) ? ~u : (u | 0x80000000u);
}

// How a warp's lanes share out moves of `units` units each: `per` moves at once,
// this lane at unit `at` of move `sub` of them (idle where sub == per).
struct RowLanes {
  int per, sub, at;
  bool more;  // a move has 64 units: twice the lanes
  __device__ __forceinline__ RowLanes(int units, int lane) {
    more = units > 32;
    const int u = more ? 32 : units > 0 ? units : 1;
    per = 32 / u;
    sub = lane / u;
    at = lane - sub * u;
    if (sub > per) sub = per;
  }
};

// Units of type T of up to 4 * per moves, on their way from row rs to row rd of
// lane m for move m; `base` is the lane's place in row 0.
template <typename T>
struct RowCopy {
  T v[4];
  uint32_t to[4];
  __device__ __forceinline__ void load(const RowLanes &l, int m0, int count, uint32_t rs, uint32_t rd,
                                       const T *base, int row_bytes) {
#pragma unroll
    for (int a = 0; a < 4; ++a) {
      const int m = m0 + a * l.per + l.sub;
      const uint32_t from = __shfl_sync(0xffffffffu, rs, m & 31);
      to[a] = __shfl_sync(0xffffffffu, rd, m & 31);
      if (m >= count || l.sub >= l.per) to[a] = kNowhere;
      if (to[a] != kNowhere)
        v[a] = *reinterpret_cast<const T *>(reinterpret_cast<const uint8_t *>(base) +
                                            static_cast<unsigned long long>(from) * row_bytes);
    }
  }
  __device__ __forceinline__ void store(T *base, int row_bytes) const {
#pragma unroll
    for (int a = 0; a < 4; ++a)
      if (to[a] != kNowhere)
        *reinterpret_cast<T *>(reinterpret_cast<uint8_t *>(base) +
                               static_cast<unsigned long long>(to[a]) * row_bytes) = v[a];
  }
};

__global__ void __launch_bounds__(kEvictThreads, 2) kv_evict_kernel(const EvictParams p) {
  extern __shared__ uint32_t smem[];
  __shared__ uint32_t hist[2][256];                  // added up over the copies
  __shared__ uint32_t copies[kEvictCopies][256];
  __shared__ __align__(16) uint32_t total[256];      // over the cluster
  __shared__ uint32_t found[3];                      // digit, slots wanted within it, slots
  __shared__ uint32_t near[kEvictPool], pool[kEvictPool];  // keys around the last kept one: here, of all
  __shared__ int near_count;
  __shared__ int warp_count[2][kEvictWarps];
  __shared__ int cta_count[3];                       // ties, holes, movers
  uint32_t *keys = smem, *list = smem + p.seg_max;   // holes first, then movers

  cg::cluster_group cluster = cg::this_cluster();
  const int C = static_cast<int>(cluster.num_blocks());
  const int rank = static_cast<int>(cluster.block_rank());
  const int row = static_cast<int>(blockIdx.x) / C;
  const int b = row / p.c.H, h = row - b * p.c.H;
  const int tid = threadIdx.x, warp = tid / 32, lane = tid & 31;
  wait_for_previous_grid();

  const int len = p.lens[b];
  const int room = p.c.width * p.c.S;
  const int n = len < 0 ? 0 : len < room ? len : room;
  const int left = n < p.budget ? n : p.budget;
  if (rank == 0 && h == 0 && tid == 0) {
    p.new_lens[b] = left;
    if (len > room && p.c.status) atomicOr(p.c.status, 1);
  }
  const long long base = static_cast<long long>(row) * p.state_width;
  const float *w = p.weights + base;
  const int *pos = p.positions + base;
  float *new_w = p.new_weights + base;
  int *new_pos = p.new_positions + base;
  const int seg = ((n + C - 1) / C + 31) & ~31;
  const int lo = rank * seg < n ? rank * seg : n, hi = lo + seg < n ? lo + seg : n;
  const int cnt = hi - lo;

  if (n <= p.budget) {  // the same for the whole cluster
    for (int i = lo + tid; i < hi; i += kEvictThreads) {
      const float x = w[i];
      const int y = pos[i];
      new_w[i] = x;
      new_pos[i] = y;
    }
    return;
  }

  // The state of the slots below the new length is written now, as if all of
  // them stayed (the moves overwrite the others'), and the rest is cleared: at
  // once, or behind the moves where the buffers are the same.
  const int from = p.seen[b] - p.recent;
  const bool in_place = new_w == w || new_pos == pos;
#pragma unroll 2
  for (int i = tid; i < cnt; i += kEvictThreads) {
    const float x = w[lo + i];
    const int y = pos[lo + i];
    keys[i] = evict_key(x, y, p.sinks, from);
    if (lo + i < left) {
      new_w[lo + i] = x;
      new_pos[lo + i] = y;
    } else if (!in_place) {
      new_w[lo + i] = 0.0f;
      new_pos[lo + i] = -1;
    }
  }
  for (int i = tid; i < kEvictCopies * 256; i += kEvictThreads) copies[i / 256][i % 256] = 0u;
  if (tid == 0) near_count = 0;
  __syncthreads();

  // the key of the last kept slot, most significant byte first
  uint32_t prefix = 0u, want = static_cast<uint32_t>(left), count = 0u;
  for (int pass = 0; pass < 4 && want != count; ++pass) {
    const int shift = 24 - 8 * pass;
    for (int i = tid; i < cnt; i += kEvictThreads) {
      const uint32_t k = keys[i];
      if (pass == 0 || (k >> (shift + 8)) == (prefix >> (shift + 8)))
        atomicAdd(&copies[tid % kEvictCopies][(k >> shift) & 255u], 1u);
    }
    __syncthreads();
    if (tid < 256) {
      uint32_t sum = 0u;
#pragma unroll
      for (int i = 0; i < kEvictCopies; ++i) {
        sum += copies[i][tid];
        copies[i][tid] = 0u;
      }
      if (C == 1) total[tid] = sum;
      else hist[pass & 1][tid] = sum;  // last read two passes ago
    }
    if (C > 1) {
      cluster.sync();
      if (tid < 256) {
        uint32_t part[kEvictMaxCluster], sum = 0u;
#pragma unroll
        for (int r = 0; r < kEvictMaxCluster; ++r)
          part[r] = r < C ? *cluster.map_shared_rank(&hist[pass & 1][tid], r) : 0u;
#pragma unroll
        for (int r = 0; r < kEvictMaxCluster; ++r) sum += part[r];
        total[tid] = sum;
      }
    }
    __syncthreads();
    // lane l of the first warp goes through bins 255 - 8 l downwards
    if (warp == 0) {
      const uint4 hi = *reinterpret_cast<const uint4 *>(&total[252 - 8 * lane]);
      const uint4 lo4 = *reinterpret_cast<const uint4 *>(&total[248 - 8 * lane]);
      const uint32_t bin[8] = {hi.w, hi.z, hi.y, hi.x, lo4.w, lo4.z, lo4.y, lo4.x};
      uint32_t sum = 0u;
#pragma unroll
      for (int i = 0; i < 8; ++i) sum += bin[i];
      uint32_t before = sum;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const uint32_t x = __shfl_up_sync(0xffffffffu, before, o);
        if (lane >= o) before += x;
      }
      before -= sum;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        if (before < want && want <= before + bin[i]) {
          found[0] = static_cast<uint32_t>(255 - 8 * lane - i);
          found[1] = want - before;
          found[2] = bin[i];
        }
        before += bin[i];
      }
    }
    __syncthreads();
    prefix |= found[0] << shift;  // (written again two barriers from here)
    want = found[1];
    count = found[2];  // keys that begin with the prefix: `want` of them stay
    if (pass > 0 && pass < 3 && want != count && count <= kEvictPool) {
      // few enough to be brought together and ranked: a thread counts how many
      // are above its key
      for (int i = tid; i < cnt; i += kEvictThreads)
        if ((keys[i] >> shift) == (prefix >> shift)) near[atomicAdd(&near_count, 1)] = keys[i];
      if (C > 1) cluster.sync();
      else __syncthreads();
      const int n_of = lane < C ? *cluster.map_shared_rank(&near_count, lane) : 0;
      int end = n_of;
#pragma unroll
      for (int o = 1; o < kEvictMaxCluster; o <<= 1) {
        const int x = __shfl_up_sync(0xffffffffu, end, o);
        if (lane >= o) end += x;
      }
      if (warp < C) {  // warp r fetches rank r's
        const int n_r = __shfl_sync(0xffffffffu, n_of, warp), at = __shfl_sync(0xffffffffu, end, warp) - n_r;
        const uint32_t *from_r = cluster.map_shared_rank(near, warp);
        for (int i = lane; i < n_r; i += 32) pool[at + i] = from_r[i];
      }
      __syncthreads();
      if (tid < static_cast<int>(count)) {
        const uint32_t k = pool[tid];
        uint32_t above = 0u, alike = 0u;
        for (uint32_t i = 0; i < count; ++i) {
          above += pool[i] > k;
          alike += pool[i] == k;
        }
        if (above < want && want <= above + alike) {  // the same for all alike
          found[0] = k;
          found[1] = want - above;
          found[2] = alike;
        }
      }
      __syncthreads();
      prefix = found[0];
      want = found[1];
      count = found[2];
      break;
    }
  }
  // every key that begins with the prefix stays: no tie to be broken
  const bool all_stay = want == count;

  // slots with the last kept key: the first `want` of them stay
  const int span = ((cnt + kEvictWarps - 1) / kEvictWarps + 31) & ~31;
  const int w0 = warp * span < cnt ? warp * span : cnt;
  const int w1 = w0 + span < cnt ? w0 + span : cnt;
  int tie0 = 0;
  if (!all_stay) {
    int ties = 0;
    for (int i = w0 + lane; i < w1; i += 32) ties += keys[i] == prefix;
    ties = __reduce_add_sync(0xffffffffu, ties);
    if (lane == 0) warp_count[0][warp] = ties;
    __syncthreads();
    if (warp == 0) {
      const int sum = __reduce_add_sync(0xffffffffu, lane < kEvictWarps ? warp_count[0][lane] : 0);
      if (lane == 0) cta_count[0] = sum;
    }
    cluster.sync();
    // (lane r asks rank r, and lane i warp i)
    tie0 = lane < rank ? *cluster.map_shared_rank(&cta_count[0], lane) : 0;
    tie0 += lane < warp ? warp_count[0][lane] : 0;
    tie0 = __reduce_add_sync(0xffffffffu, tie0);
    __syncthreads();
  } else {
    want = 0x7fffffffu;
  }

  // holes and movers of this warp's slots, counted and then listed in order
  int holes = 0, movers = 0, tie = tie0;
  for (int i0 = w0; i0 < w1; i0 += 32) {
    const int i = i0 + lane;
    const bool in = i < w1;
    const uint32_t k = in ? keys[i] : 0u;
    const bool same = in && k == prefix;
    const uint32_t m = __ballot_sync(0xffffffffu, same);
    const bool keep = in && (k > prefix || (same && tie + __popc(m & ((1u << lane) - 1u)) < static_cast<int>(want)));
    tie += __popc(m);
    const bool below = lo + i < left;
    holes += __popc(__ballot_sync(0xffffffffu, in && below && !keep));
    movers += __popc(__ballot_sync(0xffffffffu, keep && !below));
  }
  if (lane == 0) {
    warp_count[0][warp] = holes;
    warp_count[1][warp] = movers;
  }
  __syncthreads();
  const int lane_holes = lane < kEvictWarps ? warp_count[0][lane] : 0;
  const int lane_movers = lane < kEvictWarps ? warp_count[1][lane] : 0;
  int hole0 = __reduce_add_sync(0xffffffffu, lane < warp ? lane_holes : 0);
  int mover0 = __reduce_add_sync(0xffffffffu, lane < warp ? lane_movers : 0);
  const int all_holes = __reduce_add_sync(0xffffffffu, lane_holes);
  const int all_movers = __reduce_add_sync(0xffffffffu, lane_movers);
  if (tid == 0) {
    cta_count[1] = all_holes;
    cta_count[2] = all_movers;
  }
  mover0 += all_holes;
  tie = tie0;
  for (int i0 = w0; i0 < w1; i0 += 32) {
    const int i = i0 + lane;
    const bool in = i < w1;
    const uint32_t k = in ? keys[i] : 0u;
    const bool same = in && k == prefix;
    const uint32_t m = __ballot_sync(0xffffffffu, same), under = (1u << lane) - 1u;
    const bool keep = in && (k > prefix || (same && tie + __popc(m & under) < static_cast<int>(want)));
    tie += __popc(m);
    const bool below = lo + i < left;
    const bool hole = in && below && !keep, mover = keep && !below;
    const uint32_t mh = __ballot_sync(0xffffffffu, hole), mm = __ballot_sync(0xffffffffu, mover);
    if (hole) list[hole0 + __popc(mh & under)] = static_cast<uint32_t>(lo + i);
    if (mover) list[mover0 + __popc(mm & under)] = static_cast<uint32_t>(lo + i);
    hole0 += __popc(mh);
    mover0 += __popc(mm);
  }
  cluster.sync();

  // first hole and first mover of every CTA: lane r asks rank r
  int holes_of = lane < C ? *cluster.map_shared_rank(&cta_count[1], lane) : 0;
  int movers_of = lane < C ? *cluster.map_shared_rank(&cta_count[2], lane) : 0;
  int hole_end = holes_of, mover_end = movers_of;
#pragma unroll
  for (int o = 1; o < kEvictMaxCluster; o <<= 1) {
    const int x = __shfl_up_sync(0xffffffffu, hole_end, o), y = __shfl_up_sync(0xffffffffu, mover_end, o);
    if (lane >= o) {
      hole_end += x;
      mover_end += y;
    }
  }
  const int moves = __shfl_sync(0xffffffffu, hole_end, C - 1);
  const int *table = p.c.table + static_cast<long long>(b) * p.c.width;
  // The cluster's warps share the moves evenly; a warp looks up to 32 of them up
  // at once, a lane each, and then copies their rows, 16 bytes a lane, four
  // lines of them in flight.  A lane's place in a row (or rows) is always the
  // same.
  const RowLanes big(p.c.row_bytes / 8, lane), small(4 * p.c.G, lane);
  uint8_t *side = big.at < p.c.row_bytes / 16 ? p.c.k + big.at * 16 : p.c.v + big.at * 16 - p.c.row_bytes;
  const int kind = p.c.G ? small.at / p.c.G : 0;
  uint16_t *scale = kind == 0   ? p.c.k_scales
                    : kind == 1 ? p.c.k_biases
                    : kind == 2 ? p.c.v_scales
                                : p.c.v_biases;
  scale += p.c.G ? small.at - kind * p.c.G : 0;
  const int each = (moves + C * kEvictWarps - 1) / (C * kEvictWarps);
  const int m_end = (rank * kEvictWarps + warp + 1) * each < moves ? (rank * kEvictWarps + warp + 1) * each : moves;
  for (int m0 = (rank * kEvictWarps + warp) * each; m0 < m_end; m0 += 32) {
    const int count = m_end - m0 < 32 ? m_end - m0 : 32;
    uint32_t rs = kNowhere, rd = kNowhere;
    // the ranks that list the move's hole and mover, and where their lists begin
    const int m = m0 + lane;
    int rh = 0, rm = 0, h0 = 0, l0 = -__shfl_sync(0xffffffffu, holes_of, 0);
#pragma unroll
    for (int r = 1; r < kEvictMaxCluster; ++r) {
      const int he = __shfl_sync(0xffffffffu, hole_end, r - 1), me = __shfl_sync(0xffffffffu, mover_end, r - 1);
      const int holes_r = __shfl_sync(0xffffffffu, holes_of, r);
      if (r < C && m >= he) {
        rh = r;
        h0 = he;
      }
      if (r < C && m >= me) {
        rm = r;
        l0 = me - holes_r;  // movers come after the rank's holes
      }
    }
    if (lane < count) {
      const int dst = static_cast<int>(cluster.map_shared_rank(list, rh)[m - h0]);
      const int src = static_cast<int>(cluster.map_shared_rank(list, rm)[m - l0]);
      const int ps = src / p.c.S, pd = dst / p.c.S;
      const int es = __ldg(table + ps), ed = __ldg(table + pd);
      const float x = w[src];
      const int y = pos[src];
      const int sp = checked_page(p.c, es), dp = checked_page(p.c, ed);
      new_w[dst] = x;
      new_pos[dst] = y;
      if (sp >= 0 && dp >= 0) {
        rs = cache_row(p.c, sp, h, src - ps * p.c.S);
        rd = cache_row(p.c, dp, h, dst - pd * p.c.S);
        // all of the rows on their way at once
        for (int i = 0; count > 4 && i < p.c.row_bytes; i += 128) {
          const unsigned long long at = static_cast<unsigned long long>(rs) * p.c.row_bytes + i;
          asm volatile("prefetch.global.L2 [%0];\n" ::"l"(p.c.k + at));
          asm volatile("prefetch.global.L2 [%0];\n" ::"l"(p.c.v + at));
        }
      }
    }
    for (int half = 0; half < (big.more ? 2 : 1); ++half) {
      // (a row of more than 32 units, of bf16 heads of 256: keys, then values)
      uint4 *rows = reinterpret_cast<uint4 *>(half ? p.c.v + big.at * 16 : side);
      RowCopy<uint4> x;
      RowCopy<uint16_t> y;
      // the first lines of both kinds together, then what is left of each
      x.load(big, 0, count, rs, rd, rows, p.c.row_bytes);
      if (p.c.G) y.load(small, 0, count, rs, rd, scale, 2 * p.c.G);
      x.store(rows, p.c.row_bytes);
      if (p.c.G) y.store(scale, 2 * p.c.G);
      for (int i = 4 * big.per; i < count; i += 4 * big.per) {
        x.load(big, i, count, rs, rd, rows, p.c.row_bytes);
        x.store(rows, p.c.row_bytes);
      }
      for (int i = 4 * small.per; p.c.G && i < count; i += 4 * small.per) {
        y.load(small, i, count, rs, rd, scale, 2 * p.c.G);
        y.store(scale, 2 * p.c.G);
      }
    }
  }
  cluster.sync();  // every mover's state has been read, and every list
  for (int i = (lo > left ? lo : left) + tid; in_place && i < hi; i += kEvictThreads) {
    new_w[i] = 0.0f;
    new_pos[i] = -1;
  }
}

}  // namespace qmvc

// ---------------------------------------------------------------------------
// C entry points
// ---------------------------------------------------------------------------

namespace {

// (an array, so that a refusal needs no memory and nothing is thrown through a C
// entry point)
thread_local char g_kv_error[512];

int kfail(int code, const char *fmt, ...) __attribute__((format(printf, 2, 3)));
int kfail(int code, const char *fmt, ...) {
  va_list ap;
  va_start(ap, fmt);
  vsnprintf(g_kv_error, sizeof g_kv_error, fmt, ap);
  va_end(ap);
  return code;
}

int kok() {
  g_kv_error[0] = 0;
  return QMV_OK;
}

bool aligned(const void *p, unsigned to) { return (reinterpret_cast<uintptr_t>(p) & (to - 1)) == 0; }

constexpr int kMaxBatch = 4096;

// Checks what every entry point shares and fills the device's view.
int check_cache(const char *f, const qmv_kv_cache *c, const int *table, int batch, int width,
                int *status, qmvc::CacheView *out) {
  if (!c || !c->k || !c->v) return kfail(QMV_ERR_NULL, "%s: the cache or its k or v is NULL", f);
  if (c->bits != 4 && c->bits != 8 && c->bits != 16)
    return kfail(QMV_ERR_UNSUPPORTED, "%s: bits=%d not in {4,8,16}", f, c->bits);
  const int D = c->head_dim, gs = c->group_size;
  if (D != 64 && D != 96 && D != 128 && D != 256)
    return kfail(QMV_ERR_UNSUPPORTED, "%s: head_dim=%d not in {64,96,128,256}", f, D);
  const bool q = c->bits != 16;
  if (q) {
    if (!c->k_scales || !c->k_biases || !c->v_scales || !c->v_biases)
      return kfail(QMV_ERR_NULL, "%s: scales and biases of a quantized cache must not be NULL", f);
    if (gs != 32 && gs != 64 && gs != 128)
      return kfail(QMV_ERR_UNSUPPORTED, "%s: group_size=%d not in {32,64,128}", f, gs);
    if (D % gs)
      return kfail(QMV_ERR_SHAPE, "%s: head_dim=%d is not a multiple of group_size=%d", f, D, gs);
  }
  if (c->num_pages <= 0 || c->num_kv_heads <= 0 || c->page_size <= 0)
    return kfail(QMV_ERR_SHAPE, "%s: num_pages=%d num_kv_heads=%d page_size=%d must be positive", f,
                 c->num_pages, c->num_kv_heads, c->page_size);
  if (c->page_size % 16)
    return kfail(QMV_ERR_UNSUPPORTED, "%s: page_size=%d is not a multiple of 16", f, c->page_size);
  if (c->num_kv_heads > 65536 ||
      static_cast<double>(c->num_pages) * c->num_kv_heads * c->page_size >= 2147483648.0)
    return kfail(QMV_ERR_UNSUPPORTED, "%s: 2^31 rows or more in the cache", f);
  if (batch < 0 || batch > kMaxBatch)
    return kfail(batch < 0 ? QMV_ERR_SHAPE : QMV_ERR_UNSUPPORTED, "%s: batch=%d not in [0,%d]", f,
                 batch, kMaxBatch);
  if (static_cast<long long>(batch) * c->num_kv_heads > (1LL << 24))
    return kfail(QMV_ERR_UNSUPPORTED, "%s: batch * num_kv_heads above 2^24", f);
  if (width <= 0 || static_cast<double>(width) * c->page_size >= 2147483648.0)
    return kfail(QMV_ERR_SHAPE, "%s: table_width=%d pages of %d slots", f, width, c->page_size);
  if (!table) return kfail(QMV_ERR_NULL, "%s: block_table must not be NULL", f);
  const void *big[] = {c->k, c->v, c->k_scales, c->k_biases, c->v_scales, c->v_biases};
  for (int i = 0; i < (q ? 6 : 2); ++i)
    if (!aligned(big[i], 16)) return kfail(QMV_ERR_ALIGN, "%s: cache buffers must be 16-byte aligned", f);
  if (!aligned(table, 4) || !aligned(status, 4))
    return kfail(QMV_ERR_ALIGN, "%s: index arrays must be 4-byte aligned", f);
  out->k = static_cast<uint8_t *>(c->k);
  out->v = static_cast<uint8_t *>(c->v);
  out->k_scales = q ? static_cast<uint16_t *>(c->k_scales) : nullptr;
  out->k_biases = q ? static_cast<uint16_t *>(c->k_biases) : nullptr;
  out->v_scales = q ? static_cast<uint16_t *>(c->v_scales) : nullptr;
  out->v_biases = q ? static_cast<uint16_t *>(c->v_biases) : nullptr;
  out->table = table;
  out->num_pages = c->num_pages;
  out->H = c->num_kv_heads;
  out->S = c->page_size;
  out->D = D;
  out->bits = c->bits;
  out->G = q ? D / gs : 0;
  out->width = width;
  out->row_bytes = D * c->bits / 8;
  out->status = status;
  return QMV_OK;
}

using qmvc::Device;

// The current device and its SM count, asked once per device.
int current_device(const char *f, Device *out) {
  static std::atomic<int> known[qmvc::kMaxDevices];  // two threads may both ask
  int d = 0;
  const cudaError_t e = cudaGetDevice(&d);
  if (e != cudaSuccess || d < 0 || d >= qmvc::kMaxDevices)
    return kfail(QMV_ERR_CUDA, "%s: no usable CUDA device (%s)", f, cudaGetErrorString(e));
  int sms = known[d].load(std::memory_order_relaxed);
  if (sms == 0) {
    const cudaError_t q = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, d);
    if (q != cudaSuccess || sms <= 0)
      return kfail(QMV_ERR_CUDA, "%s: cannot query device %d (%s)", f, d, cudaGetErrorString(q));
    known[d].store(sms, std::memory_order_relaxed);
  }
  out->id = d;
  out->sms = sms;
  return QMV_OK;
}

int launched(const char *f, cudaError_t e) {
  return e == cudaSuccess ? kok() : kfail(QMV_ERR_CUDA, "%s launch: %s", f, cudaGetErrorString(e));
}

// What kv_append and kv_read share.
int check_rows(const char *f, qmvc::RowParams &p, const void *k, const void *v, long long k_stride,
               long long v_stride, const int *lens, const int *starts, int batch, int tokens) {
  if (!k || !v || !lens) return kfail(QMV_ERR_NULL, "%s: k, v and lens must not be NULL", f);
  const long long need = static_cast<long long>(p.c.H) * p.c.D;
  if (tokens < 0) return kfail(QMV_ERR_SHAPE, "%s: num_tokens=%d", f, tokens);
  if (!starts && tokens != batch)
    return kfail(QMV_ERR_SHAPE, "%s: without token_starts num_tokens must be batch", f);
  if (k_stride < need || v_stride < need)
    return kfail(QMV_ERR_SHAPE, "%s: a token's stride is below num_kv_heads*head_dim", f);
  if (k_stride % 8 || v_stride % 8 || !aligned(k, 16) || !aligned(v, 16))
    return kfail(QMV_ERR_ALIGN, "%s: every token of k and v must be 16-byte aligned", f);
  if (!aligned(lens, 4) || !aligned(starts, 4))
    return kfail(QMV_ERR_ALIGN, "%s: index arrays must be 4-byte aligned", f);
  p.k = static_cast<uint16_t *>(const_cast<void *>(k));
  p.v = static_cast<uint16_t *>(const_cast<void *>(v));
  p.k_stride = k_stride;
  p.v_stride = v_stride;
  p.lens = lens;
  p.starts = starts;
  p.batch = batch;
  p.tokens = tokens;
  p.wide = k_stride % 16 == 0 && v_stride % 16 == 0 && aligned(k, 32) && aligned(v, 32) &&
           (p.c.bits != 16 || (aligned(p.c.k, 32) && aligned(p.c.v, 32)));
  return QMV_OK;
}

// One wave of blocks, each with a whole number of passes over as many tokens as
// its threads hold at once (a block begins with look-ups that depend on one
// another: more and shorter blocks only repeat those).
template <bool APPEND>
int row_grid(qmvc::RowParams &p, int sms) {
  const int per_token = 2 * p.c.H * (p.c.D / 16);
  const int at_once = per_token < qmvc::kRowThreads ? qmvc::kRowThreads / per_token : 1;
  const long long blocks = static_cast<long long>(qmvc::row_blocks<APPEND>()) * sms;
  long long each = (p.tokens + blocks - 1) / blocks;
  each = (each + at_once - 1) / at_once * at_once;
  p.block_tokens = static_cast<int>(each);
  return static_cast<int>((p.tokens + each - 1) / each);
}

template <bool APPEND, int BITS, int GS, int D>
cudaError_t rows_t(qmvc::RowParams &p, int sms, cudaStream_t st) {
  if constexpr (D % GS != 0) return cudaErrorInvalidValue;  // refused before
  else
    return qmvc::launch_overlapped(qmvc::kv_rows_kernel<APPEND, BITS, GS, D>, dim3(row_grid<APPEND>(p, sms)),
                                   qmvc::kRowThreads, 0, 1, st, p);
}
template <bool APPEND, int BITS, int GS>
cudaError_t rows_g(qmvc::RowParams &p, int sms, cudaStream_t st) {
  switch (p.c.D) {
    case 64: return rows_t<APPEND, BITS, GS, 64>(p, sms, st);
    case 96: return rows_t<APPEND, BITS, GS, 96>(p, sms, st);
    case 128: return rows_t<APPEND, BITS, GS, 128>(p, sms, st);
    default: return rows_t<APPEND, BITS, GS, 256>(p, sms, st);
  }
}
template <bool APPEND, int BITS>
cudaError_t rows_b(qmvc::RowParams &p, int sms, cudaStream_t st) {
  switch (p.c.D / p.c.G) {
    case 32: return rows_g<APPEND, BITS, 32>(p, sms, st);
    case 64: return rows_g<APPEND, BITS, 64>(p, sms, st);
    default: return rows_g<APPEND, BITS, 128>(p, sms, st);
  }
}
template <bool APPEND>
cudaError_t rows_launch(qmvc::RowParams &p, int sms, cudaStream_t st) {
  return p.c.bits == 4   ? rows_b<APPEND, 4>(p, sms, st)
         : p.c.bits == 8 ? rows_b<APPEND, 8>(p, sms, st)
                         : rows_g<APPEND, 16, 32>(p, sms, st);  // bf16 rows have no groups
}

// Arrays of 4-byte words in device memory: `rows` rows of `width` words, `pitch`
// words apart.
struct Words {
  const char *name;
  const void *at;
  long long rows, width, pitch;
};

// Whether two of them have a word in common.  Rows i and j do where
// -a.width < (a.at - b.at) + (i - j) * pitch < b.width; both have the pitch of
// the state arrays, or one row.
bool overlap(const Words &a, const Words &b) {
  if (a.rows * a.width == 0 || b.rows * b.width == 0) return false;
  const long long pitch = a.rows > 1 ? a.pitch : b.pitch;
  const long long d = (static_cast<long long>(reinterpret_cast<uintptr_t>(b.at)) -
                       static_cast<long long>(reinterpret_cast<uintptr_t>(a.at))) / 4;
  // the first i - j above (d - a.width) / pitch that there is
  const long long low = d - a.width;
  long long t = low / pitch - (low % pitch < 0) + 1;
  if (t < 1 - b.rows) t = 1 - b.rows;
  return t < a.rows && t * pitch < d + b.width;
}

int check_state_width(const char *f, const qmvc::CacheView &c, int state_width) {
  if (state_width < c.width * c.S)
    return kfail(QMV_ERR_SHAPE, "%s: state_width=%d is below the sequence's room of %d slots", f,
                 state_width, c.width * c.S);
  return QMV_OK;
}

}  // namespace

extern "C" {

int kv_append(const qmv_kv_cache *cache, const void *k, const void *v, long long k_stride,
              long long v_stride, const int *block_table, const int *lens,
              const int *token_starts, int batch, int num_tokens, int table_width,
              const int *seen, int *positions, float *weights, int state_width, int *d_status,
              void *stream) {
  const char *f = "kv_append";
  qmvc::RowParams p = {};
  int rc = check_cache(f, cache, block_table, batch, table_width, d_status, &p.c);
  if (!rc) rc = check_rows(f, p, k, v, k_stride, v_stride, lens, token_starts, batch, num_tokens);
  if (rc) return rc;
  if (seen || positions || weights) {
    if (!seen || !positions || !weights)
      return kfail(QMV_ERR_NULL, "%s: seen, positions and weights go together", f);
    if ((rc = check_state_width(f, p.c, state_width))) return rc;
    if (!aligned(seen, 4) || !aligned(positions, 4) || !aligned(weights, 4))
      return kfail(QMV_ERR_ALIGN, "%s: seen, positions and weights must be 4-byte aligned", f);
    p.seen = seen;
    p.positions = positions;
    p.weights = weights;
    p.state_width = state_width;
  }
  if (batch == 0 || num_tokens == 0) return kok();
  Device dev;
  if ((rc = current_device(f, &dev))) return rc;
  return launched(f, rows_launch<true>(p, dev.sms, static_cast<cudaStream_t>(stream)));
}

int kv_read(const qmv_kv_cache *cache, void *k, void *v, long long k_stride, long long v_stride,
            const int *block_table, const int *lens, const int *token_starts, int batch,
            int num_tokens, int table_width, int *d_status, void *stream) {
  const char *f = "kv_read";
  qmvc::RowParams p = {};
  int rc = check_cache(f, cache, block_table, batch, table_width, d_status, &p.c);
  if (!rc) rc = check_rows(f, p, k, v, k_stride, v_stride, lens, token_starts, batch, num_tokens);
  if (rc) return rc;
  if (batch == 0 || num_tokens == 0) return kok();
  Device dev;
  if ((rc = current_device(f, &dev))) return rc;
  return launched(f, rows_launch<false>(p, dev.sms, static_cast<cudaStream_t>(stream)));
}

// What kv_attention and its workspace query share.
static int check_attention(const char *f, const qmv_kv_cache *cache, const int *table, int batch,
                           int num_q_heads, int width, int *status, qmvc::CacheView *c) {
  int rc = check_cache(f, cache, table, batch, width, status, c);
  if (rc) return rc;
  if (num_q_heads <= 0 || num_q_heads % c->H)
    return kfail(QMV_ERR_SHAPE, "%s: num_q_heads=%d is not a positive multiple of num_kv_heads=%d", f,
                 num_q_heads, c->H);
  if (num_q_heads > 65535)
    return kfail(QMV_ERR_UNSUPPORTED, "%s: num_q_heads=%d above 65535", f, num_q_heads);
  // slots are numbered in 31 bits, the ends of tiles and of the weights' blocks behind
  // the last one among them (check_cache leaves a room below 2^31)
  if (width * c->S > 0x7fffffff - 4095)
    return kfail(QMV_ERR_UNSUPPORTED, "%s: room of %d slots above 2^31 - 4096", f, width * c->S);
  // tiles of 16 slots and (for the weights) score rows are numbered in 31 bits
  if (static_cast<double>(batch) * num_q_heads * (static_cast<double>(width) * c->S / 16 + 1) >= 2147483648.0)
    return kfail(QMV_ERR_UNSUPPORTED, "%s: batch * num_q_heads * room above 2^35", f);
  return QMV_OK;
}

static size_t attention_workspace(const qmvc::CacheView &c, int batch, int num_q_heads, bool weights,
                                  int sms) {
  return c.bits == 4   ? qmvc::attn_workspace_4(c, batch, num_q_heads, weights, sms)
         : c.bits == 8 ? qmvc::attn_workspace_8(c, batch, num_q_heads, weights, sms)
                       : qmvc::attn_workspace_16(c, batch, num_q_heads, weights, sms);
}

int kv_attention_workspace(const qmv_kv_cache *cache, int batch, int num_q_heads, int table_width,
                           int with_weights, size_t *bytes) {
  const char *f = "kv_attention_workspace";
  static const int no_table = 0;  // stands for the call's table, never read
  if (!bytes) return kfail(QMV_ERR_NULL, "%s: bytes must not be NULL", f);
  qmvc::CacheView c = {};
  int rc = check_attention(f, cache, &no_table, batch, num_q_heads, table_width, nullptr, &c);
  if (rc) return rc;
  Device dev;
  if ((rc = current_device(f, &dev))) return rc;
  *bytes = attention_workspace(c, batch, num_q_heads, with_weights != 0, dev.sms);
  return kok();
}

int kv_attention(const qmv_kv_cache *cache, const void *q, long long q_stride,
                 const int *block_table, const int *lens, void *out, int batch, int num_q_heads,
                 int table_width, float scale, float *weights, int state_width, void *workspace,
                 size_t workspace_bytes, int *d_status, void *stream) {
  const char *f = "kv_attention";
  qmvc::AttnArgs a = {};
  int rc = check_attention(f, cache, block_table, batch, num_q_heads, table_width, d_status, &a.cache);
  if (rc) return rc;
  if (!q || !lens || !out) return kfail(QMV_ERR_NULL, "%s: q, lens and out must not be NULL", f);
  if (!std::isfinite(scale)) return kfail(QMV_ERR_SHAPE, "%s: scale is not finite", f);
  if (q_stride < static_cast<long long>(num_q_heads) * a.cache.D)
    return kfail(QMV_ERR_SHAPE, "%s: q_stride is below num_q_heads*head_dim", f);
  if (q_stride % 8 || !aligned(q, 16) || !aligned(out, 16))
    return kfail(QMV_ERR_ALIGN, "%s: every row of q, and out, must be 16-byte aligned", f);
  if (!aligned(lens, 4) || !aligned(weights, 4))
    return kfail(QMV_ERR_ALIGN, "%s: lens and weights must be 4-byte aligned", f);
  if (weights && (rc = check_state_width(f, a.cache, state_width))) return rc;
  if (batch == 0) return kok();
  Device dev;
  if ((rc = current_device(f, &dev))) return rc;
  const size_t need = attention_workspace(a.cache, batch, num_q_heads, weights != nullptr, dev.sms);
  if (need && !workspace) return kfail(QMV_ERR_NULL, "%s: workspace must not be NULL", f);
  if (workspace_bytes < need)
    return kfail(QMV_ERR_SHAPE, "%s: workspace of %zu bytes, the call needs %zu", f, workspace_bytes,
                 need);
  if (!aligned(workspace, 16)) return kfail(QMV_ERR_ALIGN, "%s: workspace must be 16-byte aligned", f);
  a.q = q;
  a.q_stride = q_stride;
  a.lens = lens;
  a.out = out;
  a.batch = batch;
  a.num_q_heads = num_q_heads;
  a.scale = scale;
  a.weights = weights;
  a.state_width = state_width;
  a.workspace = workspace;
  a.stream = static_cast<cudaStream_t>(stream);
  return launched(f, a.cache.bits == 4   ? qmvc::attn_launch_4(a, dev)
                     : a.cache.bits == 8 ? qmvc::attn_launch_8(a, dev)
                                         : qmvc::attn_launch_16(a, dev));
}

int kv_evict(const qmv_kv_cache *cache, const int *block_table, const int *lens, const int *seen,
             const float *weights, const int *positions, int *new_lens, float *new_weights,
             int *new_positions, int batch, int table_width, int state_width, int budget,
             int recent, int sinks, int *d_status, void *stream) {
  const char *f = "kv_evict";
  qmvc::EvictParams p = {};
  int rc = check_cache(f, cache, block_table, batch, table_width, d_status, &p.c);
  if (rc) return rc;
  if (!lens || !seen || !weights || !positions || !new_lens || !new_weights || !new_positions)
    return kfail(QMV_ERR_NULL, "%s: a state or length array is NULL", f);
  if (budget <= 0 || recent < 0 || sinks < 0 || static_cast<long long>(recent) + sinks > budget)
    return kfail(QMV_ERR_SHAPE, "%s: budget=%d recent=%d sinks=%d: need recent + sinks <= budget", f,
                 budget, recent, sinks);
  if ((rc = check_state_width(f, p.c, state_width))) return rc;
  constexpr int kEvictSlots = 2048;
  const int room = table_width * p.c.S;
  if (room > qmvc::kEvictMaxSlots)
    return kfail(QMV_ERR_UNSUPPORTED, "%s: room of %d slots above %d", f, room, qmvc::kEvictMaxSlots);
  const void *words[] = {lens, seen, weights, positions, new_lens, new_weights, new_positions};
  for (const void *w : words)
    if (!aligned(w, 4)) return kfail(QMV_ERR_ALIGN, "%s: state and length arrays must be 4-byte aligned", f);
  // A cluster of one head may write new_lens, or its state, while those of other
  // heads have yet to read their inputs.
  const long long state_rows = static_cast<long long>(batch) * p.c.H;
  const long long table_words = static_cast<long long>(batch) * table_width;
  const Words read[] = {{"lens", lens, 1, batch, batch},
                        {"seen", seen, 1, batch, batch},
                        {"block_table", block_table, 1, table_words, table_words},
                        {"weights", weights, state_rows, room, state_width},
                        {"positions", positions, state_rows, room, state_width}};
  const Words written[] = {{"new_lens", new_lens, 1, batch, batch},
                           {"new_weights", new_weights, state_rows, room, state_width},
                           {"new_positions", new_positions, state_rows, room, state_width}};
  for (int i = 0; i < 3; ++i) {
    for (int j = 0; j < 5; ++j) {
      const bool in_place = i > 0 && j == i + 2 && written[i].at == read[j].at;
      if (!in_place && overlap(written[i], read[j]))
        return kfail(QMV_ERR_UNSUPPORTED, "%s: %s overlaps %s", f, written[i].name, read[j].name);
    }
    for (int j = 0; j < i; ++j)
      if (overlap(written[i], written[j]))
        return kfail(QMV_ERR_UNSUPPORTED, "%s: %s overlaps %s", f, written[i].name, written[j].name);
  }
  if (batch == 0) return kok();
  Device dev;
  if ((rc = current_device(f, &dev))) return rc;
  p.lens = lens;
  p.seen = seen;
  p.weights = weights;
  p.positions = positions;
  p.new_lens = new_lens;
  p.new_weights = new_weights;
  p.new_positions = new_positions;
  p.batch = batch;
  p.state_width = state_width;
  p.budget = budget;
  p.recent = recent;
  p.sinks = sinks;
  // A CTA for every kEvictSlots slots of room, up to the portable cluster size,
  // while all clusters fit the device at once (two CTAs to an SM, less what
  // clusters of 8 leave unused: 32 rows of 16384 slots took 32 us in clusters of
  // 8, which ran in two waves), and at least as many as hold the keys.
  int cluster = 1;
  const long long rows = static_cast<long long>(batch) * p.c.H;
  while (cluster < qmvc::kEvictMaxCluster && cluster * kEvictSlots < room &&
         (2 * cluster * rows <= 2 * dev.sms || room > cluster * (qmvc::kEvictMaxSlots / qmvc::kEvictMaxCluster)))
    cluster *= 2;
  p.seg_max = ((room + cluster - 1) / cluster + 31) & ~31;
  const size_t smem = 8u * static_cast<size_t>(p.seg_max);
  static qmvc::Granted granted;
  const cudaError_t e = allow_smem(qmvc::kv_evict_kernel, granted, dev, static_cast<int>(smem));
  if (e != cudaSuccess) return kfail(QMV_ERR_CUDA, "%s: shared memory: %s", f, cudaGetErrorString(e));
  return launched(f, qmvc::launch_overlapped(qmvc::kv_evict_kernel, dim3(batch * p.c.H * cluster),
                                             qmvc::kEvictThreads, smem, cluster,
                                             static_cast<cudaStream_t>(stream), p));
}

const char *qmv_kv_last_error(void) { return g_kv_error; }

}  // extern "C"
