// qmv_kv.cu -- the paged key-value cache in the packed affine format:
// kv_append (bf16 rows in, quantized or as they are), kv_read (dense bf16
// rows out), kv_evict (the slots with the least accumulated attention weight
// make room), and the C entry points, kv_attention's among them (its kernels
// are in qmv_kv_attn.cuh).  Contracts are in include/qmv.h.
//
// Append and read are streaming and element-wise: bf16 rows on one side, code
// rows, scales and biases on the other.  A warp takes 32 chunks of 8 elements
// of one token's heads (keys first, then values), so the token's sequence,
// slot and page are looked up once for the warp; a group of 32, 64 or 128
// elements is 4, 8 or 16 neighbouring lanes.
#include <cooperative_groups.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cmath>
#include <cstdarg>
#include <cstdint>
#include <cstdio>
#include <cstring>
#include <mutex>
#include <string>

#include "qmv.h"
#include "qmv_kv.h"

namespace qmvc {

namespace cg = cooperative_groups;

constexpr int kRowThreads = 256;

struct RowParams {
  CacheView c;
  uint16_t *k, *v;            // dense rows: read by append, written by read
  long long k_stride, v_stride;
  const int *lens, *starts;   // starts may be null: one token per sequence
  const int *seen;            // slot state (append), or null
  int *positions;
  float *weights;
  int batch, tokens, state_width;
};

// Where token t goes: its sequence, slot, page and place in the page.  False
// where it has none (padding, an unused row of the batch, or a bad index).
struct Place {
  int seq, slot, nth, page, at;
};

__device__ __forceinline__ bool place_of(const RowParams &p, int t, Place &o) {
  int first = t;
  o.seq = t;
  if (p.starts) {
    // the last sequence that starts at or before t
    int lo = 0, hi = p.batch;
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (__ldg(p.starts + mid) <= t) lo = mid;
      else hi = mid;
    }
    first = __ldg(p.starts + lo);
    if (t < first || t >= __ldg(p.starts + lo + 1)) return false;
    o.seq = lo;
  } else {
    first = t;
  }
  const int len = __ldg(p.lens + o.seq);
  if (len < 0) return false;
  o.nth = t - first;
  const long long slot = static_cast<long long>(len) + o.nth;
  if (slot >= static_cast<long long>(p.c.width) * p.c.S) {
    if (p.c.status) atomicOr(p.c.status, 1);
    return false;
  }
  o.slot = static_cast<int>(slot);
  const int at_page = o.slot / p.c.S;
  o.at = o.slot - at_page * p.c.S;
  o.page = checked_page(p.c, __ldg(p.c.table + static_cast<long long>(o.seq) * p.c.width + at_page));
  return o.page >= 0;
}

// ---------------------------------------------------------------------------
// The quantizer's binary32 steps, those of affine_quantize (qmv_quant.cu); the
// rows of the two are tested to be the same bits
// ---------------------------------------------------------------------------

// min(round(d / scale), n_bins), halves away from zero: the product with the
// rounded reciprocal is within 3 * 2^-24 of the quotient, so it decides the
// code except near a half-integer, where the IEEE division does.
__device__ __forceinline__ uint32_t code_of(float v, float bias, float scale, float rcp,
                                            float n_bins) {
  const float d = __fsub_rn(v, bias);
  const float t = __fmul_rn(d, rcp);
  const float r = rintf(t);
  float code = r;
  if (fabsf(__fsub_rn(t, r)) > 0.5f - fmaxf(fabsf(t), 1.0f) * 0x1p-20f)
    code = roundf(__fdiv_rn(d, scale));
  return static_cast<uint32_t>(fminf(code, n_bins));
}

// Scale and bias of a group with range [lo, hi], hi >= 0.
__device__ __forceinline__ float2 scale_bias(float lo, float hi, float n_bins) {
  const float size = fmaxf(__fdiv_rn(__fsub_rn(hi, lo), n_bins), 1e-7f);
  const bool low = fabsf(lo) > fabsf(hi);
  const float edge = low ? lo : hi, step = low ? size : -size;
  const float q0 = roundf(__fdiv_rn(edge, step));
  return q0 == 0.0f ? make_float2(step, 0.0f) : make_float2(__fdiv_rn(edge, q0), edge);
}

// ---------------------------------------------------------------------------
// Append
// ---------------------------------------------------------------------------

// 8 bf16 elements in, 8 codes out (BITS bytes); the group's first lane stores
// its scale and bias.  All lanes of the warp take part.
template <int BITS, int GS>
__device__ __forceinline__ uint2 quantize_chunk(const uint4 raw, int lane, uint16_t &s,
                                                uint16_t &b) {
  constexpr float n_bins = static_cast<float>((1 << BITS) - 1);
  const uint32_t pr[4] = {raw.x, raw.y, raw.z, raw.w};
  float v[8];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    v[2 * i] = __uint_as_float(pr[i] << 16);
    v[2 * i + 1] = __uint_as_float(pr[i] & 0xffff0000u);
  }
  float lo = __uint_as_float(0x7f7f0000u), hi = 0.0f;  // the largest finite bf16
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    lo = fminf(lo, v[i]);
    hi = fmaxf(hi, v[i]);
  }
#pragma unroll
  for (int o = 1; o < GS / 8; o <<= 1) {
    lo = fminf(lo, __shfl_xor_sync(0xffffffffu, lo, o));
    hi = fmaxf(hi, __shfl_xor_sync(0xffffffffu, hi, o));
  }
  const float2 sb = scale_bias(lo, hi, n_bins);
  s = __bfloat16_as_ushort(__float2bfloat16_rn(sb.x));
  b = __bfloat16_as_ushort(__float2bfloat16_rn(sb.y));
  const float rcp = __frcp_rn(sb.x);
  uint32_t w[2] = {0u, 0u};
#pragma unroll
  for (int i = 0; i < 8; ++i)
    w[i * BITS / 32] |= code_of(v[i], sb.y, sb.x, rcp, n_bins) << (i * BITS % 32);
  return make_uint2(w[0], w[1]);
}

template <int BITS, int GS, int D>
__global__ void __launch_bounds__(kRowThreads) kv_append_kernel(const RowParams p) {
  constexpr int kChunks = D / 8;  // chunks of a row
  const int lane = threadIdx.x & 31;
  const int side = p.c.H * kChunks;  // chunks of a token's keys
  const int per_token = (2 * side + 31) / 32;
  const long long items = static_cast<long long>(p.tokens) * per_token;
  const long long warps = static_cast<long long>(gridDim.x) * (kRowThreads / 32);
  wait_for_previous_grid();
  for (long long it = static_cast<long long>(blockIdx.x) * (kRowThreads / 32) + threadIdx.x / 32;
       it < items; it += warps) {
    const int t = static_cast<int>(it / per_token), part = static_cast<int>(it - static_cast<long long>(t) * per_token);
    Place o;
    if (!place_of(p, t, o)) continue;
    const int cc = part * 32 + lane;
    const bool live = cc < 2 * side, value = cc >= side;
    const int rest = value ? cc - side : cc;
    const int h = rest / kChunks, i = rest - h * kChunks;
    uint4 raw = make_uint4(0u, 0u, 0u, 0u);
    if (live) {
      const uint16_t *src = value ? p.v + t * p.v_stride : p.k + t * p.k_stride;
      raw = __ldg(reinterpret_cast<const uint4 *>(src) + rest);
    }
    const long long row = cache_row(p.c, o.page, live ? h : 0, o.at);
    uint8_t *dst = (value ? p.c.v : p.c.k) + row * (D * BITS / 8) + i * BITS;
    if constexpr (BITS == 16) {
      if (live) *reinterpret_cast<uint4 *>(dst) = raw;
    } else {
      uint16_t s, b;
      const uint2 w = quantize_chunk<BITS, GS>(raw, lane, s, b);
      if (live) {
        if constexpr (BITS == 4) *reinterpret_cast<uint32_t *>(dst) = w.x;
        else *reinterpret_cast<uint2 *>(dst) = w;
        if (lane % (GS / 8) == 0) {
          const long long g = row * (D / GS) + i / (GS / 8);
          (value ? p.c.v_scales : p.c.k_scales)[g] = s;
          (value ? p.c.v_biases : p.c.k_biases)[g] = b;
        }
      }
    }
    if (part == 0 && p.positions) {
      const int pos = __ldg(p.seen + o.seq) + o.nth;
      for (int hh = lane; hh < p.c.H; hh += 32) {
        const long long j = (static_cast<long long>(o.seq) * p.c.H + hh) * p.state_width + o.slot;
        p.positions[j] = pos;
        p.weights[j] = 0.0f;
      }
    }
  }
  let_next_grid_start();
}

// ---------------------------------------------------------------------------
// Read
// ---------------------------------------------------------------------------

// bf16(s * q + b) of 8 codes: the bf16 multiply-add rounds the exact value
// once; codes enter as exact bf16 numbers (those of 8 bits through binary32).
template <int BITS>
__device__ __forceinline__ uint4 dequantize_chunk(const uint2 w, uint16_t s, uint16_t b) {
  const __nv_bfloat16 sb = __ushort_as_bfloat16(s), bb = __ushort_as_bfloat16(b);
  const __nv_bfloat162 s2 = __halves2bfloat162(sb, sb), b2 = __halves2bfloat162(bb, bb);
  uint32_t out[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    __nv_bfloat162 q;
    if constexpr (BITS == 4) {
      const uint32_t m = ((w.x >> (8 * j)) & 0xfu) | (((w.x >> (8 * j + 4)) & 0xfu) << 16) | 0x43004300u;
      const uint32_t one28 = 0x43004300u;
      q = __hsub2(*reinterpret_cast<const __nv_bfloat162 *>(&m),
                  *reinterpret_cast<const __nv_bfloat162 *>(&one28));
    } else {
      const uint32_t x = j < 2 ? w.x : w.y;
      const uint32_t c0 = (x >> (16 * (j & 1))) & 0xffu, c1 = (x >> (16 * (j & 1) + 8)) & 0xffu;
      q = __floats2bfloat162_rn(__fsub_rn(__uint_as_float(0x4b000000u | c0), 8388608.0f),
                                __fsub_rn(__uint_as_float(0x4b000000u | c1), 8388608.0f));
    }
    const __nv_bfloat162 r = __hfma2(q, s2, b2);
    out[j] = *reinterpret_cast<const uint32_t *>(&r);
  }
  return make_uint4(out[0], out[1], out[2], out[3]);
}

template <int BITS, int D>
__global__ void __launch_bounds__(kRowThreads) kv_read_kernel(const RowParams p) {
  constexpr int kChunks = D / 8;
  const int lane = threadIdx.x & 31;
  const int side = p.c.H * kChunks;
  const int per_token = (2 * side + 31) / 32;
  const long long items = static_cast<long long>(p.tokens) * per_token;
  const long long warps = static_cast<long long>(gridDim.x) * (kRowThreads / 32);
  const int group_chunks = BITS == 16 ? 1 : kChunks / p.c.G;
  wait_for_previous_grid();
  for (long long it = static_cast<long long>(blockIdx.x) * (kRowThreads / 32) + threadIdx.x / 32;
       it < items; it += warps) {
    const int t = static_cast<int>(it / per_token), part = static_cast<int>(it - static_cast<long long>(t) * per_token);
    Place o;
    if (!place_of(p, t, o)) continue;
    const int cc = part * 32 + lane;
    if (cc >= 2 * side) continue;
    const bool value = cc >= side;
    const int rest = value ? cc - side : cc;
    const int h = rest / kChunks, i = rest - h * kChunks;
    const long long row = cache_row(p.c, o.page, h, o.at);
    const uint8_t *src = (value ? p.c.v : p.c.k) + row * (D * BITS / 8) + i * BITS;
    uint4 r;
    if constexpr (BITS == 16) {
      r = *reinterpret_cast<const uint4 *>(src);
    } else {
      uint2 w = make_uint2(0u, 0u);
      if constexpr (BITS == 4) w.x = *reinterpret_cast<const uint32_t *>(src);
      else w = *reinterpret_cast<const uint2 *>(src);
      const long long g = row * p.c.G + i / group_chunks;
      r = dequantize_chunk<BITS>(w, (value ? p.c.v_scales : p.c.k_scales)[g],
                                 (value ? p.c.v_biases : p.c.k_biases)[g]);
    }
    uint16_t *dst = value ? p.v + t * p.v_stride : p.k + t * p.k_stride;
    reinterpret_cast<uint4 *>(dst)[rest] = r;
  }
  let_next_grid_start();
}

// ---------------------------------------------------------------------------
// Evict
// ---------------------------------------------------------------------------

// A (sequence, kv head)'s slots are shared out over the CTAs of a cluster.
// The weights become keys in shared memory whose unsigned order is the order
// of the choice, are read from memory once, and the key of the last kept slot
// is found 8 bits at a time from a histogram added up over the cluster.  Then
// each CTA lists its evicted slots below the new length (holes) and its kept
// ones at or above it (movers), in order, and the cluster's warps move the
// i-th mover's rows into the i-th hole.
constexpr int kEvictThreads = 512;
constexpr int kEvictWarps = kEvictThreads / 32;
constexpr int kEvictMaxCluster = 8;
constexpr int kEvictMaxSlots = 196608;

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

__global__ void __launch_bounds__(kEvictThreads) kv_evict_kernel(const EvictParams p) {
  extern __shared__ uint32_t smem[];
  __shared__ uint32_t hist[2][256];
  __shared__ uint32_t found[2];                      // digit, slots wanted within it
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

  const int from = p.seen[b] - p.recent;
  for (int i = tid; i < cnt; i += kEvictThreads)
    keys[i] = evict_key(w[lo + i], pos[lo + i], p.sinks, from);
  for (int i = tid; i < 512; i += kEvictThreads) hist[i / 256][i % 256] = 0u;
  __syncthreads();

  // the key of the last kept slot, most significant byte first
  uint32_t prefix = 0u, want = static_cast<uint32_t>(left);
  for (int pass = 0; pass < 4; ++pass) {
    const int shift = 24 - 8 * pass;
    uint32_t *hg = hist[pass & 1];
    for (int i = tid; i < cnt; i += kEvictThreads) {
      const uint32_t k = keys[i];
      if (pass == 0 || (k >> (shift + 8)) == (prefix >> (shift + 8)))
        atomicAdd(&hg[(k >> shift) & 255u], 1u);
    }
    cluster.sync();
    if (warp == 0) {
      // lane l adds up bins 255 - 8 l downwards over the cluster
      uint32_t bin[8], sum = 0u;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        bin[i] = 0u;
        for (int r = 0; r < C; ++r)
          bin[i] += *cluster.map_shared_rank(&hg[255 - 8 * lane - i], r);
        sum += bin[i];
      }
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
        }
        before += bin[i];
      }
    } else {
      // the other buffer was last read before this pass's cluster.sync
      for (int i = tid - 32; i < 256; i += kEvictThreads - 32) hist[(pass + 1) & 1][i] = 0u;
    }
    __syncthreads();
    prefix |= found[0] << shift;
    want = found[1];
    __syncthreads();
  }

  // slots with the last kept key: the first `want` of them stay
  const int span = ((cnt + kEvictWarps - 1) / kEvictWarps + 31) & ~31;
  const int w0 = warp * span < cnt ? warp * span : cnt;
  const int w1 = w0 + span < cnt ? w0 + span : cnt;
  int ties = 0;
  for (int i = w0 + lane; i < w1; i += 32) ties += keys[i] == prefix;
  ties = __reduce_add_sync(0xffffffffu, ties);
  if (lane == 0) warp_count[0][warp] = ties;
  __syncthreads();
  if (tid == 0) {
    int sum = 0;
    for (int i = 0; i < kEvictWarps; ++i) sum += warp_count[0][i];
    cta_count[0] = sum;
  }
  cluster.sync();
  int tie0 = 0;
  for (int r = 0; r < rank; ++r) tie0 += *cluster.map_shared_rank(&cta_count[0], r);
  for (int i = 0; i < warp; ++i) tie0 += warp_count[0][i];
  __syncthreads();

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
  int hole0 = 0, mover0 = 0, all_holes = 0, all_movers = 0;
  for (int i = 0; i < kEvictWarps; ++i) {
    if (i == warp) {
      hole0 = all_holes;
      mover0 = all_movers;
    }
    all_holes += warp_count[0][i];
    all_movers += warp_count[1][i];
  }
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
    if (keep && below) {
      const float x = w[lo + i];
      const int y = pos[lo + i];
      new_w[lo + i] = x;
      new_pos[lo + i] = y;
    }
  }
  cluster.sync();

  // first hole and first mover of every CTA
  int hole_at[kEvictMaxCluster + 1], mover_at[kEvictMaxCluster + 1];
  hole_at[0] = mover_at[0] = 0;
#pragma unroll
  for (int r = 0; r < kEvictMaxCluster; ++r) {
    hole_at[r + 1] = hole_at[r] + (r < C ? *cluster.map_shared_rank(&cta_count[1], r) : 0);
    mover_at[r + 1] = mover_at[r] + (r < C ? *cluster.map_shared_rank(&cta_count[2], r) : 0);
  }
  const int moves = hole_at[kEvictMaxCluster];
  const int *table = p.c.table + static_cast<long long>(b) * p.c.width;
  for (int m = rank * kEvictWarps + warp; m < moves; m += C * kEvictWarps) {
    int rh = 0, rm = 0, h0 = 0, m0 = 0, nh = hole_at[1];
#pragma unroll
    for (int r = 1; r < kEvictMaxCluster; ++r) {
      if (m >= hole_at[r] && r < C) {
        rh = r;
        h0 = hole_at[r];
      }
      if (m >= mover_at[r] && r < C) {
        rm = r;
        m0 = mover_at[r];
        nh = hole_at[r + 1] - hole_at[r];
      }
    }
    const int dst = static_cast<int>(cluster.map_shared_rank(list, rh)[m - h0]);
    const int src = static_cast<int>(cluster.map_shared_rank(list, rm)[nh + m - m0]);
    if (lane == 0) {
      const float x = w[src];
      const int y = pos[src];
      new_w[dst] = x;
      new_pos[dst] = y;
    }
    const int sp = checked_page(p.c, __ldg(table + src / p.c.S));
    const int dp = checked_page(p.c, __ldg(table + dst / p.c.S));
    if (sp < 0 || dp < 0) continue;
    const long long rs = cache_row(p.c, sp, h, src % p.c.S), rd = cache_row(p.c, dp, h, dst % p.c.S);
    const int units = p.c.row_bytes / 16;
    for (int i = lane; i < 2 * units; i += 32) {
      uint8_t *side = i < units ? p.c.k : p.c.v;
      const int at = i < units ? i : i - units;
      reinterpret_cast<uint4 *>(side + rd * p.c.row_bytes)[at] =
          reinterpret_cast<const uint4 *>(side + rs * p.c.row_bytes)[at];
    }
    for (int i = lane; i < 4 * p.c.G; i += 32) {
      const int a = i / p.c.G, g = i - a * p.c.G;
      uint16_t *s = a == 0 ? p.c.k_scales : a == 1 ? p.c.k_biases : a == 2 ? p.c.v_scales : p.c.v_biases;
      s[rd * p.c.G + g] = s[rs * p.c.G + g];
    }
  }
  cluster.sync();  // every mover's state has been read, and every list
  for (int i = (lo > left ? lo : left) + tid; i < hi; i += kEvictThreads) {
    new_w[i] = 0.0f;
    new_pos[i] = -1;
  }
}

}  // namespace qmvc

// ---------------------------------------------------------------------------
// C entry points
// ---------------------------------------------------------------------------

namespace {

thread_local std::string g_kv_error;

int kfail(int code, const char *fmt, ...) __attribute__((format(printf, 2, 3)));
int kfail(int code, const char *fmt, ...) {
  char buf[512];
  va_list ap;
  va_start(ap, fmt);
  vsnprintf(buf, sizeof buf, fmt, ap);
  va_end(ap);
  g_kv_error = buf;
  return code;
}

int kok() {
  g_kv_error.clear();
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

// SM count and shared-memory limit of the current device, asked once per device.
struct Device {
  int sms = 0, smem_optin = 0;
};
int current_device(const char *f, Device *out) {
  constexpr int kMaxDevices = 64;
  static Device devs[kMaxDevices];
  static std::once_flag once[kMaxDevices];
  int d = 0;
  const cudaError_t e = cudaGetDevice(&d);
  if (e != cudaSuccess || d < 0 || d >= kMaxDevices)
    return kfail(QMV_ERR_CUDA, "%s: no usable CUDA device (%s)", f, cudaGetErrorString(e));
  std::call_once(once[d], [&] {
    if (cudaDeviceGetAttribute(&devs[d].sms, cudaDevAttrMultiProcessorCount, d) != cudaSuccess ||
        cudaDeviceGetAttribute(&devs[d].smem_optin, cudaDevAttrMaxSharedMemoryPerBlockOptin, d) !=
            cudaSuccess)
      devs[d].sms = 0;
  });
  if (devs[d].sms <= 0) return kfail(QMV_ERR_CUDA, "%s: cannot query device %d", f, d);
  *out = devs[d];
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
  return QMV_OK;
}

// One wave of 8 blocks per SM, or fewer blocks when there is less work.
int row_grid(const qmvc::RowParams &p, int sms) {
  const long long per_token = (2LL * p.c.H * (p.c.D / 8) + 31) / 32;
  const long long need = (p.tokens * per_token + qmvc::kRowThreads / 32 - 1) / (qmvc::kRowThreads / 32);
  return static_cast<int>(need < 8LL * sms ? need : 8LL * sms);
}

template <int BITS, int GS, int D>
cudaError_t append_t(const qmvc::RowParams &p, int grid, cudaStream_t st) {
  if constexpr (BITS != 16 && D % GS != 0) return cudaErrorInvalidValue;  // refused before
  else
    return qmvc::launch_overlapped(qmvc::kv_append_kernel<BITS, GS, D>, dim3(grid), qmvc::kRowThreads,
                                   0, 1, st, p);
}
template <int BITS, int GS>
cudaError_t append_g(const qmvc::RowParams &p, int grid, cudaStream_t st) {
  switch (p.c.D) {
    case 64: return append_t<BITS, GS, 64>(p, grid, st);
    case 96: return append_t<BITS, GS, 96>(p, grid, st);
    case 128: return append_t<BITS, GS, 128>(p, grid, st);
    default: return append_t<BITS, GS, 256>(p, grid, st);
  }
}
template <int BITS>
cudaError_t append_b(const qmvc::RowParams &p, int grid, cudaStream_t st) {
  const int gs = p.c.D / p.c.G;
  return gs == 32 ? append_g<BITS, 32>(p, grid, st) : gs == 64 ? append_g<BITS, 64>(p, grid, st)
                                                              : append_g<BITS, 128>(p, grid, st);
}
template <int BITS>
cudaError_t read_b(const qmvc::RowParams &p, int grid, cudaStream_t st) {
  auto kern = p.c.D == 64    ? qmvc::kv_read_kernel<BITS, 64>
              : p.c.D == 96  ? qmvc::kv_read_kernel<BITS, 96>
              : p.c.D == 128 ? qmvc::kv_read_kernel<BITS, 128>
                             : qmvc::kv_read_kernel<BITS, 256>;
  return qmvc::launch_overlapped(kern, dim3(grid), qmvc::kRowThreads, 0, 1, st, p);
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
  const int grid = row_grid(p, dev.sms);
  auto st = static_cast<cudaStream_t>(stream);
  return launched(f, p.c.bits == 4    ? append_b<4>(p, grid, st)
                     : p.c.bits == 8  ? append_b<8>(p, grid, st)
                                      : append_g<16, 32>(p, grid, st));
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
  const int grid = row_grid(p, dev.sms);
  auto st = static_cast<cudaStream_t>(stream);
  return launched(f, p.c.bits == 4   ? read_b<4>(p, grid, st)
                     : p.c.bits == 8 ? read_b<8>(p, grid, st)
                                     : read_b<16>(p, grid, st));
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
  return launched(f, a.cache.bits == 4   ? qmvc::attn_launch_4(a, dev.sms)
                     : a.cache.bits == 8 ? qmvc::attn_launch_8(a, dev.sms)
                                         : qmvc::attn_launch_16(a, dev.sms));
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
  const int room = table_width * p.c.S;
  if (room > qmvc::kEvictMaxSlots)
    return kfail(QMV_ERR_UNSUPPORTED, "%s: room of %d slots above %d", f, room, qmvc::kEvictMaxSlots);
  const void *words[] = {lens, seen, weights, positions, new_lens, new_weights, new_positions};
  for (const void *w : words)
    if (!aligned(w, 4)) return kfail(QMV_ERR_ALIGN, "%s: state and length arrays must be 4-byte aligned", f);
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
  // a CTA for every 2048 slots of room, up to the portable cluster size
  int cluster = 1;
  while (cluster < qmvc::kEvictMaxCluster && cluster * 2048 < room) cluster *= 2;
  p.seg_max = ((room + cluster - 1) / cluster + 31) & ~31;
  const size_t smem = 8u * static_cast<size_t>(p.seg_max);
  const cudaError_t e = cudaFuncSetAttribute(qmvc::kv_evict_kernel,
                                             cudaFuncAttributeMaxDynamicSharedMemorySize,
                                             static_cast<int>(smem));
  if (e != cudaSuccess) {
    cudaGetLastError();
    return kfail(QMV_ERR_CUDA, "%s: cudaFuncSetAttribute: %s", f, cudaGetErrorString(e));
  }
  return launched(f, qmvc::launch_overlapped(qmvc::kv_evict_kernel, dim3(batch * p.c.H * cluster),
                                             qmvc::kEvictThreads, smem, cluster,
                                             static_cast<cudaStream_t>(stream), p));
}

const char *qmv_kv_last_error(void) { return g_kv_error.c_str(); }

// The calls above with their arguments as 64-bit words, in order (a float as
// its bits): for the Python binding, which pays for every argument it passes.
// The words' number is the binding's to get right; it is checked here.
int qmv_kv_words(int call, int count, const long long *a) {
  auto cache = [&] { return reinterpret_cast<const qmv_kv_cache *>(a[0]); };
  auto ptr = [&](int i) { return reinterpret_cast<void *>(a[i]); };
  auto ints = [&](int i) { return reinterpret_cast<int *>(a[i]); };
  auto floats = [&](int i) { return reinterpret_cast<float *>(a[i]); };
  auto num = [&](int i) { return static_cast<int>(a[i]); };
  if (call == 0 && count == 17)
    return kv_append(cache(), ptr(1), ptr(2), a[3], a[4], ints(5), ints(6), ints(7), num(8), num(9),
                     num(10), ints(11), ints(12), floats(13), num(14), ints(15), ptr(16));
  if (call == 1 && count == 13)
    return kv_read(cache(), ptr(1), ptr(2), a[3], a[4], ints(5), ints(6), ints(7), num(8), num(9),
                   num(10), ints(11), ptr(12));
  if (call == 2 && count == 16) {
    float scale;
    const int bits = num(9);
    static_assert(sizeof scale == sizeof bits, "a float's bits");
    std::memcpy(&scale, &bits, sizeof scale);
    return kv_attention(cache(), ptr(1), a[2], ints(3), ints(4), ptr(5), num(6), num(7), num(8), scale,
                        floats(10), num(11), ptr(12), static_cast<size_t>(a[13]), ints(14), ptr(15));
  }
  if (call == 3 && count == 17)
    return kv_evict(cache(), ints(1), ints(2), ints(3), floats(4), ints(5), ints(6), floats(7), ints(8),
                    num(9), num(10), num(11), num(12), num(13), num(14), ints(15), ptr(16));
  return kfail(QMV_ERR_SHAPE, "qmv_kv_words: call %d with %d words", call, count);
}

}  // extern "C"
