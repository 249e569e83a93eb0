// qmv_kv_attn.cu -- attention of one new token per sequence over the paged
// cache: the kernels behind kv_attention.
//
// The plainest form that is right: a CTA per (sequence, query head) writes
// the scaled scores of all slots to the workspace, finds their maximum and
// sum, and adds up the values with one thread per element; a second kernel
// adds the probabilities of a kv head's query heads into the weights.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "qmv_kv.h"

namespace qmvc {

constexpr int kThreads = 256;

struct AttnParams {
  CacheView c;
  const __nv_bfloat16 *q;
  long long q_stride;
  const int *lens;
  __nv_bfloat16 *out;
  int batch, Hq, R;
  float scale;
  float *weights;
  int state_width;
  float *scores;   // [batch][Hq][room]
  float2 *stats;   // [batch][Hq]: maximum, sum
};

__device__ __forceinline__ float element(const CacheView &c, const uint8_t *codes,
                                         const uint16_t *s, const uint16_t *b, long long row, int d) {
  const uint8_t *r = codes + row * c.row_bytes;
  if (c.bits == 16) return __bfloat162float(reinterpret_cast<const __nv_bfloat16 *>(r)[d]);
  const uint32_t q = c.bits == 8 ? r[d] : (r[d / 2] >> (4 * (d & 1))) & 15u;
  const long long g = row * c.G + d / (c.D / c.G);
  return __uint_as_float(static_cast<uint32_t>(s[g]) << 16) * static_cast<float>(q) +
         __uint_as_float(static_cast<uint32_t>(b[g]) << 16);
}

template <bool MAX>
__device__ float block_reduce(float v) {
  __shared__ float part[kThreads / 32];
  for (int o = 16; o; o >>= 1) {
    const float x = __shfl_xor_sync(0xffffffffu, v, o);
    v = MAX ? fmaxf(v, x) : v + x;
  }
  __syncthreads();
  if ((threadIdx.x & 31) == 0) part[threadIdx.x / 32] = v;
  __syncthreads();
  v = part[0];
  for (int i = 1; i < kThreads / 32; ++i) v = MAX ? fmaxf(v, part[i]) : v + part[i];
  return v;
}

__device__ __forceinline__ int length_of(const AttnParams &p, int b) {
  const int len = p.lens[b], room = p.c.width * p.c.S;
  if (len > room && p.c.status) atomicOr(p.c.status, 1);
  return len < 0 ? 0 : len < room ? len : room;
}

__global__ void __launch_bounds__(kThreads) attn_kernel(const AttnParams p) {
  __shared__ float q[256];
  const int b = blockIdx.x, h = blockIdx.y, g = h / p.R, tid = threadIdx.x;
  wait_for_previous_grid();
  const int n = length_of(p, b);
  const int *table = p.c.table + static_cast<long long>(b) * p.c.width;
  for (int d = tid; d < p.c.D; d += kThreads)
    q[d] = __bfloat162float(p.q[b * p.q_stride + h * p.c.D + d]);
  __syncthreads();
  float *s = p.scores + (static_cast<long long>(b) * p.Hq + h) * p.c.width * p.c.S;
  float m = -INFINITY;
  for (int j = tid; j < n; j += kThreads) {
    const int page = checked_page(p.c, table[j / p.c.S]);
    float x = -INFINITY;
    if (page >= 0) {
      const long long row = cache_row(p.c, page, g, j % p.c.S);
      x = 0.0f;
      for (int d = 0; d < p.c.D; ++d)
        x += q[d] * element(p.c, p.c.k, p.c.k_scales, p.c.k_biases, row, d);
      x *= p.scale;
    }
    s[j] = x;
    m = fmaxf(m, x);
  }
  m = block_reduce<true>(m);
  float l = 0.0f;
  for (int j = tid; j < n; j += kThreads) l += s[j] == -INFINITY ? 0.0f : expf(s[j] - m);
  l = block_reduce<false>(l);
  if (tid == 0) p.stats[static_cast<long long>(b) * p.Hq + h] = make_float2(m, l);
  for (int d = tid; d < p.c.D; d += kThreads) {
    float o = 0.0f;
    for (int j = 0; j < n; ++j) {
      const float x = s[j];
      if (x == -INFINITY) continue;
      const long long row = cache_row(p.c, table[j / p.c.S], g, j % p.c.S);
      o += expf(x - m) * element(p.c, p.c.v, p.c.v_scales, p.c.v_biases, row, d);
    }
    p.out[(static_cast<long long>(b) * p.Hq + h) * p.c.D + d] =
        __float2bfloat16_rn(l > 0.0f ? o / l : 0.0f);
  }
}

__global__ void __launch_bounds__(kThreads) attn_weights_kernel(const AttnParams p) {
  const int b = blockIdx.x, g = blockIdx.y;
  wait_for_previous_grid();
  const int n = length_of(p, b);
  float *w = p.weights + (static_cast<long long>(b) * p.c.H + g) * p.state_width;
  for (int j = blockIdx.z * kThreads + threadIdx.x; j < n; j += kThreads * gridDim.z) {
    float sum = 0.0f;
    for (int r = 0; r < p.R; ++r) {
      const long long h = static_cast<long long>(b) * p.Hq + g * p.R + r;
      const float x = p.scores[h * p.c.width * p.c.S + j];
      if (x != -INFINITY) sum += expf(x - p.stats[h].x) / p.stats[h].y;
    }
    w[j] += sum;
  }
}

size_t attn_workspace(const CacheView &c, int batch, int num_q_heads, bool, int) {
  const size_t heads = static_cast<size_t>(batch) * num_q_heads;
  return heads * (static_cast<size_t>(c.width) * c.S * 4 + 8) + 16;
}

cudaError_t attn_launch(const AttnArgs &a, int) {
  AttnParams p = {};
  p.c = a.cache;
  p.q = static_cast<const __nv_bfloat16 *>(a.q);
  p.q_stride = a.q_stride;
  p.lens = a.lens;
  p.out = static_cast<__nv_bfloat16 *>(a.out);
  p.batch = a.batch;
  p.Hq = a.num_q_heads;
  p.R = a.num_q_heads / a.cache.H;
  p.scale = a.scale;
  p.weights = a.weights;
  p.state_width = a.state_width;
  const size_t heads = static_cast<size_t>(a.batch) * a.num_q_heads;
  p.stats = static_cast<float2 *>(a.workspace);
  p.scores = reinterpret_cast<float *>(p.stats + (heads + 1) / 2 * 2);
  cudaError_t e = launch_overlapped(attn_kernel, dim3(a.batch, a.num_q_heads), kThreads, 0, 1,
                                    a.stream, p);
  if (e == cudaSuccess && a.weights)
    e = launch_overlapped(attn_weights_kernel, dim3(a.batch, a.cache.H, 8), kThreads, 0, 1, a.stream,
                          p);
  return e;
}

}  // namespace qmvc
