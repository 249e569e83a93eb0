// qmv_affine.cuh -- the affine quantizer's binary32 steps, for affine_quantize
// (qmv_quant.cu) and kv_append (qmv_kv.cu): the range's start, a group's scale and
// bias, and its codes, an element or eight at a time.  The two write the same bits
// for every input, NaN and infinities among them.  Internal to the library.
#pragma once

#include <cuda_runtime.h>

#include <cstdint>

namespace qmva {

// Where a group's smallest value starts: the largest finite bf16 (a group of NaNs
// keeps it).
constexpr float kRangeStart = 0x1.fep127f;

// The affine map of one group from its range [lo, hi] (lo taken from kRangeStart
// down, hi from 0 up, as the page's affine_quantize starts them), in binary32 with
// IEEE divisions:
//   * the code step has magnitude max((hi - lo) / n_bins, 1e-7);
//   * the anchor is the endpoint of larger magnitude (hi on a tie); the step
//     takes the anchor's sign when the anchor is lo, the opposite sign when
//     it is hi, so codes grow away from the anchor into the range;
//   * the anchor's position on the code grid, j = round(anchor / step)
//     (halves away from zero), refines the step to anchor / j, and the
//     anchor becomes the offset -- unless j = 0, when the step stays and the
//     offset is 0.
// Returns the step (the stored scale) and the offset (the stored bias).
__device__ __forceinline__ float2 group_step_offset(float lo, float hi, float n_bins) {
  const float magnitude = fmaxf(__fdiv_rn(__fsub_rn(hi, lo), n_bins), 1e-7f);
  const bool anchor_is_lo = fabsf(lo) > fabsf(hi);
  const float anchor = anchor_is_lo ? lo : hi;
  const float step = anchor_is_lo ? magnitude : -magnitude;
  const float j = roundf(__fdiv_rn(anchor, step));
  if (j == 0.0f) return make_float2(step, 0.0f);
  return make_float2(__fdiv_rn(anchor, j), anchor);
}

// The code of one element: min(round(d / scale), n_bins) with the page's
// binary32 quotient d / scale and round-half-away.  The quotient is formed
// as d * (1 / scale) (both correctly rounded), within 3 * 2^-24 of the
// binary32 quotient relative to it; where no half-integer lies within
// 2^-20 * max(|t|, 1) of that product, both round to the same integer and
// rint gives it.  Only the rare elements near a half-integer take the IEEE
// division and roundf, so every code is the one the page's steps decide.
__device__ __forceinline__ uint32_t quantize_code(float v, float bias, float scale, float rcp,
                                                  float n_bins) {
  const float d = __fsub_rn(v, bias);
  const float tp = __fmul_rn(d, rcp);
  const float rt = rintf(tp);
  float code = rt;
  if (fabsf(__fsub_rn(tp, rt)) > 0.5f - fmaxf(fabsf(tp), 1.0f) * 0x1p-20f)
    code = roundf(__fdiv_rn(d, scale));
  return static_cast<uint32_t>(fminf(code, n_bins));
}

// The codes of 8 elements at once, the same as quantize_code's, as whole numbers.
// The product with the rounded reciprocal is within 3 * 2^-24 of the quotient,
// relative to it, so its nearest integer is the code unless it lies within that of
// a half; elements within 2^-22 * (n_bins + 1) of one take the IEEE division.
// Adding and subtracting 1.5 * 2^23 rounds to the nearest integer (|t| < 2^22).
template <int BITS>
__device__ __forceinline__ void codes_of(float (&v)[8], float bias, float scale, float rcp) {
  constexpr float n_bins = static_cast<float>((1 << BITS) - 1);
  constexpr float kSure = 0.5f - (n_bins + 1.0f) * 0x1p-22f, kRound = 12582912.0f;
  float r[8];
  float most = 0.0f;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float t = __fmul_rn(__fsub_rn(v[i], bias), rcp);
    r[i] = __fsub_rn(__fadd_rn(t, kRound), kRound);
    most = fmaxf(most, fabsf(__fsub_rn(t, r[i])));
  }
  if (most > kSure) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float d = __fsub_rn(v[i], bias);
      const float t = __fmul_rn(d, rcp);
      if (fabsf(__fsub_rn(t, r[i])) > kSure) r[i] = roundf(__fdiv_rn(d, scale));
    }
  }
#pragma unroll
  for (int i = 0; i < 8; ++i) v[i] = fminf(r[i], n_bins);
}

}  // namespace qmva
