// e2m1 codes with a power-of-two scale per block of 32 values: device code shared by
// the kernels that make them (mx.hip, mx_gemm.hip, norm.hip).
#pragma once

#include "block_codes.h"

namespace qw {

// Magnitudes as their bits order like the values, with infinities and then NaN on
// top, so that one integer maximum finds the block's largest value and whether it has
// a scale at all.
__device__ __forceinline__ uint32_t magnitude(float v) { return __float_as_uint(v) & 0x7FFFFFFFu; }

template <int N>
__device__ __forceinline__ uint32_t top_of(const float* v) {
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < N; ++i) m = max(m, magnitude(v[i]));
  return m;
}

// Max over the aligned run of LANES lanes that this lane is in.
template <int LANES>
__device__ __forceinline__ uint32_t top_among(uint32_t m) {
#pragma unroll
  for (int h = 1; h < LANES; h <<= 1) m = max(m, (uint32_t)__shfl_xor((int)m, h));
  return m;
}

// The scale byte of a block from its largest magnitude's bits: its exponent less 2,
// 0 at least; 127 for a zero block, 255 for infinities and NaN.
__device__ __forceinline__ uint32_t mx_scale(uint32_t top) {
  const uint32_t e = top >> 23;
  return top == 0 ? 127u : e == 255 ? 255u : e > 2 ? e - 2 : 0u;
}

// Codes of 8 values, first value in the low bits.  v_cvt_scalef32_pk_fp4_f32 divides
// by the power of two in the exponent bits of its scale (0 stands for 2^-127), rounds
// to nearest even and clips at 6: the definition, for every scale but 255.
__device__ __forceinline__ uint32_t mx_codes8(const float v[8], uint32_t scale) {
  const float s = __uint_as_float(scale << 23);
  uint32_t c = 0;
  c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, v[0], v[1], s, 0);
  c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, v[2], v[3], s, 1);
  c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, v[4], v[5], s, 2);
  c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, v[6], v[7], s, 3);
  return scale == 255 ? 0u : c;
}

}  // namespace qw
