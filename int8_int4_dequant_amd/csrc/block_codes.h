// e4m3 codes with a scale per block of 128 values: device code shared by the
// kernels that make or read them (block.hip, block_gemm.hip, moe.hip).
#pragma once

#include <type_traits>

#include "qw_internal.h"

namespace qw {

typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
// For memory that is written with words of one size and read with another.
typedef uint32_t u32x2_la __attribute__((ext_vector_type(2), may_alias));
typedef uint32_t u32x4_la __attribute__((ext_vector_type(4), may_alias));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef float f32x2 __attribute__((ext_vector_type(2)));

constexpr float kTop = 448.0f;  // largest e4m3 value

// A block's scale from its max|w|: IEEE fp32 division, 1 for a zero result.
__device__ __forceinline__ float block_scale(float amax) {
  const float s = amax / kTop;
  return s == 0.0f ? 1.0f : s;
}

// NaN stays NaN (fminf and fmaxf alone would make it a number).
__device__ __forceinline__ float clip_top(float v) {
  return v != v ? v : fminf(fmaxf(v, -kTop), kTop);
}

// Codes of 4 values already divided by their scale, first value in the low
// byte.  The conversion rounds to nearest even; values are within +-448 or NaN,
// so it never saturates.
__device__ __forceinline__ uint32_t codes4(float a, float b, float c, float d) {
  int r = __builtin_amdgcn_cvt_pk_fp8_f32(clip_top(a), clip_top(b), 0, false);
  r = __builtin_amdgcn_cvt_pk_fp8_f32(clip_top(c), clip_top(d), r, true);
  return (uint32_t)r;
}

__device__ __forceinline__ float bf16_lo(uint32_t v) { return __uint_as_float(v << 16); }
__device__ __forceinline__ float bf16_hi(uint32_t v) { return __uint_as_float(v & 0xFFFF0000u); }

__device__ __forceinline__ uint16_t to_bf16(float v) {
  return __builtin_bit_cast(uint16_t, (__bf16)v);  // round to nearest even
}
__device__ __forceinline__ uint32_t to_bf16x2(float a, float b) {
  return (uint32_t)to_bf16(a) | (uint32_t)to_bf16(b) << 16;
}

// One element of either type.
__device__ __forceinline__ float load1(const float* p) { return *p; }
__device__ __forceinline__ float load1(const uint16_t* p) {
  return __uint_as_float((uint32_t)*p << 16);
}
__device__ __forceinline__ void store1(float* p, float v) { *p = v; }
__device__ __forceinline__ void store1(uint16_t* p, float v) { *p = to_bf16(v); }

// 4 consecutive elements, aligned to their size.
__device__ __forceinline__ void store4(float* p, f32x4 v) { *(f32x4*)p = v; }
__device__ __forceinline__ void store4(uint16_t* p, f32x4 v) {
  *(u32x2*)p = u32x2{to_bf16x2(v[0], v[1]), to_bf16x2(v[2], v[3])};
}

// 16 bytes at the alignment of an element: rows of any length take the vector
// accesses too, which the hardware splits where it has to.
typedef float f32x4_u __attribute__((ext_vector_type(4), aligned(4)));
typedef uint32_t u32x4_u __attribute__((ext_vector_type(4), aligned(2)));

template <bool NT, typename V>
__device__ __forceinline__ V load_as(const void* p) {
  return NT ? __builtin_nontemporal_load((const V*)p) : *(const V*)p;
}
template <bool NT, typename V>
__device__ __forceinline__ void store_as(void* p, V v) {
  if (NT)
    __builtin_nontemporal_store(v, (V*)p);
  else
    *(V*)p = v;
}

// 8 consecutive elements, at a 16-byte aligned address (VEC) or any; NT: past the
// caches.
template <bool VEC, bool NT = false>
__device__ __forceinline__ void load8(const float* p, float v[8]) {
  typedef std::conditional_t<VEC, f32x4, f32x4_u> V;
  const f32x4 a = load_as<NT, V>(p), b = load_as<NT, V>(p + 4);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    v[i] = a[i];
    v[4 + i] = b[i];
  }
}
template <bool VEC, bool NT = false>
__device__ __forceinline__ void load8(const uint16_t* p, float v[8]) {
  const u32x4 a = load_as<NT, std::conditional_t<VEC, u32x4, u32x4_u>>(p);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    v[2 * i] = bf16_lo(a[i]);
    v[2 * i + 1] = bf16_hi(a[i]);
  }
}

// Elements [j, j + 8) of a row of k, zero from k on; VEC: the row is 16-byte
// aligned and k % 8 == 0, so the 8 are all there or none is.
template <bool VEC, bool NT = false, typename T>
__device__ __forceinline__ void load8_of_row(const T* row, int64_t j, int64_t k, float v[8]) {
  if (VEC ? j < k : j + 8 <= k) {
    load8<VEC, NT>(row + j, v);
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = !VEC && j + i < k ? load1(row + j + i) : 0.0f;
  }
}

// The same for a store.
template <bool VEC, bool NT = false>
__device__ __forceinline__ void store8(float* p, const float v[8]) {
  typedef std::conditional_t<VEC, f32x4, f32x4_u> V;
  store_as<NT, V>(p, V{v[0], v[1], v[2], v[3]});
  store_as<NT, V>(p + 4, V{v[4], v[5], v[6], v[7]});
}
template <bool VEC, bool NT = false>
__device__ __forceinline__ void store8(uint16_t* p, const float v[8]) {
  typedef std::conditional_t<VEC, u32x4, u32x4_u> V;
  store_as<NT, V>(p, V{to_bf16x2(v[0], v[1]), to_bf16x2(v[2], v[3]), to_bf16x2(v[4], v[5]),
                       to_bf16x2(v[6], v[7])});
}
template <bool VEC, bool NT = false, typename T>
__device__ __forceinline__ void store8_of_row(T* row, int64_t j, int64_t k, const float v[8]) {
  if (VEC ? j < k : j + 8 <= k) {
    store8<VEC, NT>(row + j, v);
  } else if (!VEC) {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (j + i < k) store1(row + j + i, v[i]);
  }
}

__device__ __forceinline__ float amax8(const float v[8]) {
  float m = 0.0f;
#pragma unroll
  for (int i = 0; i < 8; ++i) m = fmaxf(m, fabsf(v[i]));
  return m;
}

// Max over the aligned run of 16 lanes that this lane is in.
__device__ __forceinline__ float max16(float m) {
#pragma unroll
  for (int h = 1; h < 16; h <<= 1) m = fmaxf(m, __shfl_xor(m, h));
  return m;
}

// Division by a block's scale, rounded as IEEE division is.  With r the
// correctly rounded 1 / s, x r is within 1.5 ulp of x / s, one correction with
// its exact remainder brings it within 1 ulp, and a second one to the correctly
// rounded quotient (P. Markstein, "Computation of elementary functions on the
// IBM RISC System/6000 processor", 1990): 5 instructions where the general
// division takes 10, two of them at a quarter of the rate.  The remainder is
// exact as long as nothing underflows: `plain` scales only (a value too small
// for it then has the code 0 either way).  Its sign is such that -0 stays -0.
struct Divisor {
  float s, r;
  __device__ __forceinline__ explicit Divisor(float scale) : s(scale), r(1.0f / scale) {}
  __device__ __forceinline__ bool plain() const { return s >= 0x1p-60f && s <= 0x1p100f; }
  __device__ __forceinline__ float operator()(float x) const {
    float v = x * r;
    v = __builtin_fmaf(-__builtin_fmaf(v, s, -x), r, v);
    return __builtin_fmaf(-__builtin_fmaf(v, s, -x), r, v);
  }
};

// The codes of 8 values with scale s.  The quotients of a plain scale are at
// most 448 (1 + 2^-23), which converts to 448: only the others are clipped.
__device__ __forceinline__ u32x2 codes8(const float v[8], float s) {
  const Divisor by(s);
  if (by.plain()) {
    u32x2 c;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      int r = __builtin_amdgcn_cvt_pk_fp8_f32(by(v[4 * i]), by(v[4 * i + 1]), 0, false);
      r = __builtin_amdgcn_cvt_pk_fp8_f32(by(v[4 * i + 2]), by(v[4 * i + 3]), r, true);
      c[i] = (uint32_t)r;
    }
    return c;
  }
  return u32x2{codes4(v[0] / s, v[1] / s, v[2] / s, v[3] / s),
               codes4(v[4] / s, v[5] / s, v[6] / s, v[7] / s)};
}

// silu(gate) * up = gate / (1 + 2^h) * up, h = -gate log2(e), within 4 ulp for
// every gate (fp32's own subnormal steps aside).  h is kept in two parts, since
// in 24 bits alone it would cost |h| half ulps: 2^h with the part l that h has no
// bits for added in a second step.  The quotient is a product with the hardware
// reciprocal (1 ulp): the result is then rounded to 4 bits.
//
// FAR: any gate.  From h = 64 on, gate, 1 and 2^h are all taken 2^-64 times, so
// that neither the sum nor its reciprocal leaves the hardware's range (v_rcp_f32 has
// no subnormal results) before silu itself is zero, at h = 157.  From h = 190 on,
// where the sum may be infinite, and below -190, where 2^h is 0 and h may be
// infinite, there is no l to add.  Otherwise |h| < 64, with the same bits there.
template <bool FAR>
__device__ __forceinline__ float gated(float gate, float up) {
#pragma clang fp contract(off)  // h - 64 is that of the rounded h, whose rest is l
  const float h = gate * -0x1.715476p+0f;  // log2(e) to 24 bits, and the rest of it
  const float l = __builtin_fmaf(gate, -0x1.4ae0cp-26f, __builtin_fmaf(gate, -0x1.715476p+0f, -h));
  const bool far = FAR && h > 64.0f;
  const float one = far ? 0x1p-64f : 1.0f;
  const float e = __builtin_amdgcn_exp2f(far ? h - 64.0f : h);
  const bool whole = !FAR || fabsf(h) < 190.0f;
  const float sum = one + (whole ? __builtin_fmaf(e, l * 0x1.62e43p-1f, e) : e);
  return gate * one * __builtin_amdgcn_rcpf(sum) * up;
}
// N of them, with one test for all whether a gate is far (24594 rows of 1408 bf16
// values: 33 us; 36 with every gate's own test).
template <int N>
__device__ __forceinline__ void gated(const float* gate, const float* up, float* v) {
  float top = 0.0f;
#pragma unroll
  for (int i = 0; i < N; ++i) top = fmaxf(top, fabsf(gate[i]));
  if (top < 44.0f) {
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] = gated<false>(gate[i], up[i]);
  } else {
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] = gated<true>(gate[i], up[i]);
  }
}

// Thread blocks for `items` of work, `per` to a block: the kernels' loops take
// what is beyond 2^22 blocks (a launch holds fewer than 2^32 threads).
inline unsigned grid_for(int64_t items, int per) {
  const int64_t blocks = (items + per - 1) / per;
  return (unsigned)(blocks < (1 << 22) ? blocks : 1 << 22);
}

}  // namespace qw
