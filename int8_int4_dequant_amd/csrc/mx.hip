// Microscaled 4-bit codes: quantize and unpack kernels for gfx950.
//
//   scale = 2^(floor(log2 max|w|) - 2) per 32 values, code = e2m1(w / scale)
//
// Bound by HBM: a value is read once (4 or 2 bytes), 17/32 of a byte written, or
// the reverse.
#include "mx_codes.h"

namespace qw {
namespace {

// Along the rows: 4 lanes take a block, 8 values each.  Numbered along the rows, padding
// included, 64 blocks to a thread block.
template <bool VEC, typename T>
__global__ __launch_bounds__(256) void quantize_rows(const T* __restrict__ w,
                                                     uint8_t* __restrict__ codes,
                                                     uint8_t* __restrict__ scales, int64_t k,
                                                     int64_t kb, int64_t blocks) {
  for (int64_t g = (int64_t)blockIdx.x * 64 + (threadIdx.x >> 2); g < blocks;
       g += (int64_t)gridDim.x * 64) {
    const int64_t row = g / kb;
    const int64_t j = (g - row * kb) * QW_MX_BLOCK + (threadIdx.x & 3) * 8;
    float v[8];
    load8_of_row<VEC>(w + row * k, j, k, v);
    const uint32_t s = mx_scale(top_among<4>(top_of<8>(v)));
    *(uint32_t*)(codes + g * 16 + (threadIdx.x & 3) * 4) = mx_codes8(v, s);
    if ((threadIdx.x & 3) == 0) scales[g] = (uint8_t)s;
  }
}

// Down the columns: a thread block takes 256 rows of 64 columns, a thread two blocks of
// one column, which need no other thread.  The codes go through LDS, so that 128 bytes of
// an output row are written together.
constexpr int kColRows = 256, kColCols = 64, kColPitch = 144;  // LDS rows 16 bytes apart from a multiple of the banks

template <typename T>
__global__ __launch_bounds__(256) void quantize_columns(const T* __restrict__ w,
                                                        uint8_t* __restrict__ codes,
                                                        uint8_t* __restrict__ scales, int64_t n,
                                                        int64_t k, int64_t np, int64_t tiles_k,
                                                        int64_t tiles) {
  __shared__ __align__(16) uint8_t lds[kColCols][kColPitch];
  __shared__ __align__(8) uint8_t sc[kColCols][8];
  const int c = threadIdx.x & 63, part = threadIdx.x >> 6;
  for (int64_t tile = blockIdx.x; tile < tiles; tile += gridDim.x) {
    const int64_t r0 = tile / tiles_k * kColRows, c0 = tile % tiles_k * kColCols;
    const bool have = c0 + c < k;
    __syncthreads();  // the last tile's codes have been read
#pragma unroll
    for (int b = 0; b < 2; ++b) {
      const int64_t row = r0 + part * 64 + b * 32;
      const T* p = w + row * k + c0 + c;
      float v[32];
#pragma unroll
      for (int i = 0; i < 32; ++i) v[i] = have && row + i < n ? load1(p + i * k) : 0.0f;
      const uint32_t s = mx_scale(top_of<32>(v));
      u32x4 q;
#pragma unroll
      for (int i = 0; i < 4; ++i) q[i] = mx_codes8(v + 8 * i, s);
      *(u32x4_la*)&lds[c][part * 32 + b * 16] = q;
      sc[c][part * 2 + b] = (uint8_t)s;
    }
    __syncthreads();
    // 8 lanes write the 128 bytes of a row
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int row = i * 32 + (threadIdx.x >> 3), at = (threadIdx.x & 7) * 16;
      if (c0 + row < k)
        *(u32x4*)(codes + (c0 + row) * (np / 2) + r0 / 2 + at) = *(const u32x4_la*)&lds[row][at];
    }
    if (threadIdx.x < kColCols && c0 + threadIdx.x < k)
      *(u32x2*)(scales + (c0 + threadIdx.x) * (np / 32) + r0 / 32) =
          *(const u32x2_la*)sc[threadIdx.x];
  }
}

// Values of codes, 8 a lane.
template <bool VEC>
__global__ __launch_bounds__(256) void unpack(const uint8_t* __restrict__ codes,
                                              const uint8_t* __restrict__ scales,
                                              float* __restrict__ out, int64_t k, int64_t kp,
                                              int64_t eights) {
  const int64_t per = (k + 7) / 8;
  for (int64_t g = (int64_t)blockIdx.x * 256 + threadIdx.x; g < eights;
       g += (int64_t)gridDim.x * 256) {
    const int64_t row = g / per, j = (g - row * per) * 8;
    const uint32_t c = *(const uint32_t*)(codes + row * (kp / 2) + j / 2);
    const uint32_t s = scales[row * (kp / 32) + j / 32];
    // the smallest scale, 2^-127, has no exponent bits of its own
    const float by = s == 255 ? __builtin_nanf("") : s == 0 ? 0x1p-127f : __uint_as_float(s << 23);
    float v[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const uint32_t q = c >> (4 * i) & 15, e = q >> 1 & 3, m = q & 1;
      // 0, 0.5 or (1 + m / 2) 2^(e - 1)
      const float a = e == 0 ? 0.5f * (float)m
                             : __uint_as_float((126 + e) << 23 | m << 22);
      v[i] = __uint_as_float(__float_as_uint(a) | (q >> 3) << 31) * by;
    }
    store8_of_row<VEC>(out + row * k, j, k, v);
  }
}

template <typename T>
hipError_t quantize(int transpose, int64_t n, int64_t k, const T* w, uint8_t* codes,
                    uint8_t* scales, hipStream_t stream) {
  if (transpose) {
    const int64_t np = mx_pitch(n), tiles_k = (k + kColCols - 1) / kColCols;
    const int64_t tiles = np / kColRows * tiles_k;
    quantize_columns<<<grid_for(tiles, 1), 256, 0, stream>>>(w, codes, scales, n, k, np, tiles_k,
                                                             tiles);
  } else {
    const int64_t kb = mx_pitch(k) / QW_MX_BLOCK, blocks = n * kb;
    const unsigned grid = grid_for(blocks, 64);
    if (k % 8 == 0 && aligned(w, 16))
      quantize_rows<true><<<grid, 256, 0, stream>>>(w, codes, scales, k, kb, blocks);
    else
      quantize_rows<false><<<grid, 256, 0, stream>>>(w, codes, scales, k, kb, blocks);
  }
  return hipGetLastError();
}

}  // namespace

hipError_t launch_mx_quantize(int transpose, int64_t n, int64_t k, int type, const void* w,
                              uint8_t* codes, uint8_t* scales, hipStream_t stream) {
  return type == QW_F32 ? quantize(transpose, n, k, (const float*)w, codes, scales, stream)
                        : quantize(transpose, n, k, (const uint16_t*)w, codes, scales, stream);
}

hipError_t launch_mx_unpack(int64_t n, int64_t k, const uint8_t* codes, const uint8_t* scales,
                            float* out, hipStream_t stream) {
  const int64_t kp = mx_pitch(k), eights = n * ((k + 7) / 8);
  const unsigned grid = grid_for(eights, 256);
  if (k % 8 == 0 && aligned(out, 16))
    unpack<true><<<grid, 256, 0, stream>>>(codes, scales, out, k, kp, eights);
  else
    unpack<false><<<grid, 256, 0, stream>>>(codes, scales, out, k, kp, eights);
  return hipGetLastError();
}

}  // namespace qw
