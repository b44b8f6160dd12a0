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

// The same for aligned fp32 rows of whole blocks: 8 lanes take a block, 4 values each, so that
// a load of a wave is 1 KiB in one piece and may go past the caches; two of them a thread.
template <bool NT>
__global__ __launch_bounds__(256) void quantize_rows4(const float* __restrict__ w,
                                                      uint8_t* __restrict__ codes,
                                                      uint8_t* __restrict__ scales, int64_t k,
                                                      int64_t kb, int64_t blocks) {
  // blocks g and g + 32 of every 64
  for (int64_t g0 = (int64_t)blockIdx.x * 64 + (threadIdx.x >> 3); g0 < blocks;
       g0 += (int64_t)gridDim.x * 64) {
    f32x4 v[2];
    int64_t g[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      g[i] = min(g0 + 32 * i, blocks - 1);
      const int64_t row = g[i] / kb, j = (g[i] - row * kb) * QW_MX_BLOCK + (threadIdx.x & 7) * 4;
      v[i] = j < k ? load_as<NT, f32x4>(w + row * k + j) : f32x4{};
    }
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const float t[8] = {v[i][0], v[i][1], v[i][2], v[i][3], 0.0f, 0.0f, 0.0f, 0.0f};
      const uint32_t s = mx_scale(top_among<8>(top_of<4>(t)));
      *(uint16_t*)(codes + g[i] * 16 + (threadIdx.x & 7) * 2) = (uint16_t)mx_codes8(t, s);
      if ((threadIdx.x & 7) == 0) scales[g[i]] = (uint8_t)s;
    }
  }
}

// Down the columns: a thread block takes 256 rows of 64 columns, a thread 8 consecutive rows
// of 8 columns, so that 8 lanes read a run of 64 values and 4 threads have the 32 rows of a
// block.  The codes go through LDS (rows of 33 words: the 64 lanes of a write meet 64 banks),
// so that 128 bytes of an output row are written together.  2048 x 11008 bf16 take 15 us;
// one column a thread, 2 bytes a load, took 96.
constexpr int kColRows = 256, kColCols = 64, kColWords = 33;

template <typename T>
__global__ __launch_bounds__(256) void quantize_columns(const T* __restrict__ w,
                                                        uint8_t* __restrict__ codes,
                                                        uint8_t* __restrict__ scales, int64_t n,
                                                        int64_t k, int64_t np, int64_t tiles_k,
                                                        int64_t tiles) {
  __shared__ uint32_t lds[kColCols][kColWords];
  __shared__ __align__(8) uint8_t sc[kColCols][8];
  const int c8 = (threadIdx.x & 7) * 8, r8 = threadIdx.x >> 3;  // first column, row of eight
  for (int64_t tile = blockIdx.x; tile < tiles; tile += gridDim.x) {
    const int64_t r0 = tile / tiles_k * kColRows, c0 = tile % tiles_k * kColCols;
    const int64_t row = r0 + r8 * 8;
    float v[8][8];
    if (r0 + kColRows <= n && c0 + kColCols <= k) {
#pragma unroll
      for (int i = 0; i < 8; ++i) load8<false>(w + (row + i) * k + c0 + c8, v[i]);
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        load8_of_row<false>(w + min(row + i, n - 1) * k, c0 + c8, k, v[i]);
#pragma unroll
        for (int c = 0; c < 8; ++c) v[i][c] = row + i < n ? v[i][c] : 0.0f;
      }
    }
    __syncthreads();  // the last tile's codes have been read
#pragma unroll
    for (int c = 0; c < 8; ++c) {
      float col[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) col[i] = v[i][c];
      uint32_t top = top_of<8>(col);
      top = max(top, (uint32_t)__shfl_xor((int)top, 8));
      top = max(top, (uint32_t)__shfl_xor((int)top, 16));
      const uint32_t s = mx_scale(top);
      lds[c8 + c][r8] = mx_codes8(col, s);
      if ((r8 & 3) == 0) sc[c8 + c][r8 >> 2] = (uint8_t)s;
    }
    __syncthreads();
    const int word = threadIdx.x & 31;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int c = i * 8 + (threadIdx.x >> 5);
      if (c0 + c < k) *(uint32_t*)(codes + (c0 + c) * (np / 2) + r0 / 2 + word * 4) = lds[c][word];
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
    if constexpr (sizeof(T) == 4) {
      if (k % 4 || !aligned(w, 16))
        quantize_rows<false><<<grid, 256, 0, stream>>>(w, codes, scales, k, kb, blocks);
      else if (n * k >= 16ll << 20)
        quantize_rows4<true><<<grid, 256, 0, stream>>>(w, codes, scales, k, kb, blocks);
      else
        quantize_rows4<false><<<grid, 256, 0, stream>>>(w, codes, scales, k, kb, blocks);
    } else if (k % 8 == 0 && aligned(w, 16)) {
      quantize_rows<true><<<grid, 256, 0, stream>>>(w, codes, scales, k, kb, blocks);
    } else {
      quantize_rows<false><<<grid, 256, 0, stream>>>(w, codes, scales, k, kb, blocks);
    }
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
