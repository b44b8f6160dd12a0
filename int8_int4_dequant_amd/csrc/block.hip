// Block-scaled e4m3: quantize, gated quantize and unpack kernels for gfx950.
//
//   S = max|w| / 448 per block (1 if zero), code = e4m3(clip(fl32(w / S)))
//
// All three are bound by HBM: a value is read once (4 or 2 bytes) and its
// code written (1 byte), or the reverse.  16 lanes take a row of a block, 8
// values each, so a wave's loads are runs of 256 (bf16) or 512 bytes and the
// values stay in registers between the maximum and the codes.
#include "block_codes.h"

namespace qw {
namespace {

// 1 x 128 blocks: 16 blocks to a thread block, numbered along the rows.  (4 times
// as many with their loads on the way together: 17 us for 2048 x 8192 bf16
// instead of 14.)
template <bool VEC, typename T>
__global__ __launch_bounds__(256) void quantize_rows(const T* __restrict__ w,
                                                     uint8_t* __restrict__ codes,
                                                     float* __restrict__ scales, int64_t k,
                                                     int64_t kb, int64_t blocks) {
  // whole runs of 16 lanes take part or not
  for (int64_t g = (int64_t)blockIdx.x * 16 + (threadIdx.x >> 4); g < blocks;
       g += (int64_t)gridDim.x * 16) {
    const int64_t row = g / kb;
    const int64_t j = (g - row * kb) * QW_BLOCK + (threadIdx.x & 15) * 8;
    float v[8];
    load8_of_row<VEC>(w + row * k, j, k, v);
    const float s = block_scale(max16(amax8(v)));
    *(u32x2*)(codes + row * (kb * QW_BLOCK) + j) = codes8(v, s);
    if ((threadIdx.x & 15) == 0) scales[g] = s;
  }
}

// 128 x 128 blocks: one thread block each, 8 rows of 8 values a thread.
template <bool VEC, typename T>
__global__ __launch_bounds__(256) void quantize_tiles(const T* __restrict__ w,
                                                      uint8_t* __restrict__ codes,
                                                      float* __restrict__ scales, int64_t n,
                                                      int64_t k, int64_t kb, int64_t nb,
                                                      int64_t tiles) {
  __shared__ float wave_max[4];
  for (int64_t tile = blockIdx.x; tile < tiles; tile += gridDim.x) {
    const int64_t band = tile / kb;  // matrix * nb + row of blocks
    const int64_t mat = band / nb;
    const int64_t r0 = (band - mat * nb) * QW_BLOCK;
    const int64_t j = (tile - band * kb) * QW_BLOCK + (threadIdx.x & 15) * 8;
    const int64_t base = mat * n + r0;
    const int left = (int)(n - r0 < QW_BLOCK ? n - r0 : QW_BLOCK);
    const int r = threadIdx.x >> 4;
    float v[8][8];
    float m = 0.0f;
#pragma unroll
    for (int p = 0; p < 8; ++p) {
      if (r + 16 * p < left) {
        load8_of_row<VEC>(w + (base + r + 16 * p) * k, j, k, v[p]);
      } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) v[p][i] = 0.0f;
      }
      m = fmaxf(m, amax8(v[p]));
    }
#pragma unroll
    for (int h = 1; h < 64; h <<= 1) m = fmaxf(m, __shfl_xor(m, h));
    __syncthreads();  // the last tile's maxima have been read
    if ((threadIdx.x & 63) == 0) wave_max[threadIdx.x >> 6] = m;
    __syncthreads();
    m = fmaxf(fmaxf(wave_max[0], wave_max[1]), fmaxf(wave_max[2], wave_max[3]));
    const float s = block_scale(m);
#pragma unroll
    for (int p = 0; p < 8; ++p)
      if (r + 16 * p < left)
        *(u32x2*)(codes + (base + r + 16 * p) * (kb * QW_BLOCK) + j) = codes8(v[p], s);
    if (threadIdx.x == 0) scales[tile] = s;
  }
}

// 1 x 128 blocks of silu(gate) * up, gate and up the halves of a row of h.
template <bool VEC, typename T>
__global__ __launch_bounds__(256) void quantize_swiglu(const T* __restrict__ h,
                                                       const int32_t* __restrict__ used,
                                                       uint8_t* __restrict__ codes,
                                                       float* __restrict__ scales, int64_t f,
                                                       int64_t kb, int64_t blocks) {
  const int64_t most = used ? (int64_t)*used * kb : blocks;
  if (most < blocks) blocks = most;
  for (int64_t g = (int64_t)blockIdx.x * 16 + (threadIdx.x >> 4); g < blocks;
       g += (int64_t)gridDim.x * 16) {
    const int64_t row = g / kb;
    const int64_t j = (g - row * kb) * QW_BLOCK + (threadIdx.x & 15) * 8;
    float a[8], b[8];
    load8_of_row<VEC>(h + row * 2 * f, j, f, a);
    load8_of_row<VEC>(h + row * 2 * f + f, j, f, b);
    gated<8>(a, b, a);
    const float s = block_scale(max16(amax8(a)));
    *(u32x2*)(codes + row * (kb * QW_BLOCK) + j) = codes8(a, s);
    if ((threadIdx.x & 15) == 0) scales[g] = s;
  }
}

// Values of codes: 16 lanes take a row of a block, as in quantize_rows.
template <bool VEC>
__global__ __launch_bounds__(256) void unpack(const uint8_t* __restrict__ codes,
                                              const float* __restrict__ scales,
                                              float* __restrict__ out, int brows, int64_t n,
                                              int64_t k, int64_t kb, int64_t nb,
                                              int64_t blocks) {
  for (int64_t g = (int64_t)blockIdx.x * 16 + (threadIdx.x >> 4); g < blocks;
       g += (int64_t)gridDim.x * 16) {
    const int64_t row = g / kb, b = g - row * kb;
    const int64_t mat = row / n;
    const float s = scales[(mat * nb + (row - mat * n) / brows) * kb + b];
    const int64_t j = b * QW_BLOCK + (threadIdx.x & 15) * 8;
    const u32x2 c = *(const u32x2*)(codes + row * (kb * QW_BLOCK) + j);
    float v[8];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const f32x2 lo = __builtin_amdgcn_cvt_pk_f32_fp8((int)c[i], false);
      const f32x2 hi = __builtin_amdgcn_cvt_pk_f32_fp8((int)c[i], true);
      v[4 * i] = lo.x * s;
      v[4 * i + 1] = lo.y * s;
      v[4 * i + 2] = hi.x * s;
      v[4 * i + 3] = hi.y * s;
    }
    store8_of_row<VEC>(out + row * k, j, k, v);
  }
}

template <typename T>
hipError_t quantize(int brows, int64_t count, int64_t n, int64_t k, const T* w, uint8_t* codes,
                    float* scales, hipStream_t stream) {
  const bool vec = k % 8 == 0 && aligned(w, 16);
  const int64_t kb = pitch(k) / QW_BLOCK;
  if (brows == 1) {
    const int64_t blocks = count * n * kb;
    const unsigned grid = grid_for(blocks, 16);
    if (vec)
      quantize_rows<true><<<grid, 256, 0, stream>>>(w, codes, scales, k, kb, blocks);
    else
      quantize_rows<false><<<grid, 256, 0, stream>>>(w, codes, scales, k, kb, blocks);
  } else {
    const int64_t nb = (n + QW_BLOCK - 1) / QW_BLOCK;
    const int64_t tiles = count * nb * kb;
    const unsigned grid = grid_for(tiles, 1);
    if (vec)
      quantize_tiles<true><<<grid, 256, 0, stream>>>(w, codes, scales, n, k, kb, nb, tiles);
    else
      quantize_tiles<false><<<grid, 256, 0, stream>>>(w, codes, scales, n, k, kb, nb, tiles);
  }
  return hipGetLastError();
}

template <typename T>
hipError_t swiglu(int64_t rows, int64_t f, const T* h, const int32_t* used, uint8_t* codes,
                  float* scales, hipStream_t stream) {
  const int64_t kb = pitch(f) / QW_BLOCK, blocks = rows * kb;
  const unsigned grid = grid_for(blocks, 16);
  if (f % 8 == 0 && aligned(h, 16))
    quantize_swiglu<true><<<grid, 256, 0, stream>>>(h, used, codes, scales, f, kb, blocks);
  else
    quantize_swiglu<false><<<grid, 256, 0, stream>>>(h, used, codes, scales, f, kb, blocks);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_block_quantize(int brows, int64_t count, int64_t n, int64_t k, int type,
                                 const void* w, uint8_t* codes, float* scales,
                                 hipStream_t stream) {
  return type == QW_F32
             ? quantize(brows, count, n, k, (const float*)w, codes, scales, stream)
             : quantize(brows, count, n, k, (const uint16_t*)w, codes, scales, stream);
}

hipError_t launch_block_quantize_swiglu(int64_t rows, int64_t f, int type, const void* h,
                                        const int32_t* used, uint8_t* codes, float* scales,
                                        hipStream_t stream) {
  return type == QW_F32 ? swiglu(rows, f, (const float*)h, used, codes, scales, stream)
                        : swiglu(rows, f, (const uint16_t*)h, used, codes, scales, stream);
}

hipError_t launch_block_unpack(int brows, int64_t count, int64_t n, int64_t k,
                               const uint8_t* codes, const float* scales, float* out,
                               hipStream_t stream) {
  const int64_t kb = pitch(k) / QW_BLOCK, blocks = count * n * kb;
  const int64_t nb = (n + brows - 1) / brows;
  const unsigned grid = grid_for(blocks, 16);
  if (k % 8 == 0 && aligned(out, 16))
    unpack<true><<<grid, 256, 0, stream>>>(codes, scales, out, brows, n, k, kb, nb, blocks);
  else
    unpack<false><<<grid, 256, 0, stream>>>(codes, scales, out, brows, n, k, kb, nb, blocks);
  return hipGetLastError();
}

}  // namespace qw
