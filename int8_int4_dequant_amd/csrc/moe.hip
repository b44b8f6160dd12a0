// Tokens sorted by expert and back: the sort of (token, choice) slots, the
// gather of token rows into expert order (as they are or as e4m3 codes), the
// weighted combination and its gradients.
//
// All but the sort are bound by HBM: every row is read or written once, in
// 16-byte pieces.  They go token by token, so a token's row is read once for
// its topk copies, and its output is summed in registers in the order of the
// choices: no atomics, the same bits every time.
#include "block_codes.h"

#include <algorithm>

namespace qw {
namespace {

// ------------------------------------------------------------------- sort
//
// A counting sort.  A thread block takes a run of consecutive slots, each of
// its 16 waves a run within that; a wave ranks 64 slots at a time among
// themselves (the lanes with the same expert, found with one ballot for each
// bit of the expert number), so equal experts keep the order of their slots.

constexpr int kSortWaves = 16;
constexpr int kSortOne = 4096;     // slots that one block sorts alone
constexpr int kSortBlocks = 256;   // blocks at most for more of them

// Slots of one block, a multiple of 64 * kSortWaves.
int64_t sort_run(int64_t slots) {
  const int64_t unit = 64 * kSortWaves;
  if (slots <= kSortOne) return kSortOne;
  return ((slots + kSortBlocks - 1) / kSortBlocks + unit - 1) / unit * unit;
}

// The lanes that hold the same id as this one; valid for lanes with `in`.
__device__ __forceinline__ uint64_t peers_of(int id, bool in, int bits) {
  uint64_t m = __ballot(in);
  for (int b = 0; b < bits; ++b) {
    const uint64_t s = __ballot((id >> b) & 1);
    m &= (id >> b) & 1 ? s : ~s;
  }
  return m;
}

template <typename ID>
__device__ __forceinline__ int id_at(const ID* ids, int64_t slot, int64_t end, int experts) {
  if (slot >= end) return -1;
  const ID v = ids[slot];
  return v >= 0 && v < experts ? (int)v : -1;
}

// Counts [blocks][experts] of each block's slots.
template <typename ID>
__global__ __launch_bounds__(64 * kSortWaves) void sort_count(const ID* __restrict__ ids,
                                                              int64_t slots, int64_t run,
                                                              int experts, int bits,
                                                              int32_t* __restrict__ counts) {
  extern __shared__ int hist[];
  for (int e = threadIdx.x; e < experts; e += blockDim.x) hist[e] = 0;
  __syncthreads();
  const int64_t from = blockIdx.x * run, end = min(from + run, slots);
  for (int64_t base = from + (threadIdx.x & ~63); base < end; base += blockDim.x) {
    const int id = id_at(ids, base + (threadIdx.x & 63), end, experts);
    const uint64_t same = peers_of(id, id >= 0, bits);
    if (id >= 0 && (threadIdx.x & 63) == __builtin_ctzll(same)) atomicAdd(&hist[id], __popcll(same));
  }
  __syncthreads();
  for (int e = threadIdx.x; e < experts; e += blockDim.x)
    counts[(int64_t)blockIdx.x * experts + e] = hist[e];
}

// Places the slots of each block.  counts: from sort_count, or NULL for a
// single block.
template <typename ID>
__global__ __launch_bounds__(64 * kSortWaves) void sort_place(
    const ID* __restrict__ ids, int64_t slots, int64_t run, int experts, int bits,
    const int32_t* __restrict__ counts, int32_t* __restrict__ pos, int32_t* __restrict__ order,
    int32_t* __restrict__ offsets) {
  extern __shared__ int hist[];  // [kSortWaves][experts]: counts, then next rows
  __shared__ int wave_sum[kSortWaves];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int64_t from = blockIdx.x * run, end = min(from + run, slots);
  const int64_t mine = from + wave * (run / kSortWaves);
  const int64_t mine_end = min(mine + run / kSortWaves, end);
  for (int e = threadIdx.x; e < kSortWaves * experts; e += blockDim.x) hist[e] = 0;
  __syncthreads();
  for (int64_t base = mine; base < mine_end; base += 64) {
    const int id = id_at(ids, base + lane, mine_end, experts);
    const uint64_t same = peers_of(id, id >= 0, bits);
    if (id >= 0 && lane == __builtin_ctzll(same))
      atomicAdd(&hist[wave * experts + id], __popcll(same));
  }
  __syncthreads();
  // Expert e's rows in earlier blocks and in all: 1024 / `span` threads share
  // the blocks' counts, so that few loads follow each other.
  __shared__ int rows_before[QW_MOE_MAX_EXPERTS], rows_all[QW_MOE_MAX_EXPERTS];
  const int e = threadIdx.x;
  if (counts) {
    for (int i = threadIdx.x; i < experts; i += blockDim.x) rows_before[i] = rows_all[i] = 0;
    __syncthreads();
    const int span = 1 << bits, mine_e = threadIdx.x & (span - 1);
    if (mine_e < experts) {
      int some = 0, sum = 0;
#pragma unroll 4
      for (int b = threadIdx.x >> bits; b < (int)gridDim.x; b += blockDim.x >> bits) {
        const int c = counts[(int64_t)b * experts + mine_e];
        some += b < (int)blockIdx.x ? c : 0;
        sum += c;
      }
      atomicAdd(&rows_before[mine_e], some);
      atomicAdd(&rows_all[mine_e], sum);
    }
    __syncthreads();
  }
  int before = 0, total = 0;
  if (e < experts) {
    if (counts) {
      before = rows_before[e];
      total = rows_all[e];
    } else {
      for (int w = 0; w < kSortWaves; ++w) total += hist[w * experts + e];
    }
  }
  int upto = total;
#pragma unroll
  for (int h = 1; h < 64; h <<= 1) {
    const int v = __shfl_up(upto, h);
    if (lane >= h) upto += v;
  }
  if (lane == 63) wave_sum[wave] = upto;
  __syncthreads();
  int first = upto - total, all = 0;
  for (int w = 0; w < kSortWaves; ++w) {
    if (w < wave) first += wave_sum[w];
    all += wave_sum[w];
  }
  if (e < experts) {
    if (blockIdx.x == 0) offsets[e] = first;
    int next = first + before;
    for (int w = 0; w < kSortWaves; ++w) {
      const int c = hist[w * experts + e];
      hist[w * experts + e] = next;
      next += c;
    }
  }
  if (blockIdx.x == 0 && threadIdx.x == 0) offsets[experts] = all;
  __syncthreads();
  for (int64_t base = mine; base < mine_end; base += 64) {
    const int64_t slot = base + lane;
    const int id = id_at(ids, slot, mine_end, experts);
    const uint64_t same = peers_of(id, id >= 0, bits);
    const int leader = id >= 0 ? __builtin_ctzll(same) : 0;
    int row = 0;
    if (id >= 0 && lane == leader) row = atomicAdd(&hist[wave * experts + id], __popcll(same));
    row = __shfl(row, leader) + __popcll(same & ((1ull << lane) - 1));
    if (slot < mine_end) {
      pos[slot] = id >= 0 ? row : -1;
      if (order && id >= 0) order[row] = (int)slot;
    }
  }
  if (order)
    for (int64_t i = from + threadIdx.x; i < end; i += blockDim.x)
      if (i >= all) order[i] = -1;
}

template <typename ID>
hipError_t sort(int64_t slots, int64_t experts, const ID* ids, int32_t* pos, int32_t* order,
                int32_t* offsets, void* work, hipStream_t stream) {
  const int64_t run = sort_run(slots);
  // no slots: one block still writes the offsets
  const unsigned blocks = (unsigned)std::max<int64_t>((slots + run - 1) / run, 1);
  int bits = 0;
  while ((1 << bits) < experts) ++bits;
  int32_t* counts = blocks > 1 ? (int32_t*)work : nullptr;
  if (counts) {
    sort_count<<<blocks, 64 * kSortWaves, experts * 4, stream>>>(ids, slots, run, (int)experts,
                                                                 bits, counts);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  sort_place<<<blocks, 64 * kSortWaves, kSortWaves * experts * 4, stream>>>(
      ids, slots, run, (int)experts, bits, counts, pos, order, offsets);
  return hipGetLastError();
}

// ---------------------------------------------------------- gather, combine
//
// Rows are cut into pieces of 8 values; thread i takes piece i % pieces of
// token i / pieces.
//
// NT: what goes by once goes past the caches, when the rows are more than the
// caches keep for whoever comes next (8192 tokens x 8 x 4096 bf16: combine 137
// -> 110 us with loads and stores of that kind, the gather of twice as many 207
// -> 181 with stores, the gradients 217 -> 195 with loads but 235 with stores;
// 201 MB that the kernel before wrote are combined in 36 us, past the caches in 48).

constexpr int64_t kCached = 256 << 20;  // bytes

template <bool VEC, bool NT, typename T>
__global__ __launch_bounds__(256) void gather(const T* __restrict__ x,
                                              const int32_t* __restrict__ pos,
                                              T* __restrict__ xs, int topk, int64_t d,
                                              int64_t pieces, int64_t rows, int64_t items) {
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < items;
       i += (int64_t)gridDim.x * 256) {
    const int64_t token = i / pieces, j = (i - token * pieces) * 8;
    float v[8];
    load8_of_row<VEC>(x + token * d, j, d, v);
    for (int c = 0; c < topk; ++c) {
      const int64_t p = pos[token * topk + c];
      if (p >= 0 && p < rows) store8_of_row<VEC, NT>(xs + p * d, j, d, v);
    }
  }
}

// Blocks of 128 values; 16 lanes quantize one and write it to the token's rows.
template <bool VEC, typename T>
__global__ __launch_bounds__(256) void gather_block(const T* __restrict__ x,
                                                    const int32_t* __restrict__ pos,
                                                    uint8_t* __restrict__ codes,
                                                    float* __restrict__ scales, int topk,
                                                    int64_t d, int64_t kb, int64_t rows,
                                                    int64_t blocks) {
  for (int64_t g = (int64_t)blockIdx.x * 16 + (threadIdx.x >> 4); g < blocks;
       g += (int64_t)gridDim.x * 16) {
    const int64_t token = g / kb, b = g - token * kb;
    const int64_t j = b * QW_BLOCK + (threadIdx.x & 15) * 8;
    float v[8];
    load8_of_row<VEC>(x + token * d, j, d, v);
    const float s = block_scale(max16(amax8(v)));
    const u32x2 c8 = codes8(v, s);
    for (int c = 0; c < topk; ++c) {
      const int64_t p = pos[token * topk + c];
      if (p < 0 || p >= rows) continue;
      *(u32x2*)(codes + p * (kb * QW_BLOCK) + j) = c8;
      if ((threadIdx.x & 15) == 0) scales[p * kb + b] = s;
    }
  }
}

template <bool VEC, bool NT, typename T, typename YT>
__global__ __launch_bounds__(256) void combine(const T* __restrict__ ys,
                                               const int32_t* __restrict__ pos,
                                               const float* __restrict__ weights,
                                               YT* __restrict__ y, int topk, int64_t d,
                                               int64_t pieces, int64_t rows, int64_t items) {
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < items;
       i += (int64_t)gridDim.x * 256) {
    const int64_t token = i / pieces, j = (i - token * pieces) * 8;
    float s[8] = {};
    // 4 choices at a time, their rows on the way together; without a row, row 0
    // is read and left out
    for (int c0 = 0; c0 < topk; c0 += 4) {
      int64_t p[4];
      float w[4], v[4][8];
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        const int64_t slot = token * topk + min(c0 + c, topk - 1);
        p[c] = pos[slot];
        w[c] = weights ? weights[slot] : 1.0f;
        if (c0 + c >= topk || p[c] >= rows) p[c] = -1;
      }
#pragma unroll
      for (int c = 0; c < 4; ++c) load8_of_row<VEC, NT>(ys + max(p[c], (int64_t)0) * d, j, d, v[c]);
#pragma unroll
      for (int c = 0; c < 4; ++c)
#pragma unroll
        for (int u = 0; u < 8; ++u)
          s[u] = p[c] >= 0 ? __builtin_fmaf(w[c], v[c][u], s[u]) : s[u];
    }
    store8_of_row<VEC, NT>(y + token * d, j, d, s);
  }
}

// One thread block per token; 8 choices at a time share a pass over dy.
constexpr int kChoices = 8;
template <bool VEC, bool NT, typename T>
__global__ __launch_bounds__(256) void combine_backward(
    const T* __restrict__ dy, const T* __restrict__ ys, const int32_t* __restrict__ pos,
    const float* __restrict__ weights, T* __restrict__ dys, float* __restrict__ dweights,
    int topk, int64_t d, int64_t rows, int64_t t) {
  __shared__ float part[4][kChoices];
  for (int64_t token = blockIdx.x; token < t; token += gridDim.x) {
    for (int c0 = 0; c0 < topk; c0 += kChoices) {
      int64_t p[kChoices];
      float w[kChoices], dot[kChoices] = {};
#pragma unroll
      for (int c = 0; c < kChoices; ++c) {
        const bool in = c0 + c < topk;
        p[c] = in ? pos[token * topk + c0 + c] : -1;
        if (p[c] >= rows) p[c] = -1;
        w[c] = in && p[c] >= 0 && weights ? weights[token * topk + c0 + c] : 1.0f;
      }
      for (int64_t j = threadIdx.x * 8; j < d; j += 256 * 8) {
        float g[8];
        load8_of_row<VEC, NT>(dy + token * d, j, d, g);
#pragma unroll
        for (int c = 0; c < kChoices; ++c) {
          if (p[c] < 0) continue;
          if (dweights) {
            float v[8];
            load8_of_row<VEC, NT>(ys + p[c] * d, j, d, v);
#pragma unroll
            for (int u = 0; u < 8; ++u) dot[c] = __builtin_fmaf(g[u], v[u], dot[c]);
          }
          if (dys) {
            float v[8];
#pragma unroll
            for (int u = 0; u < 8; ++u) v[u] = w[c] * g[u];
            store8_of_row<VEC>(dys + p[c] * d, j, d, v);
          }
        }
      }
      if (dweights) {
#pragma unroll
        for (int c = 0; c < kChoices; ++c) {
#pragma unroll
          for (int h = 32; h > 0; h >>= 1) dot[c] += __shfl_xor(dot[c], h);
          if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6][c] = dot[c];
        }
        __syncthreads();
        const int c = threadIdx.x;
        if (c < kChoices && c0 + c < topk)
          dweights[token * topk + c0 + c] = (part[0][c] + part[1][c]) + (part[2][c] + part[3][c]);
        __syncthreads();
      }
    }
  }
}

template <typename T>
bool rows_vec(int64_t d, const T* a, const void* b) {
  return d % 8 == 0 && aligned(a, 16) && aligned(b, 16);
}

template <typename T>
hipError_t run_gather(int64_t t, int topk, int64_t d, int64_t rows, const T* x,
                      const int32_t* pos, T* xs, hipStream_t stream) {
  const int64_t pieces = (d + 7) / 8, items = t * pieces;
  const unsigned grid = grid_for(items, 256);
  if (!rows_vec(d, x, xs))
    gather<false, false><<<grid, 256, 0, stream>>>(x, pos, xs, topk, d, pieces, rows, items);
  else if (rows * d * (int64_t)sizeof(T) > kCached)
    gather<true, true><<<grid, 256, 0, stream>>>(x, pos, xs, topk, d, pieces, rows, items);
  else
    gather<true, false><<<grid, 256, 0, stream>>>(x, pos, xs, topk, d, pieces, rows, items);
  return hipGetLastError();
}

template <typename T>
hipError_t run_gather_block(int64_t t, int topk, int64_t d, int64_t rows, const T* x,
                            const int32_t* pos, uint8_t* codes, float* scales,
                            hipStream_t stream) {
  const int64_t kb = pitch(d) / QW_BLOCK, blocks = t * kb;
  const unsigned grid = grid_for(blocks, 16);
  if (d % 8 == 0 && aligned(x, 16))
    gather_block<true><<<grid, 256, 0, stream>>>(x, pos, codes, scales, topk, d, kb, rows, blocks);
  else
    gather_block<false><<<grid, 256, 0, stream>>>(x, pos, codes, scales, topk, d, kb, rows, blocks);
  return hipGetLastError();
}

template <typename T, typename YT>
hipError_t run_combine(int64_t t, int topk, int64_t d, int64_t rows, const T* ys,
                       const int32_t* pos, const float* weights, YT* y, hipStream_t stream) {
  const int64_t pieces = (d + 7) / 8, items = t * pieces;
  const unsigned grid = grid_for(items, 256);
  if (rows == 0) topk = 0;  // no row to look at
  if (!rows_vec(d, ys, y))
    combine<false, false><<<grid, 256, 0, stream>>>(ys, pos, weights, y, topk, d, pieces, rows, items);
  else if (rows * d * (int64_t)sizeof(T) > kCached)
    combine<true, true><<<grid, 256, 0, stream>>>(ys, pos, weights, y, topk, d, pieces, rows, items);
  else
    combine<true, false><<<grid, 256, 0, stream>>>(ys, pos, weights, y, topk, d, pieces, rows, items);
  return hipGetLastError();
}

template <typename T>
hipError_t run_backward(int64_t t, int topk, int64_t d, int64_t rows, const T* dy, const T* ys,
                        const int32_t* pos, const float* weights, T* dys, float* dweights,
                        hipStream_t stream) {
  const unsigned grid = grid_for(t, 1);
  // a NULL pointer is aligned
  if (d % 8 != 0 || !aligned(dy, 16) || !aligned(ys, 16) || !aligned(dys, 16))
    combine_backward<false, false>
        <<<grid, 256, 0, stream>>>(dy, ys, pos, weights, dys, dweights, topk, d, rows, t);
  else if (rows * d * (int64_t)sizeof(T) > kCached)
    combine_backward<true, true>
        <<<grid, 256, 0, stream>>>(dy, ys, pos, weights, dys, dweights, topk, d, rows, t);
  else
    combine_backward<true, false>
        <<<grid, 256, 0, stream>>>(dy, ys, pos, weights, dys, dweights, topk, d, rows, t);
  return hipGetLastError();
}

}  // namespace

int64_t moe_sort_work_bytes(int64_t slots, int64_t experts) {
  if (slots <= kSortOne) return 0;
  // at least sort()'s blocks, without their number's falls where the run grows:
  // what is enough for more slots is enough for fewer
  const int64_t blocks = std::min<int64_t>((slots + 64 * kSortWaves - 1) / (64 * kSortWaves), kSortBlocks);
  return (blocks * experts * 4 + 255) / 256 * 256;
}

hipError_t launch_moe_sort(int64_t slots, int64_t experts, int id_bytes, const void* ids,
                           int32_t* pos, int32_t* order, int32_t* offsets, void* work,
                           hipStream_t stream) {
  return id_bytes == 4
             ? sort(slots, experts, (const int32_t*)ids, pos, order, offsets, work, stream)
             : sort(slots, experts, (const int64_t*)ids, pos, order, offsets, work, stream);
}

hipError_t launch_moe_gather(int64_t t, int64_t topk, int64_t d, int64_t rows, int type,
                             const void* x, const int32_t* pos, void* xs, hipStream_t stream) {
  return type == QW_F32
             ? run_gather(t, (int)topk, d, rows, (const float*)x, pos, (float*)xs, stream)
             : run_gather(t, (int)topk, d, rows, (const uint16_t*)x, pos, (uint16_t*)xs, stream);
}

hipError_t launch_moe_gather_block(int64_t t, int64_t topk, int64_t d, int64_t rows, int type,
                                   const void* x, const int32_t* pos, uint8_t* codes,
                                   float* scales, hipStream_t stream) {
  return type == QW_F32 ? run_gather_block(t, (int)topk, d, rows, (const float*)x, pos, codes,
                                           scales, stream)
                        : run_gather_block(t, (int)topk, d, rows, (const uint16_t*)x, pos, codes,
                                           scales, stream);
}

hipError_t launch_moe_combine(int64_t t, int64_t topk, int64_t d, int64_t rows, int type,
                              const void* ys, const int32_t* pos, const float* weights,
                              int y_type, void* y, hipStream_t stream) {
  const int k = (int)topk;
  switch ((type == QW_F32 ? 0 : 2) + (y_type == QW_F32 ? 0 : 1)) {
    case 0: return run_combine(t, k, d, rows, (const float*)ys, pos, weights, (float*)y, stream);
    case 1: return run_combine(t, k, d, rows, (const float*)ys, pos, weights, (uint16_t*)y, stream);
    case 2: return run_combine(t, k, d, rows, (const uint16_t*)ys, pos, weights, (float*)y, stream);
    default:
      return run_combine(t, k, d, rows, (const uint16_t*)ys, pos, weights, (uint16_t*)y, stream);
  }
}

hipError_t launch_moe_combine_backward(int64_t t, int64_t topk, int64_t d, int64_t rows,
                                       int type, const void* dy, const void* ys,
                                       const int32_t* pos, const float* weights, void* dys,
                                       float* dweights, hipStream_t stream) {
  return type == QW_F32
             ? run_backward(t, (int)topk, d, rows, (const float*)dy, (const float*)ys, pos,
                            weights, (float*)dys, dweights, stream)
             : run_backward(t, (int)topk, d, rows, (const uint16_t*)dy, (const uint16_t*)ys, pos,
                            weights, (uint16_t*)dys, dweights, stream);
}

}  // namespace qw
