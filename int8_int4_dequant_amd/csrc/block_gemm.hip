// Products of block-scaled e4m3 matrices on the gfx950 matrix cores.
//
//   y[r][i] = sum_b sx[r][b] sw[i][b] sum_{j in b} qx[r][j] qw[i][j]
//
// Two ways to the same sum over a block of 128, each scaled afterwards and
// added to the fp32 accumulators by the vector unit (one FMA per output and
// block):
//   8-bit cores (bf16 y): one v_mfma_f32_16x16x128_f8f6f4 started from zero, at
//     twice the bf16 rate.  It aligns 8 products at a time to the largest of
//     them and drops what lies 2^-13 below it (measured: 2^16 + 2^3 is exact,
//     2^16 + 2^2 is 2^16), about 1.4e-5 of a sum's size on Gaussian data; the
//     rounding of y to bf16 is up to 2^-8 of it.
//   bf16 cores (fp32 y): codes converted to bf16, which is exact, and four
//     v_mfma_f32_16x16x32_bf16, whose sums are good to 2^-22.
// Within one MFMA the k slots are a free permutation shared by both operands:
// lane l holds row l % 16 and, with q = l / 16, bytes [16q, 16q + 16) and
// [64 + 16q, 64 + 16q + 16) of the block, so each of its two 16-byte loads is
// part of a 64-byte run.  The weight is the A operand: output lane l holds
// token l % 16 and 4 consecutive weight rows 4q..4q+3, so sx is one value per
// lane and sw (128 x 128 blocks) one per wave.
#include "block_codes.h"

#include <algorithm>
#include <cmath>
#include <type_traits>

namespace qw {
namespace {

typedef int i32x8 __attribute__((ext_vector_type(8)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));

struct GemmArgs {
  const uint8_t* codes;
  const float* scales;
  const void* x;      // float rows (row length k) or codes (row pitch kp)
  const float* xs;
  void* y;
  const int32_t* order;  // Source TOKENS: slot of a row, and slots of a token
  int topk;
  float* ys;          // gated product: y is codes and these are their scales
  const int32_t* offsets;
  int experts;
  int64_t n, k, m;    // n: weight rows of this launch
  int64_t ldy;        // outputs in a row of y
  int64_t gated;      // gated product: rows of the gate matrix, a multiple of 128
  int64_t kp;
  int kb;             // blocks along k
  int64_t nb;         // rows of scales of one weight
  int64_t tiles_m, tiles;
  int64_t chunks;     // stream kernel: blocks that share the weight rows of one tile of x
  int y_vec;          // 4 outputs of a row at a time may be stored as one
};

__device__ __forceinline__ f32x4 mfma128(i32x8 a, i32x8 b) {
  // formats 0, 0: e4m3 both; zero scale operands select the unscaled form
  return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(a, b, f32x4{0.0f, 0.0f, 0.0f, 0.0f}, 0,
                                                          0, 0, 0, 0, 0);
}

// 8 codes -> bf16, exact.
__device__ __forceinline__ bf16x8 to_bf16x8(int lo, int hi) {
  const bf16x2 a = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8((unsigned)lo, 1.0f, false);
  const bf16x2 b = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8((unsigned)lo, 1.0f, true);
  const bf16x2 c = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8((unsigned)hi, 1.0f, false);
  const bf16x2 d = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8((unsigned)hi, 1.0f, true);
  return bf16x8{a.x, a.y, b.x, b.y, c.x, c.y, d.x, d.y};
}

// One operand's fragment of a block, as its matrix instructions take it.
template <bool EXACT> struct Frag;
template <> struct Frag<false> {
  i32x8 v;
  Frag() = default;
  __device__ __forceinline__ explicit Frag(i32x8 c) : v(c) {}
};
template <> struct Frag<true> {
  bf16x8 v[4];
  Frag() = default;
  __device__ __forceinline__ explicit Frag(i32x8 c) {
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = to_bf16x8(c[2 * i], c[2 * i + 1]);
  }
};
__device__ __forceinline__ f32x4 dot128(const Frag<false>& a, const Frag<false>& b) {
  return mfma128(a.v, b.v);
}
__device__ __forceinline__ f32x4 dot128(const Frag<true>& a, const Frag<true>& b) {
  f32x4 d = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
  for (int i = 0; i < 4; ++i) d = __builtin_amdgcn_mfma_f32_16x16x32_bf16(a.v[i], b.v[i], d, 0, 0, 0);
  return d;
}

// Two products with the same weight fragment, their steps in turn.
__device__ __forceinline__ void dot128x2(const Frag<false>& a, const Frag<false>* b, f32x4* d) {
  d[0] = mfma128(a.v, b[0].v);
  d[1] = mfma128(a.v, b[1].v);
}
__device__ __forceinline__ void dot128x2(const Frag<true>& a, const Frag<true>* b, f32x4* d) {
  d[0] = d[1] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int u = 0; u < 2; ++u)
      d[u] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(a.v[i], b[u].v[i], d[u], 0, 0, 0);
}

__device__ __forceinline__ i32x8 fragment(const uint8_t* p) {
  const u32x4_la lo = *(const u32x4_la*)p, hi = *(const u32x4_la*)(p + 64);
  return i32x8{(int)lo.x, (int)lo.y, (int)lo.z, (int)lo.w,
               (int)hi.x, (int)hi.y, (int)hi.z, (int)hi.w};
}

// Rows [row, end) of the tm-th tile of `bm` rows, counted expert by expert;
// false when there are fewer tiles.  The whole wave calls it; its results are
// the same for all lanes (in scalar registers).
__device__ __forceinline__ bool grouped_tile(const GemmArgs& a, int64_t tm, int bm, int& expert,
                                             int64_t& row, int64_t& end) {
  const int lane = threadIdx.x & 63;
  const int rows = (int)a.m;
  int64_t before = 0;
  for (int c = 0; c < a.experts; c += 64) {
    int lo = 0, hi = 0;
    if (c + lane < a.experts) {
      lo = min(max(a.offsets[c + lane], 0), rows);
      hi = min(max(a.offsets[c + lane + 1], lo), rows);
    }
    const int tiles = (hi - lo + bm - 1) / bm;
    int upto = tiles;
#pragma unroll
    for (int h = 1; h < 64; h <<= 1) {
      const int v = __shfl_up(upto, h);
      if (lane >= h) upto += v;
    }
    const int total = __builtin_amdgcn_readlane(upto, 63);
    if (tm < before + total) {
      const int l = __builtin_ctzll(__ballot(tm < before + upto));
      expert = c + l;
      row = __builtin_amdgcn_readlane(lo, l) +
            (tm - before - (__builtin_amdgcn_readlane(upto, l) - __builtin_amdgcn_readlane(tiles, l))) * bm;
      end = min((int64_t)__builtin_amdgcn_readlane(hi, l), row + bm);
      return true;
    }
    before += total;
  }
  return false;
}

template <typename XT> struct is_codes { static constexpr bool value = false; };
template <> struct is_codes<uint8_t> { static constexpr bool value = true; };

// ------------------------------------------------------------ direct kernel
//
// For more rows than the stream kernel takes and too few tiles for the tiled
// one: a block computes 16 NT weight rows x 16 MT tokens, its WV waves
// share the blocks of k, take them straight from memory into registers, and add
// their sums through LDS.  Bound by the latency of its loads: PD blocks of k are on
// their way.  Behind the last block the loads go to an empty buffer and give
// zeros without touching memory, so that no branch stands between them.

__device__ __forceinline__ i32x8 buffer_fragment(__amdgpu_buffer_rsrc_t buf, uint32_t voff,
                                                 uint32_t soff) {
  const u32x4 lo = __builtin_amdgcn_raw_buffer_load_b128(buf, voff, soff, 0);
  const u32x4 hi = __builtin_amdgcn_raw_buffer_load_b128(buf, voff + 64, soff, 0);
  return i32x8{(int)lo.x, (int)lo.y, (int)lo.z, (int)lo.w,
               (int)hi.x, (int)hi.y, (int)hi.z, (int)hi.w};
}
__device__ __forceinline__ float buffer_float(__amdgpu_buffer_rsrc_t buf, uint32_t voff,
                                              uint32_t soff) {
  return __uint_as_float(__builtin_amdgcn_raw_buffer_load_b32(buf, voff, soff, 0));
}
__device__ __forceinline__ __amdgpu_buffer_rsrc_t rsrc_of(const void* base, int64_t bytes) {
  return __builtin_amdgcn_make_buffer_rsrc((void*)base, 0, (int)(uint32_t)bytes, 0x00020000);
}

template <int NT, int MT, int WV, int PD, bool EXACT, bool BROWS1, bool GROUPED, typename YT>
__global__ __launch_bounds__(WV * 64) void gemm_direct(GemmArgs a) {
  constexpr int BN = 16 * NT, BM = 16 * MT, LD = BN + 4;
  constexpr int SW = BROWS1 ? 4 * NT : 1;  // weight scales a lane needs
  static_assert(QW_BLOCK % BN == 0, "a block's weight rows lie in one 128 x 128 block");
  __shared__ __align__(16) float part[WV][BM][LD];
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int lane = threadIdx.x & 63, r = lane & 15, q = lane >> 4;
  for (int64_t tile = blockIdx.x; tile < a.tiles; tile += gridDim.x) {
    const int64_t n0 = tile / a.tiles_m * BN;
    int64_t m0 = tile % a.tiles_m * BM, end = min(m0 + BM, a.m);
    int expert = 0;
    if (GROUPED && !grouped_tile(a, tile % a.tiles_m, BM, expert, m0, end)) continue;
    const int64_t wrows = min(a.n - n0, (int64_t)BN), srow = BROWS1 ? n0 : n0 / QW_BLOCK;
    const uint8_t* wbase = a.codes + (expert * a.n + n0) * a.kp;
    const uint8_t* xbase = (const uint8_t*)a.x + m0 * a.kp;
    const float* wsbase = a.scales + (expert * a.nb + srow) * a.kb;
    const float* xsbase = a.xs + m0 * a.kb;
    i32x8 w[PD][NT], x[PD][MT];
    float sw[PD][SW], sx[PD][MT];
    // A wave's blocks of k are consecutive ones: rows are often a power of two
    // apart, and waves side by side would all ask the same few L2 channels.
    const int each = (a.kb + WV - 1) / WV, first = wave * each;
    const int last = min(first + each, a.kb);
    auto load = [&](int b, int p) {
      const bool in = b < last;
      const auto wbuf = rsrc_of(wbase, in ? wrows * a.kp : 0);
      const auto xbuf = rsrc_of(xbase, in ? (end - m0) * a.kp : 0);
      const auto wsbuf = rsrc_of(wsbase, in ? (BROWS1 ? wrows : 1) * a.kb * 4 : 0);
      const auto xsbuf = rsrc_of(xsbase, in ? (end - m0) * a.kb * 4 : 0);
#pragma unroll
      for (int i = 0; i < NT; ++i)
        w[p][i] = buffer_fragment(wbuf, (16 * i + r) * (uint32_t)a.kp + q * 16, b * QW_BLOCK);
#pragma unroll
      for (int j = 0; j < MT; ++j) {
        x[p][j] = buffer_fragment(xbuf, (16 * j + r) * (uint32_t)a.kp + q * 16, b * QW_BLOCK);
        sx[p][j] = buffer_float(xsbuf, (16 * j + r) * a.kb * 4, b * 4);
      }
#pragma unroll
      for (int c = 0; c < SW; ++c)
        sw[p][c] = buffer_float(wsbuf, BROWS1 ? (16 * (c / 4) + 4 * q + c % 4) * a.kb * 4 : 0, b * 4);
    };
#pragma unroll
    for (int p = 0; p < PD; ++p) load(first + p, p);
    f32x4 acc[NT][MT] = {};
    for (int b = first; b < last; b += PD) {
#pragma unroll
      for (int p = 0; p < PD; ++p) {
        Frag<EXACT> wf[NT];
#pragma unroll
        for (int i = 0; i < NT; ++i) wf[i] = Frag<EXACT>(w[p][i]);
#pragma unroll
        for (int j = 0; j < MT; ++j) {
          const Frag<EXACT> xf(x[p][j]);
#pragma unroll
          for (int i = 0; i < NT; ++i) {
            const f32x4 d = dot128(wf[i], xf);
#pragma unroll
            for (int c = 0; c < 4; ++c)
              acc[i][j][c] = __builtin_fmaf(d[c], sx[p][j] * sw[p][BROWS1 ? 4 * i + c : 0],
                                            acc[i][j][c]);
          }
        }
        load(b + p + PD, p);
      }
    }
    __syncthreads();  // the last tile's sums have been read
#pragma unroll
    for (int i = 0; i < NT; ++i)
#pragma unroll
      for (int j = 0; j < MT; ++j) *(f32x4*)&part[wave][16 * j + r][16 * i + 4 * q] = acc[i][j];
    __syncthreads();
    for (int o = threadIdx.x; o < BM * BN; o += WV * 64) {
      const int t = o / BN, c = o % BN;
      if (m0 + t < end && n0 + c < a.n) {
        float s = part[0][t][c];
#pragma unroll
        for (int v = 1; v < WV; ++v) s += part[v][t][c];
        store1((YT*)a.y + (m0 + t) * a.ldy + n0 + c, s);
      }
    }
  }
}

template <int NT, int MT, int WV, int PD, bool GROUPED>
hipError_t run_direct(GemmArgs a, const BlockGemm& g, hipStream_t stream) {
  constexpr int BN = 16 * NT, BM = 16 * MT;
  a.tiles_m = GROUPED ? std::min(a.m, (a.m + a.experts * (int64_t)(BM - 1)) / BM)
                      : (a.m + BM - 1) / BM;
  a.tiles = a.tiles_m * ((a.n + BN - 1) / BN);
  // a launch holds fewer than 2^32 threads: the kernel's loop takes the rest
  const unsigned grid = (unsigned)std::min<int64_t>(a.tiles, 1 << 21);
  auto go = [&](auto exact, auto brows1, auto y) {
    gemm_direct<NT, MT, WV, PD, decltype(exact)::value, decltype(brows1)::value, GROUPED, decltype(y)>
        <<<grid, WV * 64, 0, stream>>>(a);
  };
  using std::true_type;
  using std::false_type;
  const bool one = g.brows == 1;
  if (g.y_type == QW_BF16)
    one ? go(false_type{}, true_type{}, uint16_t{}) : go(false_type{}, false_type{}, uint16_t{});
  else if (g.exact)
    one ? go(true_type{}, true_type{}, 0.0f) : go(true_type{}, false_type{}, 0.0f);
  else if constexpr (GROUPED)
    one ? go(false_type{}, true_type{}, 0.0f) : go(false_type{}, false_type{}, 0.0f);
  return hipGetLastError();
}

// ------------------------------------------------------------ tiled kernel
//
// For many rows.  A block of 8 waves, WM of them along the tokens and the rest
// along the weight rows, each with 16 NF weight rows x 16 MF tokens, one block of k
// at a time through a ring of STAGES LDS buffers (2 at 256 x 256, where no more fit,
// 3 or 4 otherwise): while the matrix cores work on one, the next ones are copied
// straight from memory (buffer loads with an LDS target, 16 bytes a lane).  A wave
// keeps its MF token fragments in registers and walks its NF weight fragments.
//
// LDS rows are the 128 bytes of a block.  A phase of a 16-byte LDS read is 16
// lanes, here 16 consecutive rows at the same place in the row, and the 64
// banks hold 2 rows: piece c of row r is kept at c ^ (r / 2 % 8), so that the
// 16 lanes meet 16 different places.  The copy writes LDS in lane order, so
// the lanes fetch the pieces in that order from memory.

constexpr int kTileWaves = 8;
constexpr int kUnits = 256;  // compute units

typedef int i32x4 __attribute__((ext_vector_type(4)));

// A buffer descriptor of `bytes` from `base`: reads beyond give zeros.
__device__ __forceinline__ i32x4 buffer_of(const void* base, uint32_t bytes) {
  const uint64_t p = (uint64_t)base;
  return i32x4{(int)(uint32_t)p, (int)(uint32_t)(p >> 32), (int)bytes, 0x00020000};
}

// 16 bytes a lane from buffer + voff + soff to LDS at `lds` + 16 * lane.  The
// compiler does not see this write (it would wait for every copy in flight
// before any LDS read): landed() orders it.  Nothing else here uses m0.
__device__ __forceinline__ void copy_to_lds(i32x4 buffer, uint32_t voff, uint32_t soff,
                                            uint32_t lds) {
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tbuffer_load_dwordx4 %1, %2, %3 offen lds"
               :: "s"(lds), "v"(voff), "s"(buffer), "s"(soff) : "memory");
}
// The same, 4 bytes a lane.
__device__ __forceinline__ void copy4_to_lds(i32x4 buffer, uint32_t voff, uint32_t soff,
                                             uint32_t lds) {
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tbuffer_load_dword %1, %2, %3 offen lds"
               :: "s"(lds), "v"(voff), "s"(buffer), "s"(soff) : "memory");
}
// This wave's copies but the LEFT newest, and its LDS accesses, are done, and
// so are the block's.
template <int LEFT>
__device__ __forceinline__ void landed() {
  asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)\n\ts_barrier" :: "i"(LEFT) : "memory");
}

// This wave's LDS accesses are done, and so are the block's; copies stay on
// their way.
__device__ __forceinline__ void lds_barrier() {
  asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");
}

__device__ __forceinline__ i32x8 lds_fragment(const uint8_t* lds, int row, int q) {
  const int sw = (row >> 1) & 7;
  const u32x4 lo = *(const u32x4*)(lds + row * 128 + ((q ^ sw) << 4));
  const u32x4 hi = *(const u32x4*)(lds + row * 128 + (((q + 4) ^ sw) << 4));
  return i32x8{(int)lo.x, (int)lo.y, (int)lo.z, (int)lo.w,
               (int)hi.x, (int)hi.y, (int)hi.z, (int)hi.w};
}

// The tile of a block.  Blocks go to the 8 XCDs in turn, each with an L2 of its
// own: an XCD takes a contiguous run of the tiles, ordered in bands of 8 tile
// rows (tokens) and down each band column by column, so that the 32 tiles it
// works on together share 8 tiles of x and 4 of the weight.
__device__ __forceinline__ void tile_place(int64_t block, int64_t tiles, int64_t tiles_m,
                                           int64_t& tm, int64_t& tn) {
  const int64_t xcd = block & 7, each = tiles >> 3, extra = tiles & 7;
  const int64_t t = xcd * each + min(xcd, extra) + (block >> 3);
  const int64_t tiles_n = tiles / tiles_m;
  const int64_t band = t / (8 * tiles_n), in_band = t - band * 8 * tiles_n;
  const int64_t height = min((int64_t)8, tiles_m - band * 8);
  tn = in_band / height;
  tm = band * 8 + in_band - tn * height;
}

//
// GATED: the weight is a gate and an up matrix of a.gated rows each, one behind
// the other; the tile is 128 rows of each, and what is written is the quantized
// silu(gate) * up: a wave's 128 gate rows are one 1 x 128 block of each of its
// tokens, so half of the tokens' sums change places with the up waves through
// LDS and every wave scales and rounds half of its tokens.  A block takes tile
// after tile and has the next one's first copies on their way while it writes its
// results (24594 rows of 64 experts, 16 blocks of k: 284 -> 267 us; the other
// products, whose results take less work, lose by it: 4096^3 63 -> 67).

template <int NF, int MF, int WM, int STAGES, bool EXACT, bool BROWS1, bool GROUPED, bool GATED,
          typename YT>
__global__ __launch_bounds__(kTileWaves * 64, 2) void gemm_tiled(GemmArgs a) {
  constexpr int BN = 16 * NF * (kTileWaves / WM), BM = 16 * MF * WM, ROWS = BN + BM;
  constexpr int PAIRS = NF * MF / 2;
  constexpr bool ROTATE = NF * MF == 32 && !GROUPED;
  constexpr int SEGS = ROWS / 8 / kTileWaves;  // 8-row pieces of a wave
  static_assert(QW_BLOCK % (16 * NF) == 0, "a wave's weight rows lie in one 128 x 128 block");
  static_assert(ROWS / 8 % kTileWaves == 0 && MF % 2 == 0, "whole pieces and pairs");
  // scales of 4 blocks of k at a time (a scale's line of memory holds its
  // row's next ones), of the tile's tokens and then of its rows of blocks
  constexpr int SROWS = BM + (BROWS1 ? BN : 64);  // BM: whole pieces of 64
  static_assert(SROWS / 64 <= kTileWaves, "64 rows of scales a wave");
  __shared__ __align__(1024) uint8_t lds[STAGES][ROWS * 128];
  __shared__ __align__(16) float scales[2][4][SROWS];
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int lane = threadIdx.x & 63, r = lane & 15, q = lane >> 4;
  const int wm = wave % WM * 16 * MF, wn = wave / WM * 16 * NF;
  static_assert(!GATED || (NF == 8 && MF == 2 && WM == 4), "128 gate rows and 128 up rows");
  const int kp = (int)a.kp;
  const int64_t urows = !GATED ? 0 : BROWS1 ? a.gated : a.gated / QW_BLOCK;  // gate to up
  // One tile: what it computes, and the buffers it reads.
  struct Place {
    int64_t n0, m0, end;
    i32x4 wbuf, ubuf, xbuf, sbuf;
    int rot;
  };
  // The first tile at or behind `at` (in steps of the grid) that has rows.
  auto place = [&](int64_t& at, Place& p) {
    for (; at < a.tiles; at += gridDim.x) {
      int64_t tm, tn;
      tile_place(at, a.tiles, a.tiles_m, tm, tn);
      p.rot = ROTATE && a.kb >= 16 ? (int)((tm * 5 + tn) & 7) : 0;
      p.n0 = GATED ? tn * QW_BLOCK : tn * BN;
      p.m0 = tm * BM;
      p.end = min(p.m0 + BM, a.m);
      int expert = 0;
      if (GROUPED && !grouped_tile(a, tm, BM, expert, p.m0, p.end)) continue;
      p.wbuf = buffer_of(a.codes + (expert * a.n + p.n0) * a.kp,
                         (uint32_t)(min(a.n - p.n0, (int64_t)(GATED ? QW_BLOCK : BN)) * a.kp));
      // GATED: from 128 rows before the up rows, for the tile's rows from 128 on
      p.ubuf = buffer_of(a.codes + (expert * a.n + a.gated + p.n0 - QW_BLOCK) * a.kp,
                         (uint32_t)(2 * QW_BLOCK * a.kp));
      p.xbuf = buffer_of((const uint8_t*)a.x + p.m0 * a.kp, (uint32_t)((p.end - p.m0) * a.kp));
      const int64_t srow = BROWS1 ? p.n0 : p.n0 / QW_BLOCK;
      p.sbuf = wave * 64 < BM
          ? buffer_of(a.xs + p.m0 * a.kb, (uint32_t)((p.end - p.m0) * a.kb * 4))
          : buffer_of(a.scales + (expert * a.nb + srow) * a.kb,
                      (uint32_t)(min(a.nb - srow, urows + (BROWS1 ? BN : 2)) * a.kb * 4));
      return true;
    }
    return false;
  };
  // of the rows of scales behind x's, those from half on are the up matrix's
  const int srel = wave * 64 + lane - (wave * 64 < BM ? 0 : BM);
  const int half_rows = BROWS1 ? QW_BLOCK : 1;
  const uint32_t soff =
      (uint32_t)(srel + (GATED && wave * 64 >= BM && srel >= half_rows ? urows - half_rows : 0)) *
      a.kb * 4;
  uint32_t voff[SEGS];
#pragma unroll
  for (int s = 0; s < SEGS; ++s) {
    const int row = (wave + kTileWaves * s) * 8 + (lane >> 3);
    const int c = (lane & 7) ^ ((row >> 1) & 7);
    voff[s] = (uint32_t)(row < BN ? row : row - BN) * kp + c * 16;
  }
  const uint32_t lds0 = (uint32_t)(uintptr_t)(__attribute__((address_space(3))) uint8_t*)&lds[0][0];
  const uint32_t lds1 =
      (uint32_t)(uintptr_t)(__attribute__((address_space(3))) uint8_t*)&scales[0][0][0];
  // Tiles of the largest shape start at different blocks of k, up to 7 apart (and
  // within what an L2 holds of the rows they share): in step they would all ask
  // the same channels, with rows often a power of two apart (8192^3 484 -> 467
  // us; the other tiles, and grouped ones, lose 2 to 5 in a hundred by it).  From 16
  // blocks of k on: 2048 x 8192 with 8, 16, 32 and 64 of them 26.4 -> 27.7, 39.0 ->
  // 40.8, 70.4 -> 70.3 and 126.8 -> 123.8 us, 4096 x 8192 with 8 and 16 49.7 -> 53.0
  // and 81.4 -> 78.9.
  auto rotated = [&](const Place& p, int b) {
    if (!ROTATE) return b;
    return b + p.rot < a.kb ? b + p.rot : b + p.rot - a.kb;
  };
  // Piece s of block b.  Behind the last block there is nothing to read, but the
  // copy is issued all the same (as zeros, from an empty buffer): a branch
  // would part the products from the scaling that runs beside them.
  auto fetch = [&](const Place& p, int b, int buf, int s) {
    i32x4 from = s >= BN / 64 ? p.xbuf : GATED && s >= BN / 128 ? p.ubuf : p.wbuf;
    from.z = b < a.kb ? from.z : 0;
    const int seg = wave + kTileWaves * s;
    copy_to_lds(from, voff[s], (uint32_t)rotated(p, b) * 128,
                lds0 + buf * (ROWS * 128) + seg * 1024);
  };
  auto fetch_scales = [&](const Place& p, int b) {  // of the 4 blocks from b on
    if (wave < SROWS / 64) {
#pragma unroll
      for (int c = 0; c < 4; ++c)
        copy4_to_lds(p.sbuf, soff, (uint32_t)rotated(p, b + c) * 4,
                     lds1 + (((b >> 2) & 1) * 4 + c) * (SROWS * 4) + wave * 256);
    }
  };
  auto fetch_first = [&](const Place& p) {  // what a tile's first step takes, and more
    fetch_scales(p, 0);
#pragma unroll
    for (int c = 0; c < STAGES - 1; ++c)
#pragma unroll
      for (int s = 0; s < SEGS; ++s) fetch(p, c, c, s);
  };

  // GATED: tile after tile, the next one's first copies on their way while this
  // one's results are written.
  int64_t at = blockIdx.x;
  Place p;
  if (!place(at, p)) return;
  fetch_first(p);
  for (;;) {
    int64_t at2 = at + gridDim.x;
    Place p2;
    const bool more = GATED && place(at2, p2);
    landed<0>();
    f32x4 acc[NF][MF] = {};
    // The scales that block b's products are multiplied with: read from LDS
    // with the first fragments, joined behind the first products.
    float s[MF], sx[MF], sw = 1.0f;
    auto take_scales = [&](int b) {
      const float* sc = scales[(b >> 2) & 1][b & 3];
      if (!BROWS1) sw = sc[BM + (GATED ? wave / WM : (int)((p.n0 + wn) / QW_BLOCK - p.n0 / QW_BLOCK))];
#pragma unroll
      for (int j = 0; j < MF; ++j) sx[j] = sc[wm + 16 * j + r];
    };
    take_scales(0);
    i32x8 xr[MF];    // token fragments as they are read, and as the products take them
    Frag<EXACT> xf[MF];
#pragma unroll
    for (int j = 0; j < MF; ++j) xr[j] = lds_fragment(lds[0] + (BN + wm) * 128, 16 * j + r, q);
    xf[0] = Frag<EXACT>(xr[0]);
    xf[1] = Frag<EXACT>(xr[1]);
    i32x8 wr = lds_fragment(lds[0] + wn * 128, r, q);  // and the weight fragment
    Frag<EXACT> wf(wr);
    // a pair of products is scaled and added while the next pair runs on the
    // matrix cores: d with the scales ps (and psw) is the last pair
    f32x4 d[2] = {}, psw = {};
    float ps[2] = {};
    // The copies of block b + STAGES - 1, a few pieces with every pair: all at
    // once they would hold up the reads behind them.
    constexpr int PER = (SEGS + PAIRS - 1) / PAIRS;
    auto fetch_with = [&](int b, int buf2, int pair) {
#pragma unroll
      for (int c = 0; c < PER; ++c)
        if (pair * PER + c < SEGS) fetch(p, b + STAGES - 1, buf2, pair * PER + c);
    };
    // Copies on their way when block b + 1 has to be whole, in the last
    // fragment of block b: all of the blocks b + 2 .. b + STAGES - 2, and as many
    // pieces of block b + STAGES - 1 as went out with the pairs up to there.
    constexpr int SENT = ((NF - 1) * (MF / 2) + 1) * PER < SEGS ? ((NF - 1) * (MF / 2) + 1) * PER : SEGS;
    constexpr int LEFT = (STAGES - 3) * SEGS + SENT;
    static_assert(LEFT >= 0, "with two buffers the next block's copies all go out before");
    int buf = 0;  // b % STAGES
    for (int b = 0; b < a.kb; ++b) {
      const uint8_t* wl = lds[buf] + wn * 128;
      const int buf1 = buf + 1 < STAGES ? buf + 1 : 0;    // of block b + 1
      const int buf2 = buf > 0 ? buf - 1 : STAGES - 1;    // of block b + STAGES - 1
      if ((b & 3) == 0 && b + 4 < a.kb) fetch_scales(p, b + 4);
      f32x4 sw4 = {};
#pragma unroll
      for (int i = 0; i < NF; ++i) {
        fetch_with(b, buf2, i * (MF / 2));
        if constexpr (BROWS1) sw4 = *(const f32x4*)&scales[(b >> 2) & 1][b & 3][BM + wn + 16 * i + 4 * q];
        if (i + 1 < NF) {
          wr = lds_fragment(wl, 16 * (i + 1) + r, q);
        } else {
          // The wave holds all that it needs of this buffer: once every wave
          // does, the next step fills it again; and the next buffer is whole.
          // Scales of other blocks that are on their way only make the wait
          // longer: they are older than the copies it leaves.
          landed<LEFT>();
          wr = lds_fragment(lds[buf1] + wn * 128, r, q);
        }
#pragma unroll
        for (int j = 0; j < MF; j += 2) {
          f32x4 e[2];
          if (j > 0) fetch_with(b, buf2, i * (MF / 2) + j / 2);
          dot128x2(wf, &xf[j], e);
#pragma unroll
          for (int u = 0; u < 2; ++u) {
            if (i == NF - 1)
              xr[j + u] = lds_fragment(lds[buf1] + (BN + wm) * 128, 16 * (j + u) + r, q);
          }
          f32x4* to = j > 0 ? &acc[i][j - 2] : &acc[i > 0 ? i - 1 : NF - 1][MF - 2];
#pragma unroll
          for (int u = 0; u < 2; ++u) {
#pragma unroll
            for (int c = 0; c < 4; ++c)
              to[u][c] = __builtin_fmaf(d[u][c], BROWS1 ? ps[u] * psw[c] : ps[u], to[u][c]);
            asm volatile("" : "+v"(to[u]));  // here, not after all the products
          }
          // what the next pair takes
          if (j + 2 < MF) {
            if (i == 0) {
              xf[j + 2] = Frag<EXACT>(xr[j + 2]);
              xf[j + 3] = Frag<EXACT>(xr[j + 3]);
            }
          } else {
            wf = Frag<EXACT>(wr);
            if (i == NF - 1) {
              xf[0] = Frag<EXACT>(xr[0]);
              xf[1] = Frag<EXACT>(xr[1]);
            }
          }
#pragma unroll
          for (int u = 0; u < (EXACT ? 8 : 2); ++u) {
            __builtin_amdgcn_sched_group_barrier(0x8, 1, 0);
            __builtin_amdgcn_sched_group_barrier(0x2, EXACT ? 5 : BROWS1 ? 8 : 4, 0);
          }
          __builtin_amdgcn_sched_barrier(0);
          if (i == 0 && j == 0) {
#pragma unroll
            for (int u = 0; u < MF; ++u) s[u] = sx[u] * sw;
          }
#pragma unroll
          for (int u = 0; u < 2; ++u) {
            d[u] = e[u];
            ps[u] = s[j + u];
          }
          psw = sw4;
          if (i == NF - 1 && j + 2 == MF) take_scales(b + 1);
        }
      }
      buf = buf1;
    }
#pragma unroll
    for (int u = 0; u < 2; ++u)
#pragma unroll
      for (int c = 0; c < 4; ++c)
        acc[NF - 1][MF - 2 + u][c] = __builtin_fmaf(
            d[u][c], BROWS1 ? ps[u] * psw[c] : ps[u], acc[NF - 1][MF - 2 + u][c]);
    // All is read, and every copy has landed, the empty ones too: the ring is free.
    landed<0>();
    if (more) fetch_first(p2);
    if constexpr (GATED) {
      // 4 of the 8 fragments at a time change places in the last of the buffers,
      // which the first copies leave free.
      f32x4* const mine =
          (f32x4*)&lds[STAGES - 1][0] + ((wave % WM) * 2 + wave / WM) * (4 * 64) + lane;
      const f32x4* const other =
          (const f32x4*)&lds[STAGES - 1][0] + ((wave % WM) * 2 + 1 - wave / WM) * (4 * 64) + lane;
      static_assert(kTileWaves * 4 * 64 * 16 <= ROWS * 128, "they fit one buffer");
      auto exchange = [&](auto up) {
        constexpr int UP = decltype(up)::value;  // gate waves keep the first tokens, up waves the others
        const int64_t row = p.m0 + wm + 16 * UP + r;
        float v[NF][4], top = 0.0f;
#pragma unroll
        for (int h = 0; h < NF; h += 4) {
          if (h > 0) lds_barrier();  // the first ones have been read
#pragma unroll
          for (int i = 0; i < 4; ++i) mine[i * 64] = acc[h + i][1 - UP];
          lds_barrier();
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const f32x4 o = other[i * 64], m = acc[h + i][UP];
            const f32x4 gate = UP ? o : m, up = UP ? m : o;
            const float gates[4] = {gate[0], gate[1], gate[2], gate[3]};
            const float ups[4] = {up[0], up[1], up[2], up[3]};
            gated<4>(gates, ups, v[h + i]);
#pragma unroll
            for (int c = 0; c < 4; ++c) top = fmaxf(top, fabsf(v[h + i][c]));
          }
        }
        top = fmaxf(top, __shfl_xor(top, 16));
        top = fmaxf(top, __shfl_xor(top, 32));
        const float scale = block_scale(top);
        if (row < p.end) {
          uint8_t* const to = (uint8_t*)a.y + row * a.gated + p.n0 + 4 * q;
#pragma unroll
          for (int i = 0; i < NF; i += 2) {
            const float w[8] = {v[i][0], v[i][1], v[i][2], v[i][3],
                                v[i + 1][0], v[i + 1][1], v[i + 1][2], v[i + 1][3]};
            const u32x2 c8 = codes8(w, scale);
            *(uint32_t*)(to + 16 * i) = c8.x;
            *(uint32_t*)(to + 16 * i + 16) = c8.y;
          }
          if (q == 0) a.ys[row * (a.gated / QW_BLOCK) + p.n0 / QW_BLOCK] = scale;
        }
      };
      if (wave / WM == 0)
        exchange(std::integral_constant<int, 0>{});
      else
        exchange(std::integral_constant<int, 1>{});
    } else {
#pragma unroll
      for (int j = 0; j < MF; ++j) {
        const int64_t row = p.m0 + wm + 16 * j + r;
        if (row >= p.end) continue;
#pragma unroll
        for (int i = 0; i < NF; ++i) {
          const int64_t col = p.n0 + wn + 16 * i + 4 * q;
          YT* y = (YT*)a.y + row * a.ldy + col;
          if (a.y_vec) {
            if (col < a.n) store4(y, acc[i][j]);
          } else {
#pragma unroll
            for (int c = 0; c < 4; ++c)
              if (col + c < a.n) store1(y + c, acc[i][j][c]);
          }
        }
      }
    }
    if (!more) return;
    at = at2;
    p = p2;
  }
}

// EXACT: the bf16 cores' instances too.
template <int NF, int MF, int WM, int STAGES, bool EXACT, bool GROUPED>
hipError_t run_tiled(GemmArgs a, const BlockGemm& g, hipStream_t stream) {
  constexpr int BN = 16 * NF * (kTileWaves / WM), BM = 16 * MF * WM;
  a.tiles_m = GROUPED ? std::min(a.m, (a.m + a.experts * (int64_t)(BM - 1)) / BM)
                      : (a.m + BM - 1) / BM;
  a.tiles = a.tiles_m * ((a.n + BN - 1) / BN);
  const unsigned grid = (unsigned)a.tiles;
  a.y_vec = g.n % 4 == 0 && aligned(g.y, g.y_type == QW_BF16 ? 8 : 16);
  auto go = [&](auto exact, auto brows1, auto y) {
    gemm_tiled<NF, MF, WM, STAGES, decltype(exact)::value, decltype(brows1)::value, GROUPED, false,
               decltype(y)><<<grid, kTileWaves * 64, 0, stream>>>(a);
  };
  using std::true_type;
  using std::false_type;
  const bool one = g.brows == 1;
  if (g.y_type == QW_BF16)
    one ? go(false_type{}, true_type{}, uint16_t{}) : go(false_type{}, false_type{}, uint16_t{});
  else if constexpr (EXACT) {
    if (g.exact) one ? go(true_type{}, true_type{}, 0.0f) : go(true_type{}, false_type{}, 0.0f);
  }
  if constexpr (GROUPED) {
    if (g.y_type == QW_F32 && !g.exact)
      one ? go(false_type{}, true_type{}, 0.0f) : go(false_type{}, false_type{}, 0.0f);
  }
  return hipGetLastError();
}

// ------------------------------------------------------------ stream kernel
//
// For up to 16 rows of x (or of x per expert): bound by reading the weight
// once.  Each of a block's WV waves owns KPW consecutive blocks of k.  It
// quantizes (or loads) its part of x once, keeps it in registers, and streams
// its part of 16 weight rows after 16 weight rows past it; a weight fragment
// is replaced by a later one as soon as its product is issued, so that RING
// fragments (2 KiB each) are always on their way.  The waves' sums meet in
// LDS, once per 16 rows.  Float x costs each block one pass over its own rows
// of x instead of a launch.

// Where the float values of a row of x come from.
enum Source {
  ROWS,    // x [rows][k]
  TOKENS,  // x [tokens][k], a row is that of its slot's token (order, topk)
  GATES,   // x [rows][2 k], a row is silu of its first half times its second
};

// This wave's part of float x as fragments: 16 lanes quantize a block of k of a
// row, as quantize_rows does, 4 rows and 2 blocks at a time; the codes change
// lanes through 4 KiB of LDS of the wave's own.
template <int KPW, Source SRC, bool VEC, typename T>
__device__ __forceinline__ void quantize_part(const GemmArgs& a, int64_t m0, int64_t end, int k0,
                                              uint8_t (*lds)[16][128], float (*scale)[16],
                                              int lane, i32x8* xf, float* sx) {
  const int r = lane & 15, q = lane >> 4;
#pragma unroll
  for (int g = 0; g < KPW; g += 2) {
    constexpr int W = 2;
    for (int64_t row = m0 + q; row - q < end; row += 4) {
      int64_t from = min(row, end - 1);
      if (SRC == TOKENS) from = max(a.order[from], 0) / a.topk;
      const T* x = (const T*)a.x + from * (SRC == GATES ? 2 * a.k : a.k);
      float v[W][8];
#pragma unroll
      for (int i = 0; i < W; ++i) {
        const int64_t j = (int64_t)(k0 + g + i) * QW_BLOCK + r * 8;
        load8_of_row<VEC>(x, j, a.k, v[i]);
        if constexpr (SRC == GATES) {
          float up[8];
          load8_of_row<VEC>(x + a.k, j, a.k, up);
          gated<8>(v[i], up, v[i]);
        }
      }
#pragma unroll
      for (int i = 0; i < W; ++i) {
        const float s = block_scale(max16(amax8(v[i])));
        *(u32x2_la*)&lds[i][(int)(row - m0)][r * 8] = codes8(v[i], s);
        scale[i][(int)(row - m0)] = s;
      }
    }
#pragma unroll
    for (int i = 0; i < W; ++i) {
      xf[g + i] = fragment(&lds[i][r][q * 16]);
      sx[g + i] = scale[i][r];
    }
  }
}

template <int KPW, int WV, bool EXACT, bool BROWS1, bool GROUPED, Source SRC, bool VEC,
          typename XT, typename YT>
__global__ __launch_bounds__(WV * 64) void gemm_stream(GemmArgs a) {
  __shared__ __align__(16) float part[2][WV][16][20];
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int lane = threadIdx.x & 63, r = lane & 15, q = lane >> 4;
  const int64_t chunk = blockIdx.x / a.tiles_m;
  int64_t m0 = blockIdx.x % a.tiles_m * 16, end = min(m0 + 16, a.m);
  int expert = 0;
  if (GROUPED && !grouped_tile(a, blockIdx.x % a.tiles_m, 16, expert, m0, end)) return;
  const int64_t tiles_n = (a.n + 15) / 16;
  const int k0 = wave * KPW;
  const uint8_t* wc = a.codes + expert * a.n * a.kp + q * 16;
  const float* ws = a.scales + expert * a.nb * a.kb;
  int koff[KPW];  // byte offset of this wave's blocks of k; the last one again behind the end
#pragma unroll
  for (int i = 0; i < KPW; ++i) koff[i] = min(k0 + i, a.kb - 1) * QW_BLOCK;
  constexpr int RING = KPW > 8 ? KPW / 2 : KPW;  // weight fragments on their way
  i32x8 w[RING];
  // scales of a tile: of the wave's blocks one per lane, or 4 rows' per lane
  float sw[BROWS1 ? KPW : 1][4];
  auto load = [&](int64_t tile, int i) {
    w[i % RING] = fragment(wc + min(tile * 16 + r, a.n - 1) * a.kp + koff[i]);
  };
  auto load_scales = [&](int64_t tile) {
    if constexpr (BROWS1) {
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        const float* row = ws + min(tile * 16 + 4 * q + c, a.n - 1) * a.kb;
#pragma unroll
        for (int i = 0; i < KPW; ++i) sw[i][c] = row[min(k0 + i, a.kb - 1)];
      }
    } else {
      sw[0][0] = ws[tile / (QW_BLOCK / 16) * a.kb + min(k0 + lane % KPW, a.kb - 1)];
    }
  };
  int64_t tile = chunk;
  load_scales(tile);
#pragma unroll
  for (int i = 0; i < RING; ++i) load(tile, i);
  i32x8 xf[KPW];
  float sx[KPW];
  if constexpr (is_codes<XT>::value) {
    const int64_t row = min(m0 + r, end - 1);
#pragma unroll
    for (int i = 0; i < KPW; ++i) {
      xf[i] = fragment((const uint8_t*)a.x + row * a.kp + q * 16 + koff[i]);
      sx[i] = a.xs[row * a.kb + min(k0 + i, a.kb - 1)];
    }
  } else {
    constexpr int W = 2;
    __shared__ __align__(16) uint8_t codes[WV][W][16][128];
    __shared__ float scale[WV][W][16];
    quantize_part<KPW, SRC, VEC, XT>(a, m0, end, k0, codes[wave], scale[wave], lane, xf, sx);
  }
  const bool have = m0 + r < end;
#pragma unroll
  for (int i = 0; i < KPW; ++i)
    if (!have || k0 + i >= a.kb) {
      xf[i] = i32x8{};
      sx[i] = 0.0f;
    }
  int buf = 0;
  auto step = [&](auto more) {
    constexpr bool MORE = decltype(more)::value;  // a tile after this one
    float s[BROWS1 ? KPW : 1][4];
#pragma unroll
    for (int i = 0; i < (BROWS1 ? KPW : 1); ++i)
#pragma unroll
      for (int c = 0; c < 4; ++c) s[i][c] = sw[i][c];
    if (MORE) load_scales(tile + a.chunks);
    f32x4 acc = {};
#pragma unroll
    for (int i = 0; i < KPW; ++i) {
      if (EXACT) asm volatile("" : "+v"(xf[i]));  // converted anew: as codes it takes half the registers
      const f32x4 d = dot128(Frag<EXACT>(w[i % RING]), Frag<EXACT>(xf[i]));
      if (i + RING < KPW)
        load(tile, i + RING);
      else if (MORE)
        load(tile + a.chunks, i + RING - KPW);
      const float one = BROWS1 ? 1.0f
                               : __int_as_float(__builtin_amdgcn_readlane(__float_as_int(s[0][0]), i));
#pragma unroll
      for (int c = 0; c < 4; ++c)
        acc[c] = __builtin_fmaf(d[c], sx[i] * (BROWS1 ? s[BROWS1 ? i : 0][c] : one), acc[c]);
    }
    *(f32x4*)&part[buf][wave][r][4 * q] = acc;
    // The weight's loads stay on their way.  One barrier a tile: the other
    // buffer is written next, and read no later than the next barrier.
    lds_barrier();
    const int t = threadIdx.x >> 4, c = threadIdx.x & 15;
    if (t < 16 && m0 + t < end && tile * 16 + c < a.n) {
      float sum = part[buf][0][t][c];
#pragma unroll
      for (int v = 1; v < WV; ++v) sum += part[buf][v][t][c];
      store1((YT*)a.y + (m0 + t) * a.ldy + tile * 16 + c, sum);
    }
    buf ^= 1;
  };
  for (; tile + a.chunks < tiles_n; tile += a.chunks) step(std::true_type{});
  step(std::false_type{});
}

constexpr int kStreamWaves = 8;

template <int KPW, bool GROUPED, Source SRC, bool VEC, typename XT>
hipError_t run_stream(GemmArgs a, const BlockGemm& g, hipStream_t stream) {
  a.tiles_m = GROUPED ? std::min(a.m, (a.m + a.experts * (int64_t)15) / 16) : (a.m + 15) / 16;
  const int64_t tiles_n = (a.n + 15) / 16;
  // two blocks a compute unit where the registers allow it
  const int64_t want = KPW <= 4 ? 512 : 256;
  a.chunks = std::min(tiles_n, std::max<int64_t>(1, (want + a.tiles_m - 1) / a.tiles_m));
  const unsigned grid = (unsigned)(a.chunks * a.tiles_m);
  auto go = [&](auto exact, auto brows1, auto y) {
    gemm_stream<KPW, kStreamWaves, decltype(exact)::value, decltype(brows1)::value, GROUPED, SRC,
                VEC, XT, decltype(y)><<<grid, kStreamWaves * 64, 0, stream>>>(a);
  };
  using std::true_type;
  using std::false_type;
  const bool one = g.brows == 1;
  // fp32 results on the bf16 cores, asked for or not: they wait for memory either way
  if (g.y_type == QW_F32) {
    one ? go(true_type{}, true_type{}, 0.0f) : go(true_type{}, false_type{}, 0.0f);
  } else if constexpr (!GROUPED || is_codes<XT>::value) {
    one ? go(false_type{}, true_type{}, uint16_t{}) : go(false_type{}, false_type{}, uint16_t{});
  }
  return hipGetLastError();
}

// The stream kernel quantizes x itself up to this many rows, and up to this many
// of a wave's blocks over all rows: every block of the grid pays for it (4096 x
// 4096: 8.5 us at 1 row, 11.3 at 8, 16.8 at 16; with codes 6.4, 7.3 and 8.0, and
// 2.8 and a launch for a kernel that makes them; 28672 x 8192 at 8 rows 51.9
// against 45.6 with that kernel).
constexpr int kFusedMaxM = 8, kFusedBlocks = 32;
// Most blocks of k that the stream kernel's waves hold.  (From 9 a wave on, with a
// scale to every weight row, the scales do not all fit the registers: 17 to 57 of them
// go through memory, and 4096 x 11008 at 1 row takes 27.0 us, with 128 x 128 blocks 20.7.)
constexpr int kStreamMaxKb = 12 * kStreamWaves;

template <bool GROUPED, Source SRC, bool VEC, typename XT>
hipError_t run_stream(const GemmArgs& a, const BlockGemm& g, hipStream_t stream) {
  const int each = (a.kb + kStreamWaves - 1) / kStreamWaves;
  if (each <= 2) return run_stream<2, GROUPED, SRC, VEC, XT>(a, g, stream);
  if (each <= 4) return run_stream<4, GROUPED, SRC, VEC, XT>(a, g, stream);
  if (each <= 8) return run_stream<8, GROUPED, SRC, VEC, XT>(a, g, stream);
  return run_stream<12, GROUPED, SRC, VEC, XT>(a, g, stream);
}

GemmArgs args_of(const BlockGemm& g) {
  GemmArgs a = {};
  a.codes = g.codes;
  a.scales = g.scales;
  a.x = g.x_type < 0 ? (const void*)g.xc : g.x;
  a.xs = g.xs;
  a.y = g.y;
  a.n = a.ldy = g.n;
  a.k = g.k;
  a.m = g.m;
  a.kp = pitch(g.k);
  a.kb = (int)(a.kp / QW_BLOCK);
  a.nb = (g.n + g.brows - 1) / g.brows;
  return a;
}

// ---------------------------------------------------------------- choice
//
// Which kernel and tile: the one with the least estimated time, from what each
// takes for a round of the 256 compute units.
//   tiled   a block of k takes `step` us with all units at work (weight rows x
//           tokens): 256 x 256 1.84, 256 x 128 1.06, 128 x 256 1.07, 128 x 128
//           0.70, 128 x 64 0.55, 64 x 64 0.40; on the bf16 cores 1.78 (128 x
//           256), 1.16, 0.84 and 0.62, the larger tiles not fitting the
//           registers (from 8192^3: 470, 540, 550, 700 us and 910, 1180; 512 x
//           4096 x 4096: 24.7, 19.7, 23.3 us for the last three; 37, 29, 33).
//           3 us to start and to write y.
//   direct  a unit takes in 28 KB of scattered rows a us, and 4 us to start,
//           to join the sums and to write (64 x 4096 x 4096: 13 us with 32 x 32
//           tiles, 16 tiled; 32 x 4096 x 4096: 11.5 with 16 x 32, 13 with 32 x
//           32; 256 x 4096 x 4096: 41, tiled 16).
// A tiled product whose last round is only partly filled may be cut in two along
// the weight rows, the rest with smaller tiles (2048 x 28672 x 8192: 3.5 rounds
// of 256 x 256, 454 us; 3 rounds and one of 256 x 128, 442 us; of ten other sizes
// cut by the rule none is slower than whole, and the smallest gain is 68.4 -> 67.5
// us), for 2 us of a second launch.
// Grouped: an expert's last tile is half empty on average.
//
// Limits beside the estimate (us, the first side's and then the other's):
//   16 rows of x to the stream kernel: one fragment of x.  4096 x 4096 at 16 rows 8.0
//     and 9.7 (tiles), at 17 11.6 and 9.6; 28672 x 8192 46.6 and 53.1, 71.2 and 53.0;
//     4096 x 11008 18.3 and 17.6, 21.5 and 17.7.
//   16 rows an expert on average: its fragment again, though experts differ in size.
//     8 and 16 rows of 64 experts of 2816 x 4096, bf16 150 and 146, 173 and 170, fp32
//     151 and 183, 172 and 188, at 24 204 and 166, 201 and 212; 8 experts at 16 rows
//     29.3 and 19.7, 28.5 and 28.2.  Too many for short rows and bf16: 4096 x 1408 at 8
//     and 16 rows 92 and 86, 146 and 88, fp32 93 and 110, 149 and 122.
struct Shape {
  int bn, bm;   // weight rows x tokens of a tile
  bool tiled;
  double step;  // tiled, 8-bit cores
  double exact; // tiled, bf16 cores; 0: not taken
};
constexpr Shape kShapes[] = {
    {256, 256, true, 1.84, 0.0}, {256, 128, true, 1.06, 0.0},  {128, 256, true, 1.07, 1.78},
    {128, 128, true, 0.70, 1.16}, {128, 64, true, 0.55, 0.84}, {64, 64, true, 0.40, 0.62},
    {32, 32, false, 0.0, 0.0},    {16, 32, false, 0.0, 0.0},
};
constexpr int kShapeCount = sizeof(kShapes) / sizeof(kShapes[0]);

// The kernels beside kShapes: the stream kernel, and the direct one's 16 x 16 tiles.
enum { kStream = -1, kDirect16 = -2 };

// Estimated us of n weight rows against m rows of x (of `experts` experts); the
// tiled kernel takes a block of k at least, and a tile with each thread block.
double cost_of(const Shape& s, int64_t n, int64_t m, int64_t experts, int kb, bool exact) {
  const int64_t spare = std::min(experts, m) / 2;  // half-empty tiles
  const double tiles_m = experts ? (double)m / s.bm + spare + 1 : (double)((m + s.bm - 1) / s.bm);
  const double tiles_n = (double)((n + s.bn - 1) / s.bn);
  const double rounds = std::ceil(tiles_m * tiles_n / kUnits);
  if (!s.tiled) return 4.0 + rounds * (s.bn + s.bm) * kb * (QW_BLOCK / 28000.0);
  const int64_t most = experts ? std::min(m, m / s.bm + experts) : (int64_t)tiles_m;
  if (kb == 0 || most * tiles_n > 1 << 22) return 1e30;
  const double step = exact ? s.exact : s.step;
  return step == 0.0 ? 1e30 : rounds * (3.0 + kb * step);
}

int best_shape(int64_t n, int64_t m, int64_t experts, int kb, bool exact, double* cost) {
  int best = 0;
  *cost = 1e30;
  for (int i = 0; i < kShapeCount; ++i) {
    const double c = cost_of(kShapes[i], n, m, experts, kb, exact);
    if (c < *cost) {
      *cost = c;
      best = i;
    }
  }
  return best;
}

// How a product is run: with one shape, or (cut > 0) with `shape` up to weight row
// `cut` and with `rest` from there on.
struct Plan {
  int shape, rest;
  int64_t cut;
};

Plan plan_of(int64_t n, int64_t m, int kb, bool exact) {
  if (m <= 16) return {kb > 0 && kb <= kStreamMaxKb ? kStream : kDirect16, 0, 0};
  double cost;
  const int shape = best_shape(n, m, 0, kb, exact, &cost);
  const Shape& s = kShapes[shape];
  if (!s.tiled) return {shape, 0, 0};
  // the weight rows of whole rounds, and the rest with another shape; the cut lies
  // between blocks of 128 rows, which share a scale (a tile of 64 is half of one)
  const int64_t tiles_m = (m + s.bm - 1) / s.bm, tiles_n = (n + s.bn - 1) / s.bn;
  const int64_t whole = tiles_m * tiles_n / kUnits * kUnits / tiles_m;
  const int64_t cut = whole * s.bn / QW_BLOCK * QW_BLOCK;
  if (cut > 0 && cut < n) {
    double rest;
    const int other = best_shape(n - cut, m, 0, kb, exact, &rest);
    if (cost_of(s, cut, m, 0, kb, exact) + rest + 2.0 < cost) return {shape, other, cut};
  }
  return {shape, 0, 0};
}

int grouped_plan(int64_t n, int64_t m, int64_t experts, int kb, bool exact) {
  // an average of 16 rows an expert: each expert's weight is read about once
  if (m <= 16 * experts && kb > 0 && kb <= kStreamMaxKb) return kStream;
  double cost;
  return best_shape(n, m, experts, kb, exact, &cost);
}

template <bool GROUPED>
hipError_t run_shape(int shape, const GemmArgs& a, const BlockGemm& g, hipStream_t stream) {
  switch (shape) {
    case 0: return run_tiled<8, 4, 4, 2, false, GROUPED>(a, g, stream);
    case 1: return run_tiled<8, 2, 4, 3, false, GROUPED>(a, g, stream);
    case 2: return run_tiled<4, 4, 4, 3, true, GROUPED>(a, g, stream);
    case 3: return run_tiled<4, 2, 4, 4, true, GROUPED>(a, g, stream);
    case 4: return run_tiled<2, 2, 2, 4, true, GROUPED>(a, g, stream);
    case 5: return run_tiled<1, 2, 2, 4, true, GROUPED>(a, g, stream);
    case 6: return run_direct<2, 2, 8, 1, GROUPED>(a, g, stream);
    default: return run_direct<1, 2, 8, 2, GROUPED>(a, g, stream);
  }
}

hipError_t run_gated(GemmArgs a, const BlockGemm& g, hipStream_t stream) {
  constexpr int BM = 128;
  a.tiles_m = std::min(a.m, (a.m + a.experts * (int64_t)(BM - 1)) / BM);
  a.tiles = a.tiles_m * (a.gated / QW_BLOCK);
  const unsigned grid = (unsigned)std::min<int64_t>(a.tiles, kUnits);
  if (g.brows == 1)
    gemm_tiled<8, 2, 4, 3, false, true, true, true, float>
        <<<grid, kTileWaves * 64, 0, stream>>>(a);
  else
    gemm_tiled<8, 2, 4, 3, false, false, true, true, float>
        <<<grid, kTileWaves * 64, 0, stream>>>(a);
  return hipGetLastError();
}

// Weight rows [from, from + count) of a product.
GemmArgs part_of(GemmArgs a, const BlockGemm& g, int64_t from, int64_t count) {
  a.codes += from * a.kp;
  a.scales += from / g.brows * a.kb;
  a.y = (char*)a.y + from * (g.y_type == QW_BF16 ? 2 : 4);
  a.n = count;
  a.nb = (count + g.brows - 1) / g.brows;
  return a;
}

}  // namespace

bool block_gemm_fuses(int64_t m, int64_t k) {
  const int64_t each = (pitch(k) / QW_BLOCK + kStreamWaves - 1) / kStreamWaves;
  return m <= kFusedMaxM && pitch(k) <= kStreamMaxKb * QW_BLOCK && m * each <= kFusedBlocks;
}

hipError_t launch_block_gemm(const BlockGemm& g, hipStream_t stream) {
  const GemmArgs a = args_of(g);
  if (g.x_type >= 0) {
    const bool vec = g.k % 8 == 0 && aligned(g.x, 16);
    if (g.x_type == QW_F32)
      return vec ? run_stream<false, ROWS, true, float>(a, g, stream)
                 : run_stream<false, ROWS, false, float>(a, g, stream);
    return vec ? run_stream<false, ROWS, true, uint16_t>(a, g, stream)
               : run_stream<false, ROWS, false, uint16_t>(a, g, stream);
  }
  const Plan plan = plan_of(g.n, g.m, a.kb, g.exact);
  if (plan.shape == kStream) return run_stream<false, ROWS, true, uint8_t>(a, g, stream);
  if (plan.shape == kDirect16) return run_direct<1, 1, 8, 4, false>(a, g, stream);
  if (plan.cut == 0) return run_shape<false>(plan.shape, a, g, stream);
  const hipError_t e = run_shape<false>(plan.shape, part_of(a, g, 0, plan.cut), g, stream);
  if (e != hipSuccess) return e;
  return run_shape<false>(plan.rest, part_of(a, g, plan.cut, g.n - plan.cut), g, stream);
}

hipError_t launch_block_gemm_grouped(const BlockGemm& g, int64_t experts,
                                     const int32_t* offsets, hipStream_t stream) {
  GemmArgs a = args_of(g);
  a.experts = (int)experts;
  a.offsets = offsets;
  const int shape = grouped_plan(g.n, g.m, experts, a.kb, g.exact);
  if (shape == kStream) return run_stream<true, ROWS, true, uint8_t>(a, g, stream);
  return run_shape<true>(shape, a, g, stream);
}

namespace {
int path_of(int shape) {
  if (shape == kStream) return 1;
  return shape == kDirect16 ? 16016 : kShapes[shape].bn * 1000 + kShapes[shape].bm;
}
}  // namespace

int block_gemm_path(int64_t n, int64_t m, int64_t k, bool exact, bool rest) {
  const Plan p = plan_of(n, m, (int)(pitch(k) / QW_BLOCK), exact);
  return rest ? p.cut > 0 ? path_of(p.rest) : 0 : path_of(p.shape);
}

int block_gemm_grouped_path(int64_t n, int64_t m, int64_t k, int64_t experts, bool exact) {
  return path_of(grouped_plan(n, m, experts, (int)(pitch(k) / QW_BLOCK), exact));
}

// Few rows an expert: what a block of the stream kernel spends on quantizing them
// is less than a kernel of its own (us of the MLP with 64 experts of 4096 x 1408, fused
// and not: 200 and 229 at 2 rows an expert, 231 and 267 at 4, 269 and 267 at 8; 2048 x
// 1408 115 and 151, 133 and 136, 150 and 151; 8 experts of 4096 x 1408 38 and 40 at 1
// row, 51 and 47 at 4).
bool block_gemm_grouped_fuses(int64_t rows, int64_t experts, int64_t k) {
  return rows <= 4 * experts && k > 0 && pitch(k) <= kStreamMaxKb * QW_BLOCK;
}

hipError_t launch_block_gemm_tokens(const BlockGemm& g, int64_t experts, const int32_t* offsets,
                                    const int32_t* order, int64_t topk, hipStream_t stream) {
  GemmArgs a = args_of(g);
  a.experts = (int)experts;
  a.offsets = offsets;
  a.order = order;
  a.topk = (int)topk;
  const bool vec = g.k % 8 == 0 && aligned(g.x, 16);
  if (g.x_type == QW_F32)
    return vec ? run_stream<true, TOKENS, true, float>(a, g, stream)
               : run_stream<true, TOKENS, false, float>(a, g, stream);
  return vec ? run_stream<true, TOKENS, true, uint16_t>(a, g, stream)
             : run_stream<true, TOKENS, false, uint16_t>(a, g, stream);
}

hipError_t launch_block_gemm_gates(const BlockGemm& g, int64_t experts, const int32_t* offsets,
                                   hipStream_t stream) {
  GemmArgs a = args_of(g);
  a.experts = (int)experts;
  a.offsets = offsets;
  return g.k % 8 == 0 ? run_stream<true, GATES, true, float>(a, g, stream)
                      : run_stream<true, GATES, false, float>(a, g, stream);
}

// From 64 rows an expert on the tiles are filled well enough (us of the MLP, gated in
// the product and not: 64 experts of 2048 x 1408 171 and 176 at 32 rows an expert, 201
// and 214 at 65, 251 and 308 at 128; 8 experts of 4096 x 1408 70 and 62, 71 and 83, 79
// and 84); the blocks of the result have to be blocks of the weight's rows (f = 0 has
// no tile to launch).
bool block_gemm_gates(int64_t rows, int64_t experts, int64_t f, int64_t k) {
  return rows > 64 * experts && f > 0 && f % QW_BLOCK == 0 && k > 0;
}

hipError_t launch_block_gemm_gated(const BlockGemm& g, int64_t experts, const int32_t* offsets,
                                   float* ys, hipStream_t stream) {
  GemmArgs a = args_of(g);
  a.experts = (int)experts;
  a.offsets = offsets;
  a.gated = g.n / 2;
  a.ys = ys;
  return run_gated(a, g, stream);
}

}  // namespace qw
