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
//     rounding of y to bf16 is 2^-9.
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
  const int32_t* offsets;
  int experts;
  int64_t n, k, m;
  int64_t kp;
  int kb;             // blocks along k
  int64_t nb;         // rows of scales of one weight
  int64_t tiles_m, tiles;
  int s_vec;          // 4 scales of a row may be loaded as one
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

__device__ __forceinline__ i32x8 fragment(const uint8_t* p) {
  const u32x4 lo = *(const u32x4*)p, hi = *(const u32x4*)(p + 64);
  return i32x8{(int)lo.x, (int)lo.y, (int)lo.z, (int)lo.w,
               (int)hi.x, (int)hi.y, (int)hi.z, (int)hi.w};
}

// Rows [row, end) of the tm-th tile of `bm` rows, counted expert by expert;
// false when there are fewer tiles.  The whole wave calls it.
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
    const int total = __shfl(upto, 63);
    if (tm < before + total) {
      const int l = __builtin_ctzll(__ballot(tm < before + upto));
      expert = c + l;
      row = __shfl(lo, l) + (tm - before - (__shfl(upto, l) - __shfl(tiles, l))) * bm;
      end = min((int64_t)__shfl(hi, l), row + bm);
      return true;
    }
    before += total;
  }
  return false;
}

// The x fragment of one lane from float values: 32 values of token row p (its
// 1 x 128 block at j), quantized with the block's scale, which the 4 lanes of
// the token find together.
template <bool VEC, typename T>
__device__ __forceinline__ i32x8 quantized_fragment(const T* row, int64_t j, int64_t k, int q,
                                                    bool have, float& s) {
  float v[4][8];
  float m = 0.0f;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int64_t at = j + (i >> 1) * 64 + 16 * q + (i & 1) * 8;
    if (have) {
      load8_of_row<VEC>(row, at, k, v[i]);
    } else {
#pragma unroll
      for (int c = 0; c < 8; ++c) v[i][c] = 0.0f;
    }
    m = fmaxf(m, amax8(v[i]));
  }
  m = fmaxf(m, __shfl_xor(m, 16));
  m = fmaxf(m, __shfl_xor(m, 32));
  s = block_scale(m);
  i32x8 f;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const u32x2 c = codes8(v[i], s);
    f[2 * i] = (int)c.x;
    f[2 * i + 1] = (int)c.y;
  }
  return f;
}

template <typename XT> struct is_codes { static constexpr bool value = false; };
template <> struct is_codes<uint8_t> { static constexpr bool value = true; };

// A block computes 16 NT weight rows x 16 MT tokens; its WV waves take every
// WV-th block of k, straight from memory into registers, and add their sums
// through LDS.
template <int NT, int MT, int WV, bool EXACT, bool BROWS1, bool GROUPED, bool VEC, typename XT,
          typename YT>
__global__ __launch_bounds__(WV * 64) void gemm_direct(GemmArgs a) {
  constexpr int BN = 16 * NT, BM = 16 * MT, LD = BN + 4;
  __shared__ float part[WV][BM][LD];
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int lane = threadIdx.x & 63, r = lane & 15, q = lane >> 4;
  for (int64_t tile = blockIdx.x; tile < a.tiles; tile += gridDim.x) {
    const int64_t n0 = tile / a.tiles_m * BN;
    int64_t m0 = tile % a.tiles_m * BM, end = min(m0 + BM, a.m);
    int expert = 0;
    if (GROUPED && !grouped_tile(a, tile % a.tiles_m, BM, expert, m0, end)) continue;
    const uint8_t* wc = a.codes + expert * a.n * a.kp + q * 16;
    const float* ws = a.scales + expert * a.nb * a.kb;
    const uint8_t* wp[NT];
#pragma unroll
    for (int i = 0; i < NT; ++i) wp[i] = wc + min(n0 + 16 * i + r, a.n - 1) * a.kp;
    const float* wsp[NT][4];
#pragma unroll
    for (int i = 0; i < NT; ++i)
#pragma unroll
      for (int c = 0; c < 4; ++c)
        wsp[i][c] = BROWS1 ? ws + min(n0 + 16 * i + 4 * q + c, a.n - 1) * a.kb
                           : ws + n0 / QW_BLOCK * a.kb;
    const XT* xp[MT];
    const float* sxp[MT];
    bool have[MT];
#pragma unroll
    for (int j = 0; j < MT; ++j) {
      const int64_t row = min(m0 + 16 * j + r, end - 1);
      have[j] = m0 + 16 * j + r < end;
      if constexpr (is_codes<XT>::value) {
        xp[j] = (const XT*)a.x + row * a.kp + q * 16;
        sxp[j] = a.xs + row * a.kb;
      } else {
        xp[j] = (const XT*)a.x + row * a.k;
        sxp[j] = nullptr;
      }
    }
    f32x4 acc[NT][MT] = {};
    for (int b = wave; b < a.kb; b += WV) {
      Frag<EXACT> wf[NT];
#pragma unroll
      for (int i = 0; i < NT; ++i) wf[i] = Frag<EXACT>(fragment(wp[i] + (int64_t)b * QW_BLOCK));
#pragma unroll
      for (int j = 0; j < MT; ++j) {
        float sx;
        i32x8 xc;
        if constexpr (is_codes<XT>::value) {
          xc = fragment(xp[j] + (int64_t)b * QW_BLOCK);
          sx = sxp[j][b];
        } else {
          xc = quantized_fragment<VEC>(xp[j], (int64_t)b * QW_BLOCK, a.k, q, have[j], sx);
        }
        const Frag<EXACT> xf(xc);
#pragma unroll
        for (int i = 0; i < NT; ++i) {
          const f32x4 d = dot128(wf[i], xf);
#pragma unroll
          for (int c = 0; c < 4; ++c)
            acc[i][j][c] = __builtin_fmaf(d[c], sx * wsp[i][c][b], acc[i][j][c]);
        }
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
        for (int w = 1; w < WV; ++w) s += part[w][t][c];
        store1((YT*)a.y + (m0 + t) * a.n + n0 + c, s);
      }
    }
  }
}

template <int NT, int MT, int WV, bool GROUPED, bool VEC, typename XT>
hipError_t run_direct(GemmArgs a, const BlockGemm& g, hipStream_t stream) {
  constexpr int BN = 16 * NT, BM = 16 * MT;
  a.tiles_m = GROUPED ? std::min(a.m, (a.m + a.experts * (int64_t)(BM - 1)) / BM)
                      : (a.m + BM - 1) / BM;
  a.tiles = a.tiles_m * ((a.n + BN - 1) / BN);
  // a launch holds fewer than 2^32 threads: the kernel's loop takes the rest
  const unsigned grid = (unsigned)std::min<int64_t>(a.tiles, 1 << 21);
  auto go = [&](auto exact, auto brows1, auto y) {
    gemm_direct<NT, MT, WV, decltype(exact)::value, decltype(brows1)::value, GROUPED, VEC, XT,
                decltype(y)><<<grid, WV * 64, 0, stream>>>(a);
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
// For many rows.  A block of 8 waves computes 16 NF * 2 weight rows x 16 MF * 4
// tokens, one block of k at a time through two LDS buffers: while the matrix
// cores work on one, the next is copied to the other straight from memory
// (buffer loads with an LDS target, 16 bytes a lane).  Waves form a grid of 4 along the tokens
// and 2 along the weight; each keeps its MF token fragments in registers and
// walks its NF weight fragments.
//
// LDS rows are the 128 bytes of a block.  A phase of a 16-byte LDS read is 16
// lanes, here 16 consecutive rows at the same place in the row, and the 64
// banks hold 2 rows: piece c of row r is kept at c ^ (r / 2 % 8), so that the
// 16 lanes meet 16 different places.  The copy writes LDS in lane order, so
// the lanes fetch the pieces in that order from memory.

constexpr int kTileWaves = 8;

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
// This wave's copies and LDS accesses are done, and so are the block's.
__device__ __forceinline__ void landed() {
  asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)\n\ts_barrier" ::: "memory");
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

template <int NF, int MF, bool EXACT, bool BROWS1, bool GROUPED, typename YT>
__global__ __launch_bounds__(kTileWaves * 64, 2) void gemm_tiled(GemmArgs a) {
  constexpr int BN = 32 * NF, BM = 64 * MF, ROWS = BN + BM;
  constexpr int SEGS = ROWS / 8 / kTileWaves;  // 8-row pieces of a wave
  static_assert(QW_BLOCK % (16 * NF) == 0, "a wave's weight rows lie in one 128 x 128 block");
  static_assert(ROWS / 8 % kTileWaves == 0 && MF % 2 == 0, "whole pieces and pairs");
  __shared__ __align__(1024) uint8_t lds[2][ROWS * 128];
  // scales of 4 blocks of k at a time (a scale's line of memory holds its
  // row's next ones), of the tile's tokens and then of its rows of blocks
  constexpr int WROWS = BROWS1 ? BN : 2;
  __shared__ __align__(16) float scales[2][4][BM + WROWS];
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int lane = threadIdx.x & 63, r = lane & 15, q = lane >> 4;
  const int wm = (wave & 3) * 16 * MF, wn = (wave >> 2) * 16 * NF;
  int64_t tm, tn;
  tile_place(blockIdx.x, a.tiles, a.tiles_m, tm, tn);
  const int64_t n0 = tn * BN;
  int64_t m0 = tm * BM, end = min(m0 + BM, a.m);
  int expert = 0;
  if (GROUPED && !grouped_tile(a, tm, BM, expert, m0, end)) return;
  const int kp = (int)a.kp;
  const i32x4 wbuf = buffer_of(a.codes + (expert * a.n + n0) * a.kp,
                               (uint32_t)(min(a.n - n0, (int64_t)BN) * a.kp));
  const i32x4 xbuf = buffer_of((const uint8_t*)a.x + m0 * a.kp, (uint32_t)((end - m0) * a.kp));
  const float* ws = a.scales + expert * a.nb * a.kb;
  const int t = threadIdx.x;
  const float* my_scales =
      t < BM ? a.xs + min(m0 + t, end - 1) * a.kb
             : ws + (BROWS1 ? min(n0 + t - BM, a.n - 1) : min(n0 / QW_BLOCK + t - BM, a.nb - 1)) * a.kb;
  uint32_t voff[SEGS];
#pragma unroll
  for (int s = 0; s < SEGS; ++s) {
    const int row = (wave + kTileWaves * s) * 8 + (lane >> 3);
    const int c = (lane & 7) ^ ((row >> 1) & 7);
    voff[s] = (uint32_t)(row < BN ? row : row - BN) * kp + c * 16;
  }
  const uint32_t lds0 = (uint32_t)(uintptr_t)(__attribute__((address_space(3))) uint8_t*)&lds[0][0];
  auto fetch = [&](int b, int buf) {
#pragma unroll
    for (int s = 0; s < SEGS; ++s) {
      const int seg = wave + kTileWaves * s;
      copy_to_lds(seg * 8 < BN ? wbuf : xbuf, voff[s], (uint32_t)b * 128,
                  lds0 + buf * (ROWS * 128) + seg * 1024);
    }
  };
  f32x4 acc[NF][MF] = {};
  if (a.kb > 0) {
    float s4[4];
    auto load_scales = [&](int b) {
      if (t >= BM + WROWS) return;
      if (a.s_vec) {
        const f32x4 v = *(const f32x4*)(my_scales + b);
#pragma unroll
        for (int c = 0; c < 4; ++c) s4[c] = v[c];
      } else {
#pragma unroll
        for (int c = 0; c < 4; ++c) s4[c] = my_scales[min(b + c, a.kb - 1)];
      }
    };
    auto keep_scales = [&](int b) {
      if (t >= BM + WROWS) return;
#pragma unroll
      for (int c = 0; c < 4; ++c) scales[(b >> 2) & 1][c][t] = s4[c];
    };
    // The scales that block b's products are multiplied with: read from LDS
    // with the first fragments, joined behind the first products.
    float s[MF], sx[MF], sw = 1.0f;
    auto take_scales = [&](int b) {
      const float* sc = scales[(b >> 2) & 1][b & 3];
      if (!BROWS1) sw = sc[BM + (int)((n0 + wn) / QW_BLOCK - n0 / QW_BLOCK)];
#pragma unroll
      for (int j = 0; j < MF; ++j) sx[j] = sc[wm + 16 * j + r];
    };
    load_scales(0);
    fetch(0, 0);
    keep_scales(0);
    landed();
    if (a.kb > 1) fetch(1, 1);
    take_scales(0);
    Frag<EXACT> xf[MF];
#pragma unroll
    for (int j = 0; j < MF; ++j)
      xf[j] = Frag<EXACT>(lds_fragment(lds[0] + (BN + wm) * 128, 16 * j + r, q));
    i32x8 next = lds_fragment(lds[0] + wn * 128, r, q);
    // a pair of products is scaled and added while the next pair runs on the
    // matrix cores: d with the scales ps (and psw) is the last pair
    f32x4 d[2] = {}, psw = {};
    float ps[2] = {};
    for (int b = 0; b < a.kb; ++b) {
      const int buf = b & 1;
      const uint8_t* wl = lds[buf] + wn * 128;
      const bool more = (b & 3) == 0 && b + 4 < a.kb;
      if (more) load_scales(b + 4);
      f32x4 sw4 = {};
#pragma unroll
      for (int i = 0; i < NF; ++i) {
        const Frag<EXACT> wf(next);
        if constexpr (BROWS1) sw4 = *(const f32x4*)&scales[(b >> 2) & 1][b & 3][BM + wn + 16 * i + 4 * q];
        if (i + 1 < NF) {
          next = lds_fragment(wl, 16 * (i + 1) + r, q);
        } else {
          // The wave holds all that it needs of this buffer: once every wave
          // does, it takes the copy after next; and the other buffer is whole.
          landed();
          if (more) keep_scales(b + 4);  // these have landed too
          if (b + 2 < a.kb) fetch(b + 2, buf);
          next = lds_fragment(lds[buf ^ 1] + wn * 128, r, q);
        }
#pragma unroll
        for (int j = 0; j < MF; j += 2) {
          f32x4 e[2];
#pragma unroll
          for (int u = 0; u < 2; ++u) {
            e[u] = dot128(wf, xf[j + u]);
            if (i == NF - 1)
              xf[j + u] = Frag<EXACT>(lds_fragment(lds[buf ^ 1] + (BN + wm) * 128, 16 * (j + u) + r, q));
          }
          f32x4* to = j > 0 ? &acc[i][j - 2] : &acc[i > 0 ? i - 1 : NF - 1][MF - 2];
#pragma unroll
          for (int u = 0; u < 2; ++u) {
#pragma unroll
            for (int c = 0; c < 4; ++c)
              to[u][c] = __builtin_fmaf(d[u][c], BROWS1 ? ps[u] * psw[c] : ps[u], to[u][c]);
            asm volatile("" : "+v"(to[u]));  // here, not after all the products
          }
#pragma unroll
          for (int u = 0; u < 2; ++u) {
            __builtin_amdgcn_sched_group_barrier(0x8, EXACT ? 4 : 1, 0);
            __builtin_amdgcn_sched_group_barrier(0x2, (BROWS1 ? 8 : 4) + (EXACT ? 8 : 0), 0);
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
    }
#pragma unroll
    for (int u = 0; u < 2; ++u)
#pragma unroll
      for (int c = 0; c < 4; ++c)
        acc[NF - 1][MF - 2 + u][c] = __builtin_fmaf(
            d[u][c], BROWS1 ? ps[u] * psw[c] : ps[u], acc[NF - 1][MF - 2 + u][c]);
  }
#pragma unroll
  for (int j = 0; j < MF; ++j) {
    const int64_t row = m0 + wm + 16 * j + r;
    if (row >= end) continue;
#pragma unroll
    for (int i = 0; i < NF; ++i) {
      const int64_t col = n0 + wn + 16 * i + 4 * q;
      YT* y = (YT*)a.y + row * a.n + col;
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

template <int NF, int MF, bool GROUPED>
hipError_t run_tiled(GemmArgs a, const BlockGemm& g, hipStream_t stream) {
  constexpr int BN = 32 * NF, BM = 64 * MF;
  a.tiles_m = GROUPED ? std::min(a.m, (a.m + a.experts * (int64_t)(BM - 1)) / BM)
                      : (a.m + BM - 1) / BM;
  a.tiles = a.tiles_m * ((a.n + BN - 1) / BN);
  a.s_vec = a.kb % 4 == 0 && aligned(a.xs, 16) && aligned(a.scales, 16);
  a.y_vec = g.n % 4 == 0 && aligned(g.y, g.y_type == QW_BF16 ? 8 : 16);
  auto go = [&](auto exact, auto brows1, auto y) {
    gemm_tiled<NF, MF, decltype(exact)::value, decltype(brows1)::value, GROUPED, decltype(y)>
        <<<(unsigned)a.tiles, kTileWaves * 64, 0, stream>>>(a);
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

GemmArgs args_of(const BlockGemm& g) {
  GemmArgs a = {};
  a.codes = g.codes;
  a.scales = g.scales;
  a.x = g.x_type < 0 ? (const void*)g.xc : g.x;
  a.xs = g.xs;
  a.y = g.y;
  a.n = g.n;
  a.k = g.k;
  a.m = g.m;
  a.kp = pitch(g.k);
  a.kb = (int)(a.kp / QW_BLOCK);
  a.nb = (g.n + g.brows - 1) / g.brows;
  return a;
}

}  // namespace

hipError_t launch_block_gemm(const BlockGemm& g, hipStream_t stream) {
  const GemmArgs a = args_of(g);
  if (g.x_type >= 0) {
    const bool vec = g.k % 8 == 0 && aligned(g.x, 16);
    if (g.x_type == QW_F32)
      return vec ? run_direct<1, 1, 8, false, true, float>(a, g, stream)
                 : run_direct<1, 1, 8, false, false, float>(a, g, stream);
    return vec ? run_direct<1, 1, 8, false, true, uint16_t>(a, g, stream)
               : run_direct<1, 1, 8, false, false, uint16_t>(a, g, stream);
  }
  if (g.m <= 16) return run_direct<1, 1, 8, false, true, uint8_t>(a, g, stream);
  if (g.m > 128) return run_tiled<8, 4, false>(a, g, stream);
  return run_direct<4, 4, 4, false, true, uint8_t>(a, g, stream);
}

hipError_t launch_block_gemm_grouped(const BlockGemm& g, int64_t experts,
                                     const int32_t* offsets, hipStream_t stream) {
  GemmArgs a = args_of(g);
  a.experts = (int)experts;
  a.offsets = offsets;
  if (g.m <= 16 * experts) return run_direct<1, 1, 8, true, true, uint8_t>(a, g, stream);
  return run_direct<4, 4, 4, true, true, uint8_t>(a, g, stream);
}

}  // namespace qw
