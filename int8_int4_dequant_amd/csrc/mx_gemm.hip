// Products of microscaled 4-bit matrices on the gfx950 matrix cores.
//
//   y[r][i] = sum_b 2^(sx[r][b] + sw[i][b] - 254) sum_{j in b} qx[r][j] qw[i][j]
//
// v_mfma_scale_f32_32x32x64_f8f6f4 multiplies 4-bit codes and applies both scales of
// every block of 32 itself: a lane holds 32 consecutive values of one row, which are one
// block, and that block's scale byte.  Its sums are fp32 (measured: within 2^-23 of the
// sum of magnitudes, accumulator included, scales up to 2^20 apart).  It reaches 8.1
// PFLOP/s here with nothing else to do, the 16x16x128 form 4.5.
//
// The weight is the A operand: output lane l holds token l % 32 and, of a fragment of 32
// weight rows, 8 g + 4 (l / 32) + 0..3, g = 0..3.
#include "mx_codes.h"
#include "tiles.h"

#include <algorithm>
#include <cmath>
#include <type_traits>

namespace qw {
namespace {

typedef int i32x8 __attribute__((ext_vector_type(8)));
typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef uint32_t u32_la __attribute__((may_alias));

struct MxArgs {
  const uint8_t *w, *ws, *x, *xs;
  const void* xfloat; // stream kernel: float rows
  int64_t n, m, k;    // outputs in a row (gated: f), rows, values of a row of x
  int64_t kp2, ksp;   // bytes of a row of codes, of scales
  int kb;             // steps of 256 along k
  void* y;
  uint8_t* ys;
  int64_t yp;         // MX_GATED_CODES: values in a row of codes
  const void* dh;
  void* h;
  int64_t tiles_m, tiles;
};

// The scales are in byte S.
template <int S>
__device__ __forceinline__ f32x16 mfma64(i32x4 a, i32x4 b, f32x16 c, int sa, int sb) {
  const i32x8 a8 = __builtin_shufflevector(a, a, 0, 1, 2, 3, -1, -1, -1, -1);
  const i32x8 b8 = __builtin_shufflevector(b, b, 0, 1, 2, 3, -1, -1, -1, -1);
  return __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(a8, b8, c, 4, 4, S, sa, S, sb);
}

// ---------------------------------------------------------------- results
//
// A lane has 16 outputs of a fragment's 32.  Results of 2 bytes, and codes, are kept so that
// weight row i of a fragment is its row i with bits 2 and 3 swapped: the lane's outputs are
// then 8 consecutive ones at 8 (l / 32) and 8 at 16 + 8 (l / 32), which two lanes write as 32
// bytes (4096 x 4096 bf16 outputs of k = 512: 18.9 us; in runs of 8 bytes 26.0).
// For results of 4 bytes the runs are 4 long and 32 bytes as they are.

template <MxResult RES, typename T>
constexpr bool kSwapped = RES == MX_GATED_CODES || sizeof(T) == 2;

__device__ __forceinline__ int swapped(int row) {  // bits 2 and 3
  return (row & ~12) | (row & 4) << 1 | (row & 8) >> 1;
}

// A lane's runs of consecutive outputs: RUN of them from column at(g, half) on.
template <typename T> struct Runs {
  static constexpr int RUN = sizeof(T) == 2 ? 8 : 4;
  static __device__ __forceinline__ int at(int g, int half) { return 2 * RUN * g + RUN * half; }
};

// 16 bytes at the alignment of an element, which the hardware splits where it has to: rows
// of any length take them.
template <int RUN, typename T>
__device__ __forceinline__ void put(T* p, const float* v, int64_t left) {
  if (left >= RUN) {
    if constexpr (RUN == 8)
      store8<false>(p, v);
    else
      *(f32x4_u*)p = f32x4_u{v[0], v[1], v[2], v[3]};
  } else {
#pragma unroll
    for (int c = 0; c < RUN; ++c)
      if (c < left) store1(p + c, v[c]);
  }
}
template <int RUN, typename T>
__device__ __forceinline__ void get(const T* p, float* v, int64_t left) {
  if (left >= RUN) {
    if constexpr (RUN == 8) {
      load8<false>(p, v);
    } else {
      const f32x4_u t = *(const f32x4_u*)p;
#pragma unroll
      for (int c = 0; c < RUN; ++c) v[c] = t[c];
    }
  } else {
#pragma unroll
    for (int c = 0; c < RUN; ++c) v[c] = c < left ? load1(p + c) : 0.0f;
  }
}

// dgate and dup, h.  With e = exp(-|gate|) neither t nor 1 - t overflows or cancels;
// beyond |gate| = 200 one of them is zero in fp32.  e = 2^g as in gated(), the part of g that
// 24 bits do not hold in a second step; below 2^-64 it is kept 2^64 times, so that t is right
// down to fp32's subnormal values.
__device__ __forceinline__ void gate_gradients(float gate, float up, float dh, float& dgate,
                                               float& dup, float& h) {
#pragma clang fp contract(off)
  const float a = -fabsf(gate), g = a * 0x1.715476p+0f;  // log2(e) to 24 bits, and the rest of it
  const float l = __builtin_fmaf(a, 0x1.4ae0cp-26f, __builtin_fmaf(a, 0x1.715476p+0f, -g));
  const bool far = g < -64.0f;
  float e = __builtin_amdgcn_exp2f(far ? g + 64.0f : g);
  e = __builtin_fmaf(e, g > -190.0f ? l * 0x1.62e43p-1f : 0.0f, e);
  const float by = far ? 0x1p-64f : 1.0f;
  const float one = __builtin_amdgcn_rcpf(__builtin_fmaf(e, by, 1.0f)), other = e * one * by;
  const bool neg = gate < 0.0f;
  const float t = neg ? other : one, u = neg ? one : other;
  const float near = __builtin_amdgcn_fmed3f(gate, -200.0f, 200.0f);
  const float silu = gate * t;
  dgate = dh * up * (t * __builtin_fmaf(near, u, 1.0f));
  dup = dh * silu;
  h = silu * up;
}

// A fragment's outputs, of columns from col0 on of output row `row`.
template <typename T>
__device__ __forceinline__ void store_fragment(const MxArgs& a, f32x16 v, int64_t row,
                                               int64_t col0, int half) {
  using R = Runs<T>;
#pragma unroll
  for (int g = 0; g < 16 / R::RUN; ++g) {
    const int64_t col = col0 + R::at(g, half);
    float o[R::RUN];
#pragma unroll
    for (int c = 0; c < R::RUN; ++c) o[c] = v[R::RUN * g + c];
    put<R::RUN>((T*)a.y + row * a.n + col, o, a.n - col);
  }
}

template <MxResult RES, typename T>
__device__ __forceinline__ void store_gated(const MxArgs& a, f32x16 gate, f32x16 up, int64_t row,
                                            int64_t col0, int half, bool have) {
  using R = Runs<T>;
  constexpr int RUN = R::RUN;
  if constexpr (RES == MX_GATED_BACKWARD) {
    if (!have) return;
#pragma unroll
    for (int g = 0; g < 16 / RUN; ++g) {
      const int64_t col = col0 + R::at(g, half), left = a.n - col;
      if (left <= 0) continue;
      float dh[RUN], dg[RUN], du[RUN], h[RUN];
      get<RUN>((const T*)a.dh + row * a.n + col, dh, left);
#pragma unroll
      for (int c = 0; c < RUN; ++c)
        gate_gradients(gate[RUN * g + c], up[RUN * g + c], dh[c], dg[c], du[c], h[c]);
      put<RUN>((T*)a.y + row * 2 * a.n + col, dg, left);
      put<RUN>((T*)a.y + row * 2 * a.n + a.n + col, du, left);
      if (a.h) put<RUN>((T*)a.h + row * a.n + col, h, left);
    }
  } else {
    float v[16], p[16], q[16];
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      p[i] = gate[i];
      q[i] = up[i];
    }
    gated<16>(p, q, v);
    if constexpr (RES == MX_GATED) {
      if (!have) return;
#pragma unroll
      for (int g = 0; g < 16 / RUN; ++g) {
        const int64_t col = col0 + R::at(g, half);
        put<RUN>((T*)a.y + row * a.n + col, v + RUN * g, a.n - col);
      }
    } else {
      // The 32 values are one block: half of them in the lane 32 away.  Behind the last output
      // they are zeros, or NaN in a row of x that has a NaN scale: code 0, and there the scale 1.
      uint32_t top = top_of<16>(v);
      top = max(top, (uint32_t)__shfl_xor((int)top, 32));
      const uint32_t s = mx_scale(top);
      const uint32_t lo = mx_codes8(v, s), hi = mx_codes8(v + 8, s);
      if (have && col0 < a.yp) {
        uint8_t* const to = (uint8_t*)a.y + (row * a.yp + col0) / 2 + 4 * half;
        *(uint32_t*)to = lo;
        *(uint32_t*)(to + 8) = hi;
        if (half == 0) a.ys[(row * a.yp + col0) / 32] = (uint8_t)(col0 < a.n ? s : 127u);
      }
    }
  }
}

// A tile's results through LDS: fragments of a wave (COLS = 32 or 64 weight rows of 32 tokens)
// change lanes, so that 128 (or, 32 results of 2 bytes, 64) bytes of an output row are written
// by lanes side by side.  Rows of RB bytes, the pieces of 16 bytes swapped as those of the
// tiles below.  Against runs of 32 bytes from the registers: 4096 x 11008 x 2048 with fp32 results
// 75 -> 71 us, 4096^3 with bf16 44.4 -> 42.2, 3001 x 6001 x 1000 (rows at any alignment) 33 -> 26.
// (Past the caches: fp32 results 5 to 25 in a hundred slower, bf16 2 faster.)
template <typename T, int COLS>
struct Rows {
  static constexpr int RB = COLS * (int)sizeof(T), PIECES = RB / 16, AT_ONCE = 64 / PIECES;
  static constexpr int PER = 16 / (int)sizeof(T);  // results of a piece
  static_assert(RB == 64 || RB == 128, "a wave's part of LDS is 4 KiB");
  static __device__ __forceinline__ int place(int row, int piece) {
    return row * RB + ((piece ^ (RB == 128 ? row >> 1 & 7 : row >> 2 & 3)) << 4);
  }
  // the lane's values of fragment I
  static __device__ __forceinline__ void put(uint8_t* lds, int i, const float v[16], int r, int half) {
#pragma unroll
    for (int g = 0; g < 16 / PER; ++g) {
      uint8_t* const p = lds + place(r, i * (32 / PER) + 2 * g + half);
      if constexpr (sizeof(T) == 2)
        *(u32x4_la*)p = u32x4_la{to_bf16x2(v[8 * g], v[8 * g + 1]), to_bf16x2(v[8 * g + 2], v[8 * g + 3]),
                                 to_bf16x2(v[8 * g + 4], v[8 * g + 5]), to_bf16x2(v[8 * g + 6], v[8 * g + 7])};
      else
        *(u32x4_la*)p = u32x4_la{__float_as_uint(v[4 * g]), __float_as_uint(v[4 * g + 1]),
                                 __float_as_uint(v[4 * g + 2]), __float_as_uint(v[4 * g + 3])};
    }
  }
  // rows [0, rows) of `ld` values, from column 0 on of which `left` are there
  static __device__ __forceinline__ void store(const uint8_t* lds, T* y, int64_t ld, int rows, int64_t left, int lane) {
    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");  // the wave's own writes, by other lanes
#pragma unroll
    for (int s = 0; s < 32 / AT_ONCE; ++s) {
      const int row = s * AT_ONCE + lane / PIECES, piece = lane % PIECES;
      const u32x4 v = *(const u32x4_la*)(lds + place(row, piece));
      T* const to = y + row * ld + piece * PER;
      const int64_t there = left - piece * PER;
      if (row < rows) {
        if (there >= PER) {
          *(u32x4_u*)to = v;
        } else {
#pragma unroll
          for (int c = 0; c < PER; ++c)
            if (c < there) to[c] = __builtin_bit_cast(Parts, v).part[c];
        }
      }
    }
  }
  // The reverse: the lane's 16 values of a fragment of x (COLS = 32).
  static __device__ __forceinline__ void load(uint8_t* lds, const T* x, int64_t ld, int rows, int64_t left, int lane,
                                              int r, int half, float v[16]) {
#pragma unroll
    for (int s = 0; s < 32 / AT_ONCE; ++s) {
      const int row = s * AT_ONCE + lane / PIECES, piece = lane % PIECES;
      const T* const from = x + min(row, rows - 1) * ld + piece * PER;
      const int64_t there = left - piece * PER;
      u32x4 t = {};
      if (there >= PER) {
        t = *(const u32x4_u*)from;
      } else {
        Parts p = {};
#pragma unroll
        for (int c = 0; c < PER; ++c)
          if (c < there) p.part[c] = from[c];
        t = __builtin_bit_cast(u32x4, p);
      }
      *(u32x4_la*)(lds + place(row, piece)) = t;
    }
    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
#pragma unroll
    for (int g = 0; g < 16 / PER; ++g) {
      const Parts t = __builtin_bit_cast(Parts, *(const u32x4_la*)(lds + place(r, 2 * g + half)));
#pragma unroll
      for (int c = 0; c < PER; ++c) v[PER * g + c] = load1(&t.part[c]);
    }
  }
  struct Parts {
    T part[PER];
  };
};

// ---------------------------------------------------------------- tiled kernel
//
// A block of WN x WM waves, each with 32 NF weight rows x 32 MF tokens, 256 values of k (a
// step) at a time through a ring of STAGES LDS buffers that copies straight from memory
// fill.  Scales are copied for four steps at once (32 bytes a row), into two buffers.
//
// What bounds it: the copies take whole lines of 128 bytes, since the rate of requests is
// what limits them (alone, 256 x 256 tiles of 4096 x 4096 x 16384: 64-byte rows of half the
// step 0.51 us for 128 values of k, 128-byte rows 0.37; scales of 16 bytes a row 0.11 more).
// The products alone take 0.50 us for it, 0.82 with values that are not zero: the clock
// falls with the power that they draw.
//
// LDS rows are the 128 bytes of a step.  A phase of a 16-byte LDS read is 16 lanes, here
// 16 consecutive rows at the same place in the row, and the 64 banks hold 2 rows: piece c
// of row r is kept at c ^ (r / 2 % 8), so that the 16 lanes meet 16 different places.  The
// copy writes LDS in lane order, so the lanes fetch the pieces in that order from memory.
// The scales of 4 steps are 32 bytes a row; 32 rows have their first 16 bytes side by side
// and then their last, so that a read of a word a row meets half of the banks (11008 x 4096
// fp32 results of k = 2048 72.4 -> 71.0 us; rows of 32 bytes meet a quarter).
//
// A step has four products a fragment; of the t-th, a lane holds block 4 (l / 32) + t, so
// that byte t of one word of its row's scales goes with it.
//
// A block takes tile after tile (in steps of the grid) and the copies run on: behind the
// last step of a tile comes the first one of the next, which is on its way while the results
// are written through the other buffer.  `chunks` of 4 steps and the two buffers of their scales
// are counted through in the same way.  (With a second set of sums, results written a part
// after every few of the next tile's steps: slower, 128 x 256 tiles of 2047 x 22016 x 4096 126 ->
// 136 us, since every wait for a step's copies also waits for the writes before them.)
//
// Gated results: the tile's rows are 32 gate rows and their 32 up rows in turn, so that a
// lane holds both values of a result.

// What the waves of a block copy for a tile of BN weight rows and BM tokens.
template <int BN, int BM, int WAVES, bool GATED, bool SWAPPED>
struct Feed {
  static constexpr int ROWS = BN + BM;
  static constexpr int COLS = GATED ? BN / 2 : BN;       // outputs of a row in a tile
  static constexpr int SEGS = ROWS / 8 / WAVES;          // 8-row pieces of a wave
  static constexpr int SPER = (ROWS / 32 + WAVES - 1) / WAVES;  // 32-row pieces of scales of a wave
  static_assert(ROWS / 8 % WAVES == 0 && BN % 64 == 0 && BM % 32 == 0, "whole pieces");
  // A tile, and each piece's buffer, of which the rows behind the last one are not a part.
  struct Place {
    int64_t n0, m0;
    int rows;
    i32x4 from[SEGS], sfrom[SPER];
  };
  const MxArgs& a;
  const int wave, kb, chunks;
  int base = 0;  // which of the two buffers holds the tile's first scales
  uint32_t lds0, lds1, voff[SEGS], soff[SPER];
  Place here, then;

  // the weight row (of gate or up) that LDS row `row` holds
  static __device__ __forceinline__ int weight_row(int row) {
    const int at = GATED ? row / 64 * 32 + row % 32 : row;
    return SWAPPED ? swapped(at) : at;
  }
  __device__ __forceinline__ Feed(const MxArgs& args, int wave, int lane, uint8_t* lds, uint8_t* scales)
      : a(args), wave(wave), kb(args.kb), chunks((args.kb + 3) >> 2) {
    lds0 = (uint32_t)(uintptr_t)(__attribute__((address_space(3))) uint8_t*)lds;
    lds1 = (uint32_t)(uintptr_t)(__attribute__((address_space(3))) uint8_t*)scales;
#pragma unroll
    for (int s = 0; s < SEGS; ++s) {
      const int row = (wave + WAVES * s) * 8 + (lane >> 3);
      const int c = (lane & 7) ^ ((row >> 1) & 7);
      const int at = row >= BN ? row - BN : weight_row(row);
      voff[s] = (uint32_t)at * (uint32_t)a.kp2 + c * 16;
    }
#pragma unroll
    for (int s = 0; s < SPER; ++s) {
      const int row = (wave + WAVES * s) * 32 + (lane & 31);
      const int at = row >= BN ? row - BN : weight_row(row);
      soff[s] = (uint32_t)at * (uint32_t)a.ksp + (lane >> 5) * 16;
    }
  }
  __device__ __forceinline__ void place(int64_t tile, Place& p) const {
    int64_t tm, tn;
    const bool there = tile < a.tiles;
    tile_place(there ? tile : 0, a.tiles, a.tiles_m, tm, tn);
    p.n0 = uniform(tn) * COLS;
    p.m0 = uniform(tm) * BM;
    p.rows = __builtin_amdgcn_readfirstlane(there ? (int)min(a.m - p.m0, (int64_t)BM) : 0);
    // behind the last output (padding of a row of codes) there are no weight rows
    const int cols = __builtin_amdgcn_readfirstlane(there ? (int)max((int64_t)0, min(a.n - p.n0, (int64_t)COLS)) : 0);
    auto choose = [&](bool of_x, bool up, const uint8_t* xbase, const uint8_t* wbase, int64_t bytes) {
      return buffer_of((const uint8_t*)uniform((int64_t)(of_x ? xbase + p.m0 * bytes : wbase + (p.n0 + (up ? a.n : 0)) * bytes)),
                       __builtin_amdgcn_readfirstlane((uint32_t)((of_x ? p.rows : cols) * bytes)));
    };
#pragma unroll
    for (int s = 0; s < SEGS; ++s) {
      const int seg = wave + WAVES * s;
      p.from[s] = choose(seg >= BN / 8, GATED && seg / 4 % 2, a.x, a.w, a.kp2);
    }
#pragma unroll
    for (int s = 0; s < SPER; ++s) {
      const int seg = wave + WAVES * s;
      p.sfrom[s] = choose(seg >= BN / 32, GATED && seg % 2, a.xs, a.ws, a.ksp);
    }
  }
  // Piece S of step b into buffer `buf`.  Behind the tile's last step: of the next tile.  Behind
  // the last tile there is nothing to read, but the copy is issued all the same (as zeros,
  // from an empty buffer), so that every step has as many.
  __device__ __forceinline__ void fetch(int b, int buf, int s) const {
    if (s >= SEGS) return;
    const bool in = b < kb;
    i32x4 buffer = here.from[s];
#pragma unroll
    for (int c = 0; c < 3; ++c) buffer[c] = in ? buffer[c] : then.from[s][c];
    copy_to_lds(buffer, voff[s], (uint32_t)(in ? b : b - kb) * 128,
                lds0 + buf * (ROWS * 128) + (wave + WAVES * s) * 1024);
  }
  // The scales of steps 4 u .. 4 u + 3.
  __device__ __forceinline__ void fetch_scales(int u, bool when) const {
    const bool in = u < chunks;
#pragma unroll
    for (int s = 0; s < SPER; ++s) {
      i32x4 buffer = here.sfrom[s];
#pragma unroll
      for (int c = 0; c < 3; ++c) buffer[c] = in ? buffer[c] : then.sfrom[s][c];
      copy_to_lds_when(__builtin_amdgcn_readfirstlane(when && wave + WAVES * s < ROWS / 32 ? 1 : 0), buffer, soff[s],
                       (uint32_t)(in ? u : u - chunks) * 32,
                       lds1 + ((base + u) & 1) * (ROWS * 32) + (wave + WAVES * s) * 1024);
    }
  }
  // A block's first tile and the one behind it: their places, and the first copies.
  template <int STAGES>
  __device__ __forceinline__ void start(int64_t tile, int64_t next) {
    place(tile, here);
    place(next, then);
    fetch_scales(0, true);
    fetch_scales(1, true);
#pragma unroll
    for (int b = 0; b < STAGES; ++b)
#pragma unroll
      for (int s = 0; s < SEGS; ++s) fetch(b, b, s);
  }
};

template <int NF, int MF, int WN, int WM, int STAGES, MxResult RES, typename T>
__global__ __launch_bounds__(WN * WM * 64, 2) void mx_tiled(MxArgs a) {
  constexpr int WAVES = WN * WM, BN = 32 * NF * WN, BM = 32 * MF * WM;
  constexpr bool GATED = RES != MX_STORE;
  using F = Feed<BN, BM, WAVES, GATED, kSwapped<RES, T>>;
  constexpr int ROWS = F::ROWS, SEGS = F::SEGS;
  static_assert(!GATED || NF % 2 == 0, "gate and up rows in one wave");
  __shared__ __align__(1024) uint8_t lds[STAGES][ROWS * 128];
  __shared__ __align__(1024) uint8_t scales[2][ROWS * 32];
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int lane = threadIdx.x & 63, r = lane & 31, half = lane >> 5;
  const int wm = wave % WM * 32 * MF, wn = wave / WM * 32 * NF;
  F feed(a, wave, lane, lds[0], scales[0]);
  const int kb = a.kb;
  int64_t tile = blockIdx.x + gridDim.x;
  feed.template start<STAGES>(blockIdx.x, tile);

  i32x4 w[2][NF], x[2][MF];  // fragments of two products
  int sw[NF], sx[MF], sw2[NF], sx2[MF];
  const int swap = (r >> 1) & 7;  // the same for all rows a multiple of 32 apart
  // Read N of the fragments of product Q of the step in buffer `buf`: the first ones' first.
  auto take = [&](int buf, auto product, int n) {
    constexpr int Q = decltype(product)::value;
    const uint8_t* p = &lds[buf][r * 128 + (((4 * half + Q) ^ swap) << 4)];
    if (n < MF)
      x[Q & 1][n] = *(const i32x4*)(p + (BN + wm + 32 * n) * 128);
    else if (n < MF + NF)
      w[Q & 1][n - MF] = *(const i32x4*)(p + (wn + 32 * (n - MF)) * 128);
  };
  auto take_scale = [&](int b, int n) {
    const int u = b < kb ? b >> 2 : feed.chunks, in = b < kb ? b & 3 : 0;  // behind the last: the next tile's first
    const uint8_t* p = &scales[(feed.base + u) & 1][(in >> 1) * 512 + r * 16 + (in & 1) * 8 + 4 * half];
    if (n < MF)
      sx2[n] = *(const int*)(p + (BN + wm + 32 * n) * 32);
    else if (n < MF + NF)
      sw2[n - MF] = *(const int*)(p + (wn + 32 * (n - MF)) * 32);
  };
  constexpr int FRAGS = NF + MF, PRODUCTS = NF * MF;
  constexpr int TAKES = (FRAGS + PRODUCTS - 1) / PRODUCTS, COPIES = (SEGS + PRODUCTS - 1) / PRODUCTS;
  // Copies that may be on their way when step b + 1 has to be there: those of the
  // STAGES - 2 steps behind it.  Scales are issued before the copies of their step and at least
  // one step ahead of the wait before their use (a tile's last chunk may be one step).
  constexpr int LEFT = (STAGES - 2) * SEGS;
  static_assert(STAGES == 2, "scales have landed by then, and all copies at a tile's end");
  landed<LEFT + SEGS>();
#pragma unroll
  for (int n = 0; n < FRAGS; ++n) {
    take(0, std::integral_constant<int, 0>{}, n);
    take_scale(0, n);
  }
  int buf = 0;
  f32x16 acc[NF][MF];
  auto step = [&](int b, auto ends) {
    constexpr bool LAST = decltype(ends)::value;  // of a tile
    const int next = buf + 1 < STAGES ? buf + 1 : 0;
#pragma unroll
    for (int i = 0; i < NF; ++i) sw[i] = sw2[i];
#pragma unroll
    for (int j = 0; j < MF; ++j) sx[j] = sx2[j];
    // Product Q of all fragments, and between them what comes next.
    auto products = [&](auto product, auto between) {
      constexpr int Q = decltype(product)::value;
#pragma unroll
      for (int p = 0; p < PRODUCTS; ++p) {
        between(p);
        acc[p / MF][p % MF] = mfma64<Q>(w[Q & 1][p / MF], x[Q & 1][p % MF], acc[p / MF][p % MF],
                                        sw[p / MF], sx[p % MF]);
        __builtin_amdgcn_sched_barrier(0);
      }
    };
    auto with_reads = [&](auto product) {
      constexpr int Q = decltype(product)::value;
      products(product, [&](int p) {
#pragma unroll
        for (int n = 0; n < TAKES; ++n)
          take(buf, std::integral_constant<int, Q + 1>{}, p * TAKES + n);
      });
    };
    with_reads(std::integral_constant<int, 0>{});
    with_reads(std::integral_constant<int, 1>{});
    with_reads(std::integral_constant<int, 2>{});
    // This wave holds all that it needs of this buffer and of these scales; once every
    // wave does, they are filled again (behind a tile's last step: the buffer takes its
    // results first).
    landed<LEFT>();
    feed.fetch_scales((b >> 2) + 2, LAST || (b & 3) == 3);
    products(std::integral_constant<int, 3>{}, [&](int p) {
#pragma unroll
      for (int n = 0; n < COPIES; ++n)
        if (!LAST) feed.fetch(b + STAGES, buf, p * COPIES + n);
#pragma unroll
      for (int n = 0; n < TAKES; ++n) {
        take(next, std::integral_constant<int, 0>{}, p * TAKES + n);
        take_scale(b + 1, p * TAKES + n);
      }
    });
    if (!LAST) buf = next;
  };
  for (;;) {
#pragma unroll
    for (int i = 0; i < NF; ++i)
#pragma unroll
      for (int j = 0; j < MF; ++j) acc[i][j] = f32x16{};
    for (int b = 0; b + 1 < kb; ++b) step(b, std::false_type{});
    if (kb > 0) step(kb - 1, std::true_type{});
    // nothing to add up: the empty copies of both buffers are not on their way any more
    if (kb == 0) landed<0>();
    uint8_t* const mine = lds[buf] + wave * (ROWS * 128 / WAVES);
    static_assert(NF == 2 && ROWS * 128 / WAVES >= 4096, "a wave's part of a buffer");
#pragma unroll
    for (int j = 0; j < MF; ++j) {
      const int64_t row0 = feed.here.m0 + wm + 32 * j;
      const int there = feed.here.rows - wm - 32 * j;
      auto values = [&](int i, float* v) {
#pragma unroll
        for (int e = 0; e < 16; ++e) v[e] = acc[i][j][e];
      };
      if constexpr (RES == MX_STORE) {
        // both fragments of 2 bytes a value, one of 4
        constexpr int EACH = sizeof(T) == 2 ? 2 : 1;
#pragma unroll
        for (int i = 0; i < NF; i += EACH) {
          const int64_t col = feed.here.n0 + wn + 32 * i;
#pragma unroll
          for (int e = 0; e < EACH; ++e) {
            float v[16];
            values(i + e, v);
            Rows<T, 32 * EACH>::put(mine, e, v, r, half);
          }
          Rows<T, 32 * EACH>::store(mine, (T*)a.y + row0 * a.n + col, a.n, there, a.n - col, lane);
        }
      } else if constexpr (RES == MX_GATED_CODES) {
        store_gated<RES, T>(a, acc[0][j], acc[1][j], row0 + r, feed.here.n0 + wn / 2, half, r < there);
      } else {
        const int64_t col = feed.here.n0 + wn / 2, left = a.n - col;
        float p[16], q[16], v[16];
        values(0, p);
        values(1, q);
        if constexpr (RES == MX_GATED) {
          gated<16>(p, q, v);
          Rows<T, 32>::put(mine, 0, v, r, half);
          Rows<T, 32>::store(mine, (T*)a.y + row0 * a.n + col, a.n, there, left, lane);
        } else if (there > 0 && left > 0) {
          float d[16];
          Rows<T, 32>::load(mine, (const T*)a.dh + row0 * a.n + col, a.n, there, left, lane, r, half, d);
#pragma unroll
          for (int e = 0; e < 16; ++e) gate_gradients(p[e], q[e], d[e], v[e], d[e], p[e]);  // p: h
          T* const y = (T*)a.y + row0 * 2 * a.n + col;
          Rows<T, 32>::put(mine, 0, v, r, half);
          Rows<T, 32>::store(mine, y, 2 * a.n, there, left, lane);
          Rows<T, 32>::put(mine, 0, d, r, half);
          Rows<T, 32>::store(mine, y + a.n, 2 * a.n, there, left, lane);
          if (a.h) {
            Rows<T, 32>::put(mine, 0, p, r, half);
            Rows<T, 32>::store(mine, (T*)a.h + row0 * a.n + col, a.n, there, left, lane);
          }
        }
      }
    }
    if (tile >= a.tiles) break;
    // every wave's part of the buffer is free: the copies that its last step left out
    lds_barrier();
#pragma unroll
    for (int s = 0; s < SEGS; ++s) feed.fetch(kb - 1 + STAGES, buf, s);
    buf = buf + 1 < STAGES ? buf + 1 : 0;
    feed.here = feed.then;
    feed.base += feed.chunks;
    tile += gridDim.x;
    feed.place(tile, feed.then);
  }
  landed<0>();  // the empty copies too, before the block's LDS is another's
}

// The same for few tiles, which are bound by the latency of a step: a block's four waves
// share the four products of each step of one tile of 64 x 64, and their sums meet in LDS.
// (256 values of k take 0.31 us; 0.48 with tiles of 64 x 64 above, of two waves.)
template <int STAGES, MxResult RES, typename T>
__global__ __launch_bounds__(256, 2) void mx_split(MxArgs a) {
  constexpr bool GATED = RES != MX_STORE;
  using F = Feed<64, 64, 4, GATED, kSwapped<RES, T>>;
  constexpr int ROWS = F::ROWS, SEGS = F::SEGS, LEFT = (STAGES - 2) * SEGS;
  static_assert(STAGES == 4, "the sums take the place of four steps; scales have landed");
  __shared__ __align__(1024) uint8_t lds[STAGES][ROWS * 128];
  __shared__ __align__(1024) uint8_t scales[2][ROWS * 32];
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int lane = threadIdx.x & 63, r = lane & 31, half = lane >> 5;
  F feed(a, wave, lane, lds[0], scales[0]);
  const int kb = a.kb;
  feed.template start<STAGES>(blockIdx.x, a.tiles);

  f32x16 acc[2][2] = {};
  i32x4 f[2][4];  // fragments of two steps: weight, weight, token, token
  int sc[2][4];
  const uint8_t* const mine = &lds[0][r * 128 + (((4 * half + wave) ^ (r >> 1 & 7)) << 4)];
  auto take = [&](int b, int buf, auto parity) {
    constexpr int P = decltype(parity)::value;
    const uint8_t* sp = &scales[(b >> 2) & 1][(b >> 1 & 1) * 512 + r * 16 + (b & 1) * 8 + 4 * half];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      f[P][i] = *(const i32x4*)(mine + buf * (ROWS * 128) + 32 * i * 128);
      sc[P][i] = *(const int*)(sp + 32 * i * 32);
    }
  };
  landed<LEFT + SEGS>();
  take(0, 0, std::integral_constant<int, 0>{});
  auto step = [&](int b, auto parity) {
    constexpr int P = decltype(parity)::value;
    const int buf = b & (STAGES - 1);
    // the next step is there, and every wave has this one in registers
    landed<LEFT>();
    feed.fetch_scales((b >> 2) + 2, (b & 3) == 3);
#pragma unroll
    for (int s = 0; s < SEGS; ++s) feed.fetch(b + STAGES, buf, s);
    take(b + 1, (b + 1) & (STAGES - 1), std::integral_constant<int, 1 - P>{});
#pragma unroll
    for (int i = 0; i < 4; ++i) sc[P][i] >>= 8 * wave;
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
      for (int j = 0; j < 2; ++j)
        acc[i][j] = mfma64<0>(f[P][i], f[P][2 + j], acc[i][j], sc[P][i], sc[P][2 + j]);
    __builtin_amdgcn_sched_barrier(0);
  };
  for (int b = 0; b < kb; b += 2) {
    step(b, std::integral_constant<int, 0>{});
    if (b + 1 < kb) step(b + 1, std::integral_constant<int, 1>{});
  }
  landed<0>();
  // four fragments of four waves, a lane's values together
  f32x4* const sums = (f32x4*)&lds[0][0];
#pragma unroll
  for (int i = 0; i < 2; ++i)
#pragma unroll
    for (int j = 0; j < 2; ++j)
#pragma unroll
      for (int g = 0; g < 4; ++g)
        sums[((wave * 4 + i * 2 + j) * 4 + g) * 64 + lane] =
            f32x4{acc[i][j][4 * g], acc[i][j][4 * g + 1], acc[i][j][4 * g + 2], acc[i][j][4 * g + 3]};
  lds_barrier();
  auto joined = [&](int fragment) {
    f32x16 t;
#pragma unroll
    for (int g = 0; g < 4; ++g) {
      f32x4 v = sums[(fragment * 4 + g) * 64 + lane];
#pragma unroll
      for (int o = 1; o < 4; ++o) v += sums[((o * 4 + fragment) * 4 + g) * 64 + lane];
#pragma unroll
      for (int c = 0; c < 4; ++c) t[4 * g + c] = v[c];
    }
    return t;
  };
  const int j = wave & 1, at = 32 * j + r;
  const int64_t row = feed.here.m0 + at;
  const bool have = at < feed.here.rows;
  if constexpr (GATED) {
    if (wave < 2) store_gated<RES, T>(a, joined(j), joined(2 + j), row, feed.here.n0, half, have);
  } else {
    const f32x16 v = joined(wave);  // fragment i, j = wave / 2, wave % 2
    if (have) store_fragment<T>(a, v, row, feed.here.n0 + 32 * (wave >> 1), half);
  }
}

constexpr int kUnits = 256;  // compute units

// go(result, type) of a call's.
template <typename Go>
void with_result(const MxGemm& g, Go go) {
  auto typed = [&](auto result) { g.y_type == QW_F32 ? go(result, 0.0f) : go(result, uint16_t{}); };
  switch (g.result) {
    case MX_STORE: typed(std::integral_constant<MxResult, MX_STORE>{}); break;
    case MX_GATED: typed(std::integral_constant<MxResult, MX_GATED>{}); break;
    case MX_GATED_CODES: go(std::integral_constant<MxResult, MX_GATED_CODES>{}, 0.0f); break;
    default: typed(std::integral_constant<MxResult, MX_GATED_BACKWARD>{});
  }
}

void count_tiles(MxArgs& a, const MxGemm& g, int bn, int bm) {
  const int cols = g.result == MX_STORE ? bn : bn / 2;
  a.tiles_m = (a.m + bm - 1) / bm;
  a.tiles = a.tiles_m * (((g.result == MX_GATED_CODES ? a.yp : a.n) + cols - 1) / cols);
}

// PER_UNIT: blocks that a compute unit holds.
template <int NF, int MF, int WN, int WM, int STAGES, int PER_UNIT>
hipError_t run_tiled(MxArgs a, const MxGemm& g, hipStream_t stream) {
  count_tiles(a, g, 32 * NF * WN, 32 * MF * WM);
  // Tile after tile where there are more than the units hold; copies that run on into the
  // next tile need two chunks of scales in each.
  const unsigned grid = (unsigned)(a.kb > 4 ? std::min<int64_t>(a.tiles, kUnits * PER_UNIT) : a.tiles);
  with_result(g, [&](auto result, auto type) {
    mx_tiled<NF, MF, WN, WM, STAGES, decltype(result)::value, decltype(type)>
        <<<grid, WN * WM * 64, 0, stream>>>(a);
  });
  return hipGetLastError();
}

hipError_t run_split(MxArgs a, const MxGemm& g, hipStream_t stream) {
  count_tiles(a, g, 64, 64);
  with_result(g, [&](auto result, auto type) {
    mx_split<4, decltype(result)::value, decltype(type)><<<(unsigned)a.tiles, 256, 0, stream>>>(a);
  });
  return hipGetLastError();
}

MxArgs args_of(const MxGemm& g) {
  MxArgs a = {};
  const int64_t kp = mx_pitch(g.k);
  a.w = g.codes;
  a.ws = g.scales;
  a.x = g.xc;
  a.xs = g.xs;
  a.n = g.n;
  a.m = g.m;
  a.k = g.k;
  a.xfloat = g.x;
  a.kp2 = kp / 2;
  a.ksp = kp / 32;
  a.kb = (int)((g.k + 255) / 256);
  a.y = g.y;
  a.ys = g.ys;
  a.yp = mx_pitch(g.n);
  a.dh = g.dh;
  a.h = g.h;
  return a;
}

// ---------------------------------------------------------------- stream kernel
//
// For up to 16 MT rows of x: bound by reading the weight once.  A block takes 16 weight rows
// (gated: 16 gate and their 16 up rows) after 16 weight rows; its 8 waves share k, each
// with U consecutive units of 512 values, one line of scales a row and unit.  A wave
// quantizes (or loads) its part of x once and keeps it in registers; a unit of the weight is
// replaced by a later one as soon as its products are issued, so that RING units (4.3 KiB
// each) are always on their way.  The waves' sums meet in LDS, once for 16 weight rows.
//
// v_mfma_scale_f32_16x16x128_f8f6f4: lane l holds row l % 16 and, with q = l / 16, one block
// of 32; of product t of a unit's four, block 4 t + q, whose scale is byte q of word t.

constexpr int kStreamWaves = 8;

// What x is: rows of float values, or codes (x and xs).
template <typename XT> struct is_codes { static constexpr bool value = false; };
template <> struct is_codes<uint8_t> { static constexpr bool value = true; };

__device__ __forceinline__ f32x4 mfma128(i32x4 a, i32x4 b, f32x4 c, int sa, int sb) {
  const i32x8 a8 = __builtin_shufflevector(a, a, 0, 1, 2, 3, -1, -1, -1, -1);
  const i32x8 b8 = __builtin_shufflevector(b, b, 0, 1, 2, 3, -1, -1, -1, -1);
  return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(a8, b8, c, 4, 4, 0, sa, 0, sb);
}

// This wave's units of float x as fragments and their scales (in byte 0): the 64 lanes
// quantize a unit of a row, 8 values each, as quantize_rows does, up to 4 rows at a time; the
// codes change lanes through LDS of the wave's own.
template <int U, bool VEC, typename XT>
__device__ __forceinline__ void quantize_part(const MxArgs& a, int unit0, uint8_t (*codes)[272],
                                              int lane, i32x4 (*xf)[4], int (*sx)[4]) {
  const int r = lane & 15, q = lane >> 4, m = (int)a.m;
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const int64_t j = (int64_t)(unit0 + u) * 512 + lane * 8;
    for (int row = 0; row < m; row += 4) {
      float v[4][8];
#pragma unroll
      for (int i = 0; i < 4; ++i) load8_of_row<VEC>((const XT*)a.xfloat + min(row + i, m - 1) * a.k, j, a.k, v[i]);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const uint32_t s = mx_scale(top_among<4>(top_of<8>(v[i])));
        const uint32_t c = mx_codes8(v[i], s);
        if (row + i < m) {
          *(u32_la*)&codes[row + i][lane * 4] = c;
          if ((lane & 3) == 0) codes[row + i][256 + (lane >> 2)] = (uint8_t)s;
        }
      }
    }
    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");  // the wave's own writes, by other lanes
#pragma unroll
    for (int t = 0; t < 4; ++t)
      xf[u][t] = __builtin_bit_cast(i32x4, *(const u32x4_la*)&codes[r][(4 * t + q) * 16]);
    const i32x4 s = __builtin_bit_cast(i32x4, *(const u32x4_la*)&codes[r][256]);
#pragma unroll
    for (int t = 0; t < 4; ++t) sx[u][t] = s[t] >> 8 * q;
  }
}

template <int U, int MT, bool GATED, bool VEC, typename XT, typename T>
__global__ __launch_bounds__(kStreamWaves * 64, 2) void mx_stream(MxArgs a) {
  constexpr int H = GATED ? 2 : 1;  // weight rows of an output
  constexpr int RING = U > 4 || (GATED && U > 3) ? 2 : U;  // what the registers hold
  constexpr int BUFS = MT == 1 ? 2 : 1;
  static_assert(U % RING == 0, "the next tile's units take the places of this one's");
  __shared__ __align__(16) float part[BUFS][kStreamWaves][H][16 * MT][20];
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int lane = threadIdx.x & 63, r = lane & 15, q = lane >> 4;
  const int units = (int)(a.kp2 / 256), unit0 = wave * U;
  const int64_t tiles_n = (a.n + 15) / 16;
  i32x4 w[RING][H][4], ws[RING][H];
  // Unit u of the tile; behind the last unit, and behind the last row, the last one again.
  auto load = [&](int64_t tile, int u) {
    const int64_t at = min(unit0 + u, units - 1);
#pragma unroll
    for (int h = 0; h < H; ++h) {
      const int64_t row = min(tile * 16 + r, a.n - 1) + (h ? a.n : 0);
      const uint8_t* p = a.w + row * a.kp2 + at * 256 + q * 16;
#pragma unroll
      for (int t = 0; t < 4; ++t) w[u % RING][h][t] = *(const i32x4*)(p + 64 * t);
      ws[u % RING][h] = *(const i32x4*)(a.ws + row * a.ksp + at * 16);
    }
  };
  int64_t tile = blockIdx.x;
#pragma unroll
  for (int u = 0; u < RING; ++u) load(tile, u);
  i32x4 xf[MT][U][4];
  int sx[MT][U][4];
  if constexpr (is_codes<XT>::value) {
#pragma unroll
    for (int j = 0; j < MT; ++j) {
      const int64_t row = min((int64_t)(16 * j + r), a.m - 1);
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int64_t at = min(unit0 + u, units - 1);
#pragma unroll
        for (int t = 0; t < 4; ++t)
          xf[j][u][t] = *(const i32x4*)(a.x + row * a.kp2 + at * 256 + t * 64 + q * 16);
        const i32x4 s = *(const i32x4*)(a.xs + row * a.ksp + at * 16);
#pragma unroll
        for (int t = 0; t < 4; ++t) sx[j][u][t] = s[t] >> 8 * q;
      }
    }
  } else {
    static_assert(MT == 1, "float rows: 16 at most");
    __shared__ __align__(16) uint8_t codes[kStreamWaves][16][272];
    quantize_part<U, VEC, XT>(a, unit0, codes[wave], lane, xf[0], sx[0]);
  }
  // a row or a unit that is not there counts nothing, whatever was read in its place
#pragma unroll
  for (int j = 0; j < MT; ++j)
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
      for (int t = 0; t < 4; ++t)
        if (16 * j + r >= (int)a.m || unit0 + u >= units) {
          xf[j][u][t] = i32x4{};
          sx[j][u][t] = 127;
        }
  int buf = 0;
  auto step = [&](auto more) {
    constexpr bool MORE = decltype(more)::value;  // a tile after this one
    f32x4 acc[H][MT] = {};
#pragma unroll
    for (int u = 0; u < U; ++u) {
#pragma unroll
      for (int h = 0; h < H; ++h)
#pragma unroll
        for (int t = 0; t < 4; ++t) {
          const int s = unit0 + u < units ? ws[u % RING][h][t] >> 8 * q : 127;
#pragma unroll
          for (int j = 0; j < MT; ++j)
            acc[h][j] = mfma128(w[u % RING][h][t], xf[j][u][t], acc[h][j], s, sx[j][u][t]);
        }
      if (u + RING < U)
        load(tile, u + RING);
      else if (MORE)
        load(tile + gridDim.x, u + RING - U);
    }
#pragma unroll
    for (int h = 0; h < H; ++h)
#pragma unroll
      for (int j = 0; j < MT; ++j) *(f32x4*)&part[buf][wave][h][16 * j + r][4 * q] = acc[h][j];
    // The weight's loads stay on their way.  With two buffers one barrier a tile: the other
    // one is written next, and read no later than the next barrier.
    lds_barrier();
    for (int o = threadIdx.x; o < 256 * MT; o += kStreamWaves * 64) {
      const int t = o >> 4, c = o & 15;
      const int64_t col = tile * 16 + c;
      if (t < (int)a.m && col < a.n) {
        float sum[H];
#pragma unroll
        for (int h = 0; h < H; ++h) {
          sum[h] = part[buf][0][h][t][c];
#pragma unroll
          for (int v = 1; v < kStreamWaves; ++v) sum[h] += part[buf][v][h][t][c];
        }
        float out = sum[0];
        if constexpr (GATED) gated<1>(&sum[0], &sum[1], &out);
        store1((T*)a.y + t * a.n + col, out);
      }
    }
    if (BUFS == 1 && MORE) lds_barrier();
    buf = BUFS - 1 - buf;
  };
  for (; tile + gridDim.x < tiles_n; tile += gridDim.x) step(std::true_type{});
  step(std::false_type{});
}

template <int U, int MT, bool GATED, bool VEC, typename XT>
hipError_t run_stream(const MxArgs& a, const MxGemm& g, hipStream_t stream) {
  const int64_t tiles_n = (a.n + 15) / 16;
  // two blocks a compute unit where the registers allow it
  const unsigned grid = (unsigned)std::min<int64_t>(tiles_n, kUnits * (U * (GATED ? 2 : 1) * MT <= 2 ? 2 : 1));
  if (g.y_type == QW_F32)
    mx_stream<U, MT, GATED, VEC, XT, float><<<grid, kStreamWaves * 64, 0, stream>>>(a);
  else
    mx_stream<U, MT, GATED, VEC, XT, uint16_t><<<grid, kStreamWaves * 64, 0, stream>>>(a);
  return hipGetLastError();
}

// Units of 512 that each of the waves takes of k.
int units_of_wave(int64_t k) { return (int)((mx_pitch(k) / 512 + kStreamWaves - 1) / kStreamWaves); }

// The most units of a wave that the stream kernel takes, for MT times 16 rows of x: they stay
// in registers, and the weight's ring beside them.
template <int MT, bool GATED>
constexpr int kMostUnits = MT == 1 ? (GATED ? 4 : 6) : MT == 2 ? (GATED ? 2 : 3) : GATED ? 1 : 2;

template <int MT, bool GATED, bool VEC, typename XT>
hipError_t run_stream(const MxArgs& a, const MxGemm& g, hipStream_t stream) {
  constexpr int MOST = kMostUnits<MT, GATED>;
  const int each = units_of_wave(g.k);
  if (each <= 1) return run_stream<1, MT, GATED, VEC, XT>(a, g, stream);
  if constexpr (MOST >= 2)
    if (each <= 2) return run_stream<2, MT, GATED, VEC, XT>(a, g, stream);
  if constexpr (MOST >= 3)
    if (each <= 3) return run_stream<3, MT, GATED, VEC, XT>(a, g, stream);
  if constexpr (MOST >= 4)
    if (each <= 4) return run_stream<4, MT, GATED, VEC, XT>(a, g, stream);
  return run_stream<MOST, MT, GATED, VEC, XT>(a, g, stream);
}

template <bool GATED>
hipError_t run_stream(const MxArgs& a, const MxGemm& g, hipStream_t stream) {
  if (g.x_type < 0) {
    if (g.m <= 16) return run_stream<1, GATED, true, uint8_t>(a, g, stream);
    return g.m <= 32 ? run_stream<2, GATED, true, uint8_t>(a, g, stream)
                     : run_stream<4, GATED, true, uint8_t>(a, g, stream);
  }
  const bool vec = g.k % 8 == 0 && aligned(g.x, 16);
  if (g.x_type == QW_F32)
    return vec ? run_stream<1, GATED, true, float>(a, g, stream) : run_stream<1, GATED, false, float>(a, g, stream);
  return vec ? run_stream<1, GATED, true, uint16_t>(a, g, stream) : run_stream<1, GATED, false, uint16_t>(a, g, stream);
}

// ---------------------------------------------------------------- choice
//
// Which tile: the one with the least estimated time,
//   first + again for every further round of the compute units + step for each 256 values of
//   k of each round,
// step being `lo` with hardly a tile on the chip, `mid` with one on every unit and `hi` with as
// many as the units hold: a lone tile is bound by its own latencies, all together by the
// clock that falls with the power.  From (us, bf16 results; tokens x weight rows x k):
//                    256x256  128x256  128x128   128x64  64x64 split
//   4096 4096 16384    133.0    156.6    164.0    214.9
//   4096 4096  4096     43.7     48.5     50.0     66.2
//   2048 4096 11008     73.7     58.2     60.5     78.6     93.4
//   2048 2048  4096     30.9     21.7     18.9     19.4     23.8
//   1024 4096  4096                       18.7     20.0     23.3
//    512 4096  4096     29.1     19.5     16.2     14.1     12.6
//    128 4096  4096                       15.4     12.7      9.4
//    128 4096 11008                       31.4     26.3     17.7
// and, the same choice, for other results (4096 11008 2048 with fp32 results; 2047 tokens, 2 x 11008
// weight rows, k = 4096 gated):
//   fp32 results         74.5     84       79        96
//   gated codes         111.5    128      126       180
//   gated bf16, fp32    112.5    127      125       167
//   gradients, bf16     150.5    157      150       190
//   gradients, fp32     239      221      221       295
// The last row is the one that the choice has wrong by 8 in a hundred: with fp32 gradients 256 x 256
// tiles keep 28 registers in scratch (9 with bf16; no other tile or result any).
// (256 x 128, weight rows first, loses to 128 x 256 by 2 to 5 in a hundred; 64 x 64 with two
// waves one after the other in k takes 12.7 and 26.1 in the last two and leads nowhere.)
struct Shape {
  int bn, bm;    // weight rows x tokens of a tile
  int per_unit;  // tiles that a compute unit holds
  double first, again, lo, mid, hi;
};
constexpr Shape kShapes[] = {
    {256, 256, 1, 14.0, 4.0, 0.85, 1.91, 1.91}, {128, 256, 1, 8.5, 5.0, 0.57, 1.13, 1.13},
    {128, 128, 2, 6.0, 3.0, 0.57, 0.78, 1.19},  {128, 64, 2, 4.6, 2.5, 0.50, 0.58, 0.80},
    {64, 64, 2, 4.5, 3.0, 0.29, 0.31, 0.48},  // split
};
constexpr int kShapeCount = sizeof(kShapes) / sizeof(kShapes[0]);

// Estimated us of n weight rows against m tokens.
double cost_of(const Shape& s, int64_t n, int64_t m, int kb) {
  const int64_t tiles = ((m + s.bm - 1) / s.bm) * ((n + s.bn - 1) / s.bn);
  if (tiles > 1 << 22) return 1e30;  // a launch holds fewer than 2^32 threads
  const double slots = (double)kUnits * s.per_unit, whole = std::floor(tiles / slots);
  const double rest = tiles - whole * slots;
  // short sums end before the results of the round before are written (4096 x 4096 x 256 16.1
  // us with 256 x 256 in one round, 19.9 with 128 x 128 in two)
  const double again = s.again + (kb <= 2 ? 3.0 : 0.0);
  double us = s.first + whole * (again + kb * s.hi) - again;
  if (rest > 0) {
    const double step = rest <= kUnits ? s.lo + (s.mid - s.lo) * rest / kUnits
                                       : s.mid + (s.hi - s.mid) * (rest - kUnits) / (slots - kUnits);
    us += again + kb * step;
  }
  return us;
}

int best_shape(int64_t n, int64_t m, int kb) {
  int best = 0;
  double least = 1e31;
  for (int i = 0; i < kShapeCount; ++i) {
    const double c = cost_of(kShapes[i], n, m, kb);
    if (c < least) {
      least = c;
      best = i;
    }
  }
  return best;
}

hipError_t run_shape(int shape, const MxArgs& a, const MxGemm& g, hipStream_t stream) {
  switch (shape) {
    case 0: return run_tiled<2, 4, 4, 2, 2, 1>(a, g, stream);
    case 1: return run_tiled<2, 2, 2, 4, 2, 1>(a, g, stream);
    case 2: return run_tiled<2, 2, 2, 2, 2, 2>(a, g, stream);
    case 3: return run_tiled<2, 1, 2, 2, 2, 2>(a, g, stream);
    default: return run_split(a, g, stream);
  }
}

}  // namespace

// The products that the stream kernel takes: up to 32 rows of x wherever it holds them (us
// against the tiles: 4096 x 4096 8.0 and 12.1, 4096 x 11008 10.5 and 23.7, 28672 x 4096 15.5 and
// 16.6, 28672 x 8192 29.2 and 27.8), up to 64 where the weight has at most 16384 rows (33 rows
// of 11008 x 4096 9.0 and 12.3, of 28672 x 4096 17.0 and 16.8; 64 rows 11.1 and 12.4, 19.3 and
// 17.4), since every block reads all rows of x.
bool mx_gemm_streams(MxResult result, int64_t n, int64_t m, int64_t k) {
  if ((result != MX_STORE && result != MX_GATED) || m > 64 || k == 0) return false;
  const bool gated = result == MX_GATED;
  if (m > 32 && (gated ? 2 * n : n) > 16384) return false;
  const int most = m <= 16 ? (gated ? kMostUnits<1, true> : kMostUnits<1, false>)
                 : m <= 32 ? (gated ? kMostUnits<2, true> : kMostUnits<2, false>)
                           : (gated ? kMostUnits<4, true> : kMostUnits<4, false>);
  return units_of_wave(k) <= most;
}

// The stream kernel quantizes x itself up to this many rows times units of a wave: every
// block pays for it (28672 x 8192 at 4 rows 26.9 us, at 8 rows 31.3; with codes 26.2 and 26.7,
// and 4.7 for a kernel that makes them; 4096 x 4096 at 16 rows 9.6, 7.6 and 2.1).
bool mx_gemm_fuses(MxResult result, int64_t m, int64_t k) {
  return m <= 16 && mx_gemm_streams(result, 0, m, k) && m * units_of_wave(k) <= 8;
}

hipError_t launch_mx_gemm(const MxGemm& g, hipStream_t stream) {
  const MxArgs a = args_of(g);
  if (mx_gemm_streams(g.result, g.n, g.m, g.k))
    return g.result == MX_GATED ? run_stream<true>(a, g, stream) : run_stream<false>(a, g, stream);
  return run_shape(best_shape(g.result == MX_STORE ? g.n : 2 * g.n, g.m, a.kb), a, g, stream);
}

int mx_gemm_path(MxResult result, int64_t n, int64_t m, int64_t k) {
  if (mx_gemm_streams(result, n, m, k)) return 100 * (m <= 16 ? 1 : m <= 32 ? 2 : 4) + units_of_wave(k);
  const int shape = best_shape(result == MX_STORE ? n : 2 * n, m, (int)((k + 255) / 256));
  return shape == kShapeCount - 1 ? 2 : kShapes[shape].bn * 1000 + kShapes[shape].bm;
}

}  // namespace qw
