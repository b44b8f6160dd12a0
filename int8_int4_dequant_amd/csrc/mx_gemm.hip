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

struct MxArgs {
  const uint8_t *w, *ws, *x, *xs;
  int64_t n, m;       // outputs in a row (gated: f), rows
  int64_t kp2, ksp;   // bytes of a row of codes, of scales
  int kb;             // steps of 256 along k
  void* y;
  uint8_t* ys;
  int64_t yp;         // MX_GATED_CODES: values in a row of codes
  const void* dh;
  void* h;
  int64_t tiles_m, tiles;
  int vec;            // 16 bytes of outputs may be stored as one
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

template <int RUN, typename T>
__device__ __forceinline__ void put(T* p, const float* v, int64_t left, bool vec) {
  if (vec && left >= RUN) {
    if constexpr (RUN == 8)
      store8<true>(p, v);
    else
      store4(p, f32x4{v[0], v[1], v[2], v[3]});
  } else {
#pragma unroll
    for (int c = 0; c < RUN; ++c)
      if (c < left) store1(p + c, v[c]);
  }
}
template <int RUN, typename T>
__device__ __forceinline__ void get(const T* p, float* v, int64_t left, bool vec) {
  if (vec && left >= RUN) {
    if constexpr (RUN == 8) {
      load8<true>(p, v);
    } else {
      const f32x4 t = *(const f32x4*)p;
#pragma unroll
      for (int c = 0; c < RUN; ++c) v[c] = t[c];
    }
  } else {
#pragma unroll
    for (int c = 0; c < RUN; ++c) v[c] = c < left ? load1(p + c) : 0.0f;
  }
}

// dgate and dup, h.  With e = exp(-|gate|) neither t nor 1 - t overflows or cancels;
// beyond |gate| = 200 one of them is zero in fp32.
__device__ __forceinline__ void gate_gradients(float gate, float up, float dh, float& dgate,
                                               float& dup, float& h) {
  const float e = expf(-fabsf(gate));
  const float one = 1.0f / (1.0f + e), other = e * one;
  const bool neg = gate < 0.0f;
  const float t = neg ? other : one, u = neg ? one : other;
  const float near = fminf(fmaxf(gate, -200.0f), 200.0f);
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
    put<R::RUN>((T*)a.y + row * a.n + col, o, a.n - col, a.vec);
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
      get<RUN>((const T*)a.dh + row * a.n + col, dh, left, a.vec);
#pragma unroll
      for (int c = 0; c < RUN; ++c)
        gate_gradients(gate[RUN * g + c], up[RUN * g + c], dh[c], dg[c], du[c], h[c]);
      put<RUN>((T*)a.y + row * 2 * a.n + col, dg, left, a.vec);
      put<RUN>((T*)a.y + row * 2 * a.n + a.n + col, du, left, a.vec);
      if (a.h) put<RUN>((T*)a.h + row * a.n + col, h, left, a.vec);
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
        put<RUN>((T*)a.y + row * a.n + col, v + RUN * g, a.n - col, a.vec);
      }
    } else {
      // The 32 values are one block: half of them in the lane 32 away.
      uint32_t top = top_of<16>(v);
      top = max(top, (uint32_t)__shfl_xor((int)top, 32));
      const uint32_t s = mx_scale(top);
      const uint32_t lo = mx_codes8(v, s), hi = mx_codes8(v + 8, s);
      if (have && col0 < a.yp) {
        uint8_t* const to = (uint8_t*)a.y + (row * a.yp + col0) / 2 + 4 * half;
        *(uint32_t*)to = lo;
        *(uint32_t*)(to + 8) = hi;
        if (half == 0) a.ys[(row * a.yp + col0) / 32] = (uint8_t)s;
      }
    }
  }
}

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
//
// A step has four products a fragment; of the t-th, a lane holds block 4 (l / 32) + t, so
// that byte t of one word of its row's scales goes with it.
//
// A block takes tile after tile (in steps of the grid) and the copies run on: behind the
// last step of a tile come the first ones of the next, which are on their way while the
// results are written.  `chunks` of 4 steps and the two buffers of their scales are counted
// through in the same way.
//
// Gated results: the tile's rows are 32 gate rows and their 32 up rows in turn, so that a
// lane holds both values of a result.

template <int NF, int MF, int WN, int WM, int STAGES, MxResult RES, typename T>
__global__ __launch_bounds__(WN * WM * 64, WN * WM == 8 ? 2 : 1) void mx_tiled(MxArgs a) {
  constexpr int WAVES = WN * WM, BN = 32 * NF * WN, BM = 32 * MF * WM, ROWS = BN + BM;
  constexpr bool GATED = RES != MX_STORE;
  constexpr int COLS = GATED ? BN / 2 : BN;        // outputs of a row in a tile
  constexpr int SEGS = ROWS / 8 / WAVES;           // 8-row pieces of a wave
  constexpr int SPER = ROWS / 32 / WAVES;          // 32-row pieces of scales of a wave
  static_assert(ROWS / 32 % WAVES == 0 && BN % 64 == 0 && BM % 64 == 0, "whole pieces");
  static_assert(!GATED || NF % 2 == 0, "gate and up rows in one wave");
  __shared__ __align__(1024) uint8_t lds[STAGES][ROWS * 128];
  __shared__ __align__(1024) uint8_t scales[2][ROWS * 32];
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int lane = threadIdx.x & 63, r = lane & 31, half = lane >> 5;
  const int wm = wave % WM * 32 * MF, wn = wave / WM * 32 * NF;
  // the weight row (of gate or up) that LDS row `row` holds
  auto weight_row = [](int row) {
    const int at = GATED ? row / 64 * 32 + row % 32 : row;
    return kSwapped<RES, T> ? swapped(at) : at;
  };
  uint32_t voff[SEGS], soff[SPER];
#pragma unroll
  for (int s = 0; s < SEGS; ++s) {
    const int row = (wave + WAVES * s) * 8 + (lane >> 3);
    const int c = (lane & 7) ^ ((row >> 1) & 7);
    const int at = row >= BN ? row - BN : weight_row(row);
    voff[s] = (uint32_t)at * (uint32_t)a.kp2 + c * 16;
  }
#pragma unroll
  for (int s = 0; s < SPER; ++s) {
    const int row = (wave + WAVES * s) * 32 + (lane >> 1);
    const int at = row >= BN ? row - BN : weight_row(row);
    soff[s] = (uint32_t)at * (uint32_t)a.ksp + (lane & 1) * 16;
  }
  // A tile, and each piece's buffer, of which the rows behind the last one are not a part.
  struct Place {
    int64_t n0, m0;
    int rows;
    i32x4 from[SEGS], sfrom[SPER];
  };
  auto place = [&](int64_t tile, Place& p) {
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
  };
  const int kb = a.kb, chunks = (kb + 3) >> 2;
  Place here, then;
  place(blockIdx.x, here);
  const uint32_t lds0 = (uint32_t)(uintptr_t)(__attribute__((address_space(3))) uint8_t*)&lds[0][0];
  const uint32_t lds1 = (uint32_t)(uintptr_t)(__attribute__((address_space(3))) uint8_t*)&scales[0][0];
  // Behind the last tile there is nothing to read, but the copy is issued all the same (as
  // zeros, from an empty buffer), so that every step has as many.
  auto fetch = [&](int b, int buf, int s) {
    if (s >= SEGS) return;
    const bool in = b < kb;
    i32x4 buffer = here.from[s];
#pragma unroll
    for (int c = 0; c < 3; ++c) buffer[c] = in ? buffer[c] : then.from[s][c];
    copy_to_lds(buffer, voff[s], (uint32_t)(in ? b : b - kb) * 128,
                lds0 + buf * (ROWS * 128) + (wave + WAVES * s) * 1024);
  };
  int base = 0;  // which of the two buffers holds the tile's first scales
  auto fetch_scales = [&](int u, bool when) {  // of steps 4 u .. 4 u + 3
    const bool in = u < chunks;
#pragma unroll
    for (int s = 0; s < SPER; ++s) {
      i32x4 buffer = here.sfrom[s];
#pragma unroll
      for (int c = 0; c < 3; ++c) buffer[c] = in ? buffer[c] : then.sfrom[s][c];
      copy_to_lds_when(__builtin_amdgcn_readfirstlane(when ? 1 : 0), buffer, soff[s],
                       (uint32_t)(in ? u : u - chunks) * 32,
                       lds1 + ((base + u) & 1) * (ROWS * 32) + (wave + WAVES * s) * 1024);
    }
  };
  int64_t tile = blockIdx.x + gridDim.x;
  place(tile, then);
  fetch_scales(0, true);
  fetch_scales(1, true);
#pragma unroll
  for (int b = 0; b < STAGES; ++b)
#pragma unroll
    for (int s = 0; s < SEGS; ++s) fetch(b, b, s);

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
    const int u = b < kb ? b >> 2 : chunks, in = b < kb ? b & 3 : 0;  // behind the last: the next tile's first
    const uint8_t* p = &scales[(base + u) & 1][r * 32 + in * 8 + 4 * half];
    if (n < MF)
      sx2[n] = *(const int*)(p + (BN + wm + 32 * n) * 32);
    else if (n < MF + NF)
      sw2[n - MF] = *(const int*)(p + (wn + 32 * (n - MF)) * 32);
  };
  constexpr int FRAGS = NF + MF, PRODUCTS = NF * MF;
  constexpr int TAKES = (FRAGS + PRODUCTS - 1) / PRODUCTS, COPIES = (SEGS + PRODUCTS - 1) / PRODUCTS;
  // Copies that may be on their way when step b + 1 has to be there: those of the
  // STAGES - 2 steps behind it.  Scales are issued before the copies of their step and four
  // steps ahead of their use: they only make the wait longer.
  constexpr int LEFT = (STAGES - 2) * SEGS;
  static_assert(STAGES >= 2 && STAGES <= 4, "scales have landed by then");
  landed<LEFT + SEGS>();
#pragma unroll
  for (int n = 0; n < FRAGS; ++n) {
    take(0, std::integral_constant<int, 0>{}, n);
    take_scale(0, n);
  }
  int buf = 0;
  for (;;) {
  f32x16 acc[NF][MF] = {};
  for (int b = 0; b < kb; ++b) {
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
    // wave does, they are filled again.
    landed<LEFT>();
    fetch_scales((b >> 2) + 2, (b & 3) == 3 || b + 1 == kb);
    products(std::integral_constant<int, 3>{}, [&](int p) {
#pragma unroll
      for (int n = 0; n < COPIES; ++n) fetch(b + STAGES, buf, p * COPIES + n);
#pragma unroll
      for (int n = 0; n < TAKES; ++n) {
        take(next, std::integral_constant<int, 0>{}, p * TAKES + n);
        take_scale(b + 1, p * TAKES + n);
      }
    });
    buf = next;
  }
#pragma unroll
  for (int j = 0; j < MF; ++j) {
    const int64_t row = here.m0 + wm + 32 * j + r;
    const bool have = wm + 32 * j + r < here.rows;
    if constexpr (GATED) {
#pragma unroll
      for (int i = 0; i < NF; i += 2)
        store_gated<RES, T>(a, acc[i][j], acc[i + 1][j], row, here.n0 + (wn + 32 * i) / 2, half, have);
    } else {
      if (!have) continue;
#pragma unroll
      for (int i = 0; i < NF; ++i) store_fragment<T>(a, acc[i][j], row, here.n0 + wn + 32 * i, half);
    }
  }
  if (tile >= a.tiles) break;
  here = then;
  base += chunks;
  tile += gridDim.x;
  place(tile, then);
  }
  landed<0>();  // the empty copies too, before the block's LDS is another's
}

constexpr int kUnits = 256;  // compute units

// PER_UNIT: blocks that a compute unit holds.
template <int NF, int MF, int WN, int WM, int STAGES, int PER_UNIT>
hipError_t run_tiled(MxArgs a, const MxGemm& g, hipStream_t stream) {
  constexpr int BN = 32 * NF * WN, BM = 32 * MF * WM;
  const int cols = g.result == MX_STORE ? BN : BN / 2;
  a.tiles_m = (a.m + BM - 1) / BM;
  a.tiles = a.tiles_m * (((g.result == MX_GATED_CODES ? a.yp : a.n) + cols - 1) / cols);
  // Tile after tile where there are more than the units hold; copies that run on into the
  // next tile need two chunks of scales in each.
  const unsigned grid = (unsigned)(a.kb > 4 ? std::min<int64_t>(a.tiles, kUnits * PER_UNIT) : a.tiles);
  auto go = [&](auto result, auto type) {
    mx_tiled<NF, MF, WN, WM, STAGES, decltype(result)::value, decltype(type)>
        <<<grid, WN * WM * 64, 0, stream>>>(a);
  };
  auto typed = [&](auto result) { g.y_type == QW_F32 ? go(result, 0.0f) : go(result, uint16_t{}); };
  switch (g.result) {
    case MX_STORE: typed(std::integral_constant<MxResult, MX_STORE>{}); break;
    case MX_GATED: typed(std::integral_constant<MxResult, MX_GATED>{}); break;
    case MX_GATED_CODES: go(std::integral_constant<MxResult, MX_GATED_CODES>{}, 0.0f); break;
    default: typed(std::integral_constant<MxResult, MX_GATED_BACKWARD>{});
  }
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
  a.kp2 = kp / 2;
  a.ksp = kp / 32;
  a.kb = (int)((g.k + 255) / 256);
  a.y = g.y;
  a.ys = g.ys;
  a.yp = mx_pitch(g.n);
  a.dh = g.dh;
  a.h = g.h;
  a.vec = g.n % (g.y_type == QW_BF16 ? 8 : 4) == 0 && aligned(g.y, 16) && aligned(g.h, 16) && aligned(g.dh, 16);
  return a;
}

}  // namespace

hipError_t launch_mx_gemm(const MxGemm& g, hipStream_t stream) {
  const MxArgs a = args_of(g);
  const int64_t rows = g.result == MX_STORE ? g.n : 2 * g.n;
  auto tiles = [&](int t) { return ((g.m + t - 1) / t) * ((rows + t - 1) / t); };
  if (tiles(256) >= 256 || tiles(64) > 1 << 22) return run_tiled<2, 4, 4, 2, 2, 1>(a, g, stream);
  if (tiles(128) >= 256) return run_tiled<2, 2, 2, 2, 2, 2>(a, g, stream);
  return run_tiled<2, 1, 1, 2, 3, 2>(a, g, stream);
}

}  // namespace qw
