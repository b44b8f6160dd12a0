// RMS norm with the residual's addition, its output in float, as e4m3 codes or as
// 4-bit codes, and its gradients, for gfx950.
//
//   s = x + residual,  r = 1 / sqrt(mean(s^2) + eps),  y = s r weight
//   ds = r (u - s r^2 mean(u s)) + dsum with u = dy weight,  dweight = sum of dy s r
//
// Bound by HBM: every input is read once and every output written once.  The lanes of
// a row hold it in registers between its sum and its results, 8 values of every
// 8 LANES a lane; the block of a scale is then 16 (e4m3) or 4 (4 bits) lanes side by
// side.
#include "mx_codes.h"

namespace qw {
namespace {

enum Form { FLOAT, BLOCK, MX };

struct NormArgs {
  int64_t rows, d;
  const void *x, *res, *weight;
  void *sum, *y, *scales;
  float eps;
  int w_type, y_type;
  int64_t pitch;  // values in a row of codes, or of y
};

// 8 weights from j on of d; 1 without weights.
__device__ __forceinline__ void load_weights(const void* w, int type, int64_t j, int64_t d,
                                             float v[8]) {
  if (!w) {
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = 1.0f;
  } else if (type == QW_F32) {
    load8_of_row<false>((const float*)w, j, d, v);
  } else {
    load8_of_row<false>((const uint16_t*)w, j, d, v);
  }
}

template <typename V>
__device__ __forceinline__ V wave_sum(V v) {
#pragma unroll
  for (int h = 1; h < 64; h <<= 1) v += __shfl_xor(v, h);
  return v;
}

// Sums over the LANES lanes of a row; `part`: N values for each wave of the block.
template <int LANES, int N, typename V>
__device__ __forceinline__ void row_sum(V (&v)[N], V (*part)[N]) {
#pragma unroll
  for (int i = 0; i < N; ++i) v[i] = wave_sum(v[i]);
  if (LANES == 64) return;
  __syncthreads();  // the last sums have been read
  if ((threadIdx.x & 63) == 0)
#pragma unroll
    for (int i = 0; i < N; ++i) part[threadIdx.x >> 6][i] = v[i];
  __syncthreads();
#pragma unroll
  for (int i = 0; i < N; ++i) {
    v[i] = part[0][i];
#pragma unroll
    for (int w = 1; w < LANES / 64; ++w) v[i] += part[w][i];
  }
}

// As the type holds it.
__device__ __forceinline__ float rounded(float v, float) { return v; }
__device__ __forceinline__ float rounded(float v, uint16_t) {
  return __uint_as_float((uint32_t)to_bf16(v) << 16);
}

// 8 results of a row from j on.
template <Form FORM, bool NT>
__device__ __forceinline__ void store_results(const NormArgs& a, int64_t row, int64_t j,
                                              const float v[8]) {
  if (FORM == FLOAT) {
    if (a.y_type == QW_F32)
      store8_of_row<false, NT>((float*)a.y + row * a.d, j, a.d, v);
    else
      store8_of_row<false, NT>((uint16_t*)a.y + row * a.d, j, a.d, v);
  } else if (FORM == BLOCK) {
    const float s = block_scale(max16(amax8(v)));
    const u32x2 c = codes8(v, s);
    if (j < a.pitch) {
      *(u32x2*)((uint8_t*)a.y + row * a.pitch + j) = c;
      if (j % QW_BLOCK == 0) ((float*)a.scales)[(row * a.pitch + j) / QW_BLOCK] = s;
    }
  } else {
    const uint32_t s = mx_scale(top_among<4>(top_of<8>(v)));
    const uint32_t c = mx_codes8(v, s);
    if (j < a.pitch) {
      *(uint32_t*)((uint8_t*)a.y + (row * a.pitch + j) / 2) = c;
      if (j % QW_MX_BLOCK == 0) ((uint8_t*)a.scales)[(row * a.pitch + j) / QW_MX_BLOCK] = (uint8_t)s;
    }
  }
}

// LANES lanes a row, CH times 8 values each; CH 0: as many as there are, in two passes
// over the row.
template <int LANES, int CH, bool NT, Form FORM, typename T>
__global__ __launch_bounds__(256) void norm(NormArgs a) {
  constexpr int N = CH ? CH : 1, ROWS = 256 / LANES;
  __shared__ double part[4][1];
  const int lane = threadIdx.x % LANES;
  // all waves of a block take as many rows: the block's barriers see all of them
  for (int64_t r0 = (int64_t)blockIdx.x * ROWS; r0 < a.rows; r0 += (int64_t)gridDim.x * ROWS) {
    const int64_t row = r0 + threadIdx.x / LANES;
    if (LANES == 64 && row >= a.rows) return;
    const T* x = (const T*)a.x + row * a.d;
    const T* res = a.res ? (const T*)a.res + row * a.d : nullptr;
    T* sum = a.sum ? (T*)a.sum + row * a.d : nullptr;
    float v[N][8];
    double sq[1] = {0.0};
    auto load = [&](int64_t j, float* s) {
      load8_of_row<false, NT>(x, j, a.d, s);
      if (res) {
        float t[8];
        load8_of_row<false, NT>(res, j, a.d, t);
#pragma unroll
        for (int i = 0; i < 8; ++i) s[i] = rounded(s[i] + t[i], T{});
      }
    };
    auto first = [&](int64_t j, float* s) {
      load(j, s);
      if (sum) store8_of_row<false, NT>(sum, j, a.d, s);
#pragma unroll
      for (int i = 0; i < 8; ++i) sq[0] = __builtin_fma((double)s[i], (double)s[i], sq[0]);
    };
    if (CH) {
#pragma unroll
      for (int c = 0; c < N; ++c) first((int64_t)(c * LANES + lane) * 8, v[c]);
    } else {
      for (int64_t j = lane * 8; j < a.d; j += LANES * 8) first(j, v[0]);
    }
    row_sum<LANES>(sq, part);
    // squares and their sum in 64 bits, r in two parts, and s r with its rounding's rest: y is
    // rounded once, so that hardly one of its codes is a neighbour of the right one (HBM leaves
    // most of the time: 8192 x 8192 bf16 into e4m3 107 us so, 105 in fp32 with two roundings)
    const double r = 1.0 / __builtin_sqrt(sq[0] / (double)a.d + (double)a.eps);
    const float rh = (float)r, rl = __builtin_isinf(rh) ? 0.0f : (float)(r - (double)rh);
    auto second = [&](int64_t j, float* s) {
      float w[8];
      load_weights(a.weight, a.w_type, j, a.d, w);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float p = s[i] * rh, e = __builtin_fmaf(s[i], rl, __builtin_fmaf(s[i], rh, -p));
        // (an infinite weight meets e = 0 as a finite one)
        s[i] = __builtin_fmaf(p, w[i], e * __builtin_amdgcn_fmed3f(w[i], -__FLT_MAX__, __FLT_MAX__));
      }
      // behind the row: zeros, also of a row whose r is infinite
      if (FORM != FLOAT && j + 8 > a.d)
#pragma unroll
        for (int i = 0; i < 8; ++i) s[i] = j + i < a.d ? s[i] : 0.0f;
      store_results<FORM, NT>(a, row, j, s);
    };
    if (CH) {
#pragma unroll
      for (int c = 0; c < N; ++c) second((int64_t)(c * LANES + lane) * 8, v[c]);
    } else {
      // whole rounds of lanes: a block's lanes exchange its maximum
      for (int64_t j = lane * 8; j - lane * 8 < a.pitch; j += LANES * 8) {
        // this lane wrote what it reads here, where sum is x or the residual
        if (sum && j < a.d)
          load8_of_row<false>((const T*)sum, j, a.d, v[0]);
        else
          load(j, v[0]);
        second(j, v[0]);
      }
    }
  }
}

struct NormBackArgs {
  int64_t rows, d;
  const void *dy, *s, *weight, *dsum;
  void* ds;
  float* part;  // [grid][d]: each block's share of dweight
  float eps;
  int w_type;
};

// The rows of a block in turn; its share of dweight stays in registers (CH 0: in
// memory, each lane adding to its own).
// Bound by HBM: 8192 x 4096 bf16 66 us (4.1 TB/s), 4099 x 4096 fp32 57 (4.7), rows that start
// anywhere in a line less (4099 x 5003 fp32 89 us, 3.7).  The row's sums are fp32: the registers are
// full, and in 64 bits 8192 x 8192 bf16 would take 211 us, not 132.  Rows whose squares fp32 may not
// hold are summed a second time; for its code four chunks keep up to 6 registers in scratch,
// since one more than 168 would leave two blocks a compute unit (209 us; 131 without that code).
template <int LANES, int CH, typename T>
__global__ __launch_bounds__(256, CH == 4 ? 3 : 1) void norm_backward(NormBackArgs a) {
  constexpr int N = CH ? CH : 1, ROWS = 256 / LANES;
  __shared__ float part[4][2];
  __shared__ float join[LANES == 64 && CH ? N * 512 : 1];
  const int lane = threadIdx.x % LANES;
  float dw[N][8] = {};
  float* const mine = a.part ? a.part + (int64_t)blockIdx.x * a.d : nullptr;
  bool fresh = true;
  for (int64_t r0 = (int64_t)blockIdx.x * ROWS; r0 < a.rows; r0 += (int64_t)gridDim.x * ROWS) {
    const int64_t row = r0 + threadIdx.x / LANES;
    if (LANES == 64 && row >= a.rows) break;
    const T* dy = (const T*)a.dy + row * a.d;
    const T* s = (const T*)a.s + row * a.d;
    float u[N][8], v[N][8], sums[2] = {0.0f, 0.0f};
    auto add = [&](int64_t j, const float* g, const float* h) {
      float w[8];
      load_weights(a.weight, a.w_type, j, a.d, w);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        sums[0] = __builtin_fmaf(h[i], h[i], sums[0]);
        sums[1] = __builtin_fmaf(g[i] * w[i], h[i], sums[1]);
      }
    };
    int e = 0;  // s is taken 2^-e times
    auto load = [&](int64_t j, float* g, float* h) {
      load8_of_row<false>(dy, j, a.d, g);
      load8_of_row<false>(s, j, a.d, h);
    };
    auto scale = [&](float* h) {
#pragma unroll
      for (int i = 0; i < 8; ++i) h[i] = __builtin_ldexpf(h[i], -e);
    };
    // The row's sums, of values from memory or (CH) as they are held.
    auto sum_up = [&](bool held) {
      sums[0] = sums[1] = 0.0f;
      if (CH) {
#pragma unroll
        for (int c = 0; c < N; ++c) {
          if (held)
            scale(v[c]);
          else
            load((int64_t)(c * LANES + lane) * 8, u[c], v[c]);
          add((int64_t)(c * LANES + lane) * 8, u[c], v[c]);
        }
      } else {
        for (int64_t j = lane * 8; j < a.d; j += LANES * 8) {
          load(j, u[0], v[0]);
          if (held) scale(v[0]);
          add(j, u[0], v[0]);
        }
      }
      row_sum<LANES>(sums, part);
      return sums[0] / (float)a.d + __builtin_ldexpf(a.eps, -2 * e);
    };
    float mean = sum_up(false);
    // Squares that fp32 may not have held: again with s by a power of two, which leaves a root of
    // the mean from 2^-126 on between 2^-46 and 2^44.
    if (__builtin_expect(mean < 0x1p-80f || mean > 0x1p80f, 0)) {
      e = mean > 1.0f ? 84 : -80;
      mean = sum_up(true);
    }
    const float r = 1.0f / __builtin_sqrtf(mean), rs = __builtin_ldexpf(r, -e);  // of s 2^-e, of s
    const float f = sums[1] / (float)a.d * r * r;
    auto second = [&](int64_t j, const float* g, const float* h, float* share) {
      if (a.ds) {
        float w[8], t[8];
        load_weights(a.weight, a.w_type, j, a.d, w);
#pragma unroll
        for (int i = 0; i < 8; ++i) t[i] = 0.0f;
        if (a.dsum) load8_of_row<false>((const T*)a.dsum + row * a.d, j, a.d, t);
#pragma unroll
        for (int i = 0; i < 8; ++i)
          t[i] = __builtin_fmaf(rs, __builtin_fmaf(-h[i], f, g[i] * w[i]), t[i]);
        store8_of_row<false>((T*)a.ds + row * a.d, j, a.d, t);
      }
#pragma unroll
      for (int i = 0; i < 8; ++i) share[i] = __builtin_fmaf(g[i], h[i] * r, share[i]);
    };
    if (CH) {
#pragma unroll
      for (int c = 0; c < N; ++c) second((int64_t)(c * LANES + lane) * 8, u[c], v[c], dw[c]);
    } else {
      for (int64_t j = lane * 8; j < a.d; j += LANES * 8) {
        load(j, u[0], v[0]);
        if (e != 0) scale(v[0]);
        float share[8] = {};
        if (mine && !fresh) load8_of_row<false>(mine, j, a.d, share);
        second(j, u[0], v[0], share);
        if (mine) store8_of_row<false>(mine, j, a.d, share);
      }
      fresh = false;
    }
  }
  if (!CH || !mine) return;
  if (LANES == 64) {
    // the four waves' shares, one after the other
    for (int w = 0; w < 4; ++w) {
      __syncthreads();
      if ((int)(threadIdx.x >> 6) != w) continue;
#pragma unroll
      for (int c = 0; c < N; ++c)
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          float* to = &join[(c * 8 + i) * 64 + lane];
          *to = w == 0 ? dw[c][i] : *to + dw[c][i];
          dw[c][i] = *to;
        }
    }
    if (threadIdx.x < 192) return;  // the last wave has the sum
  }
#pragma unroll
  for (int c = 0; c < N; ++c) store8_of_row<false>(mine, (int64_t)(c * LANES + lane) * 8, a.d, dw[c]);
}

// dweight from the blocks' shares: a thread block takes 32 columns, each of its 32 halves of
// waves every 32nd share, in a fixed order.
__global__ __launch_bounds__(1024) void sum_shares(const float* __restrict__ part,
                                                   float* __restrict__ dw, int64_t d, int count) {
  __shared__ float sums[32][33];
  const int lane = threadIdx.x & 31, group = threadIdx.x >> 5;
  for (int64_t c0 = (int64_t)blockIdx.x * 32; c0 < d; c0 += (int64_t)gridDim.x * 32) {
    const int64_t c = c0 + lane;
    float s = 0.0f;
    if (c < d) {
      int i = group;
      for (; i + 7 * 32 < count; i += 8 * 32) {
        float v[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] = part[(int64_t)(i + 32 * j) * d + c];
#pragma unroll
        for (int j = 0; j < 8; ++j) s += v[j];
      }
      for (; i < count; i += 32) s += part[(int64_t)i * d + c];
    }
    __syncthreads();
    sums[group][lane] = s;
    __syncthreads();
    float t = sums[lane][group];  // share `lane` of column `group`
#pragma unroll
    for (int h = 1; h < 32; h <<= 1) t += __shfl_xor(t, h);
    if (lane == 0 && c0 + group < d) dw[c0 + group] = t;
  }
}

// Whether rows go past the caches: large ones of 2 bytes, whose lanes read whole runs of 16
// bytes (8192 x 8192 bf16 into e4m3: 115 -> 109 us; fp32 rows, a lane's 32 bytes in two
// loads, lose).
template <typename T>
bool past_caches(int64_t rows, int64_t d) {
  return sizeof(T) == 2 && d % 8 == 0 && rows * d >= 16ll << 20;
}

template <Form FORM, typename T>
hipError_t run_norm(const NormArgs& a, hipStream_t stream) {
  const int64_t lanes = (a.pitch + 7) / 8;  // chunks of 8 in a row
  auto go = [&](auto lanes_of_row, auto chunks) {
    constexpr int LANES = decltype(lanes_of_row)::value, CH = decltype(chunks)::value;
    // a row that is read twice stays in the caches
    if (CH && past_caches<T>(a.rows, a.d))
      norm<LANES, CH, CH && sizeof(T) == 2, FORM, T><<<grid_for(a.rows, 256 / LANES), 256, 0, stream>>>(a);
    else
      norm<LANES, CH, false, FORM, T><<<grid_for(a.rows, 256 / LANES), 256, 0, stream>>>(a);
  };
  using std::integral_constant;
  if (lanes <= 64)
    go(integral_constant<int, 64>{}, integral_constant<int, 1>{});
  else if (lanes <= 128)
    go(integral_constant<int, 64>{}, integral_constant<int, 2>{});
  else if (lanes <= 256)
    go(integral_constant<int, 256>{}, integral_constant<int, 1>{});
  else if (lanes <= 512)
    go(integral_constant<int, 256>{}, integral_constant<int, 2>{});
  else if (lanes <= 768)
    go(integral_constant<int, 256>{}, integral_constant<int, 3>{});
  else if (lanes <= 1024)
    go(integral_constant<int, 256>{}, integral_constant<int, 4>{});
  else if (lanes <= 1536)
    go(integral_constant<int, 256>{}, integral_constant<int, 6>{});
  else if (lanes <= 2048)
    go(integral_constant<int, 256>{}, integral_constant<int, 8>{});
  else
    go(integral_constant<int, 256>{}, integral_constant<int, 0>{});
  return hipGetLastError();
}

// Blocks of the backward kernel, each with a share of dweight: as many as are on the chip at
// once, since each takes as many rows (registers: three of a compute unit from three chunks
// on, four below; 4099 x 5003 fp32 104 us with 1024 blocks, 89 with 768).
int64_t shares_of(int64_t rows, int64_t d) {
  const int64_t most = (d + 7) / 8 > 512 ? 768 : 1024;
  return rows < most ? rows : most;
}

template <typename T>
hipError_t run_backward(const NormBackArgs& a, int grid, hipStream_t stream) {
  const int64_t lanes = (a.d + 7) / 8;
  auto go = [&](auto lanes_of_row, auto chunks) {
    norm_backward<decltype(lanes_of_row)::value, decltype(chunks)::value, T>
        <<<grid, 256, 0, stream>>>(a);
  };
  using std::integral_constant;
  if (lanes <= 64)
    go(integral_constant<int, 64>{}, integral_constant<int, 1>{});
  else if (lanes <= 128)
    go(integral_constant<int, 64>{}, integral_constant<int, 2>{});
  else if (lanes <= 256)
    go(integral_constant<int, 256>{}, integral_constant<int, 1>{});
  else if (lanes <= 512)
    go(integral_constant<int, 256>{}, integral_constant<int, 2>{});
  else if (lanes <= 768)
    go(integral_constant<int, 256>{}, integral_constant<int, 3>{});
  else if (lanes <= 1024)
    go(integral_constant<int, 256>{}, integral_constant<int, 4>{});
  else
    go(integral_constant<int, 256>{}, integral_constant<int, 0>{});
  return hipGetLastError();
}

}  // namespace

hipError_t launch_rms_norm(const RmsNorm& g, hipStream_t stream) {
  NormArgs a = {g.rows, g.d, g.x, g.res, g.weight, g.sum, g.y, g.scales, g.eps, g.w_type, g.y_type, 0};
  a.pitch = g.form == 0 ? g.d : g.form == 1 ? pitch(g.d) : mx_pitch(g.d);
  const bool f32 = g.type == QW_F32;
  switch (g.form) {
    case 0: return f32 ? run_norm<FLOAT, float>(a, stream) : run_norm<FLOAT, uint16_t>(a, stream);
    case 1: return f32 ? run_norm<BLOCK, float>(a, stream) : run_norm<BLOCK, uint16_t>(a, stream);
    default: return f32 ? run_norm<MX, float>(a, stream) : run_norm<MX, uint16_t>(a, stream);
  }
}

// A size that grows with every argument: the most shares, whatever the width.
int64_t rms_norm_shares(int64_t rows) { return rows < 1024 ? rows : 1024; }

hipError_t launch_rms_norm_backward(const RmsNormBackward& g, hipStream_t stream) {
  const int grid = (int)shares_of(g.rows, g.d);
  NormBackArgs a = {g.rows, g.d, g.dy, g.s, g.weight, g.dsum, g.ds,
                    g.dweight ? (float*)g.work : nullptr, g.eps, g.w_type};
  hipError_t e = g.type == QW_F32 ? run_backward<float>(a, grid, stream)
                                  : run_backward<uint16_t>(a, grid, stream);
  if (e != hipSuccess || !g.dweight) return e;
  sum_shares<<<grid_for(g.d, 32), 1024, 0, stream>>>(a.part, g.dweight, g.d, grid);
  return hipGetLastError();
}

}  // namespace qw
