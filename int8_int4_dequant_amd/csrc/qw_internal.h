// Internal interfaces between the C ABI (qw_api.hip) and the kernel files.
// Not installed; the public interface is include/qw.h.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "../../include/qw.h"

namespace qw {

// Problem description after validation by the C ABI.
struct Mat {
  int bits;        // 4 or 8
  int64_t group;   // elements per scale, divides n*k
  int64_t n, k;    // rows (output channels), row length (reduction axis)
};

inline bool aligned(const void* p, uintptr_t a) {
  return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0;
}

// Each launcher enqueues on `stream` and returns hipSuccess or the launch
// error.  Shapes are already validated and non-empty.
hipError_t launch_quantize_pack(const Mat& mt, const float* w, uint8_t* payload,
                                float* scales, hipStream_t stream);
hipError_t launch_quantize_pack_batched(const Mat* mts, const float* const* ws,
                                        uint8_t* const* payloads, float* const* scales,
                                        int count, hipStream_t stream);
hipError_t launch_unpack(const Mat& mt, const uint8_t* payload,
                         const float* scales, float* w_out, hipStream_t stream);
// Several matrices, each exactly as launch_unpack writes it; vector-path
// matrices of one bit width share launches (QW_BATCH_PER_LAUNCH at a time).
hipError_t launch_unpack_batched(const Mat* mts, const uint8_t* const* payloads,
                                 const float* const* scales, float* const* outs, int count,
                                 hipStream_t stream);
hipError_t launch_gemv(const Mat& mt, const uint8_t* payload, const float* scales,
                       int m, const float* x, float* y, hipStream_t stream);
hipError_t launch_gemv_batched(const Mat* mts, const uint8_t* const* payloads,
                               const float* const* scales, int m, const float* const* xs,
                               float* const* ys, int count, hipStream_t stream);
hipError_t launch_gemm(const Mat& mt, const uint8_t* payload, const float* scales,
                       int64_t m, const uint16_t* x, float* y, hipStream_t stream);
hipError_t launch_fill_zero(float* y, int64_t count, hipStream_t stream);
// x fp32 [count] -> bf16 bit patterns, round to nearest even (gemm.hip).
hipError_t launch_round_bf16(const float* x, uint16_t* xb, int64_t count, hipStream_t stream);

// GPTQ (gptq.hip).  Work buffers are caller-provided device memory of at
// least the returned sizes.
int64_t gptq_hessian_work_bytes(int64_t k, int64_t t);
hipError_t launch_gptq_hessian(int64_t k, int64_t t, const float* x, double* h, void* work,
                               hipStream_t stream);
int64_t gptq_factor_work_bytes(int64_t k);
hipError_t launch_gptq_factor(int64_t k, const double* h, double damp, double* u, int32_t* info,
                              void* work, hipStream_t stream);
int64_t gptq_quantize_work_bytes(int64_t n, int64_t k);
hipError_t launch_gptq_quantize_pack(const Mat& mt, const float* w, const double* u,
                                     uint8_t* payload, float* scales, void* work,
                                     hipStream_t stream);

// Block-scaled e4m3 (block.hip).  `brows` is 1 or QW_BLOCK; codes are 16-byte
// aligned rows of pitch(k) bytes.
inline int64_t pitch(int64_t k) { return (k + QW_BLOCK - 1) / QW_BLOCK * QW_BLOCK; }
inline int64_t block_scales(int brows, int64_t n, int64_t k) {
  return (n + brows - 1) / brows * (pitch(k) / QW_BLOCK);
}
hipError_t launch_block_quantize(int brows, int64_t count, int64_t n, int64_t k, int type,
                                 const void* w, uint8_t* codes, float* scales,
                                 hipStream_t stream);
hipError_t launch_block_quantize_swiglu(int64_t rows, int64_t f, int type, const void* h,
                                        const int32_t* used, uint8_t* codes, float* scales,
                                        hipStream_t stream);
hipError_t launch_block_unpack(int brows, int64_t count, int64_t n, int64_t k,
                               const uint8_t* codes, const float* scales, float* out,
                               hipStream_t stream);
// Whether launch_block_gemm takes float x of these sizes (k > 0) and quantizes
// it itself.
bool block_gemm_fuses(int64_t m, int64_t k);
// One product.  x_type: QW_F32 or QW_BF16 (x) or -1 (xc and xs).
struct BlockGemm {
  int brows;
  int64_t n, k, m;
  const uint8_t* codes;
  const float* scales;
  int x_type;
  const void* x;
  const uint8_t* xc;
  const float* xs;
  int y_type;
  void* y;
  bool exact;  // fp32 y: on the bf16 cores (within an expert MLP with bf16 y it goes without)
};
hipError_t launch_block_gemm(const BlockGemm& g, hipStream_t stream);
hipError_t launch_block_gemm_grouped(const BlockGemm& g, int64_t experts,
                                     const int32_t* offsets, hipStream_t stream);
// Grouped products with float x (x_type, x; y fp32, not exact) that quantize it
// themselves, for sizes that block_gemm_grouped_fuses takes: of rows that are
// still in token order (a row's token is order[row] / topk), and of rows of 2 k
// fp32 values (g.x 16-byte aligned) whose gated product is the row.
bool block_gemm_grouped_fuses(int64_t rows, int64_t experts, int64_t k);
hipError_t launch_block_gemm_tokens(const BlockGemm& g, int64_t experts, const int32_t* offsets,
                                    const int32_t* order, int64_t topk, hipStream_t stream);
hipError_t launch_block_gemm_gates(const BlockGemm& g, int64_t experts, const int32_t* offsets,
                                   hipStream_t stream);
// The grouped product with a weight of gate rows and then as many up rows (g.n
// in all), as codes of silu(gate) * up in g.y and their 1 x 128 scales in ys:
// for sizes that block_gemm_gates takes.
bool block_gemm_gates(int64_t rows, int64_t experts, int64_t f, int64_t k);
hipError_t launch_block_gemm_gated(const BlockGemm& g, int64_t experts, const int32_t* offsets,
                                   float* ys, hipStream_t stream);

// The kernel that launch_block_gemm and launch_block_gemm_grouped take, as
// qw_block_debug_path reports it.
int block_gemm_path(int64_t n, int64_t m, int64_t k, bool exact, bool rest);
int block_gemm_grouped_path(int64_t n, int64_t m, int64_t k, int64_t experts, bool exact);

// Tokens sorted by expert and back (moe.hip).
int64_t moe_sort_work_bytes(int64_t slots, int64_t experts);
hipError_t launch_moe_sort(int64_t slots, int64_t experts, int id_bytes, const void* ids,
                           int32_t* pos, int32_t* order, int32_t* offsets, void* work,
                           hipStream_t stream);
hipError_t launch_moe_gather(int64_t t, int64_t topk, int64_t d, int64_t rows, int type,
                             const void* x, const int32_t* pos, void* xs, hipStream_t stream);
hipError_t launch_moe_gather_block(int64_t t, int64_t topk, int64_t d, int64_t rows, int type,
                                   const void* x, const int32_t* pos, uint8_t* codes,
                                   float* scales, hipStream_t stream);
hipError_t launch_moe_combine(int64_t t, int64_t topk, int64_t d, int64_t rows, int type,
                              const void* ys, const int32_t* pos, const float* weights,
                              int y_type, void* y, hipStream_t stream);
hipError_t launch_moe_combine_backward(int64_t t, int64_t topk, int64_t d, int64_t rows,
                                       int type, const void* dy, const void* ys,
                                       const int32_t* pos, const float* weights, void* dys,
                                       float* dweights, hipStream_t stream);

// Which kernel family a call takes (exposed for tests through qw_debug_path).
enum Path { PATH_NONE = 0, PATH_FAST = 1, PATH_BLOCK = 2, PATH_GENERIC = 3, PATH_MATRIX = 4 };
int quantize_path(const Mat& mt, const float* w, const uint8_t* payload);
int unpack_path(const Mat& mt, const uint8_t* payload, const float* w_out);
int gemv_path(const Mat& mt, const uint8_t* payload, const float* x);
// The kernel family of a lone GEMV at 8 rows of x (PATH_MATRIX: matrix cores).
int gemv_mfma_path(const Mat& mt, const uint8_t* payload, const float* x);
// Whether qw_matmul runs the GEMV instead of the GEMM at 5..8 rows of x.
bool matmul_prefers_gemv(const Mat& mt, const uint8_t* payload, const float* x);
int gemm_path(const Mat& mt, const uint8_t* payload, const uint16_t* x);

}  // namespace qw
