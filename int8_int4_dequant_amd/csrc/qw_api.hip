// C ABI of libqw (declared in include/qw.h): argument validation and
// dispatch to the HIP kernels.  No allocation, no synchronization.
#include <string.h>

#include <cmath>
#include <mutex>
#include <vector>

#include "../../include/qw.h"
#include "qw_internal.h"

namespace {

thread_local char g_last_error[256] = {0};

int record(hipError_t e) {
  if (e == hipSuccess) return QW_OK;
  strncpy(g_last_error, hipGetErrorString(e), sizeof(g_last_error) - 1);
  g_last_error[sizeof(g_last_error) - 1] = 0;
  return QW_EHIP;
}

// 0 <= a, b and a * b <= lim (each factor bounded first, so the product
// cannot overflow).
bool within(int64_t a, int64_t b, int64_t lim = QW_MAX_ELEMENTS) {
  return a >= 0 && b >= 0 && a <= lim && b <= lim && (a == 0 || b <= lim / a);
}

// Validates bits / group / shape; fills `mt` on success.
int check_mat(int bits, int64_t group, int64_t n, int64_t k, qw::Mat* mt) {
  if (bits != 4 && bits != 8) return QW_EBITS;
  if (!within(n, k)) return QW_ESHAPE;
  if (group < 1) return QW_EGROUP;
  const int64_t count = n * k;
  if (count % group != 0) return QW_EGROUP;
  if (bits == 4 && count % 2 != 0) return QW_ESHAPE;
  mt->bits = bits;
  mt->group = group;
  mt->n = n;
  mt->k = k;
  return QW_OK;
}

}  // namespace

extern "C" {

int64_t qw_payload_bytes(int bits, int64_t n, int64_t k) {
  if ((bits != 4 && bits != 8) || !within(n, k)) return -1;
  if (bits == 4 && (n * k) % 2 != 0) return -1;
  return n * k * bits / 8;
}

int64_t qw_num_scales(int64_t group, int64_t n, int64_t k) {
  if (group < 1 || !within(n, k) || (n * k) % group != 0) return -1;
  return n * k / group;
}

const char* qw_status_string(int status) {
  switch (status) {
    case QW_OK: return "ok";
    case QW_EBITS: return "bits must be 4 or 8";
    case QW_EGROUP: return "group must be >= 1 and divide n*k";
    case QW_ESHAPE: return "invalid shape (negative, overflowing, or odd element count for int4)";
    case QW_EM: return "m out of range";
    case QW_ENULL: return "required pointer is NULL";
    case QW_EHIP: return "HIP launch failed (see qw_last_error)";
    case QW_ECOUNT: return "invalid batch count or descriptor";
    case QW_EWORK: return "work buffer missing or too small";
    case QW_EARG: return "argument out of range";
    case QW_ESCRATCH:
      return "input too large for the static scratch of qw_matmul_noalloc "
             "(m * k * 2 bytes of bf16 x above QW_MATMUL_NOALLOC_MAX_BYTES)";
    default: return "unknown status";
  }
}

const char* qw_last_error(void) { return g_last_error; }

int qw_quantize_pack(int bits, int64_t group, int64_t n, int64_t k, const float* w,
                     uint8_t* payload, float* scales, void* stream) {
  qw::Mat mt;
  int st = check_mat(bits, group, n, k, &mt);
  if (st != QW_OK) return st;
  if (n * k == 0) return QW_OK;
  if (!w || !payload || !scales) return QW_ENULL;
  return record(qw::launch_quantize_pack(mt, w, payload, scales, (hipStream_t)stream));
}

int qw_quantize_pack_batched(int count, const qw_quant_desc* descs, void* stream) {
  if (count < 0) return QW_ECOUNT;
  if (count == 0) return QW_OK;
  if (!descs) return QW_ENULL;
  for (int i = 0; i < count; ++i) {
    const qw_quant_desc& d = descs[i];
    if (d.reserved != 0) return QW_ECOUNT;
    qw::Mat mt;
    int st = check_mat(d.bits, d.group, d.n, d.k, &mt);
    if (st != QW_OK) return st;
    if (d.n * d.k > 0 && (!d.w || !d.payload || !d.scales)) return QW_ENULL;
  }
  const int kChunk = 256;
  qw::Mat mts[kChunk];
  const float* ws[kChunk];
  uint8_t* ps[kChunk];
  float* ss[kChunk];
  for (int base = 0; base < count; base += kChunk) {
    int nb = 0;
    for (int i = base; i < count && i < base + kChunk; ++i) {
      const qw_quant_desc& d = descs[i];
      if (d.n * d.k == 0) continue;
      check_mat(d.bits, d.group, d.n, d.k, &mts[nb]);
      ws[nb] = d.w;
      ps[nb] = d.payload;
      ss[nb] = d.scales;
      ++nb;
    }
    int st = record(qw::launch_quantize_pack_batched(mts, ws, ps, ss, nb, (hipStream_t)stream));
    if (st != QW_OK) return st;
  }
  return QW_OK;
}

int qw_unpack(int bits, int64_t group, int64_t n, int64_t k, const uint8_t* payload,
              const float* scales, float* w_out, void* stream) {
  qw::Mat mt;
  int st = check_mat(bits, group, n, k, &mt);
  if (st != QW_OK) return st;
  if (n * k == 0) return QW_OK;
  if (!payload || !scales || !w_out) return QW_ENULL;
  return record(qw::launch_unpack(mt, payload, scales, w_out, (hipStream_t)stream));
}

int qw_unpack_batched(int count, const qw_unpack_desc* descs, void* stream) {
  if (count < 0) return QW_ECOUNT;
  if (count == 0) return QW_OK;
  if (!descs) return QW_ENULL;
  for (int i = 0; i < count; ++i) {
    const qw_unpack_desc& d = descs[i];
    if (d.reserved != 0) return QW_ECOUNT;
    qw::Mat mt;
    int st = check_mat(d.bits, d.group, d.n, d.k, &mt);
    if (st != QW_OK) return st;
    if (d.n * d.k > 0 && (!d.payload || !d.scales || !d.w_out)) return QW_ENULL;
  }
  const int kChunk = 256;
  qw::Mat mts[kChunk];
  const uint8_t* ps[kChunk];
  const float* ss[kChunk];
  float* os[kChunk];
  for (int base = 0; base < count; base += kChunk) {
    int nb = 0;
    for (int i = base; i < count && i < base + kChunk; ++i) {
      const qw_unpack_desc& d = descs[i];
      if (d.n * d.k == 0) continue;
      check_mat(d.bits, d.group, d.n, d.k, &mts[nb]);
      ps[nb] = d.payload;
      ss[nb] = d.scales;
      os[nb] = d.w_out;
      ++nb;
    }
    int st = record(qw::launch_unpack_batched(mts, ps, ss, os, nb, (hipStream_t)stream));
    if (st != QW_OK) return st;
  }
  return QW_OK;
}

int qw_gemv(int bits, int64_t group, int64_t n, int64_t k, const uint8_t* payload,
            const float* scales, int64_t m, const float* x, float* y, void* stream) {
  qw::Mat mt;
  int st = check_mat(bits, group, n, k, &mt);
  if (st != QW_OK) return st;
  if (m < 0 || m > 8 || !within(m, n) || !within(m, k)) return QW_EM;
  if (m == 0 || n == 0) return QW_OK;
  if (!y) return QW_ENULL;
  if (k == 0) return record(qw::launch_fill_zero(y, m * n, (hipStream_t)stream));
  if (!payload || !scales || !x) return QW_ENULL;
  return record(qw::launch_gemv(mt, payload, scales, (int)m, x, y, (hipStream_t)stream));
}

int qw_gemv_batched(int count, const qw_gemv_desc* descs, int64_t m, void* stream) {
  if (count < 0) return QW_ECOUNT;
  if (count == 0) return QW_OK;
  if (!descs) return QW_ENULL;
  if (m < 0 || m > 8) return QW_EM;
  if (m == 0) return QW_OK;
  // validate everything before enqueuing anything
  for (int i = 0; i < count; ++i) {
    const qw_gemv_desc& d = descs[i];
    if (d.reserved != 0) return QW_ECOUNT;
    qw::Mat mt;
    int st = check_mat(d.bits, d.group, d.n, d.k, &mt);
    if (st != QW_OK) return st;
    if (!within(m, d.n) || !within(m, d.k)) return QW_EM;
    if (d.n == 0) continue;
    if (!d.y) return QW_ENULL;
    if (d.k > 0 && (!d.payload || !d.scales || !d.x)) return QW_ENULL;
  }
  const int kChunk = 256;
  qw::Mat mts[kChunk];
  const uint8_t* ps[kChunk];
  const float* ss[kChunk];
  const float* xs[kChunk];
  float* ys[kChunk];
  for (int base = 0; base < count; base += kChunk) {
    int nb = 0;
    for (int i = base; i < count && i < base + kChunk; ++i) {
      const qw_gemv_desc& d = descs[i];
      if (d.n == 0) continue;
      if (d.k == 0) {
        int st = record(qw::launch_fill_zero(d.y, m * d.n, (hipStream_t)stream));
        if (st != QW_OK) return st;
        continue;
      }
      check_mat(d.bits, d.group, d.n, d.k, &mts[nb]);
      ps[nb] = d.payload;
      ss[nb] = d.scales;
      xs[nb] = d.x;
      ys[nb] = d.y;
      ++nb;
    }
    int st = record(qw::launch_gemv_batched(mts, ps, ss, (int)m, xs, ys, nb, (hipStream_t)stream));
    if (st != QW_OK) return st;
  }
  return QW_OK;
}

int qw_gemv_chain(int count, const qw_gemv_desc* descs, const int32_t* stage, int64_t m,
                  void* stream) {
  if (count < 0) return QW_ECOUNT;
  if (count == 0) return QW_OK;
  if (!descs) return QW_ENULL;
  if (!stage) return QW_ECOUNT;
  if (m < 0 || m > 8) return QW_EM;
  for (int i = 1; i < count; ++i)
    if (stage[i] < stage[i - 1]) return QW_ECOUNT;
  for (int i = 0; i < count; ++i) {
    const qw_gemv_desc& d = descs[i];
    if (d.reserved != 0) return QW_ECOUNT;
    qw::Mat mt;
    int st = check_mat(d.bits, d.group, d.n, d.k, &mt);
    if (st != QW_OK) return st;
    if (!within(m, d.n) || !within(m, d.k)) return QW_EM;
    if (d.n == 0) continue;
    if (!d.y) return QW_ENULL;
    if (d.k > 0 && (!d.payload || !d.scales || !d.x)) return QW_ENULL;
  }
  if (m == 0) return QW_OK;
  // Stage by stage, in order: the zero fills of the stage's products with
  // k == 0, then one batched launch over its other products.  A y filled
  // here is read only by later stages, which are enqueued after it.
  std::vector<qw::Mat> mts;
  std::vector<const uint8_t*> ps;
  std::vector<const float*> ss, xs;
  std::vector<float*> ys;
  for (int i0 = 0; i0 < count;) {
    int i1 = i0 + 1;
    while (i1 < count && stage[i1] == stage[i0]) ++i1;
    mts.clear();
    ps.clear();
    ss.clear();
    xs.clear();
    ys.clear();
    for (int i = i0; i < i1; ++i) {
      const qw_gemv_desc& d = descs[i];
      if (d.n == 0) continue;
      if (d.k == 0) {
        int st = record(qw::launch_fill_zero(d.y, m * d.n, (hipStream_t)stream));
        if (st != QW_OK) return st;
        continue;
      }
      qw::Mat mt;
      check_mat(d.bits, d.group, d.n, d.k, &mt);
      mts.push_back(mt);
      ps.push_back(d.payload);
      ss.push_back(d.scales);
      xs.push_back(d.x);
      ys.push_back(d.y);
    }
    if (!mts.empty()) {
      int st = record(qw::launch_gemv_batched(mts.data(), ps.data(), ss.data(), (int)m,
                                              xs.data(), ys.data(), (int)mts.size(),
                                              (hipStream_t)stream));
      if (st != QW_OK) return st;
    }
    i0 = i1;
  }
  return QW_OK;
}

int qw_gemm(int bits, int64_t group, int64_t n, int64_t k, const uint8_t* payload,
            const float* scales, int64_t m, const uint16_t* x_bf16, float* y, void* stream) {
  qw::Mat mt;
  int st = check_mat(bits, group, n, k, &mt);
  if (st != QW_OK) return st;
  if (!within(m, n) || !within(m, k)) return QW_EM;
  if (m == 0 || n == 0) return QW_OK;
  if (!y) return QW_ENULL;
  if (k == 0) return record(qw::launch_fill_zero(y, m * n, (hipStream_t)stream));
  if (!payload || !scales || !x_bf16) return QW_ENULL;
  return record(qw::launch_gemm(mt, payload, scales, m, x_bf16, y, (hipStream_t)stream));
}

int64_t qw_matmul_work_bytes(int64_t m, int64_t k) {
  if (!within(m, k)) return -1;
  if (m <= QW_MATMUL_GEMV_MAX_M) return 0;
  return (m * k * 2 + 255) / 256 * 256;  // bf16 copy of x
}

}  // extern "C"

// The static scratch of qw_matmul_noalloc: each device holds its own copy
// from the library's first use on it until the process ends.  Host code
// never passes the array's name to a kernel (in host code it is only a
// stand-in for the symbol); it passes the device address looked up once per
// device with hipGetSymbolAddress.
static __device__ __align__(256) uint8_t scratch[QW_MATMUL_NOALLOC_MAX_BYTES];

namespace {

// qw_matmul with a resolved work pointer (the caller's buffer, or this
// device's static scratch).  Arguments are validated by the callers.
int matmul_with_work(const qw::Mat& mt, const uint8_t* payload, const float* scales, int64_t m,
                     const float* x, float* y, void* work, hipStream_t stream) {
  uint16_t* xb = (uint16_t*)work;
  hipError_t e = qw::launch_round_bf16(x, xb, m * mt.k, stream);
  if (e != hipSuccess) return record(e);
  return record(qw::launch_gemm(mt, payload, scales, m, xb, y, stream));
}

constexpr int kMaxDevices = 64;
std::mutex g_scratch_mu;
void* g_scratch_ptr[kMaxDevices] = {};

// This device's address of `scratch`, looked up on the first call on the
// device (the current device, on which `stream` must run).
int scratch_address(hipStream_t stream, void** out) {
  int dev = 0;
  hipError_t e = hipGetDevice(&dev);
  if (e != hipSuccess) return record(e);
  if (dev < 0 || dev >= kMaxDevices) return QW_EARG;
  if (stream) {
    hipDevice_t sdev = 0;
    e = hipStreamGetDevice(stream, &sdev);
    if (e != hipSuccess) return record(e);
    if ((int)sdev != dev) return QW_EARG;
  }
  std::lock_guard<std::mutex> lock(g_scratch_mu);
  if (!g_scratch_ptr[dev]) {
    void* p = nullptr;
    e = hipGetSymbolAddress(&p, HIP_SYMBOL(scratch));
    if (e != hipSuccess) return record(e);
    if (!p) return QW_EHIP;
    g_scratch_ptr[dev] = p;
  }
  *out = g_scratch_ptr[dev];
  return QW_OK;
}

}  // namespace

extern "C" {

int qw_matmul(int bits, int64_t group, int64_t n, int64_t k, const uint8_t* payload,
              const float* scales, int64_t m, const float* x, float* y, void* work,
              int64_t work_bytes, void* stream) {
  qw::Mat mt;
  int st = check_mat(bits, group, n, k, &mt);
  if (st != QW_OK) return st;
  if (!within(m, n) || !within(m, k)) return QW_EM;
  if (m <= QW_MATMUL_GEMV_MAX_M || (m <= 8 && qw::matmul_prefers_gemv(mt, payload, x)))
    return qw_gemv(bits, group, n, k, payload, scales, m, x, y, stream);
  if (n == 0) return QW_OK;
  if (!y) return QW_ENULL;
  if (k == 0) return record(qw::launch_fill_zero(y, m * n, (hipStream_t)stream));
  if (!payload || !scales || !x) return QW_ENULL;
  if (!work || work_bytes < qw_matmul_work_bytes(m, k)) return QW_EWORK;
  return matmul_with_work(mt, payload, scales, m, x, y, work, (hipStream_t)stream);
}

int qw_matmul_noalloc(int bits, int64_t group, int64_t n, int64_t k, const uint8_t* payload,
                      const float* scales, int64_t m, const float* x, float* y, void* stream) {
  qw::Mat mt;
  int st = check_mat(bits, group, n, k, &mt);
  if (st != QW_OK) return st;
  if (!within(m, n) || !within(m, k)) return QW_EM;
  if (m <= QW_MATMUL_GEMV_MAX_M || (m <= 8 && qw::matmul_prefers_gemv(mt, payload, x)))
    return qw_gemv(bits, group, n, k, payload, scales, m, x, y, stream);
  if (n == 0) return QW_OK;
  if (qw_matmul_work_bytes(m, k) > QW_MATMUL_NOALLOC_MAX_BYTES) return QW_ESCRATCH;
  if (!y) return QW_ENULL;
  if (k == 0) return record(qw::launch_fill_zero(y, m * n, (hipStream_t)stream));
  if (!payload || !scales || !x) return QW_ENULL;
  void* work = nullptr;
  st = scratch_address((hipStream_t)stream, &work);
  if (st != QW_OK) return st;
  return matmul_with_work(mt, payload, scales, m, x, y, work, (hipStream_t)stream);
}

int64_t qw_gptq_hessian_work_bytes(int64_t k, int64_t t) {
  if (k < 0 || k > QW_GPTQ_MAX_K || !within(t, k, QW_GPTQ_MAX_ELEMENTS)) return -1;
  return qw::gptq_hessian_work_bytes(k, t);
}

int qw_gptq_hessian(int64_t k, int64_t t, const float* x, double* h, void* work,
                    int64_t work_bytes, void* stream) {
  if (k < 0 || k > QW_GPTQ_MAX_K || !within(t, k, QW_GPTQ_MAX_ELEMENTS)) return QW_ESHAPE;
  if (k == 0 || t == 0) return QW_OK;
  if (!x || !h) return QW_ENULL;
  if (!work || work_bytes < qw::gptq_hessian_work_bytes(k, t)) return QW_EWORK;
  return record(qw::launch_gptq_hessian(k, t, x, h, work, (hipStream_t)stream));
}

int64_t qw_gptq_factor_work_bytes(int64_t k) {
  if (k < 0 || k > QW_GPTQ_MAX_K) return -1;
  return qw::gptq_factor_work_bytes(k);
}

int qw_gptq_factor(int64_t k, const double* h, double damp, double* u, int32_t* info,
                   void* work, int64_t work_bytes, void* stream) {
  if (k < 0 || k > QW_GPTQ_MAX_K) return QW_ESHAPE;
  if (!(damp >= 0.0) || !(damp < 1e300)) return QW_EARG;
  if (k == 0) return QW_OK;
  if (!h || !u) return QW_ENULL;
  if (!work || work_bytes < qw::gptq_factor_work_bytes(k)) return QW_EWORK;
  return record(qw::launch_gptq_factor(k, h, damp, u, info, work, (hipStream_t)stream));
}

int64_t qw_gptq_quantize_work_bytes(int64_t n, int64_t k) {
  if (!within(n, k, QW_GPTQ_MAX_ELEMENTS) || n > QW_GPTQ_MAX_N || k > QW_GPTQ_MAX_K) return -1;
  return qw::gptq_quantize_work_bytes(n, k);
}

int qw_gptq_quantize_pack(int bits, int64_t group, int64_t n, int64_t k, const float* w,
                          const double* u, uint8_t* payload, float* scales, void* work,
                          int64_t work_bytes, void* stream) {
  qw::Mat mt;
  int st = check_mat(bits, group, n, k, &mt);
  if (st != QW_OK) return st;
  if (!within(n, k, QW_GPTQ_MAX_ELEMENTS) || n > QW_GPTQ_MAX_N || k > QW_GPTQ_MAX_K)
    return QW_ESHAPE;
  if (k > 0 && (k % group != 0 || (bits == 4 && group % 2 != 0))) return QW_EGROUP;
  if (n * k == 0) return QW_OK;
  if (!w || !u || !payload || !scales) return QW_ENULL;
  if (!work || work_bytes < qw::gptq_quantize_work_bytes(n, k)) return QW_EWORK;
  return record(qw::launch_gptq_quantize_pack(mt, w, u, payload, scales, work,
                                              (hipStream_t)stream));
}

// ------------------------------------------------- block-scaled e4m3 codes

}  // extern "C"

namespace {

bool type_ok(int type) { return type == QW_F32 || type == QW_BF16; }

// block_rows and the sizes of `count` matrices of n x k (their code rows
// included); `shape` is the status of sizes out of range.
int check_block(int brows, int64_t count, int64_t n, int64_t k) {
  if (brows != 1 && brows != QW_BLOCK) return QW_EARG;
  if (!within(n, k) || !within(n, qw::pitch(k))) return QW_ESHAPE;
  // the codes; the scales are fewer, one for 128 of them at most
  if (!within(count, n) || !within(count * n, qw::pitch(k))) return QW_ESHAPE;
  return QW_OK;
}

// x or y side of a product: m rows of n outputs and of k inputs.
int check_rows(int64_t m, int64_t n, int64_t k) {
  if (k > QW_BLOCK_MAX_K) return QW_ESHAPE;
  return within(m, n) && within(m, k) && within(m, qw::pitch(k)) ? QW_OK : QW_EM;
}

int check_moe(int64_t t, int64_t topk, int64_t d, int64_t rows) {
  if (topk < 1) return QW_EARG;
  if (!within(t, topk, QW_MOE_MAX_SLOTS)) return QW_ESHAPE;
  if (rows < 0 || rows > QW_MOE_MAX_SLOTS) return QW_ESHAPE;
  if (!within(d, 1) || !within(t, qw::pitch(d)) || !within(rows, qw::pitch(d)))
    return QW_ESHAPE;
  return QW_OK;
}

// A part of a work buffer, 256-byte aligned relative to its start.
struct Carve {
  int64_t at = 0;
  int64_t take(int64_t bytes) {
    const int64_t here = at;
    at += (bytes + 255) / 256 * 256;
    return here;
  }
};

}  // namespace

extern "C" {

int64_t qw_block_pitch(int64_t k) { return within(k, 1) ? qw::pitch(k) : -1; }

int64_t qw_block_num_scales(int block_rows, int64_t n, int64_t k) {
  if (check_block(block_rows, 1, n, k) != QW_OK) return -1;
  return qw::block_scales(block_rows, n, k);
}

int qw_block_quantize(int block_rows, int64_t count, int64_t n, int64_t k, int type,
                      const void* w, uint8_t* codes, float* scales, void* stream) {
  int st = check_block(block_rows, count, n, k);
  if (st != QW_OK) return st;
  if (!type_ok(type)) return QW_EARG;
  if (count * n * k == 0) return QW_OK;
  if (!w || !codes || !scales) return QW_ENULL;
  if (!qw::aligned(codes, 16)) return QW_EARG;
  return record(qw::launch_block_quantize(block_rows, count, n, k, type, w, codes, scales,
                                          (hipStream_t)stream));
}

int qw_block_quantize_swiglu(int64_t rows, int64_t f, int type, const void* h,
                             const int32_t* used, uint8_t* codes, float* scales,
                             void* stream) {
  int st = check_block(1, 1, rows, f);
  if (st != QW_OK) return st;
  if (!within(rows, f, QW_MAX_ELEMENTS / 2)) return QW_ESHAPE;
  if (!type_ok(type)) return QW_EARG;
  if (rows * f == 0) return QW_OK;
  if (!h || !codes || !scales) return QW_ENULL;
  if (!qw::aligned(codes, 16)) return QW_EARG;
  return record(qw::launch_block_quantize_swiglu(rows, f, type, h, used, codes, scales,
                                                 (hipStream_t)stream));
}

int qw_block_unpack(int block_rows, int64_t count, int64_t n, int64_t k, const uint8_t* codes,
                    const float* scales, float* out, void* stream) {
  int st = check_block(block_rows, count, n, k);
  if (st != QW_OK) return st;
  if (count * n * k == 0) return QW_OK;
  if (!codes || !scales || !out) return QW_ENULL;
  if (!qw::aligned(codes, 16)) return QW_EARG;
  return record(qw::launch_block_unpack(block_rows, count, n, k, codes, scales, out,
                                        (hipStream_t)stream));
}

int qw_block_gemm(int block_rows, int64_t n, int64_t k, const uint8_t* codes,
                  const float* scales, int64_t m, const uint8_t* x_codes,
                  const float* x_scales, int y_type, void* y, void* stream) {
  int st = check_block(block_rows, 1, n, k);
  if (st != QW_OK) return st;
  st = check_rows(m, n, k);
  if (st != QW_OK) return st;
  if (!type_ok(y_type)) return QW_EARG;
  if (m * n == 0) return QW_OK;
  if (!y || (k > 0 && (!codes || !scales || !x_codes || !x_scales))) return QW_ENULL;
  if (!qw::aligned(codes, 16) || !qw::aligned(x_codes, 16)) return QW_EARG;
  qw::BlockGemm g = {block_rows, n, k, m, codes, scales, -1, nullptr, x_codes, x_scales,
                     y_type, y, y_type == QW_F32};
  return record(qw::launch_block_gemm(g, (hipStream_t)stream));
}

int64_t qw_block_matmul_work_bytes(int64_t m, int64_t k) {
  if (check_rows(m, 1, k) != QW_OK) return -1;
  if (qw::block_gemm_fuses(m, k)) return 0;
  Carve c;
  c.take(m * qw::pitch(k));
  c.take(qw::block_scales(1, m, k) * 4);
  return c.at;
}

int qw_block_matmul(int block_rows, int64_t n, int64_t k, const uint8_t* codes,
                    const float* scales, int64_t m, int x_type, const void* x, int y_type,
                    void* y, void* work, int64_t work_bytes, void* stream) {
  int st = check_block(block_rows, 1, n, k);
  if (st != QW_OK) return st;
  st = check_rows(m, n, k);
  if (st != QW_OK) return st;
  if (!type_ok(x_type) || !type_ok(y_type)) return QW_EARG;
  if (m * n == 0) return QW_OK;
  if (!y || (k > 0 && (!codes || !scales || !x))) return QW_ENULL;
  if (!qw::aligned(codes, 16)) return QW_EARG;
  qw::BlockGemm g = {block_rows, n, k, m, codes, scales, x_type, x, nullptr, nullptr,
                     y_type, y, y_type == QW_F32};
  if (k == 0 || !qw::block_gemm_fuses(m, k)) {
    const int64_t need = qw_block_matmul_work_bytes(m, k);
    if (need > 0 && (!work || work_bytes < need || !qw::aligned(work, 16))) return QW_EWORK;
    Carve c;
    uint8_t* xc = (uint8_t*)work + c.take(m * qw::pitch(k));
    float* xs = (float*)((uint8_t*)work + c.take(0));
    if (k > 0) {
      const hipError_t e = qw::launch_block_quantize(1, 1, m, k, x_type, x, xc, xs,
                                                     (hipStream_t)stream);
      if (e != hipSuccess) return record(e);
    }
    g.x_type = -1;
    g.x = nullptr;
    g.xc = xc;
    g.xs = xs;
  }
  return record(qw::launch_block_gemm(g, (hipStream_t)stream));
}

int qw_block_gemm_grouped(int block_rows, int64_t experts, int64_t n, int64_t k,
                          const uint8_t* codes, const float* scales, int64_t rows,
                          const uint8_t* x_codes, const float* x_scales,
                          const int32_t* offsets, int y_type, void* y, void* stream) {
  if (experts < 1 || experts > QW_MOE_MAX_EXPERTS) return QW_EARG;
  int st = check_block(block_rows, experts, n, k);
  if (st != QW_OK) return st;
  if (rows < 0 || rows > QW_MOE_MAX_SLOTS) return QW_EM;
  st = check_rows(rows, n, k);
  if (st != QW_OK) return st;
  if (!type_ok(y_type)) return QW_EARG;
  if (rows * n == 0) return QW_OK;
  if (!y || !offsets || (k > 0 && (!codes || !scales || !x_codes || !x_scales)))
    return QW_ENULL;
  if (!qw::aligned(codes, 16) || !qw::aligned(x_codes, 16)) return QW_EARG;
  const qw::BlockGemm g = {block_rows, n, k, rows, codes, scales, -1, nullptr, x_codes,
                           x_scales, y_type, y, y_type == QW_F32};
  return record(qw::launch_block_gemm_grouped(g, experts, offsets, (hipStream_t)stream));
}

// ------------------------------------------ tokens sorted by expert and back

int64_t qw_moe_sort_work_bytes(int64_t t, int64_t topk, int64_t experts) {
  if (topk < 1 || experts < 1 || experts > QW_MOE_MAX_EXPERTS ||
      !within(t, topk, QW_MOE_MAX_SLOTS))
    return -1;
  return qw::moe_sort_work_bytes(t * topk, experts);
}

int qw_moe_sort(int64_t t, int64_t topk, int64_t experts, int id_bytes, const void* ids,
                int32_t* pos, int32_t* order, int32_t* offsets, void* work,
                int64_t work_bytes, void* stream) {
  if (topk < 1 || experts < 1 || experts > QW_MOE_MAX_EXPERTS) return QW_EARG;
  if (id_bytes != 4 && id_bytes != 8) return QW_EARG;
  if (!within(t, topk, QW_MOE_MAX_SLOTS)) return QW_ESHAPE;
  if (!offsets || (t > 0 && (!ids || !pos))) return QW_ENULL;
  const int64_t need = qw_moe_sort_work_bytes(t, topk, experts);
  if (need > 0 && (!work || work_bytes < need || !qw::aligned(work, 4))) return QW_EWORK;
  return record(qw::launch_moe_sort(t * topk, experts, id_bytes, ids, pos, order, offsets, work,
                                    (hipStream_t)stream));
}

int qw_moe_gather(int64_t t, int64_t topk, int64_t d, int64_t rows, int type, const void* x,
                  const int32_t* pos, void* xs, void* stream) {
  int st = check_moe(t, topk, d, rows);
  if (st != QW_OK) return st;
  if (!type_ok(type)) return QW_EARG;
  if (t * d == 0 || rows == 0) return QW_OK;
  if (!x || !pos || !xs) return QW_ENULL;
  return record(qw::launch_moe_gather(t, topk, d, rows, type, x, pos, xs, (hipStream_t)stream));
}

int qw_moe_gather_block(int64_t t, int64_t topk, int64_t d, int64_t rows, int type,
                        const void* x, const int32_t* pos, uint8_t* codes, float* scales,
                        void* stream) {
  int st = check_moe(t, topk, d, rows);
  if (st != QW_OK) return st;
  if (!type_ok(type)) return QW_EARG;
  if (t * d == 0 || rows == 0) return QW_OK;
  if (!x || !pos || !codes || !scales) return QW_ENULL;
  if (!qw::aligned(codes, 16)) return QW_EARG;
  return record(qw::launch_moe_gather_block(t, topk, d, rows, type, x, pos, codes, scales,
                                            (hipStream_t)stream));
}

int qw_moe_combine(int64_t t, int64_t topk, int64_t d, int64_t rows, int type, const void* ys,
                   const int32_t* pos, const float* weights, int y_type, void* y,
                   void* stream) {
  int st = check_moe(t, topk, d, rows);
  if (st != QW_OK) return st;
  if (!type_ok(type) || !type_ok(y_type)) return QW_EARG;
  if (t * d == 0) return QW_OK;
  if (!pos || !y || (rows > 0 && !ys)) return QW_ENULL;
  return record(qw::launch_moe_combine(t, topk, d, rows, type, ys, pos, weights, y_type, y,
                                       (hipStream_t)stream));
}

int qw_moe_combine_backward(int64_t t, int64_t topk, int64_t d, int64_t rows, int type,
                            const void* dy, const void* ys, const int32_t* pos,
                            const float* weights, void* dys, float* dweights, void* stream) {
  int st = check_moe(t, topk, d, rows);
  if (st != QW_OK) return st;
  if (!type_ok(type)) return QW_EARG;
  if (t == 0) return QW_OK;
  if (!pos || (d > 0 && !dy) || (dweights && rows > 0 && d > 0 && !ys)) return QW_ENULL;
  if (!dys && !dweights) return QW_OK;
  return record(qw::launch_moe_combine_backward(t, topk, d, rows, type, dy, ys, pos, weights,
                                                dys, dweights, (hipStream_t)stream));
}

}  // extern "C"

namespace {

// The buffers of qw_moe_mlp in its work buffer, and the way it takes: few rows
// are quantized by the products themselves, many gated by the first one (on the
// 8-bit cores: for bf16 y).
struct MlpWork {
  bool few, gates;
  int64_t pos, order, offsets, sort, xc, xs, h, hc, hs, ys, bytes;
  MlpWork(int64_t t, int64_t topk, int64_t experts, int64_t d, int64_t f, int y_type) {
    const int64_t rows = t * topk;
    few = qw::block_gemm_grouped_fuses(rows, experts, d) &&
          qw::block_gemm_grouped_fuses(rows, experts, f);
    gates = y_type == QW_BF16 && qw::block_gemm_gates(rows, experts, f, d);
    // every buffer, whichever way: a size that grows with every argument, so that
    // what is enough for the largest call is enough for all smaller ones
    Carve c;
    pos = c.take(rows * 4);
    order = c.take(rows * 4);
    offsets = c.take((experts + 1) * 4);
    sort = c.take(qw::moe_sort_work_bytes(rows, experts));
    xc = c.take(rows * qw::pitch(d));
    xs = c.take(qw::block_scales(1, rows, d) * 4);
    h = c.take(rows * 2 * f * 4);
    hc = c.take(rows * qw::pitch(f));
    hs = c.take(qw::block_scales(1, rows, f) * 4);
    ys = c.take(rows * d * 4);
    bytes = c.at;
  }
};

int check_mlp(int64_t t, int64_t topk, int64_t experts, int64_t d, int64_t f) {
  if (topk < 1 || experts < 1 || experts > QW_MOE_MAX_EXPERTS) return QW_EARG;
  if (!within(t, topk, QW_MOE_MAX_SLOTS) || !within(d, 1) || !within(f, 2)) return QW_ESHAPE;
  if (d > QW_BLOCK_MAX_K || f > QW_BLOCK_MAX_K) return QW_ESHAPE;
  if (!within(t * topk, qw::pitch(d)) || !within(t * topk, 2 * qw::pitch(f))) return QW_ESHAPE;
  return QW_OK;
}

}  // namespace

extern "C" {

int64_t qw_moe_mlp_work_bytes(int64_t t, int64_t topk, int64_t experts, int64_t d, int64_t f) {
  if (check_mlp(t, topk, experts, d, f) != QW_OK) return -1;
  return MlpWork(t, topk, experts, d, f, QW_F32).bytes;
}

int qw_moe_mlp(int block_rows, int64_t experts, int64_t d, int64_t f, const uint8_t* gate_up,
               const float* gate_up_scales, const uint8_t* down, const float* down_scales,
               int64_t t, int64_t topk, int x_type, const void* x, int id_bytes,
               const void* ids, const float* weights, int y_type, void* y, void* work,
               int64_t work_bytes, void* stream) {
  int st = check_mlp(t, topk, experts, d, f);
  if (st != QW_OK) return st;
  st = check_block(block_rows, experts, 2 * f, d);
  if (st != QW_OK) return st;
  st = check_block(block_rows, experts, d, f);
  if (st != QW_OK) return st;
  if (!type_ok(x_type) || !type_ok(y_type) || (id_bytes != 4 && id_bytes != 8)) return QW_EARG;
  if (t * d == 0) return QW_OK;
  if (!x || !ids || !y || (f > 0 && (!gate_up || !gate_up_scales || !down || !down_scales)))
    return QW_ENULL;
  if (!qw::aligned(gate_up, 16) || !qw::aligned(down, 16)) return QW_EARG;
  const MlpWork at(t, topk, experts, d, f, y_type);
  if (!work || work_bytes < at.bytes || !qw::aligned(work, 16)) return QW_EWORK;
  uint8_t* const b = (uint8_t*)work;
  const int64_t rows = t * topk;
  int32_t* const pos = (int32_t*)(b + at.pos);
  int32_t* const offsets = (int32_t*)(b + at.offsets);
  int32_t* const order = at.few ? (int32_t*)(b + at.order) : nullptr;
  const hipStream_t s = (hipStream_t)stream;
  st = qw_moe_sort(t, topk, experts, id_bytes, ids, pos, order, offsets, b + at.sort,
                   at.xc - at.sort, stream);
  if (st != QW_OK) return st;
  // fp32 results either way; y's type decides how exact their sums are
  const bool exact = y_type == QW_F32;
  qw::BlockGemm up = {block_rows, 2 * f, d, rows, gate_up, gate_up_scales, x_type, x,
                      nullptr, nullptr, QW_F32, b + at.h, exact};
  qw::BlockGemm out = {block_rows, d, f, rows, down, down_scales, QW_F32, b + at.h,
                       nullptr, nullptr, QW_F32, b + at.ys, exact};
  if (at.few) {
    st = record(qw::launch_block_gemm_tokens(up, experts, offsets, order, topk, s));
    if (st != QW_OK) return st;
    st = record(qw::launch_block_gemm_gates(out, experts, offsets, s));
  } else {
    float* const xs = (float*)(b + at.xs);
    float* const hs = (float*)(b + at.hs);
    st = qw_moe_gather_block(t, topk, d, rows, x_type, x, pos, b + at.xc, xs, stream);
    if (st != QW_OK) return st;
    up.x_type = out.x_type = -1;
    up.xc = b + at.xc;
    up.xs = xs;
    out.xc = b + at.hc;
    out.xs = hs;
    if (at.gates) {
      up.y = b + at.hc;
      st = record(qw::launch_block_gemm_gated(up, experts, offsets, hs, s));
      if (st != QW_OK) return st;
    } else if (f > 0) {
      st = record(qw::launch_block_gemm_grouped(up, experts, offsets, s));
      if (st != QW_OK) return st;
      st = qw_block_quantize_swiglu(rows, f, QW_F32, b + at.h, offsets + experts, b + at.hc, hs,
                                    stream);
      if (st != QW_OK) return st;
    }
    st = record(qw::launch_block_gemm_grouped(out, experts, offsets, s));
  }
  if (st != QW_OK) return st;
  return qw_moe_combine(t, topk, d, rows, QW_F32, b + at.ys, pos, weights, y_type, y, stream);
}

int qw_block_debug_path(int op, int64_t experts, int64_t m, int64_t n, int64_t k, int y_type) {
  const bool mlp = op == 3;
  if (op < 0 || op > 3 || (op > 1 && (experts < 1 || experts > QW_MOE_MAX_EXPERTS)))
    return QW_EARG;
  if (!type_ok(y_type)) return QW_EARG;
  int st = mlp ? check_mlp(m, 1, experts, k, n) : check_block(1, op > 1 ? experts : 1, n, k);
  if (st != QW_OK) return st;
  if (op > 1 && m > QW_MOE_MAX_SLOTS) return QW_EM;
  if (!mlp) st = check_rows(m, n, k);
  if (st != QW_OK) return st;
  if (mlp) {
    const MlpWork at(m, 1, experts, k, n, y_type);
    return at.few ? 1 : at.gates ? 3 : 2;
  }
  if (op < 2) return qw::block_gemm_path(n, m, k, y_type == QW_F32, op == 1);
  return qw::block_gemm_grouped_path(n, m, k, experts, y_type == QW_F32);
}

}  // extern "C"

// ------------------------------------------- microscaled 4-bit codes, RMS norm

namespace {

// An n x k matrix and its rows of 4-bit codes.
bool mx_fits(int64_t n, int64_t k) {
  return within(n, k) && within(k, 1) && within(n, qw::mx_pitch(k));
}

// x or y side of a product: m rows of n outputs and of k inputs.
int check_mx_rows(int64_t m, int64_t n, int64_t k) {
  // rows without values are as long as the shortest, so that a launch holds every product's tiles
  if (k > QW_BLOCK_MAX_K || !mx_fits(n, k ? k : 1)) return QW_ESHAPE;
  return within(m, n) && mx_fits(m, k ? k : 1) ? QW_OK : QW_EM;
}

// The weight of a gated product, 2 f x k, and its m rows of x and of results.
int check_gated(int64_t f, int64_t k, int64_t m) {
  if (!within(f, 2) || !mx_fits(2 * f, k)) return QW_ESHAPE;
  const int st = check_mx_rows(m, 2 * f, k);
  if (st != QW_OK) return st;
  return mx_fits(m, f) ? QW_OK : QW_EM;
}

bool codes_ok(const void* codes, const void* scales) {
  return qw::aligned(codes, 16) && qw::aligned(scales, 16);
}

int check_norm(int64_t rows, int64_t d, int type, int w_type, const void* weight, float eps) {
  if (!within(rows, d)) return QW_ESHAPE;
  if (!type_ok(type) || (weight && !type_ok(w_type))) return QW_EARG;
  return std::isfinite(eps) && eps >= 0.0f ? QW_OK : QW_EARG;
}

// The buffers of qw_mx_mlp: the codes of x and of h, and h as floats for few rows.
struct MxMlpWork {
  int64_t xc, xs, hc, hs, h, bytes;
  MxMlpWork(int64_t m, int64_t d, int64_t f) {
    Carve c;
    xc = c.take(m * (qw::mx_pitch(d) / 2));
    xs = c.take(m * (qw::mx_pitch(d) / 32));
    hc = c.take(m * (qw::mx_pitch(f) / 2));
    hs = c.take(m * (qw::mx_pitch(f) / 32));
    // for every size of the call, so that what is enough for the largest is for all smaller ones
    h = c.take((m < 64 ? m : 64) * f * 4);
    bytes = c.at;
  }
};

int check_mx_mlp(int64_t m, int64_t d, int64_t f) {
  if (!within(f, 2) || !within(d, 1) || d > QW_BLOCK_MAX_K || f > QW_BLOCK_MAX_K) return QW_ESHAPE;
  if (!mx_fits(m, d) || !within(m, 2 * qw::mx_pitch(f))) return QW_EM;
  return QW_OK;
}

}  // namespace

extern "C" {

int64_t qw_mx_pitch(int64_t k) { return within(k, 1) && within(qw::mx_pitch(k), 1) ? qw::mx_pitch(k) : -1; }

int qw_mx_quantize(int transpose, int64_t n, int64_t k, int type, const void* w, uint8_t* codes,
                   uint8_t* scales, void* stream) {
  if (transpose != 0 && transpose != 1) return QW_EARG;
  if (!within(n, k) || !(transpose ? mx_fits(k, n) : mx_fits(n, k))) return QW_ESHAPE;
  if (!type_ok(type)) return QW_EARG;
  if (n * k == 0) return QW_OK;
  if (!w || !codes || !scales) return QW_ENULL;
  if (!codes_ok(codes, scales)) return QW_EARG;
  return record(qw::launch_mx_quantize(transpose, n, k, type, w, codes, scales,
                                       (hipStream_t)stream));
}

int qw_mx_unpack(int64_t n, int64_t k, const uint8_t* codes, const uint8_t* scales, float* out,
                 void* stream) {
  if (!mx_fits(n, k)) return QW_ESHAPE;
  if (n * k == 0) return QW_OK;
  if (!codes || !scales || !out) return QW_ENULL;
  if (!codes_ok(codes, scales)) return QW_EARG;
  return record(qw::launch_mx_unpack(n, k, codes, scales, out, (hipStream_t)stream));
}

int qw_mx_gemm(int64_t n, int64_t k, const uint8_t* codes, const uint8_t* scales, int64_t m,
               const uint8_t* x_codes, const uint8_t* x_scales, int y_type, void* y,
               void* stream) {
  if (!mx_fits(n, k)) return QW_ESHAPE;
  const int st = check_mx_rows(m, n, k);
  if (st != QW_OK) return st;
  if (!type_ok(y_type)) return QW_EARG;
  if (m * n == 0) return QW_OK;
  if (!y || (k > 0 && (!codes || !scales || !x_codes || !x_scales))) return QW_ENULL;
  if (!codes_ok(codes, scales) || !codes_ok(x_codes, x_scales)) return QW_EARG;
  const qw::MxGemm g = {qw::MX_STORE, n, k, m, codes, scales, x_codes, x_scales, y_type, y,
                        nullptr, nullptr, nullptr, -1, nullptr};
  return record(qw::launch_mx_gemm(g, (hipStream_t)stream));
}

int64_t qw_mx_matmul_work_bytes(int64_t m, int64_t k) {
  if (check_mx_rows(m, 1, k) != QW_OK) return -1;
  // more rows or a longer k are not taken either, so that the size grows with both
  if (qw::mx_gemm_fuses(qw::MX_STORE, m, k)) return 0;
  Carve c;
  c.take(m * (qw::mx_pitch(k) / 2));
  c.take(m * (qw::mx_pitch(k) / 32));
  return c.at;
}

int qw_mx_matmul(int64_t n, int64_t k, const uint8_t* codes, const uint8_t* scales, int64_t m,
                 int x_type, const void* x, int y_type, void* y, void* work,
                 int64_t work_bytes, void* stream) {
  if (!mx_fits(n, k)) return QW_ESHAPE;
  int st = check_mx_rows(m, n, k);
  if (st != QW_OK) return st;
  if (!type_ok(x_type) || !type_ok(y_type)) return QW_EARG;
  if (m * n == 0) return QW_OK;
  if (!y || (k > 0 && (!codes || !scales || !x))) return QW_ENULL;
  if (!codes_ok(codes, scales)) return QW_EARG;
  qw::MxGemm g = {qw::MX_STORE, n, k, m, codes, scales, nullptr, nullptr, y_type, y,
                  nullptr, nullptr, nullptr, x_type, x};
  if (!qw::mx_gemm_fuses(qw::MX_STORE, m, k)) {
    const int64_t need = qw_mx_matmul_work_bytes(m, k);
    if (need > 0 && (!work || work_bytes < need || !qw::aligned(work, 16))) return QW_EWORK;
    Carve c;
    uint8_t* const xc = (uint8_t*)work + c.take(m * (qw::mx_pitch(k) / 2));
    uint8_t* const xs = (uint8_t*)work + c.take(0);
    if (k > 0) {
      st = record(qw::launch_mx_quantize(0, m, k, x_type, x, xc, xs, (hipStream_t)stream));
      if (st != QW_OK) return st;
    }
    g.x_type = -1;
    g.x = nullptr;
    g.xc = xc;
    g.xs = xs;
  }
  return record(qw::launch_mx_gemm(g, (hipStream_t)stream));
}

int qw_rms_norm(int64_t rows, int64_t d, int type, const void* x, const void* residual,
                void* sum, int weight_type, const void* weight, float eps, int y_type, void* y,
                void* stream) {
  const int st = check_norm(rows, d, type, weight_type, weight, eps);
  if (st != QW_OK) return st;
  if (!type_ok(y_type)) return QW_EARG;
  if (rows * d == 0) return QW_OK;
  if (!x || !y) return QW_ENULL;
  return record(qw::launch_rms_norm({0, rows, d, type, x, residual, sum, weight_type, weight, eps,
                                     y_type, y, nullptr}, (hipStream_t)stream));
}

int qw_rms_norm_block(int64_t rows, int64_t d, int type, const void* x, const void* residual,
                      void* sum, int weight_type, const void* weight, float eps,
                      uint8_t* codes, float* scales, void* stream) {
  const int st = check_norm(rows, d, type, weight_type, weight, eps);
  if (st != QW_OK) return st;
  if (check_block(1, 1, rows, d) != QW_OK) return QW_ESHAPE;
  if (rows * d == 0) return QW_OK;
  if (!x || !codes || !scales) return QW_ENULL;
  if (!qw::aligned(codes, 16)) return QW_EARG;
  return record(qw::launch_rms_norm({1, rows, d, type, x, residual, sum, weight_type, weight, eps,
                                     QW_F32, codes, scales}, (hipStream_t)stream));
}

int qw_rms_norm_mx(int64_t rows, int64_t d, int type, const void* x, const void* residual,
                   void* sum, int weight_type, const void* weight, float eps, uint8_t* codes,
                   uint8_t* scales, void* stream) {
  const int st = check_norm(rows, d, type, weight_type, weight, eps);
  if (st != QW_OK) return st;
  if (!mx_fits(rows, d)) return QW_ESHAPE;
  if (rows * d == 0) return QW_OK;
  if (!x || !codes || !scales) return QW_ENULL;
  if (!codes_ok(codes, scales)) return QW_EARG;
  return record(qw::launch_rms_norm({2, rows, d, type, x, residual, sum, weight_type, weight, eps,
                                     QW_F32, codes, scales}, (hipStream_t)stream));
}

int64_t qw_rms_norm_backward_work_bytes(int64_t rows, int64_t d) {
  return within(rows, d) ? qw::rms_norm_shares(rows) * d * 4 : -1;
}

int qw_rms_norm_backward(int64_t rows, int64_t d, int type, const void* dy, const void* s,
                         int weight_type, const void* weight, float eps, const void* dsum,
                         void* ds, float* dweight, void* work, int64_t work_bytes,
                         void* stream) {
  const int st = check_norm(rows, d, type, weight_type, weight, eps);
  if (st != QW_OK) return st;
  if (d == 0 || (!ds && !dweight)) return QW_OK;
  if (rows == 0)
    return dweight ? record(qw::launch_fill_zero(dweight, d, (hipStream_t)stream)) : QW_OK;
  if (!dy || !s) return QW_ENULL;
  const int64_t need = qw_rms_norm_backward_work_bytes(rows, d);
  if (dweight && (!work || work_bytes < need || !qw::aligned(work, 16))) return QW_EWORK;
  return record(qw::launch_rms_norm_backward({rows, d, type, dy, s, weight_type, weight, eps, dsum,
                                              ds, dweight, work}, (hipStream_t)stream));
}

int qw_mx_gated(int64_t f, int64_t k, const uint8_t* codes, const uint8_t* scales, int64_t m,
                const uint8_t* x_codes, const uint8_t* x_scales, int h_type, void* h,
                void* stream) {
  const int st = check_gated(f, k, m);
  if (st != QW_OK) return st;
  if (!type_ok(h_type)) return QW_EARG;
  if (m * f == 0) return QW_OK;
  if (!h || (k > 0 && (!codes || !scales || !x_codes || !x_scales))) return QW_ENULL;
  if (!codes_ok(codes, scales) || !codes_ok(x_codes, x_scales)) return QW_EARG;
  const qw::MxGemm g = {qw::MX_GATED, f, k, m, codes, scales, x_codes, x_scales, h_type, h,
                        nullptr, nullptr, nullptr, -1, nullptr};
  return record(qw::launch_mx_gemm(g, (hipStream_t)stream));
}

int qw_mx_gated_codes(int64_t f, int64_t k, const uint8_t* codes, const uint8_t* scales,
                      int64_t m, const uint8_t* x_codes, const uint8_t* x_scales,
                      uint8_t* h_codes, uint8_t* h_scales, void* stream) {
  const int st = check_gated(f, k, m);
  if (st != QW_OK) return st;
  if (m * f == 0) return QW_OK;
  if (!h_codes || !h_scales || (k > 0 && (!codes || !scales || !x_codes || !x_scales)))
    return QW_ENULL;
  if (!codes_ok(codes, scales) || !codes_ok(x_codes, x_scales) || !codes_ok(h_codes, h_scales))
    return QW_EARG;
  const qw::MxGemm g = {qw::MX_GATED_CODES, f, k, m, codes, scales, x_codes, x_scales, QW_F32,
                        h_codes, h_scales, nullptr, nullptr, -1, nullptr};
  return record(qw::launch_mx_gemm(g, (hipStream_t)stream));
}

int qw_mx_gated_backward(int64_t f, int64_t k, const uint8_t* codes, const uint8_t* scales,
                         int64_t m, const uint8_t* x_codes, const uint8_t* x_scales, int type,
                         const void* dh, void* dgate_up, void* h, void* stream) {
  const int st = check_gated(f, k, m);
  if (st != QW_OK) return st;
  if (!type_ok(type)) return QW_EARG;
  if (m * f == 0) return QW_OK;
  if (!dh || !dgate_up || (k > 0 && (!codes || !scales || !x_codes || !x_scales)))
    return QW_ENULL;
  if (!codes_ok(codes, scales) || !codes_ok(x_codes, x_scales)) return QW_EARG;
  const qw::MxGemm g = {qw::MX_GATED_BACKWARD, f, k, m, codes, scales, x_codes, x_scales, type,
                        dgate_up, nullptr, dh, h, -1, nullptr};
  return record(qw::launch_mx_gemm(g, (hipStream_t)stream));
}

int64_t qw_mx_mlp_work_bytes(int64_t m, int64_t d, int64_t f) {
  if (check_mx_mlp(m, d, f) != QW_OK) return -1;
  return MxMlpWork(m, d, f).bytes;
}

int qw_mx_mlp(int64_t d, int64_t f, const uint8_t* gate_up, const uint8_t* gate_up_scales,
              const uint8_t* down, const uint8_t* down_scales, int64_t m, int x_type,
              const void* x, int y_type, void* y, void* work, int64_t work_bytes,
              void* stream) {
  int st = check_mx_mlp(m, d, f);
  if (st != QW_OK) return st;
  st = check_gated(f, d, m);
  if (st != QW_OK) return st;
  if (!mx_fits(d, f)) return QW_ESHAPE;
  st = check_mx_rows(m, d, f);
  if (st != QW_OK) return st;
  if (!type_ok(x_type) || !type_ok(y_type)) return QW_EARG;
  if (m * d == 0) return QW_OK;
  if (!x || !y || (f > 0 && (!gate_up || !gate_up_scales || !down || !down_scales)))
    return QW_ENULL;
  if (!codes_ok(gate_up, gate_up_scales) || !codes_ok(down, down_scales)) return QW_EARG;
  const MxMlpWork at(m, d, f);
  if (!work || work_bytes < at.bytes || !qw::aligned(work, 16)) return QW_EWORK;
  uint8_t* const b = (uint8_t*)work;
  const hipStream_t s = (hipStream_t)stream;
  // few rows: gated values as floats, the sums of both products shared by waves
  const bool few = qw::mx_gemm_streams(qw::MX_GATED, f, m, d) && qw::mx_gemm_streams(qw::MX_STORE, d, m, f);
  qw::MxGemm up = {qw::MX_GATED, f, d, m, gate_up, gate_up_scales, b + at.xc, b + at.xs, QW_F32,
                   b + at.h, nullptr, nullptr, nullptr, -1, nullptr};
  if (few && qw::mx_gemm_fuses(qw::MX_GATED, m, d)) {
    up.x_type = x_type;
    up.x = x;
  } else {
    st = qw_mx_quantize(0, m, d, x_type, x, b + at.xc, b + at.xs, stream);
    if (st != QW_OK) return st;
  }
  if (!few) {
    up.result = qw::MX_GATED_CODES;
    up.y = b + at.hc;
    up.ys = b + at.hs;
  }
  if (f > 0) {
    st = record(qw::launch_mx_gemm(up, s));
    if (st != QW_OK) return st;
  }
  qw::MxGemm out = {qw::MX_STORE, d, f, m, down, down_scales, b + at.hc, b + at.hs, y_type, y,
                    nullptr, nullptr, nullptr, -1, nullptr};
  if (few && qw::mx_gemm_fuses(qw::MX_STORE, m, f)) {
    out.x_type = QW_F32;
    out.x = b + at.h;
  } else if (few) {
    st = qw_mx_quantize(0, m, f, QW_F32, b + at.h, b + at.hc, b + at.hs, stream);
    if (st != QW_OK) return st;
  }
  return record(qw::launch_mx_gemm(out, s));
}

int qw_mx_debug_path(int op, int64_t m, int64_t n, int64_t k) {
  if (op < 0 || op > 4) return QW_EARG;
  if (op == 0 || op == 4) {
    if (!mx_fits(n, k)) return QW_ESHAPE;
    const int st = check_mx_rows(m, n, k);
    if (st != QW_OK) return st;
    if (op == 4) return qw::mx_gemm_fuses(qw::MX_STORE, m, k) ? 1 : 2;
    return qw::mx_gemm_path(qw::MX_STORE, n, m, k);
  }
  const int st = check_gated(n, k, m);
  if (st != QW_OK) return st;
  return qw::mx_gemm_path(op == 1 ? qw::MX_GATED : op == 2 ? qw::MX_GATED_CODES : qw::MX_GATED_BACKWARD,
                          n, m, k);
}

// Which kernel family a call with these arguments would take (1 = fast,
// 2 = block, 3 = generic, 4 = matrix-core GEMV; for op 5, 1 = GEMV and
// 2 = GEMM; negative = invalid arguments).  Used by the tests to make sure
// every family is exercised.
int qw_debug_path(int op, int bits, int64_t group, int64_t n, int64_t k, const void* a,
                  const void* b) {
  qw::Mat mt;
  int st = check_mat(bits, group, n, k, &mt);
  if (st != QW_OK) return st;
  switch (op) {
    case 0: return qw::quantize_path(mt, (const float*)a, (const uint8_t*)b);
    case 1: return qw::unpack_path(mt, (const uint8_t*)a, (const float*)b);
    case 2: return qw::gemv_path(mt, (const uint8_t*)a, (const float*)b);
    case 3: return qw::gemm_path(mt, (const uint8_t*)a, (const uint16_t*)b);
    case 4: return qw::gemv_mfma_path(mt, (const uint8_t*)a, (const float*)b);
    case 5: return qw::matmul_prefers_gemv(mt, (const uint8_t*)a, (const float*)b) ? 1 : 2;
    default: return QW_ECOUNT;
  }
}

}  // extern "C"
