/*
 * Host-side check of the entry points of include/qw_mx.h, as abi_fuzz.c does it
 * for the others: built with AddressSanitizer and UndefinedBehaviorSanitizer on
 * the host code of libqw by tests/test_host_sanitizers_mx.py, on a machine
 * without a GPU.
 *
 * Part 1 calls each entry point with arguments whose status is known, part 2
 * draws arguments from edge values with a seeded generator and checks that every
 * call returns a documented status and that the sizes asked for agree with the
 * calls that need them.  With no GPU, calls that pass validation run the
 * dispatch code on the host up to the kernel launch, which fails with QW_EHIP.
 * Pointers are fake device addresses that the host code never dereferences; if a
 * GPU is visible only calls that fail validation are made.
 */
#include <stdint.h>
#include <stdio.h>
#include <stdlib.h>

#include "qw_mx.h"

/* from the HIP runtime (C linkage; hipError_t is an enum) */
int hipGetDeviceCount(int* count);

static int g_fail = 0;
static long g_calls = 0;
static long g_hist[16];

static void fail(const char* what, long long got) {
  printf("FAIL: %s: %lld\n", what, got);
  ++g_fail;
}

static void seen(int st) {
  ++g_calls;
  if (st > 0 || st < -10)
    fail("undocumented status", st);
  else
    ++g_hist[-st];
}

#define EXPECT(call, want)                                                               \
  do {                                                                                   \
    const int64_t v_ = (call);                                                           \
    ++g_calls;                                                                           \
    if (v_ != (int64_t)(want)) {                                                         \
      printf("FAIL line %d: %s returned %lld, expected %lld\n", __LINE__, #call,         \
             (long long)v_, (long long)(want));                                          \
      ++g_fail;                                                                          \
    }                                                                                    \
  } while (0)

/* fake device addresses: 256-aligned, 4-aligned, unaligned */
#define PA ((void*)(uintptr_t)0x7f0000000000ull)
#define P4 ((void*)(uintptr_t)0x7f0000000004ull)
#define P1 ((void*)(uintptr_t)0x7f0000000001ull)

static const int64_t MAXE = QW_MAX_ELEMENTS;

static void fixed_cases(int launches_ok) {
  EXPECT(qw_mx_pitch(MAXE), MAXE);
  EXPECT(qw_mx_pitch(MAXE + 1), -1);
  EXPECT(qw_mx_pitch(INT64_MAX), -1);
  EXPECT(qw_mx_matmul_work_bytes(MAXE, 1), -1);
  EXPECT(qw_mx_matmul_work_bytes(4, QW_BLOCK_MAX_K + 1), -1);
  EXPECT(qw_mx_mlp_work_bytes(4, QW_BLOCK_MAX_K, QW_BLOCK_MAX_K) > 0, 1);
  EXPECT(qw_mx_mlp_work_bytes(INT64_MAX, 4, 4), -1);
  EXPECT(qw_rms_norm_backward_work_bytes(INT64_MAX, INT64_MAX), -1);
  EXPECT(qw_mx_quantize(0, MAXE, 1, QW_F32, PA, PA, PA, 0), QW_ESHAPE);
  EXPECT(qw_mx_quantize(1, 1, MAXE, QW_F32, PA, PA, PA, 0), QW_ESHAPE);
  EXPECT(qw_mx_gemm(MAXE / 512, 512, PA, PA, 1 << 10, PA, PA, QW_F32, PA, 0), QW_EM);
  EXPECT(qw_mx_gemm(8, 512, PA, PA, INT64_MAX, PA, PA, QW_F32, PA, 0), QW_EM);
  EXPECT(qw_mx_gated(MAXE / 512, 512, PA, PA, 4, PA, PA, QW_F32, PA, 0), QW_ESHAPE);
  EXPECT(qw_mx_gated(INT64_MAX, 512, PA, PA, 4, PA, PA, QW_F32, PA, 0), QW_ESHAPE);
  EXPECT(qw_mx_mlp(QW_BLOCK_MAX_K, QW_BLOCK_MAX_K, PA, PA, PA, PA, 4, QW_F32, PA, QW_F32, PA, PA,
                   INT64_MAX, 0),
         QW_ESHAPE);
  if (!launches_ok) return;
  /* one call of every way that the dispatch takes, at ordinary and at limit sizes */
  static const int64_t ms[] = {1, 8, 9, 16, 17, 32, 33, 64, 300, 4096, 1 << 20, MAXE / 512};
  static const int64_t shapes[][2] = {{1, 1}, {4096, 4096}, {28672, 8192}, {17, 128 * 97},
                                      {1, QW_BLOCK_MAX_K}, {65536, 130}, {30, 0},
                                      {MAXE / 1024, 3}, {2, 20000}};
  for (int i = 0; i < 12; ++i)
    for (int j = 0; j < 9; ++j)
      for (int type = 0; type < 2; ++type) {
        const int64_t m = ms[i], n = shapes[j][0], k = shapes[j][1];
        if (m > MAXE / (2 * n) || m > MAXE / (2 * qw_mx_pitch(k) + 1) || m > MAXE / (2 * qw_mx_pitch(n))) continue;
        const int64_t work = qw_mx_matmul_work_bytes(m, k);
        EXPECT(qw_mx_gemm(n, k, PA, PA, m, PA, PA, type, PA, 0), QW_EHIP);
        EXPECT(qw_mx_gemm(n, k, PA, PA, m, PA, PA, type, P4, 0), QW_EHIP);
        EXPECT(qw_mx_matmul(n, k, PA, PA, m, type, PA, type, PA, PA, work, 0), QW_EHIP);
        EXPECT(qw_mx_matmul(n, k, PA, PA, m, type, P4, type, P4, PA, work, 0), QW_EHIP);
        if (work > 0)
          EXPECT(qw_mx_matmul(n, k, PA, PA, m, type, PA, type, PA, PA, work - 1, 0), QW_EWORK);
        EXPECT(qw_mx_gated(n, k, PA, PA, m, PA, PA, type, PA, 0), QW_EHIP);
        EXPECT(qw_mx_gated_codes(n, k, PA, PA, m, PA, PA, PA, PA, 0), QW_EHIP);
        EXPECT(qw_mx_gated_backward(n, k, PA, PA, m, PA, PA, type, PA, PA, PA, 0), QW_EHIP);
        EXPECT(qw_mx_gated_backward(n, k, PA, PA, m, PA, PA, type, P4, P4, 0, 0), QW_EHIP);
        for (int t = 0; t < 2; ++t)
          EXPECT(qw_mx_quantize(t, n, k, type, P4, PA, PA, 0), k ? QW_EHIP : QW_OK);
        EXPECT(qw_mx_unpack(n, k, PA, PA, P4, 0), k ? QW_EHIP : QW_OK);
        if (n <= QW_BLOCK_MAX_K && qw_mx_mlp_work_bytes(m, k, n) >= 0) {
          const int64_t w = qw_mx_mlp_work_bytes(m, k, n);
          EXPECT(qw_mx_mlp(k, n, PA, PA, PA, PA, m, type, PA, type, PA, PA, w, 0),
                 k ? QW_EHIP : QW_OK);
          if (k)
            EXPECT(qw_mx_mlp(k, n, PA, PA, PA, PA, m, type, P4, type, P4, PA, w - 1, 0), QW_EWORK);
        }
      }
  static const int64_t ds[] = {1, 500, 1024, 1030, 4096, 5003, 16384, 16392, 70000, 1 << 24};
  for (int i = 0; i < 12; ++i)
    for (int j = 0; j < 10; ++j)
      for (int type = 0; type < 2; ++type) {
        const int64_t rows = ms[i], d = ds[j];
        if (rows > MAXE / qw_mx_pitch(d)) continue;
        const int64_t work = qw_rms_norm_backward_work_bytes(rows, d);
        EXPECT(qw_rms_norm(rows, d, type, PA, 0, 0, 0, 0, 1e-6f, 1 - type, P4, 0), QW_EHIP);
        EXPECT(qw_rms_norm(rows, d, type, P4, PA, PA, 1, PA, 0.0f, type, PA, 0), QW_EHIP);
        EXPECT(qw_rms_norm_block(rows, d, type, PA, PA, P4, 0, PA, 1e-6f, PA, PA, 0), QW_EHIP);
        EXPECT(qw_rms_norm_mx(rows, d, type, PA, PA, P4, 0, PA, 1e-6f, PA, PA, 0), QW_EHIP);
        EXPECT(qw_rms_norm_backward(rows, d, type, PA, PA, 0, P4, 1e-6f, PA, PA, PA, PA, work, 0),
               QW_EHIP);
        EXPECT(qw_rms_norm_backward(rows, d, type, P4, P4, 1, 0, 1e-6f, 0, P4, 0, 0, 0, 0),
               QW_EHIP);
        EXPECT(qw_rms_norm_backward(rows, d, type, PA, PA, 0, 0, 1e-6f, 0, 0, PA, PA, work - 1, 0),
               QW_EWORK);
      }
  EXPECT(qw_rms_norm_backward(0, 40, QW_F32, 0, 0, 0, 0, 1e-6f, 0, 0, PA, 0, 0, 0), QW_EHIP);
}

/* ------------------------------------------------------------ fuzz */

static uint64_t g_rng = 0x9E3779B97F4A7C15ull;
static uint64_t rnd(void) { /* xorshift64* */
  g_rng ^= g_rng >> 12;
  g_rng ^= g_rng << 25;
  g_rng ^= g_rng >> 27;
  return g_rng * 0x2545F4914F6CDD1Dull;
}

static const int64_t kDims[] = {-1, 0, 1, 2, 7, 8, 100, 127, 128, 511, 512, 513, 1408, 4096, 28672,
                                1ll << 20, 1ll << 22, (1ll << 22) + 1, (1ll << 31) - 1, 1ll << 31,
                                1ll << 36, INT64_MAX - 511, INT64_MAX};
static const int64_t kMs[] = {-1, 0, 1, 2, 8, 9, 16, 17, 60, 300, 4099, 1ll << 20, 1ll << 30,
                              (1ll << 30) + 1, 1ll << 31, INT64_MAX};
#define PICK(v) (v[rnd() % (sizeof(v) / sizeof(v[0]))])
/* mostly sane values, so that whole calls get through */
#define MOSTLY(v, lo, count) (rnd() % 4 ? v[(lo) + rnd() % (count)] : PICK(v))

static void* ptr(void) {
  static void* const p[] = {PA, PA, PA, PA, P4, P1, 0};
  return p[rnd() % 7];
}
static int type(void) { return rnd() % 16 ? (int)(rnd() % 2) : (int)(rnd() % 5) - 2; }

static float eps(void) {
  static const float e[] = {1e-6f, 1e-5f, 0.0f, 1.0f, -1.0f, 1.0f / 0.0f, 0.0f / 0.0f};
  return rnd() % 4 ? e[rnd() % 4] : e[rnd() % 7];
}

static void fuzz(long iters, int launches_ok) {
  for (long it = 0; it < iters; ++it) {
    const int64_t n = MOSTLY(kDims, 2, 12), k = MOSTLY(kDims, 1, 14), m = MOSTLY(kMs, 1, 10);
    const int64_t bytes = rnd() % 2 ? INT64_MAX : ((int64_t)(rnd() % 5) - 1) * (1 << 20);
    void* const out = launches_ok ? ptr() : 0; /* without it every call with work to do fails */
    const int op = (int)(rnd() % 17);
    int st = 0;
    switch (op) {
      case 0:
        st = qw_mx_quantize(rnd() % 8 ? (int)(rnd() % 2) : (int)(rnd() % 9) - 4, n, k, type(), ptr(),
                            out, ptr(), 0);
        break;
      case 1: st = qw_mx_unpack(n, k, ptr(), ptr(), out, 0); break;
      case 2: st = qw_mx_gemm(n, k, ptr(), ptr(), m, ptr(), ptr(), type(), out, 0); break;
      case 3:
        st = qw_mx_matmul(n, k, ptr(), ptr(), m, type(), ptr(), type(), out, ptr(), bytes, 0);
        break;
      case 4: st = qw_mx_gated(n, k, ptr(), ptr(), m, ptr(), ptr(), type(), out, 0); break;
      case 5: st = qw_mx_gated_codes(n, k, ptr(), ptr(), m, ptr(), ptr(), out, ptr(), 0); break;
      case 6:
        st = qw_mx_gated_backward(n, k, ptr(), ptr(), m, ptr(), ptr(), type(), ptr(), out, ptr(), 0);
        break;
      case 7:
        st = qw_mx_mlp(k, n, ptr(), ptr(), ptr(), ptr(), m, type(), ptr(), type(), out, ptr(), bytes,
                       0);
        break;
      case 8:
        st = qw_rms_norm(m, k, type(), ptr(), ptr(), ptr(), type(), ptr(), eps(), type(), out, 0);
        break;
      case 9:
        st = qw_rms_norm_block(m, k, type(), ptr(), ptr(), ptr(), type(), ptr(), eps(), out, ptr(), 0);
        break;
      case 10:
        st = qw_rms_norm_mx(m, k, type(), ptr(), ptr(), ptr(), type(), ptr(), eps(), out, ptr(), 0);
        break;
      case 11:
        st = qw_rms_norm_backward(m, k, type(), launches_ok ? ptr() : 0, ptr(), type(), ptr(), eps(),
                                  ptr(), out, launches_ok ? ptr() : 0, ptr(), bytes, 0);
        break;
      default: {
        int64_t v;
        ++g_calls;
        if (op == 12)
          v = qw_mx_pitch(k);
        else if (op == 13)
          v = qw_mx_matmul_work_bytes(m, k);
        else if (op == 14)
          v = qw_mx_mlp_work_bytes(m, k, n);
        else if (op == 15)
          v = qw_rms_norm_backward_work_bytes(m, k);
        else {
          v = qw_mx_debug_path((int)(rnd() % 7) - 1, m, n, k);
          if (v < -10 || v > 256256) fail("qw_mx_debug_path", v);
          continue;
        }
        if (v < -1) fail("a size", v);
        continue;
      }
    }
    seen(st);
  }
}

int main(int argc, char** argv) {
  const long iters = argc > 1 ? atol(argv[1]) : 20000;
  int devices = 0;
  if (hipGetDeviceCount(&devices) != 0) devices = 0;
  const int launches_ok = devices == 0;
  if (!launches_ok) printf("a GPU is visible: only calls that fail validation are made\n");
  fixed_cases(launches_ok);
  fuzz(iters, launches_ok);
  printf("abi_fuzz_mx: %ld calls, %d failures; statuses:", g_calls, g_fail);
  for (int i = 0; i <= 10; ++i) printf(" %d:%ld", -i, g_hist[i]);
  printf("\n");
  return g_fail ? 1 : 0;
}
