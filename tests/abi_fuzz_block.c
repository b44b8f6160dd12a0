/*
 * Host-side check of the block-scaled and expert entry points of the C ABI
 * (include/qw.h), as abi_fuzz.c does it for the others: built with
 * AddressSanitizer and UndefinedBehaviorSanitizer on the host code of libqw by
 * tests/test_host_sanitizers_block.py, on a machine without a GPU.
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

#include "qw.h"

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
  EXPECT(qw_block_pitch(MAXE), MAXE);
  EXPECT(qw_block_pitch(MAXE + 1), -1);
  EXPECT(qw_block_num_scales(1, MAXE / 128, 128), MAXE / 128);
  EXPECT(qw_block_num_scales(1, MAXE / 128 + 1, 128), -1);
  EXPECT(qw_block_num_scales(128, INT64_MAX, INT64_MAX), -1);
  EXPECT(qw_block_matmul_work_bytes(MAXE, 1), -1);
  EXPECT(qw_block_matmul_work_bytes(4, QW_BLOCK_MAX_K + 1), -1);
  EXPECT(qw_moe_sort_work_bytes(QW_MOE_MAX_SLOTS, 1, 512) > 0, 1);
  EXPECT(qw_moe_sort_work_bytes(QW_MOE_MAX_SLOTS + 1, 1, 512), -1);
  EXPECT(qw_moe_sort_work_bytes(INT64_MAX, INT64_MAX, 1), -1);
  EXPECT(qw_moe_mlp_work_bytes(QW_MOE_MAX_SLOTS, 1, 8, 128, 128), -1); /* rows of codes */
  EXPECT(qw_moe_mlp_work_bytes(4, 2, 8, QW_BLOCK_MAX_K + 1, 4), -1);
  EXPECT(qw_moe_mlp_work_bytes(4, 2, 8, 4, QW_BLOCK_MAX_K + 1), -1);
  EXPECT(qw_moe_mlp_work_bytes(4, 2, 8, QW_BLOCK_MAX_K, QW_BLOCK_MAX_K) > 0, 1);

  EXPECT(qw_block_quantize(128, 2, MAXE, 1, QW_F32, PA, PA, PA, 0), QW_ESHAPE);
  EXPECT(qw_block_quantize(128, INT64_MAX, 2, 2, QW_F32, PA, PA, PA, 0), QW_ESHAPE);
  EXPECT(qw_block_quantize_swiglu(1, MAXE, QW_F32, PA, 0, PA, PA, 0), QW_ESHAPE);
  EXPECT(qw_block_gemm(1, MAXE / 128, 128, PA, PA, 1 << 10, PA, PA, QW_F32, PA, 0), QW_EM);
  EXPECT(qw_block_gemm(1, 8, 128, PA, PA, INT64_MAX, PA, PA, QW_F32, PA, 0), QW_EM);
  EXPECT(qw_block_gemm_grouped(1, 512, MAXE / 128, 128, PA, PA, 4, PA, PA, PA, QW_F32, PA, 0),
         QW_ESHAPE);
  EXPECT(qw_moe_gather(QW_MOE_MAX_SLOTS, 2, 8, 8, QW_F32, PA, PA, PA, 0), QW_ESHAPE);
  EXPECT(qw_moe_combine(4, 2, MAXE, 8, QW_F32, PA, PA, 0, QW_F32, PA, 0), QW_ESHAPE);
  EXPECT(qw_moe_mlp(128, 512, QW_BLOCK_MAX_K, QW_BLOCK_MAX_K, PA, PA, PA, PA, 4, 2, QW_F32, PA,
                    4, PA, 0, QW_F32, PA, PA, INT64_MAX, 0),
         QW_ESHAPE);
  EXPECT(qw_block_debug_path(0, 0, INT64_MAX, INT64_MAX, INT64_MAX, QW_F32), QW_ESHAPE);
  if (!launches_ok) return;
  /* one call of every way that the dispatch takes, at ordinary and at limit sizes */
  static const int64_t ms[] = {1, 9, 16, 17, 64, 300, 4096, 1 << 20};
  static const int64_t shapes[][2] = {{1, 1}, {4096, 4096}, {28672, 8192}, {17, 128 * 97},
                                      {1, QW_BLOCK_MAX_K}, {65536, 130}, {30, 0}};
  for (int i = 0; i < 8; ++i)
    for (int j = 0; j < 7; ++j)
      for (int br = 1; br <= 128; br += 127)
        for (int type = 0; type < 2; ++type) {
          const int64_t m = ms[i], n = shapes[j][0], k = shapes[j][1];
          if (m * n > MAXE || m * qw_block_pitch(k) > MAXE) continue;
          const int64_t work = qw_block_matmul_work_bytes(m, k);
          EXPECT(qw_block_gemm(br, n, k, PA, PA, m, PA, PA, type, PA, 0), QW_EHIP);
          EXPECT(qw_block_matmul(br, n, k, PA, PA, m, type, PA, type, PA, PA, work, 0), QW_EHIP);
          EXPECT(qw_block_matmul(br, n, k, PA, PA, m, type, P4, type, P4, PA, work, 0), QW_EHIP);
          if (work > 0)
            EXPECT(qw_block_matmul(br, n, k, PA, PA, m, type, PA, type, PA, PA, work - 1, 0),
                   QW_EWORK);
          EXPECT(qw_block_gemm_grouped(br, 7, n, k, PA, PA, m, PA, PA, PA, type, PA, 0), QW_EHIP);
          EXPECT(qw_block_quantize(br, 3, n, k, type, P4, PA, PA, 0), k ? QW_EHIP : QW_OK);
          EXPECT(qw_block_unpack(br, 3, n, k, PA, PA, P4, 0), k ? QW_EHIP : QW_OK);
        }
  static const int64_t ts[] = {1, 4, 40, 400, 5000, 300000};
  for (int i = 0; i < 6; ++i)
    for (int type = 0; type < 2; ++type)
      for (int64_t f = 0; f < 400; f += 100 + 28 * (f == 100)) {
        const int64_t t = ts[i], sort = qw_moe_sort_work_bytes(t, 2, 60);
        const int64_t work = qw_moe_mlp_work_bytes(t, 2, 60, 520, f);
        EXPECT(qw_moe_sort(t, 2, 60, 8, PA, PA, PA, PA, PA, sort, 0), QW_EHIP);
        EXPECT(qw_moe_mlp(128, 60, 520, f, PA, PA, PA, PA, t, 2, type, PA, 4, PA, PA, type, PA,
                          PA, work, 0),
               QW_EHIP);
        EXPECT(qw_moe_mlp(128, 60, 520, f, PA, PA, PA, PA, t, 2, type, PA, 4, PA, PA, type, PA,
                          PA, work - 1, 0),
               QW_EWORK);
        EXPECT(qw_moe_gather(t, 2, f + 1, 2 * t, type, PA, PA, PA, 0), QW_EHIP);
        EXPECT(qw_moe_gather_block(t, 2, f + 1, 2 * t, type, PA, PA, PA, PA, 0), QW_EHIP);
        EXPECT(qw_moe_combine(t, 2, f + 1, 2 * t, type, PA, PA, PA, 1 - type, PA, 0), QW_EHIP);
        EXPECT(qw_moe_combine(t, 2, f + 1, 0, type, 0, PA, PA, 1 - type, PA, 0), QW_EHIP);
        EXPECT(qw_moe_combine_backward(t, 2, f, 2 * t, type, PA, PA, PA, 0, PA, PA, 0), QW_EHIP);
        EXPECT(qw_block_quantize_swiglu(t, f, type, P4, PA, PA, PA, 0), f ? QW_EHIP : QW_OK);
      }
}

/* ------------------------------------------------------------ fuzz */

static uint64_t g_rng = 0x9E3779B97F4A7C15ull;
static uint64_t rnd(void) { /* xorshift64* */
  g_rng ^= g_rng >> 12;
  g_rng ^= g_rng << 25;
  g_rng ^= g_rng >> 27;
  return g_rng * 0x2545F4914F6CDD1Dull;
}

static const int64_t kDims[] = {-1, 0, 1, 2, 7, 8, 100, 127, 128, 129, 300, 1408, 4096, 28672,
                                1ll << 20, 1ll << 22, (1ll << 22) + 1, (1ll << 31) - 1, 1ll << 31,
                                1ll << 36, INT64_MAX - 127, INT64_MAX};
static const int64_t kMs[] = {-1, 0, 1, 2, 8, 9, 16, 17, 60, 300, 4099, 1ll << 20, 1ll << 30,
                              (1ll << 30) + 1, 1ll << 31, INT64_MAX};
static const int64_t kTops[] = {-1, 0, 1, 2, 3, 8, 17, 1ll << 30, INT64_MAX};
static const int64_t kExperts[] = {-1, 0, 1, 2, 8, 60, 512, 513, 1ll << 31, INT64_MAX};
#define PICK(v) (v[rnd() % (sizeof(v) / sizeof(v[0]))])
/* mostly sane values, so that whole calls get through */
#define MOSTLY(v, lo, count) (rnd() % 4 ? v[(lo) + rnd() % (count)] : PICK(v))

static void* ptr(void) {
  static void* const p[] = {PA, PA, PA, PA, P4, P1, 0};
  return p[rnd() % 7];
}
static int type(void) { return rnd() % 16 ? (int)(rnd() % 2) : (int)(rnd() % 5) - 2; }

static void fuzz(long iters, int launches_ok) {
  for (long it = 0; it < iters; ++it) {
    const int br = rnd() % 8 ? (rnd() % 2 ? 128 : 1) : (int)(rnd() % 200) - 50;
    const int64_t n = MOSTLY(kDims, 2, 12), k = MOSTLY(kDims, 1, 14), m = MOSTLY(kMs, 1, 10);
    const int64_t topk = MOSTLY(kTops, 2, 5), e = MOSTLY(kExperts, 2, 5);
    const int64_t d = MOSTLY(kDims, 1, 12), rows = MOSTLY(kMs, 1, 11);
    const int64_t bytes = rnd() % 2 ? INT64_MAX : ((int64_t)(rnd() % 5) - 1) * (1 << 20);
    const int ids = rnd() % 8 ? 4 << rnd() % 2 : (int)(rnd() % 20) - 4;
    void* const out = launches_ok ? ptr() : 0; /* without it every call with work to do fails */
    const int op = (int)(rnd() % 18);
    int st = 0;
    switch (op) {
      case 0: st = qw_block_quantize(br, topk, n, k, type(), ptr(), out, ptr(), 0); break;
      case 1: st = qw_block_quantize_swiglu(m, d, type(), ptr(), ptr(), out, ptr(), 0); break;
      case 2: st = qw_block_unpack(br, topk, n, k, ptr(), ptr(), out, 0); break;
      case 3: st = qw_block_gemm(br, n, k, ptr(), ptr(), m, ptr(), ptr(), type(), out, 0); break;
      case 4:
        st = qw_block_matmul(br, n, k, ptr(), ptr(), m, type(), ptr(), type(), out, ptr(), bytes,
                             0);
        break;
      case 5:
        st = qw_block_gemm_grouped(br, e, n, k, ptr(), ptr(), rows, ptr(), ptr(), ptr(), type(),
                                   out, 0);
        break;
      case 6:
        st = qw_moe_sort(m, topk, e, ids, ptr(), ptr(), ptr(), out, ptr(), bytes, 0);
        break;
      case 7: st = qw_moe_gather(m, topk, d, rows, type(), ptr(), ptr(), out, 0); break;
      case 8:
        st = qw_moe_gather_block(m, topk, d, rows, type(), ptr(), ptr(), out, ptr(), 0);
        break;
      case 9:
        st = qw_moe_combine(m, topk, d, rows, type(), ptr(), ptr(), ptr(), type(), out, 0);
        break;
      case 10:
        st = qw_moe_combine_backward(m, topk, d, rows, type(), ptr(), ptr(),
                                     launches_ok ? ptr() : 0, ptr(), out, ptr(), 0);
        break;
      case 11:
        st = qw_moe_mlp(br, e, d, n, ptr(), ptr(), ptr(), ptr(), m, topk, type(), ptr(), ids,
                        ptr(), ptr(), type(), out, ptr(), bytes, 0);
        break;
      default: {
        int64_t v;
        ++g_calls;
        if (op == 12)
          v = qw_block_pitch(k);
        else if (op == 13)
          v = qw_block_num_scales(br, n, k);
        else if (op == 14)
          v = qw_block_matmul_work_bytes(m, k);
        else if (op == 15)
          v = qw_moe_sort_work_bytes(m, topk, e);
        else if (op == 16)
          v = qw_moe_mlp_work_bytes(m, topk, e, d, n);
        else {
          v = qw_block_debug_path((int)(rnd() % 6) - 1, e, m, n, k, type());
          if (v < -10 || v > 256256) fail("qw_block_debug_path", v);
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
  printf("abi_fuzz_block: %ld calls, %d failures; statuses:", g_calls, g_fail);
  for (int i = 0; i <= 10; ++i) printf(" %d:%ld", -i, g_hist[i]);
  printf("\n");
  return g_fail ? 1 : 0;
}
